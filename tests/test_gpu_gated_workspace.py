"""The gated products' workspaces: a call brings what the kernel that takes it uses."""
import gc

import pytest
import torch

import moe_ragged_bf16_amd as mdg
from _gated import DEV, bf16, kernel_of, offsets

pytestmark = pytest.mark.gpu
HEAD, PARTIALS = 8192, 256 * 256 * 256 * 4      # the tile kernel's plan, and its partial tiles at most

# m, experts, f, k (n in the gradient)
SIZES = [(2, 8, 14336, 4096), (1, 1, 8, 8), (40, 64, 1536, 2048), (488, 64, 1536, 2048), (300, 2, 136, 72),
         (3001, 16, 1000, 2000), (16384, 8, 14336, 4096), (2600, 1, 2176, 1000), (9000, 4, 1608, 40), (0, 3, 64, 64)]


def test_the_queries_follow_the_kernel():
    seen = set()
    for m, e, f, k in SIZES:
        for op, query in (("fwd", lambda: mdg.gated_gemm_fwd_workspace_bytes(m, f, k, e)),
                          ("dgrad", lambda: mdg.gated_gemm_dgrad_workspace_bytes(m, k, f, e))):
            tile = kernel_of(op, m, e, k, f) == "tile"
            seen.add((op, tile))
            assert HEAD < query() <= HEAD + PARTIALS if tile else query() == HEAD, (op, m, e, f, k)
    assert len(seen) == 4


def operands(m, e, f, k):
    g = torch.Generator(device=DEV)
    g.manual_seed(m + f)
    sizes = [m // e + (i < m % e) for i in range(e)]
    return (bf16((m, k), g), bf16((e, 2 * f, k), g, 2 / k ** 0.5), bf16((m, k), g), bf16((e, k, f), g, 1 / f ** 0.5),
            offsets(sizes))


@pytest.mark.parametrize("m,e,f,k", [s for s in SIZES if s[0] < 16384])
def test_a_workspace_of_just_that_size(m, e, f, k):
    x, w, dy, w2, offs = operands(m, e, f, k)
    want = mdg.grouped_gated_gemm_fwd(x, w, offs, keep=True)
    dwant = mdg.grouped_gated_gemm_dgrad(dy, w2, want.gate_up, offs)
    for op, need, call, out in (
            ("fwd", mdg.gated_gemm_fwd_workspace_bytes(m, f, k, e),
             lambda ws: mdg.grouped_gated_gemm_fwd(x, w, offs, workspace=ws).h, want.h),
            ("dgrad", mdg.gated_gemm_dgrad_workspace_bytes(m, k, f, e),
             lambda ws: mdg.grouped_gated_gemm_dgrad(dy, w2, want.gate_up, offs, workspace=ws), dwant)):
        around = torch.full((need + 4096,), 77, dtype=torch.uint8, device=DEV)
        ws = around[:need]
        assert torch.equal(call(ws), out)
        assert torch.all(around[need:] == 77)
        if kernel_of(op, m, e, k, f) != "tile":
            assert torch.all(ws == 77)                       # (the other kernels use none of it)
        with pytest.raises(ValueError, match="workspace too small"):
            call(ws[:need - 256])


def test_a_token_needs_its_outputs_only():
    x, w, _, _, offs = operands(2, 8, 1024, 512)
    mdg.grouped_gated_gemm_fwd(x, w, offs)
    gc.collect()
    torch.cuda.synchronize()
    torch.cuda.reset_peak_memory_stats()
    before = torch.cuda.memory_allocated()
    r = mdg.grouped_gated_gemm_fwd(x, w, offs)
    assert torch.cuda.max_memory_allocated() - before == HEAD + r.h.numel() * 2
