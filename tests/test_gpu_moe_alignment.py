"""Routing of tensors whose memory starts anywhere their type allows: the accesses
change, the values and their bits do not."""
import pytest
import torch

import moe_ragged_bf16_amd as mdg

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def moved(t, by):
    """t's values in memory that starts `by` elements into an allocation."""
    out = torch.empty(t.numel() + by, dtype=t.dtype, device=t.device)[by:].view(t.shape)
    out.copy_(t)
    assert out.is_contiguous() and out.data_ptr() % 16 == by * t.element_size() % 16
    return out


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("T,E,k", [(1, 8, 2), (7, 16, 3), (5, 256, 8), (300, 128, 4), (1001, 64, 8), (9000, 8, 2),
                                   (33, 1024, 32), (70, 528, 5), (40, 12, 3)])
def test_unaligned_logits(T, E, k, dtype):
    g = torch.Generator(device=DEV)
    g.manual_seed(T + E)
    logits = torch.randn((T, E), generator=g, device=DEV).to(dtype)
    mask = torch.rand(T, generator=g, device=DEV) > 0.2
    dw, dl = torch.randn((T, k), generator=g, device=DEV), torch.full((), 0.3, device=DEV)
    for normalize in (True, False):
        want = mdg.moe_route_fwd(logits, k, normalize=normalize, token_mask=mask)
        grad = mdg.moe_route_bwd(dw, dl, logits, want, normalize=normalize)
        for by in (1, 2, 3, 4, 7):
            l = moved(logits, by)
            got = mdg.moe_route_fwd(l, k, normalize=normalize, token_mask=moved(mask, by))
            for a, b in zip(got, want):
                assert torch.equal(a, b)
            r = mdg.MoeRoute(*(moved(t, 1) if t.dim() else t for t in want))
            assert torch.equal(mdg.moe_route_bwd(moved(dw, 1), moved(dl[None], 1)[0], l, r, normalize=normalize), grad)


def test_unaligned_idx_of_a_plan_and_refused_rows():
    idx = torch.randint(-1, 9, (700, 3), dtype=torch.int32, device=DEV)
    want = mdg.moe_plan(idx, 9)
    for by in (1, 3):
        for a, b in zip(mdg.moe_plan(moved(idx, by), 9), want):
            assert torch.equal(a, b)
    x = moved(torch.randn((700, 64), device=DEV), 1)                # rows start on 16 bytes
    with pytest.raises(mdg.MdgError, match="status 1"):
        mdg.moe_dispatch_fwd(x, want)
