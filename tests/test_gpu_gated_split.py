"""The gated products where units left over after whole rounds of the GPU are cut along
the reduction and joined by a second kernel: every output element against the 64-bit
oracle, for launches of pieces only and of whole units and pieces, for each form of the
tile kernel, both activations, with the projections kept and without.  The plan that ran is read from
the workspace's head.  Bounds: tests/_gated.py (fp32 sums in any order)."""
import pytest
import torch

import moe_ragged_bf16_amd as mdg
from _gated import DEV, bf16, check_dgrad, check_fwd, offsets, up, variant_of

pytestmark = pytest.mark.gpu
SLOTS = 256                      # units of a round, and partial tiles of the workspace
MANY = [0] * 37


def plan_of(op, sizes, m, n, f):
    """(units, units that are cut, pieces of each), restated from the library's rule; n: k in the forward."""
    cols = up(f, 128 if op == "fwd" else 256)
    total, slots = sum(up(s, 256) for s in sizes) * cols, min((up(m, 256) + len(sizes)) * cols * 8, SLOTS)
    tail = total % SLOTS
    split = min(SLOTS // tail, 8, up(up(n, 32), 4), slots // tail) if tail else 1
    return total, tail if split > 1 else 0, split


# rows of the groups and of no group, f, k (n in the gradient)
FWD = [
    # pieces only: whole and partial stages, 2 to 8 pieces
    ([300, 0, 700], 39_000, 264, 264), ([300, 0, 700], 39_000, 264, 256), ([1, 256, 515], 39_000, 392, 2048),
    ([100], 40_000, 264, 1032), ([300, 0, 700] + MANY[1:] + [150], 10_850, 560, 512),
    # whole units and pieces
    ([4200, 100], 500, 2040, 264), ([4200, 100], 500, 2048, 512), ([4200, 100] + MANY + [30], 7670, 2048, 384),
    ([4097, 0, 255], 500, 1928, 136),
]
DGRAD = [
    ([300, 0, 700], 39_000, 264, 264), ([300, 0, 700], 39_000, 264, 256), ([1, 256, 515], 39_000, 392, 2048),
    ([100], 40_000, 520, 1032), ([4200, 100], 500, 4088, 264), ([4200, 100], 500, 4096, 512), ([4097, 0, 255], 500, 3848, 136),
]


def test_the_sizes_cut_units_in_every_form():
    got = set()
    for op, cases in (("fwd", FWD), ("dgrad", DGRAD)):
        for sizes, pad, f, n in cases:
            m = sum(sizes) + pad
            form, (total, tail, split) = variant_of(op, m, len(sizes), n, f), plan_of(op, sizes, m, n, f)
            assert form[1] == "tile" and split > 1, (op, sizes, f, n)
            got.add((*form, "both" if total > tail else "pieces"))
    assert got == {(*form, plan) for plan in ("pieces", "both") for form in (
        ("fwd", "tile", False, False), ("fwd", "tile", False, True), ("fwd", "tile", True, True),
        ("dgrad", "tile", False, True), ("dgrad", "tile", True, True))}
    assert {plan_of("fwd", s, sum(s) + p, n, f)[2] for s, p, f, n in FWD} >= {2, 3, 4, 8}


def gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def stale(need):
    """A workspace whose partial tiles are NaN: what a call does not write it may not read."""
    return torch.full((need,), 255, dtype=torch.uint8, device=DEV)


def check_plan(ws, op, sizes, m, n, f):
    _, tail, split = plan_of(op, sizes, m, n, f)
    assert ws[:8].view(torch.int32).tolist() == [tail, split]


@pytest.mark.parametrize("name", ["silu", "gelu_tanh"])
@pytest.mark.parametrize("keep", [True, False])
@pytest.mark.parametrize("sizes,pad,f,k", FWD)
def test_fwd(sizes, pad, f, k, keep, name):
    rows, g = sum(sizes), gen(f + k)
    m, e = rows + pad, len(sizes)
    x, w, offs = bf16((m, k), g), bf16((e, 2 * f, k), g, 2 / k ** 0.5), offsets(sizes)
    ws = stale(mdg.gated_gemm_fwd_workspace_bytes(m, f, k, e))
    h = torch.full((m, f), 7.0, dtype=torch.bfloat16, device=DEV)
    r = mdg.grouped_gated_gemm_fwd(x, w, offs, activation=name, keep=keep, out=h, workspace=ws)
    check_plan(ws, "fwd", sizes, m, k, f)
    check_fwd(x, w, offs, name, h, r.gate_up, rows)
    assert torch.all(h[rows:] == 7.0)
    again = mdg.grouped_gated_gemm_fwd(x, w, offs, activation=name, keep=not keep)
    assert torch.equal(again.h[:rows], h[:rows])


@pytest.mark.parametrize("name", ["silu", "gelu_tanh"])
@pytest.mark.parametrize("sizes,pad,f,n", DGRAD)
def test_dgrad(sizes, pad, f, n, name):
    rows, g = sum(sizes), gen(f + n)
    m, e = rows + pad, len(sizes)
    dy, w2, gate_up, offs = bf16((m, n), g), bf16((e, n, f), g, 1 / f ** 0.5), bf16((m, 2 * f), g), offsets(sizes)
    ws = stale(mdg.gated_gemm_dgrad_workspace_bytes(m, n, f, e))
    d = torch.full((m, 2 * f), 7.0, dtype=torch.bfloat16, device=DEV)
    mdg.grouped_gated_gemm_dgrad(dy, w2, gate_up, offs, activation=name, out=d, workspace=ws)
    check_plan(ws, "dgrad", sizes, m, n, f)
    check_dgrad(dy, w2, gate_up, offs, name, d, rows)
    assert torch.all(d[rows:] == 7.0)
    assert torch.equal(mdg.grouped_gated_gemm_dgrad(dy, w2, gate_up, offs, activation=name)[:rows], d[:rows])
