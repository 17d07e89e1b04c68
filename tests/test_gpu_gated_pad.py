"""Batches with rows of no group (a buffer's unused end) that hold NaN, in inputs, in output
gradients and in the memory the calls get for what they keep: nothing of it reaches
another row, a weight's gradient or a main_grad, in any kernel of the chain."""
import pytest
import torch

import moe_ragged_bf16_amd as mdg
from _gated import DEV, bf16, offsets, variant_of

pytestmark = pytest.mark.gpu

CASES = [([3, 0, 2], 20, 72, 64, 40), ([0, 0, 0], 33, 72, 64, 40), ([40, 0, 301], 21, 136, 72, 64), ([255, 1, 0, 130], 700, 264, 96, 72),
         ([900, 1101, 700], 500, 1608, 96, 72), ([0, 0, 0], 9000, 1608, 96, 72), ([2048, 0, 3001], 63, 2048, 64, 1000),
         ([2048, 0, 3001], 63, 2056, 72, 1032)]


def test_the_cases_reach_every_kernel():
    got = {variant_of(op, sum(s) + p, len(s), n if op == "dgrad" else k, f)[:2]
           for s, p, f, k, n in CASES for op in ("fwd", "dgrad")}
    assert got == {("fwd", "small"), ("fwd", "mid"), ("fwd", "tile"), ("dgrad", "mid"), ("dgrad", "tile")}


@pytest.mark.parametrize("sizes,pad,f,k,n", CASES)
@pytest.mark.parametrize("fuse", [False, True])
def test_nan_in_rows_of_no_group(sizes, pad, f, k, n, fuse):
    g = torch.Generator(device=DEV)
    g.manual_seed(f)
    rows, e = sum(sizes), len(sizes)
    m, offs = rows + pad, offsets(sizes)
    x, dy = bf16((m, k), g), bf16((m, n), g)
    w, w2 = bf16((e, 2 * f, k), g, 2 / k ** 0.5), bf16((e, n, f), g, 1 / f ** 0.5)

    def step(x, dy, w=w, w2=w2):
        a, b, c = (t.clone().requires_grad_() for t in (x, w, w2))
        b.main_grad, c.main_grad = (torch.ones(t.shape, device=DEV) for t in (b, c))
        y = mdg.grouped_gated_ffn(a, b, c, offs, fuse_wgrad_accumulation=fuse)
        y.backward(dy)
        return [t.clone() for t in ((y.detach(), a.grad, b.main_grad, c.main_grad) if fuse else
                                    (y.detach(), a.grad, b.grad, c.grad))]

    zeros = [t.clone() for t in (x, dy)]
    for t in zeros:
        t[rows:] = 0
    want = step(*zeros)
    nan = float("nan")
    for t in (x, dy):
        t[rows:] = nan
    step(*(torch.full_like(t, nan) for t in (x, dy, w, w2)))     # (its memory is what the next calls get)
    got = step(x, dy)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert torch.all(got[0][rows:] == 0) and torch.all(got[1][rows:] == 0)
