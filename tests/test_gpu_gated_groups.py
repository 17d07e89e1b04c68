"""The gated products over more groups than a wave's lanes hold, in every kernel: rows in
the first and the last groups and around each wave's first and last ones, offsets that
fall there, every output element against the 64-bit oracle.  Bounds: tests/_gated.py."""
import numpy as np
import pytest
import torch

import moe_ragged_bf16_amd as mdg
from _gated import DEV, bf16, check_dgrad, check_fwd, offsets, variant_of

pytestmark = pytest.mark.gpu

# product, kernel (and tile), groups, rows in groups, rows of none, f, k (n in the gradient)
CASES = [
    ("fwd", "small", 257, 300, 0, 56, 40), ("fwd", "small", 1000, 24, 0, 264, 264), ("fwd", "small", 1024, 900, 0, 24, 72),
    ("fwd", ("mid", 64), 257, 1500, 8800, 24, 72),
    ("fwd", ("mid", 128), 1000, 3000, 0, 136, 40), ("fwd", ("mid", 128), 1024, 2500, 100, 72, 200),
    ("fwd", "tile", 1024, 3000, 262_000, 136, 40),
    ("dgrad", ("mid", 64), 257, 700, 30, 136, 72), ("dgrad", ("mid", 64), 1024, 860, 0, 24, 40),
    ("dgrad", ("mid", 128), 1000, 2000, 0, 72, 136), ("dgrad", ("mid", 128), 1024, 3000, 50, 264, 40),
    ("dgrad", "tile", 1024, 3000, 300_000, 136, 40),
]


def sizes_of(groups, rows, seed):
    """Rows in about a tenth of the groups, and in those at the ends of each wave's (64 threads of 4 groups)."""
    rng = np.random.default_rng(seed)
    ends = [g for w in range(0, groups, 256) for g in (w - 1, w, w + 1)] + [groups - 1, groups - 2, 3, 4]
    p = (rng.random(groups) < 0.1) * rng.random(groups)
    p[[g for g in ends if 0 <= g < groups]] = 0.5
    return rng.multinomial(rows, p / p.sum())


def form_of(op, m, e, n, f):
    v = variant_of(op, m, e, n, f)
    return v[1] if v[1] != "mid" else v[1:]


@pytest.mark.parametrize("op,form,groups,rows,pad,f,n", CASES)
@pytest.mark.parametrize("name", ["silu", "gelu_tanh"])
def test_many_groups(op, form, groups, rows, pad, f, n, name):
    m = rows + pad
    assert form_of(op, m, groups, n, f) == form
    g = torch.Generator(device=DEV)
    g.manual_seed(groups + rows)
    sizes = sizes_of(groups, rows, rows)
    good = offsets(sizes)
    # what falls, is negative or lies past the rows acts as its clamped form
    bad = good.clone()
    for at in range(256, groups, 256):
        if sizes[at] == 0:
            continue
        bad[at - 1] = good[at]                               # group `at` loses its rows to the one before
        bad[at] = good[at] - 1 if at % 512 else -3
    if not pad:
        bad[-1] = 10 ** 6
    for offs in (good, bad):
        if op == "fwd":
            x, w = bf16((m, n), g), bf16((groups, 2 * f, n), g, 2 / n ** 0.5)
            h = torch.full((m, f), 7.0, dtype=torch.bfloat16, device=DEV)
            r = mdg.grouped_gated_gemm_fwd(x, w, offs, activation=name, keep=True, out=h)
            check_fwd(x, w, offs, name, h, r.gate_up, rows)
            assert torch.all(h[rows:] == 7.0)
        else:
            dy, w2, gate_up = bf16((m, n), g), bf16((groups, n, f), g, 1 / f ** 0.5), bf16((m, 2 * f), g)
            d = torch.full((m, 2 * f), 7.0, dtype=torch.bfloat16, device=DEV)
            mdg.grouped_gated_gemm_dgrad(dy, w2, gate_up, offs, activation=name, out=d)
            check_dgrad(dy, w2, gate_up, offs, name, d, rows)
            assert torch.all(d[rows:] == 7.0)
