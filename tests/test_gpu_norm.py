"""The norms around a block on the GPU against the 64-bit oracle: every value at sizes
around the kernels' layouts, every combination of what may be left out, gradients
against the formula and against differences, special values, streams, graphs.

Tolerances (u = 2^-24).  A row's sum passes at most 40 roundings (16 a lane, 6 in a wave, 16
waves), so a mean of squares is off by 40 u of itself and 1 / rms by 20 u + 4 u: 32 u.
x = v / rms: 34 u.  z: 36 u.  out = fma(scale gate, z, residual): 40 u |scale gate z| + u |out|.
normed: 36 u.  With M = mean |g x| (g = dnormed weight) the mean is off by 110 u M, so
do = dout + (g - x mean) / rms by 160 u (|g| + |x| M) / rms + 3 u |dout|, and A = sum do z by
120 u sum (|dout| + |g| / rms) |z| + 300 u M / rms sum |x z|.  A sum of n terms over tokens: (n + 100) u
sum |terms|.  Results lie between the roundings of the interval's ends to their type.
"""
import itertools

import numpy as np
import pytest
import torch

import moe_ragged_bf16_amd as mdg
from oracle import norm as ref

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
U = 2.0 ** -24
BF, FP = torch.bfloat16, torch.float32


def f64(t):
    return None if t is None else t.detach().double().cpu().numpy()


def inside(got, want, tol, what=""):
    lo = np.nextafter((want - tol).astype(np.float32), np.float32(-np.inf))
    hi = np.nextafter((want + tol).astype(np.float32), np.float32(np.inf))
    if got.dtype == BF:
        lo, hi = (torch.from_numpy(v).to(BF).float().numpy() for v in (lo, hi))
    g = got.detach().float().cpu().numpy()
    ok = (lo <= g) & (g <= hi)
    assert ok.all(), (what, int((~ok).sum()), np.argwhere(~ok)[:3].tolist(), g[~ok][:3], want[~ok][:3], tol[~ok][:3])


def make(T, H, dtype, wdtype, seed, with_y=True, weight=True, post=True, gate=True):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    r = lambda *s, scale=1.0: torch.randn(s, generator=g, device=DEV) * scale
    return {"residual": r(T, H, scale=2.0).to(dtype), "y": r(T, H).to(dtype) if with_y else None,
            "weight": (1 + r(H, scale=0.3)).to(wdtype) if weight else None,
            "post_weight": (1 + r(H, scale=0.3)).to(wdtype) if post and with_y else None,
            "gate": r(T) if gate and with_y else None,
            "dout": r(T, H).to(dtype), "dnormed": r(T, H).to(dtype) if weight else None}


def check(c, scale, eps, got, grads=None, dout=True):
    n = {k: f64(v) for k, v in c.items()}
    H = n["residual"].shape[1]
    y, w, wp, gate = n["y"], n["weight"], n["post_weight"], n["gate"]
    g = scale * (np.ones((n["residual"].shape[0], 1)) if gate is None else gate[:, None])
    if y is not None:
        z = y if wp is None else ref.norm(y, wp, eps)
        want = n["residual"] + g * z
        inside(got.out, want, 40 * U * np.abs(g * z) + U * np.abs(want), "out")
        if wp is not None:
            inside(got.post_rstd, (1 / ref.rms(y, eps))[:, 0], 32 * U * (1 / ref.rms(y, eps))[:, 0], "post_rstd")
    else:
        assert got.out is c["residual"]
    out = f64(got.out)
    if w is not None:
        want = ref.norm(out, w, eps)
        inside(got.normed, want, 36 * U * np.abs(want), "normed")
    if grads is None:
        return
    dn, d = n["dnormed"], n["dout"] if dout else None
    do, dy, dw, dp, dg = ref.block_grad(d, dn, out, y, w, wp, gate, scale, eps)
    T, ad = out.shape[0], np.zeros(out.shape) if d is None else np.abs(d)
    r = 1 / ref.rms(out, eps)
    x, gx = out * r, np.zeros(out.shape)
    if dn is not None:
        gx = np.abs(dn * w)
    M = (gx * np.abs(x)).mean(axis=1, keepdims=True)
    te = 160 * U * r * (gx + np.abs(x) * M) + 3 * U * ad
    inside(grads.dresidual, do, te, "dresidual")
    if w is not None:
        tw = np.zeros(H) if dn is None else ((T + 100) * U * np.abs(dn * x)).sum(axis=0)
        inside(grads.dweight, dw, tw + 1e-38, "dweight")
    else:
        assert grads.dweight is None
    if y is None:
        assert grads.dy is None and grads.dgate is None and grads.dpost_weight is None
        return
    ta = 120 * U * ((ad + r * gx) * np.abs(z)).sum(1) + 300 * U * (M * r)[:, 0] * np.abs(x * z).sum(1)
    if gate is not None:
        inside(grads.dgate, dg, np.abs(scale) * ta + 4 * U * np.abs(dg), "dgate")
    dz = np.abs(g * do)
    tz = np.abs(g) * te + 3 * U * dz
    if wp is None:
        inside(grads.dy, dy, tz, "dy")
        return
    ry = 1 / ref.rms(y, eps)
    yh, A = np.abs(y * ry), np.abs((do * z).sum(axis=1, keepdims=True))
    back = np.abs(g) * A / H
    ty = ry * (np.abs(wp) * tz + yh * np.abs(g) * ta[:, None] / H + 60 * U * (dz * np.abs(wp) + yh * back))
    inside(grads.dy, dy, ty, "dy")
    tp = (tz * yh).sum(axis=0) + ((T + 100) * U * dz * yh).sum(axis=0)
    inside(grads.dpost_weight, dp, tp, "dpost_weight")


def run(c, scale, eps, dout=True, dnormed=True):
    how = {k: c[k] for k in ("weight", "post_weight", "gate")}
    got = mdg.block_norm_fwd(c["residual"], c["y"], scale=scale, eps=eps, **how)
    grads = mdg.block_norm_bwd(c["dout"] if dout else None, c["dnormed"] if dnormed else None, got, c["y"], scale=scale,
                               **how)
    return got, grads


@pytest.mark.parametrize("dtype,wdtype", [(BF, BF), (BF, FP), (FP, FP), (FP, BF)])
@pytest.mark.parametrize("T,H", [(1, 8), (3, 40), (5, 512), (4, 520), (9, 1016), (2, 1024), (7, 1032), (130, 2048), (33, 2056),
                                 (1, 4096), (700, 4104), (17, 7168), (3, 8192), (2, 8200), (600, 16384)])
def test_sizes(T, H, dtype, wdtype):
    c = make(T, H, dtype, wdtype, T + H)
    got, grads = run(c, 0.7, 1e-6)
    check(c, 0.7, 1e-6, got, grads)
    again, grads2 = run(c, 0.7, 1e-6)
    for a, b in zip(tuple(got) + tuple(grads), tuple(again) + tuple(grads2)):
        assert torch.equal(a, b)


@pytest.mark.parametrize("T,H", [(6, 72), (2100, 264), (40, 2304), (5, 16376)])
@pytest.mark.parametrize("dtype", [BF, FP])
def test_every_combination(T, H, dtype):
    for with_y, weight, post, gate in itertools.product((True, False), repeat=4):
        if not with_y and (post or gate or not weight):
            continue
        c = make(T, H, dtype, dtype, T, with_y, weight, post, gate)
        got, grads = run(c, -0.5, 1e-5)
        check(c, -0.5, 1e-5, got, grads)
        assert (got.normed is None) == (not weight) and (got.post_rstd is None) == (not post)
        if weight:
            got, grads = run(c, -0.5, 1e-5, dout=False)
            check(c, -0.5, 1e-5, got, grads, dout=False)
            _, grads = run(c, -0.5, 1e-5, dnormed=False)
            check({**c, "dnormed": None}, -0.5, 1e-5, got, grads)
            assert torch.all(grads.dweight == 0)


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("T,H", [(4095, 1032), (4096, 1032), (5001, 2048)])
def test_long_calls_around_the_rule_for_blocks(T, H, dtype):
    c = make(T, H, dtype, FP, T)
    got, grads = run(c, 0.25, 1e-6)
    check(c, 0.25, 1e-6, got, grads)
    _, grads2 = run(c, 0.25, 1e-6)
    assert all(torch.equal(a, b) for a, b in zip(grads, grads2))


def test_many_rows_of_a_narrow_width():
    c = make(70001, 24, BF, FP, 5)
    got, grads = run(c, 1.0, 1e-6)
    check(c, 1.0, 1e-6, got, grads)


@pytest.mark.parametrize("H", [64, 2048])
def test_no_tokens(H):
    c = make(0, H, BF, BF, 1)
    got, grads = run(c, 1.0, 1e-6)
    assert got.out.shape == got.normed.shape == (0, H) and got.rstd.shape == (0,)
    assert torch.all(grads.dweight == 0) and torch.all(grads.dpost_weight == 0) and grads.dweight.shape == (H,)
    assert grads.dy.shape == (0, H) and grads.dgate.shape == (0,)


@pytest.mark.parametrize("dtype", [BF, FP])
def test_special_rows_stay_where_they_are(dtype):
    """Rows of zeros, and NaN or infinities in one row, change no other row; a row of
    zeros is normed to zeros; a row whose squares overflow is divided by infinity."""
    c = make(40, 1040, dtype, dtype, 4)
    base, gbase = run(c, 1.0, 1e-6)
    d = {k: None if v is None else v.clone() for k, v in c.items()}
    d["y"][3] = 0
    d["residual"][3] = 0
    d["y"][7, 5] = float("nan")
    d["residual"][9, 1000] = float("inf")
    d["residual"][11] = 3e38
    got, grads = run(d, 1.0, 1e-6)
    rows = [i for i in range(40) if i not in (3, 7, 9, 11)]
    for a, b in ((got.out, base.out), (got.normed, base.normed), (got.rstd, base.rstd), (grads.dresidual, gbase.dresidual),
                 (grads.dy, gbase.dy), (grads.dgate, gbase.dgate)):
        assert torch.equal(a[rows], b[rows])
    assert torch.all(got.out[3] == 0) and torch.all(got.normed[3] == 0) and torch.isfinite(grads.dresidual[3]).all()
    assert got.out[7].isnan().all() and got.normed[7].isnan().all() and got.normed[9, 1000].isnan()
    assert torch.all(got.rstd[11] == 0) and torch.all(got.normed[11] == 0)


def test_normed_is_the_norm_of_out_as_stored():
    c = make(50, 4104, BF, BF, 8)
    got, _ = run(c, 0.3, 1e-6)
    alone = mdg.block_norm_fwd(got.out, weight=c["weight"])
    assert torch.equal(alone.normed, got.normed) and torch.equal(alone.rstd, got.rstd) and alone.out is got.out


@pytest.mark.parametrize("dtype", [BF, FP])
def test_autograd_is_the_single_calls(dtype):
    c = make(65, 1160, dtype, dtype, 9)
    names = ("residual", "y", "weight", "post_weight", "gate")
    leaves = {k: c[k].clone().requires_grad_() for k in names}
    out, normed = mdg.block_norm(leaves["residual"], leaves["y"], weight=leaves["weight"],
                                 post_weight=leaves["post_weight"], gate=leaves["gate"], scale=0.4)
    torch.autograd.backward([out, normed], [c["dout"], c["dnormed"]])
    got, grads = run(c, 0.4, 1e-6)
    assert torch.equal(out, got.out) and torch.equal(normed, got.normed)
    for k, g in zip(names, grads):
        assert torch.equal(leaves[k].grad, g), k
    # one of the outputs used, strided gradients, some inputs constant
    x = c["residual"].clone().requires_grad_()
    out, normed = mdg.block_norm(x, c["y"], weight=c["weight"], post_weight=c["post_weight"], gate=c["gate"], scale=0.4)
    strided = torch.cat([c["dnormed"], c["dnormed"]], 1)[:, :1160]
    g, = torch.autograd.grad(normed, x, strided, retain_graph=True)
    _, want = run(c, 0.4, 1e-6, dout=False)
    assert torch.equal(g, want.dresidual)
    g, = torch.autograd.grad(out, x, c["dout"])
    assert torch.equal(g, c["dout"])
    # before a block: the residual itself and its norm
    x, w = c["residual"].clone().requires_grad_(), c["weight"].clone().requires_grad_()
    out, normed = mdg.block_norm(x, weight=w)
    assert out is x
    (out.float() * c["dout"].float() + normed.float() * c["dnormed"].float()).sum().backward()
    b = mdg.block_norm_bwd(None, c["dnormed"], mdg.block_norm_fwd(c["residual"], weight=c["weight"]), weight=c["weight"])
    assert torch.equal(w.grad, b.dweight) and torch.equal(x.grad, c["dout"] + b.dresidual)


def test_gradients_against_differences():
    """fp32 rows: directional derivatives against central differences of the oracle in 64
    bits; the gradients carry fp32 roundings (bounds above), 1e-5 of their norm is outside
    them by far."""
    T, H, eps, scale = 6, 136, 1e-6, 0.8
    c = make(T, H, FP, FP, 10)
    _, grads = run(c, scale, eps)
    names = ("residual", "y", "weight", "post_weight", "gate")
    base, do, dn = [f64(c[k]) for k in names], f64(c["dout"]), f64(c["dnormed"])

    def value(r, y, w, p, g):
        out, normed = ref.block(r, y, w, p, g, scale, eps)
        return float((out * do).sum() + (normed * dn).sum())

    rng = np.random.default_rng(0)
    for i, g in enumerate(grads):
        v = rng.normal(size=base[i].shape)
        e = 1e-6
        hi, lo = list(base), list(base)
        hi[i], lo[i] = base[i] + e * v, base[i] - e * v
        want = (value(*hi) - value(*lo)) / (2 * e)
        got = float((f64(g) * v).sum())
        assert abs(got - want) <= 1e-5 * np.linalg.norm(f64(g)) * np.linalg.norm(v), (names[i], got, want)


def test_other_stream_and_graph_replay():
    c = make(300, 2056, BF, BF, 12)
    want, gwant = run(c, 0.5, 1e-6)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got, grads = run(c, 0.5, 1e-6)
    side.synchronize()
    for a, b in zip(tuple(got) + tuple(grads), tuple(want) + tuple(gwant)):
        assert torch.equal(a, b)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got, grads = run(c, 0.5, 1e-6)
    for i in range(4):
        new = make(300, 2056, BF, BF, 20 + i)
        for k, v in c.items():
            v.copy_(new[k])
        torch.cuda.synchronize()
        graph.replay()
        want, gwant = run(c, 0.5, 1e-6)
        torch.cuda.synchronize()
        for a, b in zip(tuple(got) + tuple(grads), tuple(want) + tuple(gwant)):
            assert torch.equal(a, b)


def test_rows_of_more_than_4_gib():
    T, H = 160_000, 16384                     # 5.2 GB a tensor
    g = torch.Generator(device=DEV)
    g.manual_seed(3)
    x = torch.empty((T, H), dtype=BF, device=DEV)
    x[:5], x[-300:] = (torch.randn((n, H), generator=g, device=DEV) for n in (5, 300))
    x[5:-300] = 1
    w = torch.randn(H, generator=g, device=DEV)
    got = mdg.block_norm_fwd(x, weight=w)
    alone = mdg.block_norm_fwd(x[-300:].clone(), weight=w)
    assert torch.equal(got.normed[-300:], alone.normed) and torch.equal(got.rstd[-300:], alone.rstd)
    b = mdg.block_norm_bwd(None, x, got, weight=w)
    ba = mdg.block_norm_bwd(None, x[-300:].clone(), alone, weight=w)
    assert torch.equal(b.dresidual[-300:], ba.dresidual)


def test_refusals_on_the_device():
    c = make(6, 64, BF, BF, 1)
    r, y, w = c["residual"], c["y"], c["weight"]
    fwd, bwd = mdg.block_norm_fwd, mdg.block_norm_bwd
    got = fwd(r, y, weight=w)
    flat = torch.zeros(7 * 64 + 8, dtype=BF, device=DEV)
    for error, call in (
            (ValueError, lambda: fwd(r)),
            (ValueError, lambda: fwd(r, weight=w, gate=c["gate"])),
            (ValueError, lambda: fwd(r, weight=w, post_weight=w)),
            (TypeError, lambda: fwd(r.half(), weight=w)),
            (TypeError, lambda: fwd(r, y.float(), weight=w)),
            (ValueError, lambda: fwd(r, y[:5], weight=w)),
            (ValueError, lambda: fwd(r, weight=w[:32])),
            (TypeError, lambda: fwd(r, y, weight=w, post_weight=w.float())),
            (TypeError, lambda: fwd(r, y, gate=c["gate"].to(BF))),
            (ValueError, lambda: fwd(r, y, gate=c["gate"][:5])),
            (ValueError, lambda: fwd(r.t(), weight=w)),
            (ValueError, lambda: fwd(r.cpu(), weight=w)),
            (TypeError, lambda: fwd(r, y, weight=w, scale=torch.ones((), device=DEV))),
            (mdg.MdgError, lambda: fwd(r, y, weight=w, scale=float("inf"))),
            (mdg.MdgError, lambda: fwd(r, y, weight=w, eps=-1.0)),
            (mdg.MdgError, lambda: fwd(flat[:6 * 60].view(6, 60), weight=flat[:60])),
            (mdg.MdgError, lambda: fwd(flat[4:4 + 6 * 64].view(6, 64), weight=w)),
            (mdg.MdgError, lambda: fwd(torch.zeros((1, 16392), dtype=BF, device=DEV),
                                       weight=torch.zeros(16392, dtype=BF, device=DEV))),
            (ValueError, lambda: bwd(None, None, got, y, weight=w)),
            (ValueError, lambda: bwd(r, r, got, y)),
            (ValueError, lambda: bwd(r, r, got, y, weight=w, post_weight=w)),
            (ValueError, lambda: bwd(r, None, fwd(r, y, gate=c["gate"]), gate=c["gate"])),
            (TypeError, lambda: bwd(r.float(), None, got, y, weight=w))):
        with pytest.raises(error):
            call()
