"""Operands, bounds and checks of the gated feed-forward's tests.

Tolerances (u = 2^-24).  A sum of n products is off by at most (n + 2) u sum
|products|.  s(q) by es = 2 u (|q| + 3) of itself.  |act'| <= 1.13, so h = act(a) b is off by at
most (1.13 |b| da + |act(a)| db + 1.13 da db) + (es + 4 u) |h|.  The slope s + a s (1 - s) q' is off by at
most (1 + |a q'|) s (es + 8 u): each of its factors carries es or a rounding, and 1 - s an
absolute s es + u.  An s below the smallest normal number (TINY = 2^-126) is 0 in the kernels
(the hardware's reciprocal gives no subnormals), so s carries an absolute TINY beside
es, which reaches h as |a b| TINY, da as |dh b| (1 + |a q'|) TINY and db as |dh a| TINY.  bf16 results lie between the bf16 roundings of the interval's ends.
"""
import numpy as np
import torch

from oracle import gated as ref

DEV = "cuda:0"
U = 2.0 ** -24
TINY = 2.0 ** -126
C = np.sqrt(2.0 / np.pi)


def bf16(shape, gen, scale=1.0):
    return (torch.randn(shape, generator=gen, device=DEV) * scale).to(torch.bfloat16)


def f64(t):
    return t.detach().double().cpu().numpy()


def offsets(sizes):
    return torch.tensor(np.cumsum(sizes), dtype=torch.int32, device=DEV)


def inside(got, want, tol, what=""):
    lo = np.nextafter((want - tol).astype(np.float32), np.float32(-np.inf))
    hi = np.nextafter((want + tol).astype(np.float32), np.float32(np.inf))
    lo, hi = (torch.from_numpy(v).to(torch.bfloat16).float().numpy() for v in (lo, hi))
    g = got.detach().float().cpu().numpy()
    ok = (lo <= g) & (g <= hi)
    assert ok.all(), (what, int((~ok).sum()), np.argwhere(~ok)[:3].tolist(), g[~ok][:3], want[~ok][:3], tol[~ok][:3])


def q_of(a, name):
    if name == "silu":
        return a, np.ones_like(a)
    return 2 * C * (a + 0.044715 * a ** 3), 2 * C * (1 + 0.134145 * a * a)


def check_fwd(x, w, offs, name, h, gate_up, rows):
    """h and gate_up (or None) of the first `rows` rows."""
    xn, wn, k = f64(x)[:rows], f64(w), x.shape[1]
    o = offs.cpu().numpy()
    a, b = ref.projections(xn, wn, o)
    ta, tb = (t * (k + 2) * U for t in ref.projections(np.abs(xn), np.abs(wn), o))
    if gate_up is not None:
        inside(gate_up[:rows], np.concatenate([a, b], 1), np.concatenate([ta, tb], 1), "gate_up")
    want = ref.hidden(a, b, name)
    es = 2 * U * (np.abs(q_of(a, name)[0]) + 3)
    tol = 1.13 * np.abs(b) * ta + np.abs(ref.act(a, name)) * tb + 1.13 * ta * tb + (es + 4 * U) * np.abs(want) + np.abs(a * b) * TINY
    inside(h[:rows], want, tol + 1e-38, "h")


def check_dgrad(dy, w_down, gate_up, offs, name, d, rows):
    f, o, n = w_down.shape[2], offs.cpu().numpy(), dy.shape[1]
    gu = f64(gate_up)[:rows]
    a, b = gu[:, :f], gu[:, f:]
    dh, want = ref.gate_up_grad(f64(dy)[:rows], f64(w_down), a, b, o, name)
    t, _ = ref.gate_up_grad(np.abs(f64(dy)[:rows]), np.abs(f64(w_down)), a, b, o, name)
    t = t * (n + 2) * U
    q, dq = q_of(a, name)
    es = 2 * U * (np.abs(q) + 3)
    s = 1 / (1 + np.exp(-q))
    slope, act = np.abs(ref.act_grad(a, name)), np.abs(ref.act(a, name))
    err = (1 + np.abs(a) * dq) * (s * (es + 8 * U) + TINY)
    ta = np.abs(b) * (slope * t + (np.abs(dh) + t) * err) + 3 * U * np.abs(dh * b) * slope
    tb = act * t + (np.abs(dh) + t) * (act * (es + 4 * U) + np.abs(a) * TINY)
    inside(d[:rows], want, np.concatenate([ta, tb], 1) + 1e-38, "dgate_up")


def up(a, b):
    return -(-a // b)


def mid_tile(op, m, e, f, cus=256):
    """The middle kernel's tiles, restated from the library's rule."""
    tiles = (m // 64 + min(e, m)) * up(f, 32 if op == "fwd" else 64)
    return 64 if tiles * 2 <= (4 if op == "fwd" else 7) * cus else 128


def kernel_of(op, m, e, n, f, cus=256):
    """The kernel that takes a call ("small", "mid", "tile"), restated from the library's rule; n: k in
    the forward."""
    active = min(e, m)
    half_tiles = (m // 128 + active) * up(f, 128 if op == "fwd" else 256)
    if op == "fwd":
        units = (active + m // 64) * up(f, 16)
        if (m <= 32 * active and units * 4 <= 5 * cus) or (m <= 16 * active and units <= 8 * cus):
            return "small"
        return "mid" if m < 256 * active or half_tiles * 4 <= (9 if n <= 1024 else 5) * cus else "tile"
    if mid_tile(op, m, e, f, cus) == 64:
        return "mid" if n <= 2560 else "tile"
    if m < 96 * active or (half_tiles <= cus and n <= 2048):
        return "mid"
    return "mid" if half_tiles * 4 <= 9 * cus and n <= 1024 else "tile"


def variant_of(op, m, e, n, f):
    """The kernel and its form: the middle kernel's tiles; the tile kernel's partial stages and stages in pairs."""
    k = kernel_of(op, m, e, n, f)
    if k == "mid":
        return (op, k, mid_tile(op, m, e, f))
    if k == "small":
        return (op, k)
    return (op, k, n % 32 != 0, op == "dgrad" or n % 32 != 0 or m >= 1024 * e)
