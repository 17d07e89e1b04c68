"""Plain NumPy implementation, in 64 bits, of the experts' gated feed-forward and its
gradients (written from the formulas; shares no code with the GPU path).

Expert e, rows s:t: a = x W[e, :F]^T, b = x W[e, F:]^T, h = act(a) b, y = h W2[e]^T;
act is SiLU, a / (1 + exp(-a)), or the tanh form of GELU, a (1 + tanh(c (a + 0.044715
a^3))) / 2 with c = sqrt(2 / pi).
"""
from __future__ import annotations

import numpy as np

__all__ = ["act", "act_grad", "groups", "projections", "hidden", "down", "gate_up_grad", "product_grads"]

_C = np.sqrt(2.0 / np.pi)


def _logistic(a, name):
    """(s, 1 - s, the derivative of its argument).  (1 + tanh v) / 2 = 1 / (1 + exp(-2 v)): the
    right side, as 1 + tanh v cancels for negative v (at v = -16 half a percent is lost in
    64 bits)."""
    q, dq = (a, np.ones_like(a)) if name == "silu" else \
        (2.0 * _C * (a + 0.044715 * a ** 3), 2.0 * _C * (1.0 + 0.134145 * a * a))
    return 1.0 / (1.0 + np.exp(-q)), 1.0 / (1.0 + np.exp(q)), dq


def act(a, name):
    with np.errstate(over="ignore", invalid="ignore"):
        return a * _logistic(a, name)[0]


def act_grad(a, name):
    with np.errstate(over="ignore", invalid="ignore"):
        s, rest, dq = _logistic(a, name)
        return s + a * s * rest * dq


def groups(offs, rows):
    """Slices of the groups for offsets read as the kernels read them."""
    end, out = 0, []
    for o in offs:
        start, end = end, max(end, min(max(int(o), 0), rows))
        out.append(slice(start, end))
    return out


def projections(x, w, offs):
    """(a, b) [M, F], NaN in rows of no group."""
    f = w.shape[1] // 2
    out = np.full((x.shape[0], 2 * f), np.nan)
    for e, g in enumerate(groups(offs, x.shape[0])):
        out[g] = x[g] @ w[e].T
    return out[:, :f], out[:, f:]


def hidden(a, b, name):
    return act(a, name) * b


def down(h, w2, offs):
    out = np.full((h.shape[0], w2.shape[1]), np.nan)
    for e, g in enumerate(groups(offs, h.shape[0])):
        out[g] = h[g] @ w2[e].T
    return out


def gate_up_grad(dy, w2, a, b, offs, name):
    """(dh [M, F], [da, db] [M, 2 F])."""
    dh = np.full(a.shape, np.nan)
    for e, g in enumerate(groups(offs, dy.shape[0])):
        dh[g] = dy[g] @ w2[e]
    return dh, np.concatenate([dh * b * act_grad(a, name), dh * act(a, name)], axis=1)


def product_grads(g, x, w, offs):
    """Gradients of rows x and weights w [E, N, K] of the product x W^T for its gradient g."""
    dx, dw = np.zeros(x.shape), np.zeros(w.shape)
    for e, r in enumerate(groups(offs, x.shape[0])):
        dx[r] = g[r] @ w[e]
        dw[e] = g[r].T @ x[r]
    return dx, dw
