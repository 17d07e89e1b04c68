"""Plain NumPy implementation, in 64 bits, of routing, the plan, dispatch and
combine and their gradients (written from the formulas; shares no code with the
GPU path).

Routing of logits l [T, E]: expert e is available to token t when the token is
kept and l[t, e] != -inf; p is the softmax over the available experts (0 for a
token without any); the k largest available logits are chosen, ties to the lower
expert; weights are the softmax over the chosen ones (normalize) or their p.
With c_e the slots that chose e, R the tokens with an available expert and S_e =
sum_t p[t, e]: loss = E / (k R^2) sum_e c_e S_e.
"""
from __future__ import annotations

import numpy as np

__all__ = ["route", "route_grad", "plan", "dispatch", "dispatch_grad", "combine", "combine_grad"]


def _softmax(logits, mask):
    l = np.array(logits, dtype=np.float64)
    if mask is not None:
        l[~np.asarray(mask, dtype=bool)] = -np.inf
    with np.errstate(invalid="ignore"):
        big = l.max(axis=1, keepdims=True) if l.shape[0] else np.zeros((0, 1))
        live = big[:, 0] != -np.inf
        p = np.zeros_like(l)
        ex = np.exp(l[live] - big[live])
        p[live] = ex / ex.sum(axis=1, keepdims=True)
    return l, live, p


def route(logits, k, normalize=True, mask=None):
    """(weight [T, k], idx [T, k], counts [E], loss, balance [E])."""
    l, live, p = _softmax(logits, mask)
    T, E = l.shape
    # NaN above everything, then the value, then the lower expert
    rank = np.where(np.isnan(l), np.inf, l)
    idx = np.empty((T, k), dtype=np.int64)
    for t in range(T):
        idx[t] = np.lexsort((np.arange(E), -rank[t], ~np.isnan(l[t])))[:k]
    there = np.take_along_axis(l, idx, 1) != -np.inf
    weight = np.where(there, np.take_along_axis(p, idx, 1), 0.0)
    if normalize:
        s = weight.sum(axis=1, keepdims=True)
        weight = np.where(there, weight / np.where(s == 0, 1.0, s), 0.0)
    idx = np.where(there, idx, -1)
    counts = np.bincount(idx[idx >= 0], minlength=E)
    R = int(live.sum())
    balance = E * counts / (k * float(R) ** 2) if R else np.zeros(E)
    return weight, idx, counts, float((balance * p.sum(axis=0)).sum()), balance


def route_grad(logits, k, dweight, dloss, normalize=True, mask=None):
    """d (sum dweight * weight + dloss * loss) / d logits, by the chain rule through p."""
    weight, idx, _, _, balance = route(logits, k, normalize, mask)
    _, _, p = _softmax(logits, mask)
    T, E = p.shape
    dp = np.tile(dloss * balance, (T, 1))
    for t in range(T):
        sel = idx[t] >= 0
        e, w, dw = idx[t][sel], weight[t][sel], np.asarray(dweight[t], dtype=np.float64)[sel]
        if normalize:
            s = p[t, e].sum()
            dp[t, e] += (dw - (w * dw).sum()) / (s if s else 1.0)
        else:
            dp[t, e] += dw
    return p * (dp - (p * dp).sum(axis=1, keepdims=True))


def plan(idx, num_experts):
    """(offs [E], dest like idx): rows sorted by expert, then by slot."""
    flat = np.asarray(idx).reshape(-1)
    ok = (flat >= 0) & (flat < num_experts)
    slots = np.nonzero(ok)[0]
    slots = slots[np.argsort(flat[slots], kind="stable")]
    dest = np.full(flat.shape, -1, dtype=np.int64)
    dest[slots] = np.arange(slots.size)
    return np.cumsum(np.bincount(flat[ok], minlength=num_experts)), dest.reshape(np.shape(idx))


def dispatch(x, dest):
    rows = np.zeros((dest.size, x.shape[1]))
    for t, j in zip(*np.nonzero(dest >= 0)):
        rows[dest[t, j]] = x[t]
    return rows


def dispatch_grad(drows, dest):
    return combine(drows, np.ones(dest.shape), dest)


def combine(y, weight, dest):
    out = np.zeros((dest.shape[0], y.shape[1]))
    for t, j in zip(*np.nonzero(dest >= 0)):
        out[t] += np.float64(weight[t, j]) * y[dest[t, j]]
    return out


def combine_grad(dout, y, weight, dest):
    """(dy, dweight)."""
    dy, dw = np.zeros(y.shape), np.zeros(dest.shape)
    for t, j in zip(*np.nonzero(dest >= 0)):
        dy[dest[t, j]] = np.float64(weight[t, j]) * dout[t]
        dw[t, j] = (np.asarray(dout[t], dtype=np.float64) * y[dest[t, j]]).sum()
    return dy, dw
