"""Plain NumPy implementation, in 64 bits, of the norms around a block, of the
gradients' norm and of clipping (written from the formulas; shares no code with the
GPU path).

z = y or y / rms(y) * post; out = residual + scale gate z, stored by `store` (the
rounding to the rows' type); normed = out / rms(out) * weight, rms(v) = sqrt(mean(v^2)
+ eps).
"""
from __future__ import annotations

import math

import numpy as np

__all__ = ["rms", "norm", "norm_grad", "block", "block_grad", "total_norm", "clipped"]


def rms(v, eps):
    return np.sqrt((v * v).mean(axis=1, keepdims=True) + eps)


def norm(v, weight, eps):
    return v / rms(v, eps) * weight


def norm_grad(v, weight, g, eps):
    """(dv, dweight) of norm(v, weight) for its gradient g."""
    r = rms(v, eps)
    gw = g * weight
    return gw / r - v * (gw * v).mean(axis=1, keepdims=True) / r ** 3, (g * v / r).sum(axis=0)


def block(residual, y, weight, post, gate, scale, eps, store=lambda v: v):
    """(out, normed or None)."""
    out = residual
    if y is not None:
        z = y if post is None else norm(y, post, eps)
        out = store(residual + scale * (1.0 if gate is None else gate[:, None]) * z)
    return out, None if weight is None else norm(out, weight, eps)


def block_grad(dout, dnormed, out, y, weight, post, gate, scale, eps):
    """(dresidual, dy, dweight, dpost, dgate), None for what is not there."""
    do, dw = np.zeros(out.shape) if dout is None else dout, None
    if weight is not None:
        dv, dw = norm_grad(out, weight, np.zeros(out.shape) if dnormed is None else dnormed, eps)
        do = do + dv
    if y is None:
        return do, None, dw, None, None
    dz = scale * (1.0 if gate is None else gate[:, None]) * do
    z = y if post is None else norm(y, post, eps)
    dgate = None if gate is None else scale * (do * z).sum(axis=1)
    if post is None:
        return do, dz, dw, None, dgate
    dy, dpost = norm_grad(y, post, dz, eps)
    return do, dy, dw, dpost, dgate


def total_norm(grads):
    """sqrt of the sum of squares over all arrays, exactly rounded sums of each array's."""
    return math.sqrt(math.fsum(float(np.square(g.astype(np.longdouble)).sum()) for g in grads))


def clipped(g, norm, max_norm, eps=1e-6):
    by = min(1.0, max_norm / (norm + eps)) if math.isfinite(norm) else 1.0
    return g * by
