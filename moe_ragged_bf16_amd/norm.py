"""The norms before and after a block, with the block's gate and the scaled residual.

    out, n = block_norm(x, weight=w)                          # before a block: n = norm(x) (out is x)
    y = block(n)
    out, n = block_norm(x, y, post_weight=wp, gate=g, scale=s, weight=w)   # after it, and before the next

    z = y, or y / rms(y) * post_weight
    out = residual + scale * gate[t] * z                       # in the residual's type
    normed = out / rms(out) * weight                           # of out as stored

with rms(v) = sqrt(mean(v^2) + eps) over a token's row, in fp32.  ``block_norm`` is
differentiable in every tensor; ``block_norm_fwd`` and ``_bwd`` are the single
calls it is made of, which record nothing for autograd.  Every step runs in the
library's gfx950 kernels and is bitwise reproducible; all raise
NotImplementedError under ``torch.jit.trace``, which cannot see the calls.
"""
from __future__ import annotations

from typing import NamedTuple, Optional, Tuple

import torch

from ._capi import native, refuse_tracing
from .ops import incoming_gradient

__all__ = ["BlockNorm", "BlockNormGrads", "block_norm", "block_norm_fwd", "block_norm_bwd"]


class BlockNorm(NamedTuple):
    out: torch.Tensor                   # [tokens, hidden]: the residual stream (the residual itself without y)
    normed: Optional[torch.Tensor]      # [tokens, hidden], with a weight
    rstd: Optional[torch.Tensor]        # [tokens] fp32: 1 / rms(out), with a weight
    post_rstd: Optional[torch.Tensor]   # [tokens] fp32: 1 / rms(y), with a post_weight


class BlockNormGrads(NamedTuple):
    dresidual: Optional[torch.Tensor]
    dy: Optional[torch.Tensor]
    dweight: Optional[torch.Tensor]
    dpost_weight: Optional[torch.Tensor]
    dgate: Optional[torch.Tensor]


def block_norm_fwd(residual: torch.Tensor, y: Optional[torch.Tensor] = None, *,
                   weight: Optional[torch.Tensor] = None, post_weight: Optional[torch.Tensor] = None,
                   gate: Optional[torch.Tensor] = None, scale: float = 1.0, eps: float = 1e-6) -> BlockNorm:
    """out and normed (above) of residual and y [tokens, hidden], both bf16 or
    both fp32; hidden a multiple of 8, up to 16384, and up to 4,000,000 tokens.  weight and post_weight
    [hidden] are both bf16 or both fp32, in either type; gate [tokens] is fp32.
    Without y there is only the norm of the residual, which needs a weight."""
    refuse_tracing("block_norm_fwd")
    return BlockNorm(*native.norm_fwd(residual, y, weight, post_weight, gate, scale, eps))


def _bwd(dout, dnormed, norm, y, weight, post_weight, gate, scale, need) -> BlockNormGrads:
    return BlockNormGrads(*native.norm_bwd(dout, dnormed, norm.out, norm.rstd, norm.post_rstd, y, weight, post_weight,
                                           gate, scale, need))


def block_norm_bwd(dout: Optional[torch.Tensor], dnormed: Optional[torch.Tensor], norm: BlockNorm,
                   y: Optional[torch.Tensor] = None, *, weight: Optional[torch.Tensor] = None,
                   post_weight: Optional[torch.Tensor] = None, gate: Optional[torch.Tensor] = None,
                   scale: float = 1.0) -> BlockNormGrads:
    """The gradients of everything the forward was given (the others None), for
    the gradients of out and of normed, either of which may be None (zero).
    ``norm`` is what ``block_norm_fwd`` returned for the same arguments.
    dweight and dpost_weight are sums over the tokens in fp32, rounded once to
    the weights' type."""
    refuse_tracing("block_norm_bwd")
    need = 1 | 2 * (y is not None) | 4 * (weight is not None) | 8 * (post_weight is not None) | 16 * (gate is not None)
    return _bwd(dout, dnormed, norm, y, weight, post_weight, gate, scale, need)


class _BlockNorm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, residual, y, weight, post_weight, gate, scale, eps):
        r = block_norm_fwd(residual, y, weight=weight, post_weight=post_weight, gate=gate, scale=scale, eps=eps)
        ctx.set_materialize_grads(False)
        with_z = post_weight is not None or gate is not None
        ctx.with_y, ctx.scale = y is not None, scale
        # (without a norm or a gate on it, y's gradient does not need y, nor any out without a norm of it)
        ctx.save_for_backward(r.out if weight is not None else None, y if with_z else None, weight, post_weight, gate, r.rstd, r.post_rstd)
        return (r.normed,) if y is None else (r.out, r.normed)

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, *grads):
        out, y, weight, post_weight, gate, rstd, post_rstd = ctx.saved_tensors
        dout, dnormed = grads if ctx.with_y else (None, grads[0])
        if dout is None and dnormed is None:
            return (None,) * 7
        dout, dnormed = (None if g is None else incoming_gradient(g) for g in (dout, dnormed))
        need = sum(1 << i for i in range(5) if ctx.needs_input_grad[i])
        g = _bwd(dout, dnormed, BlockNorm(out, None, rstd, post_rstd), y, weight, post_weight, gate, ctx.scale, need)
        return (*g, None, None)


def block_norm(residual: torch.Tensor, y: Optional[torch.Tensor] = None, *, weight: Optional[torch.Tensor] = None,
               post_weight: Optional[torch.Tensor] = None, gate: Optional[torch.Tensor] = None, scale: float = 1.0,
               eps: float = 1e-6) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """(out, normed) of ``block_norm_fwd``, differentiable in residual, y, weight,
    post_weight and gate; normed is None without a weight, and out is the
    residual itself without y.  Kept for the gradient: out with a weight, y with a
    post_weight or a gate, and those."""
    got = _BlockNorm.apply(residual, y, weight, post_weight, gate, scale, eps)
    return (residual, got[0]) if y is None else got
