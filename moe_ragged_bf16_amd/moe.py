"""Around the expert products: routing, the plan, rows dispatched and combined.

    route = moe_route(logits, top_k)              # weight, idx, counts, loss
    plan = moe_plan(route.idx, num_experts)       # offs, dest
    rows = moe_dispatch(x, plan)                  # [tokens * top_k, hidden], sorted by expert
    y = cake_grouped_det_mm(rows, w, plan.offs)   # the expert products of this package
    out = moe_combine(y, route.weight, plan)      # [tokens, hidden]

``moe_route``, ``moe_dispatch`` and ``moe_combine`` are differentiable (``weight``
and ``loss`` by the logits; rows by x; ``out`` by y and the weights); the
``_fwd`` / ``_bwd`` functions are the single calls they are made of, which record
nothing for autograd (neither gradients nor forward-mode tangents).  Every
step runs in the library's gfx950 kernels, reads the routing on the device only
(no host synchronisation) and is bitwise reproducible.  ``torch.jit.trace``
cannot see the library's calls: ``moe_plan`` and the single calls raise
NotImplementedError under it.
"""
from __future__ import annotations

from typing import NamedTuple, Optional, Tuple

import torch

from ._capi import native, refuse_tracing

__all__ = ["MoeRoute", "MoePlan", "moe_route", "moe_route_fwd", "moe_route_bwd", "moe_plan", "moe_dispatch",
           "moe_dispatch_fwd", "moe_dispatch_bwd", "moe_combine", "moe_combine_fwd", "moe_combine_bwd"]

_named = tuple.__new__  # (a NamedTuple from its fields' tuple, without its Python constructor)


class MoeRoute(NamedTuple):
    weight: torch.Tensor   # [tokens, top_k] fp32
    idx: torch.Tensor      # [tokens, top_k] int32, -1: no expert
    counts: torch.Tensor   # [experts] int32
    loss: torch.Tensor     # [] fp32
    balance: torch.Tensor  # [experts] fp32: the loss's derivative by each expert's probability sum


class MoePlan(NamedTuple):
    offs: torch.Tensor     # [experts] int32, cumulative end offsets
    dest: torch.Tensor     # [tokens, top_k] int32: the slot's row, -1: none


# ------------------------------------------------------------------------------------- routing
def moe_route_fwd(logits: torch.Tensor, top_k: int, *, normalize: bool = True,
                  token_mask: Optional[torch.Tensor] = None) -> MoeRoute:
    """Softmax top-k routing of logits [tokens, experts] (bf16 or fp32).

    idx: the top_k largest logits of each token, largest first, ties to the
    lower expert; an expert whose logit is -inf, and every expert of a token
    whose ``token_mask`` [tokens] (bool) is False, cannot be chosen, and slots
    left over hold -1 and weight 0.  weight: the softmax over the chosen experts
    (``normalize``) or the chosen entries of the softmax over all.  counts:
    slots of each expert.  loss: E / (top_k R^2) sum_e counts_e S_e, with R the
    tokens that have an expert and S_e their summed probability of e (0 without
    such tokens); it is 1 when the routing is even.
    """
    refuse_tracing("moe_route_fwd")
    return _named(MoeRoute, native.route_fwd(logits, top_k, normalize, token_mask))


def moe_route_bwd(dweight: Optional[torch.Tensor], dloss: Optional[torch.Tensor], logits: torch.Tensor,
                  route: MoeRoute, *, normalize: bool = True) -> torch.Tensor:
    """dlogits [tokens, experts] (logits' type) for the gradients of
    ``route.weight`` (fp32 [tokens, top_k]) and ``route.loss`` (fp32 scalar on
    the device); either may be None (zero).  ``route`` is what
    ``moe_route_fwd(logits, ..., normalize=normalize)`` returned."""
    refuse_tracing("moe_route_bwd")
    return native.route_bwd(dweight, dloss, logits, route.weight, route.idx, route.balance, normalize)


class _Route(torch.autograd.Function):
    @staticmethod
    def forward(ctx, logits, top_k, normalize, token_mask):
        r = _named(MoeRoute, native.route_fwd(logits, top_k, normalize, token_mask))
        ctx.save_for_backward(logits, *r)
        ctx.normalize = normalize
        ctx.mark_non_differentiable(r.idx, r.counts, r.balance)
        ctx.set_materialize_grads(False)
        return tuple(r)

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dweight, _idx, _counts, dloss, _balance):
        logits, *r = ctx.saved_tensors
        if dweight is None and dloss is None:
            return None, None, None, None
        dweight = None if dweight is None else dweight.contiguous()
        return moe_route_bwd(dweight, dloss, logits, MoeRoute(*r), normalize=ctx.normalize), None, None, None


def moe_route(logits: torch.Tensor, top_k: int, *, normalize: bool = True,
              token_mask: Optional[torch.Tensor] = None) -> MoeRoute:
    """``moe_route_fwd``, with ``weight`` and ``loss`` differentiable in logits
    (``idx``, ``counts`` and ``balance`` are constants)."""
    return MoeRoute(*_Route.apply(logits, top_k, normalize, token_mask))


# ---------------------------------------------------------------------------------- plan, rows
def moe_plan(idx: torch.Tensor, num_experts: int) -> MoePlan:
    """The plan that sorts the slots of idx [tokens, top_k] (int32) by expert,
    keeping their order within an expert: ``offs`` [num_experts] as the grouped
    products take it and ``dest`` [tokens, top_k], each slot's row.  Entries
    outside [0, num_experts) have no row (dest -1)."""
    refuse_tracing("moe_plan")
    return _named(MoePlan, native.plan(idx, num_experts))


def moe_dispatch_fwd(x: torch.Tensor, plan: MoePlan) -> torch.Tensor:
    """rows [tokens * top_k, hidden]: rows[dest[t, j]] = x[t] (bf16 or fp32);
    rows from offs[E-1] on, which no slot has, are zero."""
    refuse_tracing("moe_dispatch_fwd")
    return native.dispatch_fwd(x, plan.offs, plan.dest)


def moe_dispatch_bwd(drows: torch.Tensor, plan: MoePlan) -> torch.Tensor:
    """dx [tokens, hidden] = sum_j drows[dest[t, j]], in fp32, rounded once."""
    refuse_tracing("moe_dispatch_bwd")
    return native.dispatch_bwd(drows, plan.offs, plan.dest)


def moe_combine_fwd(y: torch.Tensor, weight: torch.Tensor, plan: MoePlan) -> torch.Tensor:
    """out [tokens, hidden] = sum_j weight[t, j] y[dest[t, j]], in fp32, rounded
    once; slots without a row add nothing."""
    refuse_tracing("moe_combine_fwd")
    return native.combine_fwd(y, weight, plan.offs, plan.dest)


def moe_combine_bwd(dout: torch.Tensor, y: torch.Tensor, weight: torch.Tensor,
                    plan: MoePlan) -> Tuple[torch.Tensor, torch.Tensor]:
    """(dy, dweight): dy[dest[t, j]] = weight[t, j] dout[t] (rows no slot has:
    zero) and dweight[t, j] = <dout[t], y[dest[t, j]]> in fp32."""
    refuse_tracing("moe_combine_bwd")
    return native.combine_bwd(dout, y, weight, plan.offs, plan.dest)


class _Dispatch(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, offs, dest):
        ctx.save_for_backward(offs, dest)
        return native.dispatch_fwd(x, offs, dest)

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, drows):
        return moe_dispatch_bwd(drows.contiguous(), MoePlan(*ctx.saved_tensors)), None, None


class _Combine(torch.autograd.Function):
    @staticmethod
    def forward(ctx, y, weight, offs, dest):
        ctx.save_for_backward(y, weight, offs, dest)
        return native.combine_fwd(y, weight, offs, dest)

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dout):
        y, weight, offs, dest = ctx.saved_tensors
        dy, dweight = moe_combine_bwd(dout.contiguous(), y, weight, MoePlan(offs, dest))
        return dy, dweight, None, None


def moe_dispatch(x: torch.Tensor, plan: MoePlan) -> torch.Tensor:
    """``moe_dispatch_fwd``, differentiable in x."""
    return _Dispatch.apply(x, plan.offs, plan.dest)


def moe_combine(y: torch.Tensor, weight: torch.Tensor, plan: MoePlan) -> torch.Tensor:
    """``moe_combine_fwd``, differentiable in y and weight."""
    return _Combine.apply(y, weight, plan.offs, plan.dest)
