"""Around the expert products: routing, the plan, rows dispatched and combined.

    route = moe_route(logits, top_k)              # weight, idx, counts, loss
    plan = moe_plan(route.idx, num_experts)       # offs, dest
    rows = moe_dispatch(x, plan)                  # [tokens * top_k, hidden], sorted by expert
    y = cake_grouped_det_mm(rows, w, plan.offs)   # the expert products of this package
    out = moe_combine(y, route.weight, plan)      # [tokens, hidden]

``moe_route``, ``moe_dispatch`` and ``moe_combine`` are differentiable (``weight``
and ``loss`` by the logits; rows by x; ``out`` by y and the weights); the
``_fwd`` / ``_bwd`` functions are the single calls they are made of.  Every
step runs in the library's gfx950 kernels, reads the routing on the device only
(no host synchronisation) and is bitwise reproducible.
"""
from __future__ import annotations

from typing import NamedTuple, Optional, Tuple

import torch

from . import _capi
from .ops import _need, _same_device

__all__ = ["MoeRoute", "MoePlan", "moe_route", "moe_route_fwd", "moe_route_bwd", "moe_plan", "moe_dispatch",
           "moe_dispatch_fwd", "moe_dispatch_bwd", "moe_combine", "moe_combine_fwd", "moe_combine_bwd"]

try:  # the allocation torch's own compiled programs make: half the host time of torch.empty
    from torch._C._dynamo.guards import _empty_strided_cuda
except ImportError:  # pragma: no cover
    _empty_strided_cuda = None

_CODES = {torch.bfloat16: _capi.MDG_BF16, torch.float32: _capi.MDG_FP32}


class MoeRoute(NamedTuple):
    weight: torch.Tensor   # [tokens, top_k] fp32
    idx: torch.Tensor      # [tokens, top_k] int32, -1: no expert
    counts: torch.Tensor   # [experts] int32
    loss: torch.Tensor     # [] fp32
    balance: torch.Tensor  # [experts] fp32: the loss's derivative by each expert's probability sum


class MoePlan(NamedTuple):
    offs: torch.Tensor     # [experts] int32, cumulative end offsets
    dest: torch.Tensor     # [tokens, top_k] int32: the slot's row, -1: none


def _check(t: torch.Tensor, name: str, dtype, ndim: int, like: Optional[torch.Tensor] = None) -> None:
    """_need and _same_device at the cost of one test where all is well."""
    if isinstance(t, torch.Tensor) and t.dtype is dtype and t.dim() == ndim and t.is_cuda and t.is_contiguous() and \
            (like is None or t.get_device() == like.get_device()):
        return
    _need(t, name, dtype, ndim)
    _same_device(like, t)


def _need_float(t: torch.Tensor, name: str) -> int:
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    code = _CODES.get(t.dtype)
    if code is None:
        raise TypeError(f"{name} must be bfloat16 or float32, got {t.dtype}")
    _check(t, name, t.dtype, 2)
    return code


def _allocator(like: torch.Tensor):
    """f(size, stride, dtype): an uninitialised tensor on like's device."""
    if _empty_strided_cuda is not None and like.get_device() == torch._C._cuda_getDevice():
        return _empty_strided_cuda
    return lambda size, stride, dtype: torch.empty_strided(size, stride, dtype=dtype, device=like.device)


_entries = {}


def _entry(name: str):
    f = _entries.get(name)
    if f is None:
        f = _entries[name] = getattr(_capi.load_library(), name)
    return f


def _call(name: str, t: torch.Tensor, *args) -> None:
    """Calls a library entry on t's device, with its current stream as the last argument."""
    index = t.get_device()
    if index == torch._C._cuda_getDevice():
        st = _entry(name)(*args, torch._C._cuda_getCurrentRawStream(index))
    else:
        with torch.cuda.device(index):
            st = _entry(name)(*args, torch._C._cuda_getCurrentRawStream(index))
    if st:
        _capi.check(name, st)


def _scratch(new, need: int) -> Tuple[Optional[torch.Tensor], int]:
    """A workspace of `need` bytes (kept alive by the caller until the launch) and its address."""
    if need == 0:
        return None, 0
    t = new((need,), (1,), torch.uint8)
    return t, t.data_ptr()


def _plain_int(v, name: str) -> int:
    if isinstance(v, bool) or not isinstance(v, int):
        raise TypeError(f"{name} must be an int")
    return v


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
    code = _need_float(logits, "logits")
    _plain_int(top_k, "top_k")
    if not isinstance(normalize, bool):
        raise TypeError("normalize must be a bool")
    T, E = logits.shape
    if not 1 <= top_k <= E:
        raise ValueError(f"top_k must be between 1 and the number of experts {E}, got {top_k}")
    mask = 0
    if token_mask is not None:
        _check(token_mask, "token_mask", torch.bool, 1, logits)
        if token_mask.shape[0] != T:
            raise ValueError(f"token_mask must have {T} entries")
        mask = token_mask.data_ptr()
    new = _allocator(logits)
    weight = new((T, top_k), (top_k, 1), torch.float32)
    idx = new((T, top_k), (top_k, 1), torch.int32)
    counts = new((E,), (1,), torch.int32)
    loss = new((), (), torch.float32)
    balance = new((E,), (1,), torch.float32)
    need = _entry("moe_route_fwd_workspace_bytes")(T, E)
    ws, wp = _scratch(new, need)
    _call("moe_route_fwd", logits, logits.data_ptr(), code, mask, weight.data_ptr(), idx.data_ptr(), counts.data_ptr(),
          loss.data_ptr(), balance.data_ptr(), T, E, top_k, normalize, wp, need)
    return MoeRoute(weight, idx, counts, loss, balance)


def moe_route_bwd(dweight: Optional[torch.Tensor], dloss: Optional[torch.Tensor], logits: torch.Tensor,
                  route: MoeRoute, *, normalize: bool = True) -> torch.Tensor:
    """dlogits [tokens, experts] (logits' type) for the gradients of
    ``route.weight`` (fp32 [tokens, top_k]) and ``route.loss`` (fp32 scalar on
    the device); either may be None (zero).  ``route`` is what
    ``moe_route_fwd(logits, ..., normalize=normalize)`` returned."""
    code = _need_float(logits, "logits")
    T, E = logits.shape
    _check(route.weight, "route.weight", torch.float32, 2, logits)
    _check(route.idx, "route.idx", torch.int32, 2, logits)
    _check(route.balance, "route.balance", torch.float32, 1, logits)
    k = route.idx.shape[1]
    if tuple(route.idx.shape) != (T, k) or tuple(route.weight.shape) != (T, k) or route.balance.shape[0] != E:
        raise ValueError("route does not belong to logits of this shape")
    dw = dl = 0
    if dweight is not None:
        _check(dweight, "dweight", torch.float32, 2, logits)
        if tuple(dweight.shape) != (T, k):
            raise ValueError(f"dweight must have shape {(T, k)}")
        dw = dweight.data_ptr()
    if dloss is not None:
        _check(dloss, "dloss", torch.float32, 0, logits)
        dl = dloss.data_ptr()
    out = _allocator(logits)((T, E), (E, 1), logits.dtype)
    _call("moe_route_bwd", logits, logits.data_ptr(), code, route.weight.data_ptr(), route.idx.data_ptr(),
          route.balance.data_ptr(), dw, dl, out.data_ptr(), T, E, k, int(normalize))
    return out


class _Route(torch.autograd.Function):
    @staticmethod
    def forward(ctx, logits, top_k, normalize, token_mask):
        r = moe_route_fwd(logits, top_k, normalize=normalize, token_mask=token_mask)
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
    _check(idx, "idx", torch.int32, 2)
    _plain_int(num_experts, "num_experts")
    T, k = idx.shape
    if k < 1 or num_experts < 1:
        raise ValueError("idx needs at least one column and num_experts at least one expert")
    new = _allocator(idx)
    offs = new((num_experts,), (1,), torch.int32)
    dest = new((T, k), (k, 1), torch.int32)
    need = _entry("moe_plan_workspace_bytes")(T, k, num_experts)
    ws, wp = _scratch(new, need)
    _call("moe_plan", idx, idx.data_ptr(), offs.data_ptr(), dest.data_ptr(), T, k, num_experts, wp, need)
    return MoePlan(offs, dest)


def _need_plan(plan: MoePlan, t: torch.Tensor) -> Tuple[int, int, int]:
    offs, dest = plan
    _check(offs, "plan.offs", torch.int32, 1, t)
    _check(dest, "plan.dest", torch.int32, 2, t)
    T, k = dest.shape
    return T, k, offs.shape[0]


def _need_rows(t: torch.Tensor, name: str, rows: int) -> None:
    if t.shape[0] != rows:
        raise ValueError(f"{name} must have {rows} rows, got {t.shape[0]}")


def moe_dispatch_fwd(x: torch.Tensor, plan: MoePlan) -> torch.Tensor:
    """rows [tokens * top_k, hidden]: rows[dest[t, j]] = x[t] (bf16 or fp32);
    rows from offs[E-1] on, which no slot has, are zero."""
    code = _need_float(x, "x")
    T, k, E = _need_plan(plan, x)
    _need_rows(x, "x", T)
    H = x.shape[1]
    rows = _allocator(x)((T * k, H), (H, 1), x.dtype)
    _call("moe_dispatch_fwd", x, x.data_ptr(), plan.dest.data_ptr(), plan.offs.data_ptr(), rows.data_ptr(),
          T, k, E, H, code)
    return rows


def moe_dispatch_bwd(drows: torch.Tensor, plan: MoePlan) -> torch.Tensor:
    """dx [tokens, hidden] = sum_j drows[dest[t, j]], in fp32, rounded once."""
    code = _need_float(drows, "drows")
    T, k, _ = _need_plan(plan, drows)
    _need_rows(drows, "drows", T * k)
    H = drows.shape[1]
    dx = _allocator(drows)((T, H), (H, 1), drows.dtype)
    _call("moe_dispatch_bwd", drows, drows.data_ptr(), plan.dest.data_ptr(), dx.data_ptr(), T, k, H, code)
    return dx


def moe_combine_fwd(y: torch.Tensor, weight: torch.Tensor, plan: MoePlan) -> torch.Tensor:
    """out [tokens, hidden] = sum_j weight[t, j] y[dest[t, j]], in fp32, rounded
    once; slots without a row add nothing."""
    code = _need_float(y, "y")
    T, k, _ = _need_plan(plan, y)
    _need_rows(y, "y", T * k)
    _need_weight(weight, y, T, k)
    H = y.shape[1]
    out = _allocator(y)((T, H), (H, 1), y.dtype)
    _call("moe_combine_fwd", y, y.data_ptr(), weight.data_ptr(), plan.dest.data_ptr(), out.data_ptr(), T, k, H,
          code)
    return out


def _need_weight(weight: torch.Tensor, like: torch.Tensor, T: int, k: int) -> None:
    _check(weight, "weight", torch.float32, 2, like)
    if tuple(weight.shape) != (T, k):
        raise ValueError(f"weight must have shape {(T, k)}")


def moe_combine_bwd(dout: torch.Tensor, y: torch.Tensor, weight: torch.Tensor,
                    plan: MoePlan) -> Tuple[torch.Tensor, torch.Tensor]:
    """(dy, dweight): dy[dest[t, j]] = weight[t, j] dout[t] (rows no slot has:
    zero) and dweight[t, j] = <dout[t], y[dest[t, j]]> in fp32."""
    code = _need_float(y, "y")
    T, k, E = _need_plan(plan, y)
    _need_rows(y, "y", T * k)
    _need_weight(weight, y, T, k)
    H = y.shape[1]
    _check(dout, "dout", y.dtype, 2, y)
    if tuple(dout.shape) != (T, H):
        raise ValueError(f"dout must have shape {(T, H)}")
    new = _allocator(y)
    dy = new((T * k, H), (H, 1), y.dtype)
    dweight = new((T, k), (k, 1), torch.float32)
    _call("moe_combine_bwd", y, dout.data_ptr(), y.data_ptr(), weight.data_ptr(), plan.dest.data_ptr(),
          plan.offs.data_ptr(), dy.data_ptr(), dweight.data_ptr(), T, k, E, H, code)
    return dy, dweight


class _Dispatch(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, offs, dest):
        ctx.save_for_backward(offs, dest)
        return moe_dispatch_fwd(x, MoePlan(offs, dest))

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, drows):
        return moe_dispatch_bwd(drows.contiguous(), MoePlan(*ctx.saved_tensors)), None, None


class _Combine(torch.autograd.Function):
    @staticmethod
    def forward(ctx, y, weight, offs, dest):
        ctx.save_for_backward(y, weight, offs, dest)
        return moe_combine_fwd(y, weight, MoePlan(offs, dest))

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
