"""The experts' gated feed-forward: both projections, the activation and their
product in one kernel, and the gradient through the down product in another.

    y = grouped_gated_ffn(rows, w_gate_up, w_down, offs)      # differentiable

    h = grouped_gated_gemm_fwd(rows, w_gate_up, offs).h       # serving: the first half,
    y = grouped_det_gemm_fwd(h, w_down, offs)                 # then the down product

For expert e: a = x W_gate^T, b = x W_up^T, h = act(a) b, y = h W_down^T, with
W_gate and W_up the first and the second half of w_gate_up[e]'s rows.  act is
``"silu"`` (a s(a), s the logistic function) or ``"gelu_tanh"`` (0.5 a (1 +
tanh(sqrt(2/pi) (a + 0.044715 a^3)))).  h is rounded once, from the fp32 sums a
and b.  For the gradient the forward keeps a and b in bf16 (``gate_up``) and h;
the backward takes act and its derivative at those bf16 values.

``grouped_gated_gemm_fwd`` and ``_dgrad`` record nothing for autograd.  All raise
NotImplementedError under ``torch.jit.trace``, which cannot see the library's
calls.  Sums repeat bit for bit in calls of the same sizes and offsets; in calls
of other sizes the same row can get different bits.
"""
from __future__ import annotations

from typing import NamedTuple, Optional

import torch

from . import _capi
from ._capi import native, refuse_tracing
from .autograd import _fused_main_grad, _fused_wgrad, _main_grad
from .ops import incoming_gradient

__all__ = ["GatedRows", "grouped_gated_gemm_fwd", "grouped_gated_gemm_dgrad", "grouped_gated_ffn",
           "gated_gemm_fwd_workspace_bytes", "gated_gemm_dgrad_workspace_bytes"]

_ACTIVATIONS = {"silu": _capi.MDG_SILU, "gelu_tanh": _capi.MDG_GELU_TANH}


class GatedRows(NamedTuple):
    h: torch.Tensor                          # [M, F] bf16
    gate_up: Optional[torch.Tensor] = None   # [M, 2 F] bf16: a and b, where kept


def _code(activation: str) -> int:
    try:
        return _ACTIVATIONS[activation]
    except (KeyError, TypeError):
        raise ValueError(f"activation must be one of {sorted(_ACTIVATIONS)}, got {activation!r}") from None


def gated_gemm_fwd_workspace_bytes(m_rows: int, f: int, k: int, num_groups: int) -> int:
    """Bytes of workspace of ``grouped_gated_gemm_fwd`` on the current device."""
    return int(_capi.load_library().grouped_gated_gemm_fwd_workspace_bytes(m_rows, f, k, num_groups))


def gated_gemm_dgrad_workspace_bytes(m_rows: int, n: int, f: int, num_groups: int) -> int:
    """Bytes of workspace of ``grouped_gated_gemm_dgrad`` on the current device."""
    return int(_capi.load_library().grouped_gated_gemm_dgrad_workspace_bytes(m_rows, n, f, num_groups))


def grouped_gated_gemm_fwd(x: torch.Tensor, w: torch.Tensor, offs: torch.Tensor, *, activation: str = "silu",
                           keep: bool = False, out: Optional[torch.Tensor] = None,
                           workspace: Optional[torch.Tensor] = None) -> GatedRows:
    """h [M, F] = act(X W_gate[e]^T) * (X W_up[e]^T) of each group's rows, bf16 x
    [M, K] and w [E, 2 F, K] (gate rows, then up rows; F and K multiples of 8; up to
    4,000,000 rows and 1024 experts).
    ``keep``: also gate_up [M, 2 F], both projections in bf16, for
    ``grouped_gated_gemm_dgrad``; h has the same bits either way.  offs as in
    ``grouped_det_gemm_fwd``; rows past offs[E-1] are not written.  ``out``: h's
    tensor; ``workspace`` (uint8, at least ``gated_gemm_fwd_workspace_bytes()``)
    is allocated per call when not given."""
    refuse_tracing("grouped_gated_gemm_fwd")
    return GatedRows(*native.gated_fwd(x, w, offs, _code(activation), keep, out, workspace))


def grouped_gated_gemm_dgrad(dy: torch.Tensor, w_down: torch.Tensor, gate_up: torch.Tensor, offs: torch.Tensor, *,
                             activation: str = "silu", out: Optional[torch.Tensor] = None,
                             workspace: Optional[torch.Tensor] = None) -> torch.Tensor:
    """dgate_up [M, 2 F]: the gradients of a and b for the gradient dy [M, N] of
    y = h W_down[e]^T, with w_down [E, N, F] and gate_up as the forward kept it.
    dh = dY W_down[e] stays in fp32 inside the call."""
    refuse_tracing("grouped_gated_gemm_dgrad")
    return native.gated_dgrad(dy, w_down, gate_up, offs, _code(activation), out, workspace)


class _GatedFfn(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, w, w_down, offs, code, fuse, record):
        need_x, need_w, need_down = (record and n for n in ctx.needs_input_grad[:3])
        through = need_x or need_w                     # (the gradients through the down product)
        y, h, gate_up = native.ffn_fwd(x, w, w_down, offs, code, through + 2 * need_down)
        if through or need_down:                       # what the wanted gradients read
            ctx.save_for_backward(x if need_w else None, w if need_x else None, w_down if through else None, offs, h,
                                  gate_up)
        ctx.code, ctx.fuse, ctx.experts = code, fuse, w.shape[0]
        # (the caller's weights themselves, whose main_grad the backward reads)
        ctx.w_objs = (w, w_down) if fuse else (None, None)
        return y

    @staticmethod
    def backward(ctx, dy):
        if torch.is_grad_enabled():
            raise NotImplementedError("grouped_gated_ffn has no double backward (create_graph=True)")
        x, w, w_down, offs, h, gate_up = ctx.saved_tensors
        dy = incoming_gradient(dy)
        need_x, need_w, need_down = ctx.needs_input_grad[:3]
        if not ctx.fuse:
            dx, dw, dw_down, _ = native.ffn_bwd(dy, w_down, gate_up, offs, ctx.code, x, w, h, ctx.experts,
                                                need_x + 2 * need_w + 4 * need_down)
            return dx, dw, dw_down, None, None, None, None
        read = (("the output gradient", dy), ("x", x), ("offs", offs), ("w", w), ("w_down", w_down), ("h", h),
                ("gate_up", gate_up))
        read = tuple((name, t) for name, t in read if t is not None)
        mgs = [_fused_main_grad(o, "grouped_gated_ffn", read) if need else None
               for o, need in zip(ctx.w_objs, (need_w, need_down))]
        dx, _, _, d = native.ffn_bwd(dy, w_down, gate_up, offs, ctx.code, x, w, h, ctx.experts, need_x + 8 * need_w)
        dw = _fused_wgrad(ctx.w_objs[0], mgs[0], d, x, offs) if need_w else None
        dw_down = _fused_wgrad(ctx.w_objs[1], mgs[1], dy, h, offs) if need_down else None
        return dx, dw, dw_down, None, None, None, None


@torch.compiler.disable
def _apply_eagerly(x, w, w_down, offs, code, fuse):
    # (the library's calls are opaque to torch.compile: out of its graphs)
    # (grad mode is off inside forward, and needs_input_grad does not follow it)
    return _GatedFfn.apply(x, w, w_down, offs, code, fuse, torch.is_grad_enabled())


def grouped_gated_ffn(x: torch.Tensor, w_gate_up: torch.Tensor, w_down: torch.Tensor, offs: torch.Tensor, *,
                      activation: str = "silu", fuse_wgrad_accumulation: bool = False) -> torch.Tensor:
    """Differentiable gated feed-forward of each group's rows: y [M, N] =
    (act(X W_gate[e]^T) * (X W_up[e]^T)) W_down[e]^T, bf16 x [M, K], w_gate_up
    [E, 2 F, K] and w_down [E, N, F] (K, F and N multiples of 8); rows past
    offs[E-1] are zero, and so is their gradient.

    The weights' gradients are in the weights' type, or, with
    ``fuse_wgrad_accumulation``, added into both weights' ``main_grad`` by the
    wgrad kernel's epilogue, by the rules of ``cake_grouped_det_mm``.  A call
    keeps what the gradients of the tensors that require one will read (w_down's h;
    x's and w_gate_up's gate_up and w_down; x's w_gate_up, w_gate_up's x), nothing
    without grad mode.  There is no double backward."""
    refuse_tracing("grouped_gated_ffn")
    if torch.compiler.is_compiling():
        raise NotImplementedError("grouped_gated_ffn cannot be compiled by torch.compile")
    if not isinstance(fuse_wgrad_accumulation, bool):
        raise ValueError(f"fuse_wgrad_accumulation must be a bool, got {type(fuse_wgrad_accumulation).__name__}")
    code = _code(activation)
    if fuse_wgrad_accumulation and torch.is_grad_enabled() and torch._C._current_autograd_node() is None:
        for w in (w_gate_up, w_down):
            if isinstance(w, torch.Tensor) and w.requires_grad:
                _main_grad(w, "forward", "grouped_gated_ffn")
    return _apply_eagerly(x, w_gate_up, w_down, offs, code, fuse_wgrad_accumulation)
