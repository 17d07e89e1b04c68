"""The norm of all gradients, and the gradients clipped by it.

    norm = clip_grads([p.main_grad for p in parameters], max_norm=1.0)

    norm = grad_norm(grads)                       # where a norm spans several processes:
    total = ...                                   # all-reduce norm^2, take the root,
    clip_grads(grads, 1.0, norm=total)            # and scale by it

norm = sqrt(sum of g^2 over all tensors), squares and sums in 64 bits; every
gradient is multiplied by min(1, max_norm / (norm + 1e-6)), as
``torch.nn.utils.clip_grad_norm_`` does, except that a norm which is not finite
leaves the gradients as they are.  Nothing waits for the device: the norm stays
there.  The sums' order is fixed by the tensors' sizes, so results repeat bit for
bit.  A captured call works on the tensors it was captured with.
"""
from __future__ import annotations

from typing import Optional, Sequence

import torch

from ._capi import native, refuse_tracing

__all__ = ["grad_norm", "clip_grads"]


def grad_norm(grads: Sequence[torch.Tensor]) -> torch.Tensor:
    """The norm of the tensors (bf16 or fp32, of any shape, one at least, on one
    device, without gaps or overlaps between their elements), an fp32 scalar on
    the device."""
    refuse_tracing("grad_norm")
    return native.grad_norm(grads)


def clip_grads(grads: Sequence[torch.Tensor], max_norm: float, *, norm: Optional[torch.Tensor] = None,
               out: Optional[Sequence[torch.Tensor]] = None) -> torch.Tensor:
    """Clips the gradients (as ``grad_norm`` takes them) in place, or into ``out``:
    tensors of the same types, shapes and strides.  Returns their norm from
    before, an fp32 scalar on the device.  ``norm``: an fp32 scalar on the device
    to clip by in place of the gradients' own norm; it is returned.  Tensors that
    are written may not share memory with each other or with other gradients."""
    refuse_tracing("clip_grads")
    return native.clip_grads(grads, max_norm, norm, out)
