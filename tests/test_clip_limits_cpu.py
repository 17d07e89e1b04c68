"""The largest gradient lists, without a GPU: every call here is refused before any
device access, whatever its pointers hold."""
import pytest

import moe_ragged_bf16_amd as mdg
from moe_ragged_bf16_amd._capi import MDG_EUNSUPPORTED, MDG_FP32, Gradient

P = [0x100000000 * i for i in range(1, 4)]
LARGEST = 2 ** 36                     # values of a tensor, 2^23 pieces of 32 KiB in fp32
WORKGROUPS = 1024                     # of a launch, at most


def pieces(n):
    """Gradients (aliases of one tensor: only read) of n pieces in all."""
    whole, rest = divmod(n, 2 ** 23)
    return [(P[0], P[0], LARGEST, MDG_FP32, 0)] * whole + [(P[0], P[0], rest * 8192, MDG_FP32, 0)] * (rest > 0)


@pytest.mark.parametrize("n", [2 ** 31 - WORKGROUPS, 2 ** 31 - WORKGROUPS // 2, 2 ** 31 - 1])
def test_a_walk_that_passes_32_bits_is_refused(n):
    """A workgroup walks pieces b, b + grid, ... in 32 bits: the count behind its last piece
    has to fit as well."""
    lib, rows = mdg.load_library(), pieces(n)
    table, need = (Gradient * len(rows))(*rows), lib.grad_norm_workspace_bytes(len(rows))
    assert lib.grad_norm(table, len(rows), P[1], P[2], need, None) == MDG_EUNSUPPORTED
    assert lib.grad_clip(table, len(rows), 1.0, None, P[1], P[2], need, None) == MDG_EUNSUPPORTED
