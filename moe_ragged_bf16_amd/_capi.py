"""ctypes loader of the gfx950 HIP library (``libmoe_ragged_bf16.so``).

Argument marshalling only.  The library is required: if it is missing or fails
to load, every call raises; there is no fallback implementation.
"""
from __future__ import annotations

import ctypes
import os
import threading
from typing import Optional

from torch._C import _is_tracing

from . import build as _build

MDG_OK, MDG_EINVAL, MDG_EUNSUPPORTED, MDG_EOVERLAP, MDG_EWORKSPACE, MDG_EHIP, MDG_ENOMEM = range(7)
MDG_BF16, MDG_FP32, MDG_E4M3 = range(3)
MDG_SILU, MDG_GELU_TANH = range(2)

EXPORTED = (
    "grouped_det_gemm_abi_version",
    "grouped_det_gemm_status_string",
    "grouped_det_gemm_fwd",
    "grouped_det_gemm_dgrad",
    "grouped_det_gemm_fwd_noalloc",
    "grouped_det_gemm_fwd_workspace_bytes",
    "grouped_det_gemm_dgrad_workspace_bytes",
    "grouped_det_gemm_wgrad",
    "grouped_det_gemm_wgrad_workspace_bytes",
    "grouped_det_gemm_wgrad_chunk_rows",
    "grouped_det_gemm_zero_pad_rows",
    "grouped_det_gemm_prepare_fwd",
    "grouped_det_gemm_prepare_dgrad",
    "grouped_det_gemm_prepare_wgrad",
    "grouped_det_gemm_launch",
    "grouped_det_gemm_launch_info",
    "grouped_det_gemm_launch_free",
    "moe_route_fwd",
    "moe_route_fwd_workspace_bytes",
    "moe_route_bwd",
    "moe_plan",
    "moe_plan_workspace_bytes",
    "moe_dispatch_fwd",
    "moe_dispatch_bwd",
    "moe_combine_fwd",
    "moe_combine_bwd",
    "grouped_fp8_quantize_rows",
    "grouped_fp8_quantize_weight",
    "grouped_fp8_gemm_fwd",
    "grouped_fp8_gemm_fwd_workspace_bytes",
    "grouped_gated_gemm_fwd",
    "grouped_gated_gemm_fwd_workspace_bytes",
    "grouped_gated_gemm_dgrad",
    "grouped_gated_gemm_dgrad_workspace_bytes",
    "block_norm_fwd",
    "block_norm_bwd",
    "block_norm_bwd_workspace_bytes",
    "grad_norm",
    "grad_norm_workspace_bytes",
    "grad_clip",
)


class LaunchInfo(ctypes.Structure):
    """mdg_launch_info of the C header."""
    _fields_ = [("op", ctypes.c_int32), ("device", ctypes.c_int32), ("kernels", ctypes.c_int32),
                ("gemm_grid", ctypes.c_int32), ("dw_dtype", ctypes.c_int32), ("accumulate", ctypes.c_int32),
                ("chunk_rows", ctypes.c_int32), ("tail_slots", ctypes.c_int32),
                ("workspace_bytes", ctypes.c_int64)]


class Gradient(ctypes.Structure):
    """mdg_gradient of the C header."""
    _fields_ = [("data", ctypes.c_void_p), ("out", ctypes.c_void_p), ("elements", ctypes.c_int64),
                ("dtype", ctypes.c_int32), ("reserved", ctypes.c_int32)]


_lock = threading.Lock()
_lib = None


class MdgError(RuntimeError):
    """A non-OK status returned by the C ABI."""

    def __init__(self, entry: str, status: int, message: str):
        super().__init__(f"{entry}: status {status}: {message}")
        self.entry = entry
        self.status = status


def load_library(path: Optional[str] = None) -> ctypes.CDLL:
    """Load (once) and return the library, with argument types declared.  It is
    required: a missing or unloadable library raises (no fallback exists)."""
    global _lib
    with _lock:
        if _lib is not None:
            return _lib
        path = path or _build.LIB_PATH
        if not os.path.exists(path):
            raise ImportError(
                f"{path} is missing: build the HIP library first "
                "(python -m moe_ragged_bf16_amd.build)")
        lib = ctypes.CDLL(path)
        i32, i64, vp, sz = ctypes.c_int32, ctypes.c_int64, ctypes.c_void_p, ctypes.c_size_t
        lib.grouped_det_gemm_abi_version.restype = ctypes.c_int
        lib.grouped_det_gemm_abi_version.argtypes = []
        lib.grouped_det_gemm_status_string.restype = ctypes.c_char_p
        lib.grouped_det_gemm_status_string.argtypes = [ctypes.c_int]
        for name in ("grouped_det_gemm_fwd", "grouped_det_gemm_dgrad"):
            f = getattr(lib, name)
            f.restype = ctypes.c_int
            f.argtypes = [vp, vp, vp, vp, i64, i64, i64, i32, vp, sz, vp]
        lib.grouped_det_gemm_fwd_noalloc.restype = ctypes.c_int
        lib.grouped_det_gemm_fwd_noalloc.argtypes = [vp, vp, vp, vp, i64, i64, i64, i32, vp]
        for name in ("grouped_det_gemm_fwd_workspace_bytes", "grouped_det_gemm_dgrad_workspace_bytes"):
            f = getattr(lib, name)
            f.restype = sz
            f.argtypes = [i64, i64, i64, i32]
        lib.grouped_det_gemm_wgrad.restype = ctypes.c_int
        lib.grouped_det_gemm_wgrad.argtypes = [vp, vp, vp, vp, ctypes.c_int, ctypes.c_int,
                                               i64, i64, i64, i32, vp, sz, vp]
        lib.grouped_det_gemm_wgrad_workspace_bytes.restype = sz
        lib.grouped_det_gemm_wgrad_workspace_bytes.argtypes = [i64, i64, i64, i32]
        lib.grouped_det_gemm_wgrad_chunk_rows.restype = i64
        lib.grouped_det_gemm_wgrad_chunk_rows.argtypes = [i64, i64, i64, i32]
        lib.grouped_det_gemm_zero_pad_rows.restype = ctypes.c_int
        lib.grouped_det_gemm_zero_pad_rows.argtypes = [vp, vp, i64, i64, i32, vp]
        pp = ctypes.POINTER(vp)
        for name in ("grouped_det_gemm_prepare_fwd", "grouped_det_gemm_prepare_dgrad"):
            f = getattr(lib, name)
            f.restype = ctypes.c_int
            f.argtypes = [vp, vp, vp, vp, i64, i64, i64, i32, vp, sz, pp]
        lib.grouped_det_gemm_prepare_wgrad.restype = ctypes.c_int
        lib.grouped_det_gemm_prepare_wgrad.argtypes = [vp, vp, vp, vp, ctypes.c_int, ctypes.c_int,
                                                       i64, i64, i64, i32, vp, sz, pp]
        lib.grouped_det_gemm_launch.restype = ctypes.c_int
        lib.grouped_det_gemm_launch.argtypes = [vp, vp]
        lib.grouped_det_gemm_launch_info.restype = ctypes.c_int
        lib.grouped_det_gemm_launch_info.argtypes = [vp, ctypes.POINTER(LaunchInfo)]
        lib.grouped_det_gemm_launch_free.restype = None
        lib.grouped_det_gemm_launch_free.argtypes = [vp]
        st, f32 = ctypes.c_int, ctypes.c_float
        for name, res, args in (
                ("moe_route_fwd_workspace_bytes", sz, [i64, i32]),
                ("moe_route_fwd", st, [vp, st, vp, vp, vp, vp, vp, vp, i64, i32, i32, st, vp, sz, vp]),
                ("moe_route_bwd", st, [vp, st, vp, vp, vp, vp, vp, vp, i64, i32, i32, st, vp]),
                ("moe_plan_workspace_bytes", sz, [i64, i32, i32]),
                ("moe_plan", st, [vp, vp, vp, i64, i32, i32, vp, sz, vp]),
                ("moe_dispatch_fwd", st, [vp, vp, vp, vp, i64, i32, i32, i64, st, vp]),
                ("moe_dispatch_bwd", st, [vp, vp, vp, i64, i32, i64, st, vp]),
                ("moe_combine_fwd", st, [vp, vp, vp, vp, i64, i32, i64, st, vp]),
                ("moe_combine_bwd", st, [vp, vp, vp, vp, vp, vp, vp, i64, i32, i32, i64, st, vp]),
                ("grouped_fp8_quantize_rows", st, [vp, st, vp, vp, i64, i64, vp]),
                ("grouped_fp8_quantize_weight", st, [vp, st, vp, vp, vp, vp, i32, i64, i64, vp]),
                ("grouped_fp8_gemm_fwd_workspace_bytes", sz, [i64, i64, i64, i32, st]),
                ("grouped_fp8_gemm_fwd", st, [vp, st, vp, vp, vp, vp, vp, i64, i64, i64, i32, vp, sz, vp]),
                ("grouped_gated_gemm_fwd_workspace_bytes", sz, [i64, i64, i64, i32]),
                ("grouped_gated_gemm_fwd", st, [vp, vp, vp, vp, vp, st, i64, i64, i64, i32, vp, sz, vp]),
                ("grouped_gated_gemm_dgrad_workspace_bytes", sz, [i64, i64, i64, i32]),
                ("grouped_gated_gemm_dgrad", st, [vp, vp, vp, vp, vp, st, i64, i64, i64, i32, vp, sz, vp]),
                ("block_norm_fwd", st, [vp] * 9 + [i64, i64, st, st, f32, f32, vp]),
                ("block_norm_bwd_workspace_bytes", sz, [i64, i64]),
                ("block_norm_bwd", st, [vp] * 14 + [i64, i64, st, st, f32, vp, sz, vp]),
                ("grad_norm_workspace_bytes", sz, [i64]),
                ("grad_norm", st, [ctypes.POINTER(Gradient), i64, vp, vp, sz, vp]),
                ("grad_clip", st, [ctypes.POINTER(Gradient), i64, f32, vp, vp, vp, sz, vp])):
            f = getattr(lib, name)
            f.restype, f.argtypes = res, args
        _lib = lib
        return lib


def status_string(status: int) -> str:
    return load_library().grouped_det_gemm_status_string(status).decode()


def check(entry: str, status: int) -> None:
    if status != MDG_OK:
        raise MdgError(entry, status, status_string(status))


def refuse_tracing(call: str) -> None:
    """Raises under torch.jit.trace: it would record only the allocation of the
    outputs, not the library's call that fills them."""
    if _is_tracing():
        raise NotImplementedError(f"{call} cannot be traced by torch.jit.trace")


class _Native:
    """The calls of binding.cpp (``native.plan(idx, num_experts)``, ...), bound
    at the first use to the library's entries."""

    def __getattr__(self, name: str):
        import torch
        try:
            from . import _binding
        except ImportError as e:
            raise ImportError(f"{_build.BINDING_PATH} is missing or does not load ({e}): build it first "
                              "(python -m moe_ragged_bf16_amd.build)") from e
        lib = load_library()
        _binding.setup({n: ctypes.cast(getattr(lib, n), ctypes.c_void_p).value for n in _binding.entries()},
                       torch._C._cuda_getCurrentRawStream, check)
        self.__dict__.update({n: f for n, f in vars(_binding).items() if callable(f)})
        return self.__dict__[name]


native = _Native()
