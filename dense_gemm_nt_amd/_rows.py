"""ctypes binding of the C ABI in include/gemm_rows.h (argument marshalling only)."""
from __future__ import annotations

import ctypes
import os

from ._lib import PKG, GemmEpilogue

LIB_PATH = os.path.join(PKG, "libgemm_rows.so")

GEMM_TAIL_KEEP, GEMM_TAIL_ZERO = 0, 1

# Every symbol include/gemm_rows.h declares.
EXPORTS = ("gemm_lora_workspace", "gemm_run_lora", "gemm_lora_backward_workspace",
           "gemm_run_lora_backward", "gemm_route_workspace", "gemm_run_route",
           "gemm_run_route_backward", "gemm_run_routed", "gemm_run_routed_wgrad")


class GemmAdapters(ctypes.Structure):
    _fields_ = [("A", ctypes.c_void_p), ("B", ctypes.c_void_p), ("scale", ctypes.c_void_p),
                ("ids", ctypes.c_void_p), ("num_adapters", ctypes.c_int64),
                ("rank", ctypes.c_int64), ("a_stride", ctypes.c_int64), ("a_ld", ctypes.c_int64),
                ("b_stride", ctypes.c_int64), ("b_ld", ctypes.c_int64)]


class GemmRouting(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("ids", "weights", "counts", "offsets", "order",
                                               "tokens", "loss")]


_lib = None


def lib():
    """The loaded HIP library; raises if it has not been built (there is no fallback)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise RuntimeError("libgemm_rows.so is not built; run `python -m dense_gemm_nt_amd.build` "
                           "or __graft_entry__.build() first")
    import torch  # noqa: F401  (first, for the HIP runtime that it carries)
    L = ctypes.CDLL(LIB_PATH)
    vp, i64, ci = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int
    out64 = ctypes.POINTER(i64)
    ad, epi, rt = ctypes.POINTER(GemmAdapters), ctypes.POINTER(GemmEpilogue), ctypes.POINTER(GemmRouting)
    L.gemm_lora_workspace.argtypes = [i64] * 5 + [out64]
    L.gemm_run_lora.argtypes = [vp] * 3 + [i64] * 6 + [ci] * 2 + [ad, epi, vp, i64, vp]
    L.gemm_lora_backward_workspace.argtypes = [i64] * 5 + [out64]
    L.gemm_run_lora_backward.argtypes = [vp] * 6 + [i64] * 7 + [ci] * 3 + [ad, vp, i64, vp]
    L.gemm_route_workspace.argtypes = [i64] * 3 + [out64]
    L.gemm_run_route.argtypes = [vp, vp] + [i64] * 4 + [ci] * 2 + [rt, vp, i64, vp]
    L.gemm_run_route_backward.argtypes = [vp, rt, vp, vp, vp] + [i64] * 5 + [ci] * 2 + [vp]
    L.gemm_run_routed.argtypes = [vp] * 4 + [i64] * 8 + [ci] * 4 + [vp]
    L.gemm_run_routed_wgrad.argtypes = [vp] * 4 + [i64] * 6 + [ci] * 2 + [vp]
    for name in EXPORTS:
        getattr(L, name).restype = ci
    _lib = L
    return L


def workspace_bytes(fn, *sizes):
    """(status, bytes) of one of the *_workspace functions."""
    n = ctypes.c_int64()
    return getattr(lib(), fn)(*sizes, ctypes.byref(n)), n.value
