"""ctypes binding of the C ABI in include/gemm_layer.h (argument marshalling only)."""
from __future__ import annotations

import ctypes
import os

from ._lib import PKG, GemmEpilogue

LIB_PATH = os.path.join(PKG, "libgemm_layer.so")

GATES = {"relu": 1, "gelu": 2, "silu": 3}

# Every symbol include/gemm_layer.h declares.
EXPORTS = ("gemm_gated_workspace", "gemm_run_gated", "gemm_gated_backward_workspace",
           "gemm_gated_backward_workspace_of", "gemm_run_gated_backward", "gemm_run_quantize_int8",
           "gemm_int8_workspace", "gemm_run_int8", "gemm_orthogonalize_workspace",
           "gemm_run_orthogonalize")

_lib = None


def lib():
    """The loaded HIP library; raises if it has not been built (there is no fallback)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise RuntimeError("libgemm_layer.so is not built; run `python -m dense_gemm_nt_amd.build` "
                           "or __graft_entry__.build() first")
    import torch  # noqa: F401  (first, for the HIP runtime that it carries)
    L = ctypes.CDLL(LIB_PATH)
    vp, i64, ci = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int
    out64 = ctypes.POINTER(i64)
    L.gemm_gated_workspace.argtypes = [i64] * 3 + [out64]
    L.gemm_run_gated.argtypes = [vp] * 4 + [i64] * 7 + [ci] * 3 + [vp, i64, vp]
    L.gemm_gated_backward_workspace.argtypes = [i64] * 3 + [out64]
    L.gemm_gated_backward_workspace_of.argtypes = [i64] * 3 + [ci, out64]
    L.gemm_run_gated_backward.argtypes = [vp] * 7 + [i64] * 8 + [ci] * 4 + [vp, i64, vp]
    L.gemm_run_quantize_int8.argtypes = [vp] * 3 + [i64] * 4 + [ci, vp]
    L.gemm_int8_workspace.argtypes = [i64] * 3 + [out64]
    L.gemm_run_int8.argtypes = [vp] * 3 + [i64] * 6 + [ci, vp, i64, vp, i64, ctypes.POINTER(GemmEpilogue),
                                                       vp, i64, vp]
    L.gemm_orthogonalize_workspace.argtypes = [i64] * 3 + [out64]
    L.gemm_run_orthogonalize.argtypes = [vp] * 2 + [i64] * 7 + [ci] * 2 + [i64, ctypes.POINTER(ctypes.c_float),
                                                                          ctypes.c_double, vp, i64, vp]
    for name in EXPORTS:
        getattr(L, name).restype = ci
    _lib = L
    return L


def workspace_bytes(fn, *sizes):
    """(status, bytes) of one of the *_workspace functions."""
    n = ctypes.c_int64()
    return getattr(lib(), fn)(*sizes, ctypes.byref(n)), n.value
