"""The products of a feed-forward layer (include/gemm_layer.h) on CUDA tensors:

- the gated block act(x Wg^T) * (x Wu^T) and its gradients: ``gemm_gated``,
  ``gemm_gated_backward``;
- the product in 8-bit integers with a scale for each token and output channel:
  ``quantize_int8``, ``gemm_int8``;
- the orthogonalized update of a weight (Newton-Schulz products): ``orthogonalize``.

Every call runs on the tensors' device, on its current stream, with workspaces and
results from torch's allocator, so calls on several streams do not share any
memory, and a captured call (``torch.cuda.graph``) replays with what its input
tensors then hold.
"""
from __future__ import annotations

import ctypes
import functools

from . import _layer, _lib
from .rows import _code, _index, _matrix, _on, _out, _ptr, _vector


# (a function of the sizes only; calls repeat them)
@functools.lru_cache(maxsize=256)
def _workspace_bytes(fn, *sizes):
    st, n = _layer.workspace_bytes(fn, *sizes)
    if st:
        _lib.check(st, "%s%s" % (fn, sizes))
    return n


def _span(t, unit):
    """(first byte, bytes from there to the last one's end, bytes of a row, from row to row or 0 with
    one row) of a matrix or vector of unit stride."""
    rows, row = (t.shape[0], t.shape[1] * unit) if t.dim() == 2 else (1, t.numel() * unit)
    step = t.stride(0) * unit if rows > 1 else 0
    return t.data_ptr(), (rows - 1) * step + row if rows and row else 0, row, step


def _apart(out, **operands):
    """Refuses an `out` that shares memory with an operand, which blocks still read when others
    store.  (Column ranges of one buffer's rows are apart.)"""
    at, size, row, step = _span(out, out.element_size())
    for name, t in operands.items():
        if t is None:
            continue
        at2, size2, row2, step2 = _span(t, t.element_size())
        if not size or not size2 or at + size <= at2 or at2 + size2 <= at:
            continue
        every = step or step2
        if every and (step2 or step) == every and (at2 - at) % every >= row and (at - at2) % every >= row2:
            continue
        raise ValueError("out overlaps %s" % name)


def _gate(activation):
    code = _layer.GATES.get(activation)
    if code is None:
        raise ValueError("activation must be one of %s, got %r" % (sorted(_layer.GATES), activation))
    return code


def _block(x, Wg, Wu):
    """(M, F, K, device index) of a gated block's checked operands."""
    if x.dim() != 2 or Wg.dim() != 2 or Wu.dim() != 2:
        raise ValueError("x, Wg and Wu must be 2-D")
    M, K = x.shape
    F = Wg.shape[0]
    if Wg.dtype != x.dtype or Wu.dtype != x.dtype:
        raise TypeError("x, Wg and Wu must share a dtype")
    index = _index(x)
    if not Wg.get_device() == Wu.get_device() == index:
        _on(index, Wg=Wg, Wu=Wu)
    return M, F, K, index


def gemm_gated(x, Wg, Wu, activation="silu", out=None, out_dtype=None):
    """h = act(x Wg^T) * (x Wu^T) for x [M, K] and Wg, Wu [F, K] (bfloat16 or float16, unit
    stride along K): [M, F] of out_dtype (default: x's), activation "silu", "gelu" (the
    exact form) or "relu".  Both sums are FP32 and h is rounded once.  K a multiple
    of 8."""
    import torch
    M, F, K, index = _block(x, Wg, Wu)
    if torch._C._cuda_getDevice() != index:
        with torch.cuda.device(index):
            return gemm_gated(x, Wg, Wu, activation, out, out_dtype)
    act = _gate(activation)
    ldx, ldg, ldu = _matrix("x", x, M, K), _matrix("Wg", Wg, F, K), _matrix("Wu", Wu, F, K)
    if out is None:
        out = torch.empty((M, F), dtype=out_dtype or x.dtype, device=x.device)
        ldh = F
    else:
        ldh = _matrix("out", _out("out", out, (M, F), x.device), M, F)
        _apart(out, x=x, Wg=Wg, Wu=Wu)
    n = _workspace_bytes("gemm_gated_workspace", M, F, K)
    ws = torch.empty(n, dtype=torch.uint8, device=x.device) if n else None
    st = _layer.lib().gemm_run_gated(
        x.data_ptr(), Wg.data_ptr(), Wu.data_ptr(), out.data_ptr(), M, F, K, ldx, ldg, ldu, ldh, _code(x.dtype),
        _code(out.dtype), act, _ptr(ws), n, torch._C._cuda_getCurrentRawStream(index))
    if st:
        _lib.check(st, "gemm_gated(M=%d, F=%d, K=%d)" % (M, F, K))
    return out


def gemm_gated_backward(dh, x, Wg, Wu, activation="silu", grad_dtype=None, dx_dtype=None, need_dx=True,
                        need_weights=True):
    """(dx, dWg, dWu) of gemm_gated for dh [M, F]: dx [M, K] of dx_dtype and dWg, dWu [F, K]
    of grad_dtype (defaults: x's).  Only the operands are needed: the two sums are
    computed again.  The gradients of the two sums are rounded to x's type once, so
    FP32 results hold no more than that; float16's are held in units of each row of dh for
    dx and of each column for the weights' gradients, so that neither large or small values of
    dh nor large sums end its range (include/gemm_layer.h).  An infinity or NaN in dh reaches
    its row of dx and its column's rows of dWg and dWu.  need_dx or need_weights False: that
    part is not computed, and None."""
    import torch
    M, F, K, index = _block(x, Wg, Wu)
    if dh.dim() != 2:
        raise ValueError("dh must be 2-D")
    if dh.dtype != x.dtype:
        raise TypeError("dh and x must share a dtype")
    if dh.get_device() != index:
        _on(index, dh=dh)
    if torch._C._cuda_getDevice() != index:
        with torch.cuda.device(index):
            return gemm_gated_backward(dh, x, Wg, Wu, activation, grad_dtype, dx_dtype, need_dx, need_weights)
    act = _gate(activation)
    ldx, ldg, ldu = _matrix("x", x, M, K), _matrix("Wg", Wg, F, K), _matrix("Wu", Wu, F, K)
    lddh = _matrix("dh", dh, M, F)
    dt, dev = x.dtype, x.device
    gdt, xdt = grad_dtype or dt, dx_dtype or dt
    dx = torch.empty((M, K), dtype=xdt, device=dev) if need_dx else None
    dWg = torch.empty((F, K), dtype=gdt, device=dev) if need_weights else None
    dWu = torch.empty((F, K), dtype=gdt, device=dev) if need_weights else None
    n = _workspace_bytes("gemm_gated_backward_workspace_of", M, F, K, _code(dt))
    ws = torch.empty(n, dtype=torch.uint8, device=dev)
    st = _layer.lib().gemm_run_gated_backward(
        dh.data_ptr(), x.data_ptr(), Wg.data_ptr(), Wu.data_ptr(), _ptr(dx) or None, _ptr(dWg) or None,
        _ptr(dWu) or None, M, F, K, lddh, ldx, ldg, ldu, K, _code(dt), _code(xdt), _code(gdt), act, ws.data_ptr(),
        n, torch._C._cuda_getCurrentRawStream(index))
    if st:
        _lib.check(st, "gemm_gated_backward(M=%d, F=%d, K=%d)" % (M, F, K))
    return dx, dWg, dWu


def quantize_int8(x):
    """(codes, scale) of the rows of x [M, K] (bfloat16, float16 or float32): scale float32 [M],
    a row's largest magnitude over 127, and codes int8 [M, K], x / scale to the nearest
    integer (even at a tie).  A row of zeros has scale 0, one with an infinity or NaN scale
    NaN; both have codes 0."""
    import torch
    if x.dim() != 2:
        raise ValueError("x must be 2-D")
    M, K = x.shape
    index = _index(x)
    if torch._C._cuda_getDevice() != index:
        with torch.cuda.device(index):
            return quantize_int8(x)
    ldx = _matrix("x", x, M, K)
    codes = torch.empty((M, K), dtype=torch.int8, device=x.device)
    scale = torch.empty(M, dtype=torch.float32, device=x.device)
    st = _layer.lib().gemm_run_quantize_int8(x.data_ptr(), codes.data_ptr(), scale.data_ptr(), M, K, ldx, K,
                                             _code(x.dtype), torch._C._cuda_getCurrentRawStream(index))
    if st:
        _lib.check(st, "quantize_int8(M=%d, K=%d)" % (M, K))
    return codes, scale


def _scale(name, s, n, torch):
    if s.dtype != torch.float32 or not s.is_contiguous() or (s.numel() != 1 and s.shape != (n,)):
        raise ValueError("%s must be one float32 value or a contiguous vector of %d" % (name, n))
    return s.numel()


def gemm_int8(A, B, scale_a, scale_b, out=None, out_dtype=None, alpha=1.0, beta=0.0, bias=None,
              bias_along="n", activation="none"):
    """C = act(alpha * y + beta * C_old + bias), y[m, n] = scale_a[m] scale_b[n] (A[m] . B[n]), for
    int8 A [M, K] (quantize_int8's codes) and B [N, K], scales float32 [M] and [N] (or one
    value each): [M, N] of out_dtype (default bfloat16).  The integer sums are exact, and taken
    to FP32 once.  K a multiple of 16 below 2^17; the epilogue as gemm_nt's."""
    import torch
    if A.dim() != 2 or B.dim() != 2 or A.shape[1] != B.shape[1]:
        raise ValueError("A must be [M, K] and B [N, K], got %s and %s" % (tuple(A.shape), tuple(B.shape)))
    if A.dtype != torch.int8 or B.dtype != torch.int8:
        raise TypeError("A and B must be int8")
    M, K = A.shape
    N = B.shape[0]
    index = _index(A)
    if torch._C._cuda_getDevice() != index:
        with torch.cuda.device(index):
            return gemm_int8(A, B, scale_a, scale_b, out, out_dtype, alpha, beta, bias, bias_along, activation)
    if not B.get_device() == scale_a.get_device() == scale_b.get_device() == index or bias is not None:
        _on(index, B=B, scale_a=scale_a, scale_b=scale_b, bias=bias)
    lda, ldb = _matrix("A", A, M, K), _matrix("B", B, N, K)
    na, nb = _scale("scale_a", scale_a, M, torch), _scale("scale_b", scale_b, N, torch)
    if out is None:
        if beta != 0.0:
            raise ValueError("beta != 0 reads the prior C: pass it as `out`")
        out = torch.empty((M, N), dtype=out_dtype or torch.bfloat16, device=A.device)
        ldc = N
    else:
        ldc = _matrix("out", _out("out", out, (M, N), A.device), M, N)
        _apart(out, A=A, B=B, scale_a=scale_a, scale_b=scale_b, bias=bias)
    epi = None
    if not (alpha == 1.0 and beta == 0.0 and bias is None and activation == "none"):
        if bias is not None:
            _vector("bias", bias, N if bias_along == "n" else M, torch.float32)
        epi = _lib.epilogue(alpha, beta, bias.data_ptr() if bias is not None else 0,
                            bias_along if bias is not None else "none", activation)
    n = _workspace_bytes("gemm_int8_workspace", M, N, K)
    ws = torch.empty(n, dtype=torch.uint8, device=A.device) if n else None
    st = _layer.lib().gemm_run_int8(
        A.data_ptr(), B.data_ptr(), out.data_ptr(), M, N, K, lda, ldb, ldc, _code(out.dtype), scale_a.data_ptr(),
        na, scale_b.data_ptr(), nb, ctypes.byref(epi) if epi is not None else None, _ptr(ws), n,
        torch._C._cuda_getCurrentRawStream(index))
    if st:
        _lib.check(st, "gemm_int8(M=%d, N=%d, K=%d)" % (M, N, K))
    return out


@functools.lru_cache(maxsize=16)
def _floats(values):
    return (ctypes.c_float * len(values))(*values)


def _coefficients(coefficients, steps):
    """The steps' triples as a host array."""
    flat = tuple(coefficients)
    if len(flat) == 3 and not any(map(_is_triple, flat)):
        flat = flat * steps
    elif len(flat) == steps and all(map(_is_triple, flat)):
        flat = tuple(v for t in flat for v in t)
    else:
        raise ValueError("coefficients must be (a, b, c) or %d such triples" % steps)
    # (numbers, not what holds them: a tensor's element may change between calls)
    return _floats(tuple(map(float, flat)))


def _is_triple(t):
    return getattr(t, "shape", None) == (3,) or isinstance(t, (tuple, list)) and len(t) == 3


def orthogonalize(G, steps=5, coefficients=(3.4445, -4.7750, 2.0315), eps=1e-7, out=None, out_dtype=None):
    """The orthogonalized update of G [m, n] or of a stack [B, m, n] (bfloat16, float16 or
    float32, unit stride along the last axis): X = G / (||G|| + eps), then `steps` times
    X = a X + b (X X^T) X + c (X X^T)^2 X, which takes every singular value s to
    a s + b s^3 + c s^5 and leaves the singular vectors.  `coefficients` is (a, b, c), or
    one such triple a step.  Of out_dtype (default bfloat16).  X is kept to 22 bits and
    multiplied in float16: about 1e-3 of the exact iteration off (relative) where the
    coefficients keep the singular values below 2.  `out` may be G itself."""
    import torch
    if G.dim() not in (2, 3):
        raise ValueError("G must be [m, n] or [B, m, n]")
    index = _index(G)
    if torch._C._cuda_getDevice() != index:
        with torch.cuda.device(index):
            return orthogonalize(G, steps, coefficients, eps, out, out_dtype)
    steps = int(steps)
    if steps < 0:
        raise ValueError("steps must not be negative")
    values = _coefficients(coefficients, steps)
    B = G.shape[0] if G.dim() == 3 else 1
    m, n = G.shape[-2:]

    def strides(name, t):
        if B and m and n and t.stride(-1) != 1 and n > 1:
            raise ValueError("%s needs unit stride along its last axis" % name)
        return t.stride(-2) if m > 1 else n, t.stride(0) if G.dim() == 3 and B > 1 else 0
    ldg, g_step = strides("G", G)
    if out is None:
        out = torch.empty(G.shape, dtype=out_dtype or torch.bfloat16, device=G.device)
    else:
        _out("out", out, G.shape, G.device)
    ldu, u_step = strides("out", out)
    if B > 1 and m and n and u_step < (m - 1) * ldu + n and not (u_step >= n and ldu >= (B - 1) * u_step + n):
        raise ValueError("out's matrices overlap")
    ws_bytes = _workspace_bytes("gemm_orthogonalize_workspace", B, m, n)
    ws = torch.empty(ws_bytes, dtype=torch.uint8, device=G.device) if ws_bytes else None
    st = _layer.lib().gemm_run_orthogonalize(
        G.data_ptr(), out.data_ptr(), B, m, n, ldg, ldu, g_step, u_step, _code(G.dtype), _code(out.dtype), steps,
        values, eps, _ptr(ws), ws_bytes, torch._C._cuda_getCurrentRawStream(index))
    if st:
        _lib.check(st, "orthogonalize(B=%d, m=%d, n=%d)" % (B, m, n))
    return out
