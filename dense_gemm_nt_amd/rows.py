"""Products whose weight depends on the row (include/gemm_rows.h) on CUDA tensors:

- a shared projection with low-rank adapters picked per row: ``gemm_lora``,
  ``gemm_lora_backward``;
- the top-k router with its balance loss and per-expert counts: ``route_topk``,
  ``route_topk_backward``;
- the experts' products over rows sorted by expert: ``gemm_routed``,
  ``gemm_routed_wgrad``.

What picks the weight stays on the device: no call reads it on the host.  Every
call runs on the tensors' device, on its current stream, with workspaces and
results from torch's allocator, so calls on several streams do not share any
memory, and a captured call (``torch.cuda.graph``) replays with what its input
tensors then hold.
"""
from __future__ import annotations

import collections
import ctypes
import functools

from . import _lib, _rows
from .api import _code as _code_of_name

Routing = collections.namedtuple("Routing", "ids weights counts offsets order tokens loss "
                                            "renormalize")
Routing.__doc__ = """What route_topk gives for T tokens, E experts, k choices (int32 but for
weights and loss): ids [T, k] (-1: none), weights [T, k] float32, counts [E],
offsets [E + 1], order [T * k] (the pairs t * k + j by expert, stable; those
without an expert last), tokens [1] (how many were routed), loss (float32
scalar), and the call's `renormalize`."""


@functools.lru_cache(maxsize=None)
def _code(dtype):
    return _code_of_name(dtype)


def _on(index, **tensors):
    for name, t in tensors.items():
        if t is not None and t.get_device() != index:
            raise ValueError("%s is on %s, expected cuda:%d" % (name, t.device, index))


# A small call's time is the host's, so the calls below ask torch for the current
# device and stream as plain integers (a third of a microsecond for both, where
# the stream object alone takes more than one), read what they check from the tensors
# directly, and make error messages only for errors.

def _index(t):
    """The device index of a CUDA tensor."""
    index = t.get_device()
    if index < 0:
        raise ValueError("expected CUDA tensors, got one on %s" % t.device)
    return index


def _matrix(name, X, rows, cols):
    """Leading dimension of a [rows, cols] tensor with unit stride along its columns.  A single
    row's stride is never used (and may be anything: the last token of a prompt is
    such a view), so that it is not held to the limits of one."""
    if X.shape != (rows, cols):
        raise ValueError("%s must be [%d, %d], got %s" % (name, rows, cols, tuple(X.shape)))
    ld, step = X.stride()
    if step != 1 and cols > 1 and rows > 0:
        raise ValueError("%s needs unit stride along its columns" % name)
    return ld if rows > 1 else cols


def _vector(name, v, n, dtype):
    if v.dtype != dtype or v.shape != (n,) or not v.is_contiguous():
        raise ValueError("%s must be a contiguous %s vector of %d values" % (name, dtype, n))


def _out(name, out, shape, dev):
    if out.shape != shape or out.device != dev:
        raise ValueError("%s must be %s on %s" % (name, list(shape), dev))
    return out


# (a function of the sizes only; calls repeat them)
@functools.lru_cache(maxsize=256)
def _workspace_bytes(fn, *sizes):
    st, n = _rows.workspace_bytes(fn, *sizes)
    if st:
        _lib.check(st, "%s%s" % (fn, sizes))
    return n


def _ptr(t):
    return t.data_ptr() if t is not None else None


def _adapters(A, B, ids, scale, M, N, K, dtype, index, torch):
    """A checked GemmAdapters of A [L, R, K], B [L, N, R], ids [M], scale [L]."""
    if A.dim() != 3 or B.shape != (A.shape[0], N, A.shape[1]) or A.shape[2] != K:
        raise ValueError("adapters must be A [L, R, %d] and B [L, %d, R], got %s and %s"
                         % (K, N, tuple(A.shape), tuple(B.shape)))
    L, R, _ = A.shape
    if A.dtype != dtype or B.dtype != dtype:
        raise TypeError("the adapters must have the operands' dtype %s" % dtype)
    if not A.get_device() == B.get_device() == ids.get_device() == scale.get_device() == index:
        _on(index, A=A, B=B, ids=ids, scale=scale)
    _vector("ids", ids, M, torch.int32)
    _vector("scale", scale, L, torch.float32)
    a_step, a_ld, a_unit = A.stride()
    b_step, b_ld, b_unit = B.stride()
    if (a_unit != 1 and K > 1 and A.numel()) or (b_unit != 1 and R > 1 and B.numel()):
        raise ValueError("A and B need unit stride along their last axis")
    if R <= 1:
        a_ld = K
    if N <= 1:
        b_ld = R
    if L <= 1:                         # a single adapter's stride is never used
        a_step = b_step = 0
    return _rows.GemmAdapters(A.data_ptr(), B.data_ptr(), scale.data_ptr(), ids.data_ptr(), L, R,
                              a_step, a_ld, b_step, b_ld)


def gemm_lora(x, W, A, B, ids, scale, out=None, out_dtype=None, alpha=1.0, beta=0.0, bias=None,
              bias_along="n", activation="none"):
    """y[m] = act(alpha (x[m] W^T + scale[a] (x[m] A[a]^T) B[a]^T) + beta y_old[m] + bias),
    a = ids[m], for x [M, K] and W [N, K] (bfloat16 or float16), A [L, R, K] and
    B [L, N, R] of their dtype, ids int32 [M] (outside 0 .. L - 1: no adapter)
    and scale float32 [L].  R a multiple of 8 up to 128, K a multiple of 8.  beta != 0
    needs `out` holding y_old; the epilogue as gemm_nt's."""
    import torch
    if x.dim() != 2 or W.dim() != 2:
        raise ValueError("x and W must be 2-D")
    M, K = x.shape
    N = W.shape[0]
    index = _index(x)
    if torch._C._cuda_getDevice() != index:
        with torch.cuda.device(index):
            return gemm_lora(x, W, A, B, ids, scale, out, out_dtype, alpha, beta, bias, bias_along,
                             activation)
    dt = x.dtype
    if W.dtype != dt:
        raise TypeError("x and W must share a dtype")
    if W.get_device() != index or bias is not None:
        _on(index, W=W, bias=bias)
    ldx, ldw = _matrix("x", x, M, K), _matrix("W", W, N, K)
    ad = _adapters(A, B, ids, scale, M, N, K, dt, index, torch)
    if out is None:
        if beta != 0.0:
            raise ValueError("beta != 0 reads the prior y: pass it as `out`")
        out = torch.empty((M, N), dtype=out_dtype or dt, device=x.device)
        ldy = N
    else:
        ldy = _matrix("out", _out("out", out, (M, N), x.device), M, N)
    epi = None
    if not (alpha == 1.0 and beta == 0.0 and bias is None and activation == "none"):
        if bias is not None:
            _vector("bias", bias, N if bias_along == "n" else M, torch.float32)
        epi = _lib.epilogue(alpha, beta, bias.data_ptr() if bias is not None else 0,
                            bias_along if bias is not None else "none", activation)
    L, R = A.shape[:2]
    n = _workspace_bytes("gemm_lora_workspace", M, N, K, L, R)
    ws = torch.empty(n, dtype=torch.uint8, device=x.device) if n else None
    st = _rows.lib().gemm_run_lora(
        x.data_ptr(), W.data_ptr(), out.data_ptr(), M, N, K, ldx, ldw, ldy, _code(dt), _code(out.dtype),
        ctypes.byref(ad), ctypes.byref(epi) if epi is not None else None, _ptr(ws), n,
        torch._C._cuda_getCurrentRawStream(index))
    if st:
        _lib.check(st, "gemm_lora(M=%d, N=%d, K=%d, L=%d, R=%d)" % (M, N, K, L, R))
    return out


def gemm_lora_backward(dy, x, W, A, B, ids, scale, grad_dtype=None, dx_dtype=None, need_dx=True,
                       need_adapters=True):
    """(dx, dA, dB) of gemm_lora without an epilogue, W frozen, for dy [M, N]: dx [M, K]
    of dx_dtype (default: x's), dA [L, R, K] and dB [L, N, R] of grad_dtype
    (default float32; zeros for adapters without a row).  need_dx or
    need_adapters False: that part is not computed, and None.  N and K
    multiples of 8, at most 1024 adapters."""
    import torch
    if dy.dim() != 2 or x.dim() != 2 or W.dim() != 2:
        raise ValueError("dy, x and W must be 2-D")
    M, K = x.shape
    N = W.shape[0]
    index, dev = _index(x), x.device
    if torch._C._cuda_getDevice() != index:
        with torch.cuda.device(index):
            return gemm_lora_backward(dy, x, W, A, B, ids, scale, grad_dtype, dx_dtype, need_dx,
                                      need_adapters)
    dt = x.dtype
    if W.dtype != dt or dy.dtype != dt:
        raise TypeError("dy, x and W must share a dtype")
    if not dy.get_device() == W.get_device() == index:
        _on(index, dy=dy, W=W)
    lddy, ldx, ldw = _matrix("dy", dy, M, N), _matrix("x", x, M, K), _matrix("W", W, N, K)
    ad = _adapters(A, B, ids, scale, M, N, K, dt, index, torch)
    L, R = A.shape[:2]
    gdt, xdt = grad_dtype or torch.float32, dx_dtype or dt
    dx = torch.empty((M, K), dtype=xdt, device=dev) if need_dx else None
    dA = torch.empty((L, R, K), dtype=gdt, device=dev) if need_adapters else None
    dB = torch.empty((L, N, R), dtype=gdt, device=dev) if need_adapters else None
    n = _workspace_bytes("gemm_lora_backward_workspace", M, N, K, L, R)
    ws = torch.empty(n, dtype=torch.uint8, device=dev) if n else None
    st = _rows.lib().gemm_run_lora_backward(
        dy.data_ptr(), x.data_ptr(), W.data_ptr(), _ptr(dx), _ptr(dA) or None, _ptr(dB) or None, M, N,
        K, lddy, ldx, ldw, K, _code(dt), _code(xdt), _code(gdt), ctypes.byref(ad), _ptr(ws), n,
        torch._C._cuda_getCurrentRawStream(index))
    if st:
        _lib.check(st, "gemm_lora_backward(M=%d, N=%d, K=%d, L=%d, R=%d)" % (M, N, K, L, R))
    return dx, dA, dB


def _mask(mask, T):
    import torch
    if mask is None:
        return None
    if mask.dtype not in (torch.bool, torch.uint8) or tuple(mask.shape) != (T,) or \
            not mask.is_contiguous():
        raise ValueError("mask must be a contiguous bool or uint8 vector of %d values" % T)
    return mask


def route_topk(logits, top_k, mask=None, renormalize=True):
    """The top_k experts of each token of logits [T, E] (bfloat16, float16 or float32):
    a Routing.  Weights are softmax probabilities, divided by their sum over
    the choices where `renormalize`; equal logits go to the lower expert; a
    logit of -inf closes an expert to its token.  Tokens whose mask (bool or
    uint8 [T]) is 0 are left out.  loss = E sum_e f_e P_e with f_e the share of
    choices that fell on e and P_e the mean probability of e, over the routed
    tokens."""
    import torch
    if logits.dim() != 2:
        raise ValueError("logits must be [T, E]")
    T, E = logits.shape
    k = int(top_k)
    index = _index(logits)
    if torch._C._cuda_getDevice() != index:
        with torch.cuda.device(index):
            return route_topk(logits, k, mask, renormalize)
    ld = _matrix("logits", logits, T, E)
    if mask is not None:
        _on(index, mask=_mask(mask, T))
    n = _workspace_bytes("gemm_route_workspace", T, E, k)
    # Up to 256 KB in one allocation, the workspace first: two more are 3 us of a call whose
    # kernels take no longer than the host (4099 tokens, 4 choices 19.2 us against 23.0).
    # Beyond that the workspace, the results of T k values and those of E apart, so that who
    # keeps one (a loss, the counts) does not keep the others' memory.
    nk, words, few, dev = T * k, n // 4, 2 * E + 3, logits.device
    if words + 3 * nk + few <= 65536:
        buf = torch.empty(words + 3 * nk + few, dtype=torch.int32, device=dev)
        ws = buf.data_ptr()
        p = ws + n
        at = p + 12 * nk
        _, ids, order, weights, counts, offsets, tokens, loss = buf.split_with_sizes(
            (words, nk, nk, nk, E, E + 1, 1, 1))
    else:
        space = torch.empty(words, dtype=torch.int32, device=dev)
        most, small = (torch.empty(m, dtype=torch.int32, device=dev) for m in (3 * nk, few))
        ws, p, at = space.data_ptr(), most.data_ptr(), small.data_ptr()
        ids, order, weights = most.split_with_sizes((nk, nk, nk))
        counts, offsets, tokens, loss = small.split_with_sizes((E, E + 1, 1, 1))
    c_out = _rows.GemmRouting(p, p + 8 * nk, at, at + 4 * E, p + 4 * nk, at + 8 * E + 4, at + 8 * E + 8)
    st = _rows.lib().gemm_run_route(logits.data_ptr(), _ptr(mask), T, E, ld, k, 1 if renormalize else 0,
                                    _code(logits.dtype), ctypes.byref(c_out), ws, n,
                                    torch._C._cuda_getCurrentRawStream(index))
    if st:
        _lib.check(st, "route_topk(T=%d, E=%d, k=%d)" % (T, E, k))
    # (.data: tensors of their own, so that one changed in place is not taken by autograd for
    # a change of the others)
    f32 = torch.float32
    return Routing(ids.view(T, k).data, weights.view(f32).view(T, k).data, counts.data, offsets.data,
                   order.data, tokens.data, loss.view(f32).view(()).data, bool(renormalize))


def route_topk_backward(logits, routing, grad_weights=None, grad_loss=None, out=None):
    """The gradient in the logits of `routing` = route_topk(logits, ...): of its
    weights (grad_weights float32 [T, k]) and its loss (grad_loss, a float32
    scalar tensor), either None for zero; counts are constants.  Of the logits'
    dtype; zeros for tokens that were not routed and closed experts."""
    import torch
    if logits.dim() != 2 or routing.ids.dim() != 2 or routing.ids.shape[0] != logits.shape[0] or \
            routing.counts.shape[0] != logits.shape[1]:
        raise ValueError("routing does not belong to these logits")
    T, E = logits.shape
    k = routing.ids.shape[1]
    index = _index(logits)
    if torch._C._cuda_getDevice() != index:
        with torch.cuda.device(index):
            return route_topk_backward(logits, routing, grad_weights, grad_loss, out)
    ld = _matrix("logits", logits, T, E)
    ids, weights, counts, _, _, tokens, _, renormalize = routing
    for t, n, dt in ((ids, T * k, torch.int32), (weights, T * k, torch.float32), (counts, E, torch.int32),
                     (tokens, 1, torch.int32)):
        if t.dtype != dt or t.numel() != n or not t.is_contiguous() or t.get_device() != index:
            raise ValueError("the routing is not what route_topk gave for these logits")
    if grad_weights is not None or grad_loss is not None:
        _on(index, grad_weights=grad_weights, grad_loss=grad_loss)
    if grad_weights is not None and (grad_weights.dtype != torch.float32 or
                                     tuple(grad_weights.shape) != (T, k) or
                                     not grad_weights.is_contiguous()):
        raise ValueError("grad_weights must be contiguous float32 [%d, %d]" % (T, k))
    if grad_loss is not None and (grad_loss.dtype != torch.float32 or grad_loss.numel() != 1):
        raise ValueError("grad_loss must be one float32 value")
    if out is None:
        out = torch.empty((T, E), dtype=logits.dtype, device=logits.device)
        ldd = E
    else:
        ldd = _matrix("out", _out("out", out, (T, E), logits.device), T, E)
        if out.dtype != logits.dtype:
            raise TypeError("out must have the logits' dtype")
    c_in = _rows.GemmRouting(ids.data_ptr(), weights.data_ptr(), counts.data_ptr(), None, None,
                             tokens.data_ptr(), None)
    st = _rows.lib().gemm_run_route_backward(
        logits.data_ptr(), ctypes.byref(c_in), _ptr(grad_weights), _ptr(grad_loss), out.data_ptr(), T, E,
        ld, ldd, k, 1 if renormalize else 0, _code(logits.dtype),
        torch._C._cuda_getCurrentRawStream(index))
    if st:
        _lib.check(st, "route_topk_backward(T=%d, E=%d, k=%d)" % (T, E, k))
    return out


def gemm_routed(x, W, offsets, out=None, out_dtype=None):
    """C[i] = x[i] W[e]^T for offsets[e] <= i < offsets[e + 1]: x [S, K] rows sorted by
    expert, W [E, N, K], offsets int32 [E + 1] on the device (route_topk's).  W[e]
    is K-major (unit stride along K) or a transposed view of [E, K, N] (unit
    stride along N): gemm_routed(dy, W.transpose(1, 2), offsets) is the gradient
    in x of gemm_routed(x, W, offsets).  Rows of no expert (before offsets[0], behind
    offsets[E]) are zero in a new result, and left as they are in `out`."""
    import torch
    if x.dim() != 2 or W.dim() != 3 or W.shape[2] != x.shape[1]:
        raise ValueError("x must be [S, K] and W [E, N, K], got %s and %s"
                         % (tuple(x.shape), tuple(W.shape)))
    S, K = x.shape
    E, N, _ = W.shape
    index = _index(x)
    if torch._C._cuda_getDevice() != index:
        with torch.cuda.device(index):
            return gemm_routed(x, W, offsets, out, out_dtype)
    dt = x.dtype
    if W.dtype != dt:
        raise TypeError("x and W must share a dtype")
    if not W.get_device() == offsets.get_device() == index:
        _on(index, W=W, offsets=offsets)
    _vector("offsets", offsets, E + 1, torch.int32)
    ldx = _matrix("x", x, S, K)
    w_stride, w_row, w_col = W.stride()
    if W.numel() == 0:
        layout, ldw = _lib.GEMM_K_MAJOR, max(K, 1)
    elif w_col == 1 and (N == 1 or w_row >= K):
        layout, ldw = _lib.GEMM_K_MAJOR, w_row if N > 1 else K
    elif w_row == 1 and (K == 1 or w_col >= N):
        layout, ldw = _lib.GEMM_MN_MAJOR, w_col if K > 1 else max(N, w_col)
    else:
        raise ValueError("W's strides %s are neither K-major nor MN-major" % (W.stride(),))
    if out is None:
        tail = _rows.GEMM_TAIL_ZERO
        out = torch.empty((S, N), dtype=out_dtype or dt, device=x.device)
        ldc = N
    else:
        tail = _rows.GEMM_TAIL_KEEP
        ldc = _matrix("out", _out("out", out, (S, N), x.device), S, N)
    st = _rows.lib().gemm_run_routed(
        x.data_ptr(), W.data_ptr(), out.data_ptr(), offsets.data_ptr(), S, N, K, E, ldx, ldw,
        w_stride if E > 1 else 0, ldc, layout, _code(dt), _code(out.dtype), tail,
        torch._C._cuda_getCurrentRawStream(index))
    if st:
        _lib.check(st, "gemm_routed(S=%d, N=%d, K=%d, E=%d)" % (S, N, K, E))
    return out


def gemm_routed_wgrad(dy, x, offsets, out_dtype=None):
    """dW [E, N, K]: dW[e] = sum over e's rows i of dy[i]^T x[i], for dy [S, N] and
    x [S, K] sorted by expert and offsets int32 [E + 1] on the device; zeros for an
    expert without rows.  N and K multiples of 8; out_dtype defaults to x's."""
    import torch
    if x.dim() != 2 or dy.dim() != 2 or dy.shape[0] != x.shape[0]:
        raise ValueError("dy must be [S, N] and x [S, K], got %s and %s"
                         % (tuple(dy.shape), tuple(x.shape)))
    S, K = x.shape
    N = dy.shape[1]
    index = _index(x)
    if torch._C._cuda_getDevice() != index:
        with torch.cuda.device(index):
            return gemm_routed_wgrad(dy, x, offsets, out_dtype)
    if x.dtype != dy.dtype:
        raise TypeError("dy and x must share a dtype")
    if offsets.dim() != 1 or offsets.shape[0] < 1:
        raise ValueError("offsets must be [E + 1]")
    E = offsets.shape[0] - 1
    if not dy.get_device() == offsets.get_device() == index:
        _on(index, dy=dy, offsets=offsets)
    _vector("offsets", offsets, E + 1, torch.int32)
    lddy, ldx = _matrix("dy", dy, S, N), _matrix("x", x, S, K)
    out = torch.empty((E, N, K), dtype=out_dtype or x.dtype, device=x.device)
    st = _rows.lib().gemm_run_routed_wgrad(
        dy.data_ptr(), x.data_ptr(), out.data_ptr(), offsets.data_ptr(), S, N, K, E, lddy, ldx,
        _code(x.dtype), _code(out.dtype), torch._C._cuda_getCurrentRawStream(index))
    if st:
        _lib.check(st, "gemm_routed_wgrad(S=%d, N=%d, K=%d, E=%d)" % (S, N, K, E))
    return out
