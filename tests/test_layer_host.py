"""The C ABI of a feed-forward layer's products without a device: its symbols, the
workspace sizes, and every refusal (which comes before any device call, so the
addresses here are never read); and the Python calls' own refusals."""
import ctypes
import os
import re

import pytest
import torch

from dense_gemm_nt_amd import _layer, _lib

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
P = 0x10000                 # an aligned address that nothing reads
OK, INVALID, UNSUPPORTED, MISALIGNED = 0, 1, 2, 3


@pytest.fixture(scope="module")
def L():
    from dense_gemm_nt_amd import build
    if build.stale_layer():
        build.build_layer()
    return _layer.lib()


def test_every_declared_symbol_is_there(L):
    text = open(os.path.join(ROOT, "include", "gemm_layer.h")).read()
    declared = sorted(set(re.findall(r"^gemm_status_t\s+(gemm_\w+)\(", text, re.M)))
    assert declared == sorted(_layer.EXPORTS)
    for name in declared:
        assert hasattr(L, name), name


def test_the_calls_are_public():
    import dense_gemm_nt_amd as g
    for name in ("gemm_gated", "gemm_gated_backward", "quantize_int8", "gemm_int8", "orthogonalize"):
        assert name in g.__all__ and callable(getattr(g, name)) and getattr(g, name).__doc__


def _gated(L, **kw):
    d = dict(x=P, Wg=P, Wu=P, h=P, M=8, F=32, K=64, ldx=64, ldg=64, ldu=64, ldh=32, in_dt=0, out_dt=0, act=3, ws=0, n=0)
    d.update(kw)
    return L.gemm_run_gated(d["x"], d["Wg"], d["Wu"], d["h"], d["M"], d["F"], d["K"], d["ldx"], d["ldg"], d["ldu"],
                            d["ldh"], d["in_dt"], d["out_dt"], d["act"], d["ws"], d["n"], None)


@pytest.mark.parametrize("kw,want", [
    (dict(M=-1), INVALID), (dict(F=-1), INVALID), (dict(K=-8), INVALID), (dict(K=60), UNSUPPORTED),
    (dict(in_dt=2), UNSUPPORTED), (dict(in_dt=3), UNSUPPORTED), (dict(out_dt=7), UNSUPPORTED),
    (dict(act=0), INVALID), (dict(act=4), INVALID), (dict(x=None), INVALID), (dict(Wg=None), INVALID),
    (dict(Wu=None), INVALID), (dict(h=None), INVALID), (dict(ldx=56), INVALID), (dict(ldg=56), INVALID),
    (dict(ldu=56), INVALID), (dict(ldh=31), INVALID), (dict(ldx=68), MISALIGNED), (dict(ldu=68), MISALIGNED),
    (dict(x=P + 8), MISALIGNED), (dict(Wu=P + 2), MISALIGNED), (dict(h=P + 1), MISALIGNED),
    (dict(ldg=1 << 22), UNSUPPORTED), (dict(M=1 << 30), UNSUPPORTED), (dict(F=1 << 21), UNSUPPORTED),
    (dict(ldh=(1 << 31) - 1), UNSUPPORTED),
    (dict(M=1 << 29, F=1 << 18, ldh=1 << 18), UNSUPPORTED),           # launches too large
    (dict(K=8192, ldx=8192, ldg=8192, ldu=8192), INVALID),            # the workspace is missing
    (dict(K=8192, ldx=8192, ldg=8192, ldu=8192, ws=P, n=64), INVALID),                     # or too small
    (dict(K=8192, ldx=8192, ldg=8192, ldu=8192, ws=P + 16, n=1 << 30), MISALIGNED),
    (dict(M=0), OK), (dict(F=0), OK),        # nothing to do, and nothing is enqueued
])
def test_gated_refuses(L, kw, want):
    assert _gated(L, **kw) == want


def _backward(L, **kw):
    d = dict(dh=P, x=P, Wg=P, Wu=P, dx=P, dWg=P, dWu=P, M=8, F=32, K=64, lddh=32, ldx=64, ldg=64, ldu=64, lddx=64,
             in_dt=0, dx_dt=0, g_dt=2, act=3, ws=0, n=0)
    d.update(kw)
    return L.gemm_run_gated_backward(d["dh"], d["x"], d["Wg"], d["Wu"], d["dx"], d["dWg"], d["dWu"], d["M"], d["F"],
                                     d["K"], d["lddh"], d["ldx"], d["ldg"], d["ldu"], d["lddx"], d["in_dt"],
                                     d["dx_dt"], d["g_dt"], d["act"], d["ws"], d["n"], None)


@pytest.mark.parametrize("kw,want", [
    (dict(M=-1), INVALID), (dict(K=60), UNSUPPORTED), (dict(in_dt=2), UNSUPPORTED), (dict(dx_dt=3), UNSUPPORTED),
    (dict(g_dt=4), UNSUPPORTED), (dict(act=7), INVALID), (dict(dh=None), INVALID), (dict(x=None), INVALID),
    (dict(Wg=None), INVALID), (dict(Wu=None), INVALID), (dict(dWg=None), INVALID), (dict(dWu=None), INVALID),
    (dict(lddh=24), INVALID), (dict(lddx=63), INVALID), (dict(dh=P + 1), MISALIGNED), (dict(dx=P + 1), MISALIGNED),
    (dict(dWg=P + 2), MISALIGNED), (dict(ldx=68), MISALIGNED), (dict(F=1 << 21), UNSUPPORTED),
    (dict(lddh=(1 << 31) - 1), UNSUPPORTED),
    (dict(), INVALID), (dict(ws=P, n=256), INVALID), (dict(ws=P + 8, n=1 << 30), MISALIGNED),
    (dict(dx=None, dWg=None, dWu=None), OK),              # nothing is asked for
    (dict(dWg=None, dWu=None, M=0), OK), (dict(dx=None, F=0), OK), (dict(K=0), OK),
])
def test_backward_refuses(L, kw, want):
    assert _backward(L, **kw) == want


def _quantize(L, **kw):
    d = dict(x=P, q=P, s=P, M=4, K=64, ldx=64, ldq=64, dt=0)
    d.update(kw)
    return L.gemm_run_quantize_int8(d["x"], d["q"], d["s"], d["M"], d["K"], d["ldx"], d["ldq"], d["dt"], None)


@pytest.mark.parametrize("kw,want", [
    (dict(M=-1), INVALID), (dict(K=-1), INVALID), (dict(dt=3), UNSUPPORTED), (dict(M=1 << 30), UNSUPPORTED),
    (dict(K=(1 << 31) - 1, ldx=1 << 31, ldq=1 << 31), UNSUPPORTED), (dict(x=None), INVALID), (dict(q=None), INVALID),
    (dict(s=None), INVALID), (dict(ldx=63), INVALID), (dict(ldq=63), INVALID), (dict(x=P + 1), MISALIGNED),
    (dict(x=P + 2, dt=2), MISALIGNED), (dict(s=P + 2), MISALIGNED), (dict(M=0, x=None), OK),
])
def test_quantize_refuses(L, kw, want):
    assert _quantize(L, **kw) == want


def _int8(L, epi=None, **kw):
    d = dict(A=P, B=P, C=P, M=8, N=32, K=64, lda=64, ldb=64, ldc=32, out_dt=0, sa=P, na=8, sb=P, nb=32, ws=0, n=0)
    d.update(kw)
    return L.gemm_run_int8(d["A"], d["B"], d["C"], d["M"], d["N"], d["K"], d["lda"], d["ldb"], d["ldc"], d["out_dt"],
                           d["sa"], d["na"], d["sb"], d["nb"], ctypes.byref(epi) if epi is not None else None,
                           d["ws"], d["n"], None)


@pytest.mark.parametrize("kw,want", [
    (dict(M=-1), INVALID), (dict(N=-1), INVALID), (dict(K=-16), INVALID), (dict(K=40), UNSUPPORTED),
    (dict(K=1 << 17, lda=1 << 17, ldb=1 << 17), UNSUPPORTED), (dict(out_dt=3), UNSUPPORTED), (dict(A=None), INVALID),
    (dict(B=None), INVALID), (dict(C=None), INVALID), (dict(sa=None), INVALID), (dict(sb=None), INVALID),
    (dict(na=7), INVALID), (dict(nb=31), INVALID), (dict(lda=48), INVALID), (dict(ldc=31), INVALID),
    (dict(lda=72), MISALIGNED), (dict(B=P + 8), MISALIGNED), (dict(C=P + 1), MISALIGNED), (dict(sa=P + 2), MISALIGNED),
    (dict(lda=1 << 23), UNSUPPORTED), (dict(M=1 << 30, na=1 << 30), UNSUPPORTED),
    (dict(K=16384, lda=16384, ldb=16384), INVALID),       # the workspace is missing
    (dict(K=16384, lda=16384, ldb=16384, ws=P + 8, n=1 << 30), MISALIGNED),
    (dict(M=0), OK), (dict(N=0), OK),
])
def test_int8_refuses(L, kw, want):
    assert _int8(L, **kw) == want


def test_int8_refuses_epilogues(L):
    assert _int8(L, _lib.GemmEpilogue(1.0, 0.0, None, 1, 0)) == INVALID       # a bias axis, no bias
    assert _int8(L, _lib.GemmEpilogue(1.0, 0.0, None, 0, 9)) == INVALID
    assert _int8(L, _lib.GemmEpilogue(float("inf"), 0.0, None, 0, 0)) == UNSUPPORTED


def _ortho(L, abc=(1.5, -0.5, 0.0), **kw):
    d = dict(G=P, U=P, B=2, m=32, n=48, ldg=48, ldu=48, gs=32 * 48, us=32 * 48, in_dt=2, out_dt=0, steps=1, eps=1e-7, ws=0,
             nb=0)
    d.update(kw)
    c = (ctypes.c_float * 3)(*abc) if abc else None
    return L.gemm_run_orthogonalize(d["G"], d["U"], d["B"], d["m"], d["n"], d["ldg"], d["ldu"], d["gs"], d["us"],
                                    d["in_dt"], d["out_dt"], d["steps"], c, d["eps"], d["ws"], d["nb"], None)


@pytest.mark.parametrize("kw,want", [
    (dict(B=-1), INVALID), (dict(m=-1), INVALID), (dict(n=-1), INVALID), (dict(steps=-1), INVALID),
    (dict(abc=None), INVALID), (dict(gs=-1), INVALID), (dict(us=-1), INVALID), (dict(eps=-1.0), INVALID),
    (dict(eps=float("nan")), INVALID), (dict(in_dt=3), UNSUPPORTED), (dict(out_dt=4), UNSUPPORTED),
    (dict(m=(1 << 20) + 1), UNSUPPORTED), (dict(B=65536), UNSUPPORTED), (dict(abc=(1.0, float("inf"), 0.0)), UNSUPPORTED),
    (dict(G=None), INVALID), (dict(U=None), INVALID), (dict(ldg=47), INVALID), (dict(ldu=47), INVALID),
    (dict(G=P + 2), MISALIGNED), (dict(U=P + 1), MISALIGNED), (dict(), INVALID), (dict(ws=P, nb=64), INVALID),
    (dict(ws=P + 8, nb=1 << 30), MISALIGNED), (dict(B=60000, m=1 << 14, n=1 << 14, ldg=1 << 14, ldu=1 << 14, ws=P, nb=1 << 60), UNSUPPORTED),
    (dict(B=0), OK), (dict(m=0), OK), (dict(n=0), OK),
])
def test_orthogonalize_refuses(L, kw, want):
    kw = dict(kw)
    assert _ortho(L, kw.pop("abc", (1.5, -0.5, 0.0)), **kw) == want


def test_workspaces(L):
    def size(fn, *a):
        st, n = _layer.workspace_bytes(fn, *a)
        assert st == OK, (fn, a, st)
        return n
    assert size("gemm_gated_workspace", 0, 32, 64) == 0 and size("gemm_gated_workspace", 4096, 4096, 64) == 0
    assert size("gemm_gated_workspace", 1, 512, 4096) > 0
    assert size("gemm_int8_workspace", 1, 8192, 8192) == 0            # no tiles, no K splits
    assert size("gemm_int8_workspace", 16, 8192, 8192) > 0
    for a in ((0, 8, 16), (3, 0, 16), (3, 8, 0), (0, 0, 0)):          # no product, no plan
        assert size("gemm_gated_backward_workspace", *a) >= 0 and size("gemm_gated_workspace", *a) >= 0
        assert size("gemm_int8_workspace", *a) >= 0 and size("gemm_orthogonalize_workspace", *a) >= 0
    # both weights' gradients side by side, to whole groups of eight
    assert size("gemm_gated_backward_workspace", 1000, 1001, 64) >= 1000 * 2016 * 2
    one = size("gemm_orthogonalize_workspace", 1, 1000, 2047)
    assert 1024 * 2048 * 6 <= one < 1024 * 2048 * 40 and size("gemm_orthogonalize_workspace", 3, 1000, 2047) > 2 * one // 2
    for fn, a in (("gemm_gated_workspace", (1, -1, 8)), ("gemm_int8_workspace", (1, 1, -16)),
                  ("gemm_gated_backward_workspace", (-1, 1, 8)), ("gemm_orthogonalize_workspace", (1, -2, 2))):
        assert _layer.workspace_bytes(fn, *a)[0] == INVALID
    for fn in ("gemm_gated_workspace", "gemm_int8_workspace", "gemm_gated_backward_workspace", "gemm_orthogonalize_workspace"):
        assert getattr(L, fn)(1, 16, 16, None) == INVALID


def test_calls_refuse_what_is_not_theirs():
    import dense_gemm_nt_amd as g
    x, W = torch.zeros(4, 16, dtype=torch.bfloat16), torch.zeros(8, 16, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        g.gemm_gated(x, W, W)                               # not on a device
    with pytest.raises(TypeError):
        g.gemm_gated(x, W, W.half())
    with pytest.raises(ValueError):
        g.gemm_gated(x[0], W, W)
    with pytest.raises(ValueError):
        g.gemm_gated_backward(x, x, W, W)
    with pytest.raises(ValueError):
        g.quantize_int8(x)
    q = torch.zeros(4, 16, dtype=torch.int8)
    with pytest.raises(TypeError):
        g.gemm_int8(q, q.float(), torch.ones(4), torch.ones(4))
    with pytest.raises(ValueError):
        g.gemm_int8(q, torch.zeros(4, 32, dtype=torch.int8), torch.ones(4), torch.ones(4))
    with pytest.raises(ValueError):
        g.orthogonalize(torch.zeros(3))
    with pytest.raises(ValueError):
        g.orthogonalize(torch.zeros(3, 4))


def test_coefficients_are_taken_as_numbers():
    from dense_gemm_nt_amd import layer
    t = torch.tensor([1.0, 2.0, 3.0])
    assert list(layer._coefficients(t, 2)) == [1, 2, 3, 1, 2, 3]
    scalars = list(t)                                       # (views: the same objects with other values)
    assert list(layer._coefficients(scalars, 1)) == [1, 2, 3]
    t += 1
    assert list(layer._coefficients(scalars, 1)) == [2, 3, 4] and list(layer._coefficients(t, 1)) == [2, 3, 4]
    assert list(layer._coefficients([(1, 2, 3), [4, 5, 6], t], 3)) == [1, 2, 3, 4, 5, 6, 2, 3, 4]
    assert list(layer._coefficients(torch.ones(3, 3), 3)) == [1] * 9
    assert list(layer._coefficients((1, 2, 3), 0)) == [] and list(layer._coefficients([], 0)) == []
    for bad, steps in (((1, 2), 2), ((1, 2, 3, 4), 4), ([(1, 2, 3)], 2), ([(1, 2)] * 2, 2), ([(1, 2, 3), 1, 2], 3)):
        with pytest.raises(ValueError):
            layer._coefficients(bad, steps)


def test_outputs_that_overlap_operands_are_refused():
    from dense_gemm_nt_amd import layer
    buf = torch.zeros(8, 64)
    a, b = buf[:, :24], buf[:, 24:56]
    layer._apart(a, x=b)                                    # columns of the same rows
    layer._apart(b, x=a, y=None, z=torch.zeros(3))
    layer._apart(buf[:4], x=buf[4:])
    layer._apart(buf[:1, :8], x=buf[0, 8:16], y=buf[1, :8])
    layer._apart(buf[:, 16:24], x=buf[1:, :16])
    layer._apart(buf[3:4, :8], x=buf[:, 8:16]), layer._apart(buf[:, 8:16], x=buf[3, :8])
    layer._apart(buf[:0], x=buf), layer._apart(buf[:, :0], x=buf)
    for out, x in ((a, a), (a, buf[:, 23:30]), (buf[:, 23:30], a), (buf[:4], buf[3:]), (buf[1:3, 8:], buf[2:, :9]),
                   (buf.view(16, 32)[2:5], buf[1]), (buf[2:3], buf[:, 5:6]), (buf[:, 5:6], buf[2:3])):
        with pytest.raises(ValueError):
            layer._apart(out, x=x)
