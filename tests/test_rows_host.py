"""The C ABI of the row-indexed products without a device: its symbols, the
workspace sizes, and every refusal (which comes before any device call, so the
addresses here are never read)."""
import ctypes
import os
import re

import pytest

from dense_gemm_nt_amd import _lib, _rows
from dense_gemm_nt_amd._rows import GemmAdapters, GemmRouting

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
P = 0x10000                 # an aligned address that nothing reads
OK, INVALID, UNSUPPORTED, MISALIGNED = 0, 1, 2, 3


@pytest.fixture(scope="module")
def L():
    from dense_gemm_nt_amd import build
    if build.stale_rows():
        build.build_rows()
    return _rows.lib()


def test_every_declared_symbol_is_there(L):
    text = open(os.path.join(ROOT, "include", "gemm_rows.h")).read()
    declared = sorted(set(re.findall(r"^gemm_status_t\s+(gemm_\w+)\(", text, re.M)))
    assert declared == sorted(_rows.EXPORTS)
    for name in declared:
        assert hasattr(L, name), name


def _adapters(**kw):
    d = dict(A=P, B=P, scale=P, ids=P, num_adapters=3, rank=16, a_stride=16 * 64, a_ld=64,
             b_stride=32 * 16, b_ld=16)
    d.update(kw)
    return GemmAdapters(**d)


def _lora(L, ad=None, epi=None, **kw):
    d = dict(x=P, W=P, y=P, M=8, N=32, K=64, ldx=64, ldw=64, ldy=32, in_dt=0, out_dt=0, ws=0, n=0)
    d.update(kw)
    return L.gemm_run_lora(d["x"], d["W"], d["y"], d["M"], d["N"], d["K"], d["ldx"], d["ldw"], d["ldy"],
                           d["in_dt"], d["out_dt"], ctypes.byref(ad) if ad is not None else None,
                           ctypes.byref(epi) if epi is not None else None, d["ws"], d["n"], None)


@pytest.mark.parametrize("kw,want", [
    (dict(M=-1), INVALID), (dict(N=-1), INVALID), (dict(K=-8), INVALID), (dict(K=60), UNSUPPORTED),
    (dict(in_dt=2), UNSUPPORTED), (dict(in_dt=3), UNSUPPORTED), (dict(out_dt=7), UNSUPPORTED),
    (dict(x=None), INVALID), (dict(W=None), INVALID), (dict(y=None), INVALID),
    (dict(ldx=56), INVALID), (dict(ldw=56), INVALID), (dict(ldy=31), INVALID),
    (dict(ldx=68), MISALIGNED), (dict(x=P + 8), MISALIGNED), (dict(W=P + 2), MISALIGNED),
    (dict(y=P + 1), MISALIGNED), (dict(ldw=1 << 22), UNSUPPORTED), (dict(M=1 << 31), UNSUPPORTED),
    (dict(M=1 << 30), UNSUPPORTED), (dict(M=1 << 29, N=1 << 17, ldy=1 << 17), UNSUPPORTED),    # launches too large
    (dict(), INVALID),                       # the workspace is missing
    (dict(ws=P, n=64), INVALID),             # or too small
    (dict(ws=P + 16, n=1 << 30), MISALIGNED),
    (dict(M=0), OK), (dict(N=0), OK),        # nothing to do, and nothing is enqueued
])
def test_lora_refuses(L, kw, want):
    assert _lora(L, _adapters(), **kw) == want


@pytest.mark.parametrize("kw,want", [
    (dict(rank=12), UNSUPPORTED), (dict(rank=136), UNSUPPORTED), (dict(rank=-8), INVALID),
    (dict(num_adapters=-1), INVALID), (dict(A=None), INVALID), (dict(B=None), INVALID),
    (dict(scale=None), INVALID), (dict(ids=None), INVALID), (dict(a_ld=56), INVALID),
    (dict(b_ld=8), INVALID), (dict(a_ld=68), MISALIGNED), (dict(b_ld=20), MISALIGNED),
    (dict(a_stride=4), MISALIGNED), (dict(b_stride=4), MISALIGNED), (dict(a_stride=-8), INVALID),
    (dict(A=P + 4), MISALIGNED), (dict(B=P + 4), MISALIGNED), (dict(ids=P + 2), MISALIGNED),
    (dict(scale=P + 1), MISALIGNED),
])
def test_lora_refuses_adapters(L, kw, want):
    assert _lora(L, _adapters(**kw)) == want


def test_lora_refuses_other(L):
    assert _lora(L, None) == INVALID
    assert _lora(L, _adapters(), _lib.GemmEpilogue(1.0, 0.0, None, 1, 0)) == INVALID      # a bias axis, no bias
    assert _lora(L, _adapters(), _lib.GemmEpilogue(1.0, 0.0, None, 0, 9)) == INVALID
    assert _lora(L, _adapters(), _lib.GemmEpilogue(float("inf"), 0.0, None, 0, 0)) == UNSUPPORTED
    # B of an adapter past what a buffer load can address
    assert _lora(L, _adapters(b_ld=1 << 20, b_stride=0), N=1 << 11, ldy=1 << 11) == UNSUPPORTED


def _backward(L, ad=None, **kw):
    d = dict(dy=P, x=P, W=P, dx=P, dA=P, dB=P, M=8, N=32, K=64, lddy=32, ldx=64, ldw=64, lddx=64, in_dt=0,
             dx_dt=0, g_dt=2, ws=0, n=0)
    d.update(kw)
    return L.gemm_run_lora_backward(d["dy"], d["x"], d["W"], d["dx"], d["dA"], d["dB"], d["M"], d["N"], d["K"],
                                    d["lddy"], d["ldx"], d["ldw"], d["lddx"], d["in_dt"], d["dx_dt"], d["g_dt"],
                                    ctypes.byref(ad or _adapters()), d["ws"], d["n"], None)


@pytest.mark.parametrize("kw,want", [
    (dict(N=36, lddy=40), UNSUPPORTED), (dict(K=60), UNSUPPORTED), (dict(M=-1), INVALID),
    (dict(in_dt=2), UNSUPPORTED), (dict(dx_dt=3), UNSUPPORTED), (dict(g_dt=4), UNSUPPORTED),
    (dict(dy=None), INVALID), (dict(x=None), INVALID), (dict(W=None), INVALID),
    (dict(dA=None), INVALID), (dict(dB=None), INVALID),      # one without the other
    (dict(lddy=24), INVALID), (dict(lddx=63), INVALID), (dict(lddy=36), MISALIGNED),
    (dict(dx=P + 1), MISALIGNED), (dict(dA=P + 2), MISALIGNED),
    (dict(), INVALID), (dict(ws=P, n=256), INVALID), (dict(ws=P + 8, n=1 << 30), MISALIGNED),
])
def test_lora_backward_refuses(L, kw, want):
    assert _backward(L, **kw) == want


def test_lora_backward_refuses_many_adapters(L):
    assert _backward(L, _adapters(num_adapters=1025)) == UNSUPPORTED


def _route(L, out=None, **kw):
    d = dict(x=P, mask=None, T=4, E=8, ld=8, k=2, renorm=1, dt=2, ws=0, n=0)
    d.update(kw)
    out = GemmRouting(P, P, P, P, P, P, P) if out is None else out
    return L.gemm_run_route(d["x"], d["mask"], d["T"], d["E"], d["ld"], d["k"], d["renorm"], d["dt"],
                            ctypes.byref(out), d["ws"], d["n"], None)


@pytest.mark.parametrize("kw,want", [
    (dict(T=-1), INVALID), (dict(E=0, ld=8), UNSUPPORTED), (dict(E=1025, ld=1025), UNSUPPORTED),
    (dict(k=0), UNSUPPORTED), (dict(k=9), UNSUPPORTED), (dict(E=100, ld=100, k=65), UNSUPPORTED),
    (dict(k=-1), INVALID), (dict(T=1 << 30, k=2), UNSUPPORTED), (dict(dt=3), UNSUPPORTED),
    (dict(ld=7), INVALID), (dict(x=None), INVALID), (dict(x=P + 2), MISALIGNED), (dict(), INVALID),
    (dict(ws=P, n=8), INVALID), (dict(ws=P + 4, n=1 << 20), MISALIGNED),
])
def test_route_refuses(L, kw, want):
    assert _route(L, **kw) == want


@pytest.mark.parametrize("field", [n for n, _ in GemmRouting._fields_])
def test_route_needs_every_output(L, field):
    out = GemmRouting(P, P, P, P, P, P, P)
    setattr(out, field, None)
    assert _route(L, out) == INVALID
    setattr(out, field, P + 2)
    assert _route(L, out) == MISALIGNED


def _route_backward(L, inp=None, **kw):
    d = dict(x=P, gw=None, gl=None, dl=P, T=4, E=8, ld=8, ldd=8, k=2, dt=2)
    d.update(kw)
    inp = GemmRouting(P, P, P, P, P, P, P) if inp is None else inp
    return L.gemm_run_route_backward(d["x"], ctypes.byref(inp), d["gw"], d["gl"], d["dl"], d["T"], d["E"], d["ld"],
                                     d["ldd"], d["k"], 1, d["dt"], None)


@pytest.mark.parametrize("kw,want", [
    (dict(T=-1), INVALID), (dict(E=1025, ld=1025, ldd=1025), UNSUPPORTED), (dict(k=9), UNSUPPORTED),
    (dict(dt=4), UNSUPPORTED), (dict(ld=7), INVALID), (dict(ldd=7), INVALID), (dict(x=None), INVALID),
    (dict(dl=None), INVALID), (dict(gw=P + 1), MISALIGNED), (dict(gl=P + 2), MISALIGNED),
    (dict(dl=P + 2), MISALIGNED), (dict(T=0), OK),
])
def test_route_backward_refuses(L, kw, want):
    assert _route_backward(L, **kw) == want


def _routed(L, **kw):
    d = dict(x=P, W=P, C=P, off=P, rows=8, N=32, K=64, E=4, ldx=64, ldw=64, ws=32 * 64, ldc=32, layout=0, in_dt=0,
             out_dt=0, tail=0)
    d.update(kw)
    return L.gemm_run_routed(d["x"], d["W"], d["C"], d["off"], d["rows"], d["N"], d["K"], d["E"], d["ldx"], d["ldw"],
                             d["ws"], d["ldc"], d["layout"], d["in_dt"], d["out_dt"], d["tail"], None)


@pytest.mark.parametrize("kw,want", [
    (dict(rows=-1), INVALID), (dict(N=-1), INVALID), (dict(K=-8), INVALID), (dict(E=-1), INVALID),
    (dict(E=1025), UNSUPPORTED), (dict(K=60), UNSUPPORTED), (dict(in_dt=2), UNSUPPORTED),
    (dict(out_dt=3), UNSUPPORTED), (dict(layout=2), INVALID), (dict(tail=2), INVALID), (dict(ws=-8), INVALID),
    (dict(ws=2052), MISALIGNED), (dict(x=None), INVALID), (dict(W=None), INVALID), (dict(C=None), INVALID),
    (dict(off=None), INVALID), (dict(off=P + 2), MISALIGNED), (dict(ldx=56), INVALID), (dict(ldw=56), INVALID),
    (dict(layout=1, ldw=24), INVALID), (dict(ldc=31), INVALID), (dict(x=P + 8), MISALIGNED),
    (dict(ldw=68), MISALIGNED), (dict(C=P + 1), MISALIGNED), (dict(rows=0), OK), (dict(N=0), OK),
])
def test_routed_refuses(L, kw, want):
    assert _routed(L, **kw) == want


def _wgrad(L, **kw):
    d = dict(dy=P, x=P, dW=P, off=P, rows=8, N=32, K=64, E=4, lddy=32, ldx=64, in_dt=0, out_dt=2)
    d.update(kw)
    return L.gemm_run_routed_wgrad(d["dy"], d["x"], d["dW"], d["off"], d["rows"], d["N"], d["K"], d["E"], d["lddy"],
                                   d["ldx"], d["in_dt"], d["out_dt"], None)


@pytest.mark.parametrize("kw,want", [
    (dict(N=36, lddy=40), UNSUPPORTED), (dict(K=60), UNSUPPORTED), (dict(E=1025), UNSUPPORTED),
    (dict(rows=-1), INVALID), (dict(in_dt=2), UNSUPPORTED), (dict(dy=None), INVALID), (dict(x=None), INVALID),
    (dict(dW=None), INVALID), (dict(off=None), INVALID), (dict(lddy=24), INVALID), (dict(ldx=68), MISALIGNED),
    (dict(dW=P + 2), MISALIGNED), (dict(E=0), OK), (dict(N=0), OK), (dict(K=0), OK),
])
def test_routed_wgrad_refuses(L, kw, want):
    assert _wgrad(L, **kw) == want


def test_workspace_sizes(L):
    b = _rows.workspace_bytes
    assert b("gemm_lora_workspace", 0, 32, 64, 3, 16) == (OK, 0)
    assert b("gemm_lora_workspace", 8, 32, 60, 3, 16)[0] == UNSUPPORTED
    assert L.gemm_lora_workspace(8, 32, 64, 3, 16, None) == INVALID
    # no adapters: only what the projection's K splits need
    assert b("gemm_lora_workspace", 512, 4096, 4096, 0, 0)[1] < b("gemm_lora_workspace", 512, 4096, 4096, 3, 16)[1]
    assert b("gemm_lora_backward_workspace", 0, 32, 64, 3, 16) == (OK, 0)
    assert b("gemm_lora_backward_workspace", 8, 36, 64, 3, 16)[0] == UNSUPPORTED
    assert b("gemm_lora_backward_workspace", 8, 32, 64, 1025, 16)[0] == UNSUPPORTED
    assert b("gemm_route_workspace", 8, 8, 9)[0] == UNSUPPORTED
    for T in (0, 1, 64, 65, 100000):
        st, n = b("gemm_route_workspace", T, 64, 8)
        assert st == OK and 0 < n < 1 << 20
    for M in (1, 31, 500, 5000, 1 << 20):
        for fn in ("gemm_lora_workspace", "gemm_lora_backward_workspace"):
            st, n = b(fn, M, 4096, 4096, 8, 64)
            assert st == OK and n % 256 == 0 and n >= M * 64 * 4


def test_cleared_words_of_the_largest_grid(L, tmp_path):
    """Which counters a thread of the low-rank products' kernels clears, at the most rows that are
    accepted (below 2^30; 64 a block of 256 threads, two products of K splits): a number past 2^31
    must not come out negative, below every count, nor a step of 2^32 as zero."""
    import subprocess
    from dense_gemm_nt_amd import build
    assert _lora(L, _adapters(), M=1 << 30) == UNSUPPORTED and _lora(L, _adapters(), M=(1 << 30) - 1) == INVALID
    src = tmp_path / "walk.cpp"
    src.write_text('''
#include <cstdio>
#include <initializer_list>
#include "rows_index.hpp"
int main()
{
    const uint32_t gx = ((1u << 30) - 1 + 63) / 64;
    for (uint32_t gz : {1u, 2u, 8u, 32u})
        for (uint32_t x : {0u, 1u << 23, gx - 1})
            for (uint32_t z : {0u, gz - 1}) {
                const gnt::Walk w = gnt::clear_walk(x, 0, z, gx, 1, gz, 256, 255);
                printf("%u %u %u %lld %lld\\n", x, z, gz, (long long)w.first, (long long)w.step);
            }
}
''')
    exe = str(tmp_path / "walk")
    subprocess.run(["g++", "-std=c++17", "-I" + build.ROWS, str(src), "-o", exe], check=True)
    gx = (1 << 24)
    out = subprocess.run([exe], check=True, capture_output=True, text=True).stdout.split("\n")[:-1]
    assert len(out) == 24
    for line in out:
        x, z, gz, first, step = map(int, line.split())
        assert first == (z * gx + x) * 256 + 255 and step == gx * gz * 256
    # and the kernels go by it: nothing else in them writes counters
    text = open(os.path.join(build.ROWS, "rows_lora.hip")).read()
    assert text.count("pair.counters[") == 1 and text.count("    clear_counters(pair);") == 2
