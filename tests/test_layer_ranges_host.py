"""The layer products' workspaces, against what their parts need; no device."""
import ctypes

import pytest

from dense_gemm_nt_amd import _layer, _lib

BF16, FP16, FP32 = 0, 1, 2
OK, INVALID, UNSUPPORTED = 0, 1, 2


@pytest.fixture(scope="module", autouse=True)
def library():
    from dense_gemm_nt_amd import build
    if build.stale():
        build.build()
    if build.stale_layer():
        build.build_layer()
    return _layer.lib()


def size(fn, *a):
    st, n = _layer.workspace_bytes(fn, *a)
    assert st == OK, (fn, a, st)
    return n


@pytest.mark.parametrize("M,F,K", [(1, 1, 8), (1000, 1001, 64), (777, 1408, 2048), (8192, 8192, 4096), (100000, 40, 16)])
def test_gradients_of_each_type(M, F, K):
    """One copy of both sums' gradients, or of FP16 two and the units; without a type the larger."""
    one = M * ((F + 7) // 8 * 16) * 2                      # whole groups of eight of each
    b, f = (size("gemm_gated_backward_workspace_of", M, F, K, dt) for dt in (BF16, FP16))
    assert b >= one and f >= b + one + 2 * M + 2 * F + 4 * (M + F)
    assert size("gemm_gated_backward_workspace", M, F, K) == f


def test_gradients_workspace_refuses():
    w = _layer.workspace_bytes
    assert w("gemm_gated_backward_workspace_of", 8, 8, 8, FP32)[0] == UNSUPPORTED
    assert w("gemm_gated_backward_workspace_of", -1, 8, 8, FP16)[0] == INVALID
    assert w("gemm_gated_backward_workspace_of", 8, 8, 4, BF16)[0] == UNSUPPORTED
    assert _layer.lib().gemm_gated_backward_workspace_of(8, 8, 8, BF16, None) == INVALID
    # no rows or columns: no units
    for a in ((0, 8, 16), (3, 0, 16), (0, 0, 0)):
        assert size("gemm_gated_backward_workspace_of", *a, FP16) == size("gemm_gated_backward_workspace_of", *a, BF16)


def _splits(M, N, K):
    """The least that K splits of the library's own plan need: their partials, whole tiles' where the
    kernel sums them, and a counter a tile."""
    p = _lib.GemmPlan()
    assert _lib.lib().gemm_plan(M, N, K, BF16, FP32, ctypes.byref(p)) == OK and p.splits > 1
    if p.inreduce:
        return p.splits * p.tiles * p.block_m * p.block_n * 4 + 4 * p.tiles
    return p.splits * M * N * 4


@pytest.mark.parametrize("M,F,K", [(1, 512, 4096), (33, 1024, 8192), (64, 2048, 4096), (100, 1408, 8192)])
def test_splits_of_a_gated_block(M, F, K):
    """(up to 128 rows its plan is the library's, of both weights' columns)"""
    assert size("gemm_gated_workspace", M, F, K) >= _splits(M, 2 * F, K)


@pytest.mark.parametrize("M,N,K", [(3, 1024, 16384), (33, 1024, 16384), (100, 2816, 16384), (16, 8192, 8192)])
def test_splits_of_an_integer_product(M, N, K):
    """(two codes to an element of the tiles)"""
    assert size("gemm_int8_workspace", M, N, K) >= _splits(M, N, K // 2)


@pytest.mark.parametrize("B,m,n", [(1, 1000, 2047), (3, 1000, 2047), (3, 2047, 1000), (12, 2048, 768), (1, 1, 1)])
def test_updates(B, m, n):
    """Of each matrix X's first parts twice and its second, and two squares, in whole 64s; of a stack
    that many of all."""
    r, k = (-(-min(m, n) // 64) * 64, -(-max(m, n) // 64) * 64)
    got = size("gemm_orthogonalize_workspace", B, m, n)
    assert got >= B * (3 * r * k + 2 * r * r) * 2 + 8 * B
    assert got < B * (5 * r * k + 2 * r * r) * 2 + (160 << 20)      # (X transposed twice; bounded partials)


def test_nothing_to_do_needs_nothing():
    for a in ((0, 8, 16), (3, 0, 16), (0, 0, 0)):
        assert size("gemm_gated_workspace", *a) == 0 and size("gemm_int8_workspace", *a) == 0
        assert size("gemm_orthogonalize_workspace", *a) == 0
        assert size("gemm_gated_backward_workspace", *a) == 0
    assert size("gemm_orthogonalize_workspace", 3, 8, 0) == 0
    # K = 0: the results are written, from nothing
    assert size("gemm_gated_workspace", 3, 8, 0) == 0 and size("gemm_int8_workspace", 3, 8, 0) == 0
