"""The layer products' workspaces, against what their parts need; no device."""
import pytest

from dense_gemm_nt_amd import _layer

BF16, FP16, FP32 = 0, 1, 2
OK, INVALID, UNSUPPORTED = 0, 1, 2


@pytest.fixture(scope="module", autouse=True)
def library():
    from dense_gemm_nt_amd import build
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
