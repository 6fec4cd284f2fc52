"""Quantization and the product in 8-bit integers against their formulas in 64 bits."""
import pytest
import torch

from oracle import layer as o
from tests.rows_util import U, check, randn, rounded

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF16, FP16, FP32 = torch.bfloat16, torch.float16, torch.float32


def _codes(*shape, seed, lo=-128, hi=128):
    return torch.randint(lo, hi, shape, generator=torch.Generator().manual_seed(seed)).to(torch.int8)


def _scales(n, seed):
    return torch.rand(n, generator=torch.Generator().manual_seed(seed)) * 0.02 + 1e-4


@pytest.mark.parametrize("M,K", [(1, 1), (1, 16), (5, 100), (3, 2048), (9, 2049), (2, 8192), (2, 8200), (3, 20011), (1000, 512),
                                 (70, 4096), (1, 28672)])
@pytest.mark.parametrize("dt", [BF16, FP16, FP32])
def test_quantize(M, K, dt):
    import dense_gemm_nt_amd as g
    x = (randn(M, K, seed=M + K) * torch.exp(randn(M, 1, seed=M))).to(dt)
    codes, scale = g.quantize_int8(x.to(DEV))
    rc, rs = o.quantize(x)
    assert codes.dtype == torch.int8 and scale.dtype == FP32
    assert torch.equal(scale.cpu(), rs) and torch.equal(codes.cpu(), rc)


SIZES = [(1, 1, 16), (1, 8192, 8192), (3, 77, 1040), (33, 1001, 272), (64, 9000, 80), (70, 515, 4112), (128, 4096, 144),
         (200, 1027, 8208), (256, 333, 272), (300, 4100, 528), (512, 1024, 16384), (257, 2049, 1040), (777, 1408, 2048),
         (640, 129, 1392), (1025, 5000, 80), (700, 5600, 656), (2, 3, 131056), (2, 1030, 2064),
         (1868, 9480, 1152), (1113, 13080, 1056)]


@pytest.mark.parametrize("M,N,K", SIZES)
@pytest.mark.parametrize("out", [BF16, FP16, FP32])
def test_int8(M, N, K, out):
    import dense_gemm_nt_amd as g
    A, B, sa, sb = _codes(M, K, seed=1), _codes(N, K, seed=2), _scales(M, 3), _scales(N, 4)
    y = g.gemm_int8(A.to(DEV), B.to(DEV), sa.to(DEV), sb.to(DEV), out_dtype=out)
    ref, s = o.int8(A, B, sa, sb)
    # a K split's sum, two products and the splits' additions, each within 2^-23 of what they
    # round (at most 16 splits)
    check(y, ref, rounded(ref, 20 * U * s, out), "y")


@pytest.mark.parametrize("M,N,K", SIZES)
def test_int8_exact(M, N, K):
    """Powers of two as scales and sums below 2^24: every bit is the formula's."""
    import dense_gemm_nt_amd as g
    A, B = _codes(M, K, seed=5, lo=-4, hi=5), _codes(N, K, seed=6, lo=-4, hi=5)
    sa = 2.0 ** _codes(M, seed=7, lo=-5, hi=6).float()
    sb = 2.0 ** _codes(N, seed=8, lo=-5, hi=6).float()
    y = g.gemm_int8(A.to(DEV), B.to(DEV), sa.to(DEV), sb.to(DEV), out_dtype=FP32)
    assert torch.equal(y.cpu().double(), o.int8(A, B, sa, sb)[0])
