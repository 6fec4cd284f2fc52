"""The gated block and its gradients against their formulas in 64 bits."""
import pytest
import torch

from oracle import layer as o
from tests.rows_util import TINY, U, check, half_step, randn, rounded

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF16, FP16, FP32 = torch.bfloat16, torch.float16, torch.float32
ACTS = ("silu", "gelu", "relu")

# M, F, K: each tile, K splits summed in the kernel and by a second pass, edges
SIZES = [
    (1, 1, 8), (1, 520, 64), (1, 512, 4096), (3, 77, 1032), (33, 1001, 264), (64, 9000, 72), (70, 515, 2056),
    (128, 4096, 136), (200, 1027, 4104), (256, 333, 264), (300, 4100, 264), (512, 1024, 8192), (257, 2049, 520),
    (777, 1408, 2048), (640, 129, 1400), (1025, 2500, 72), (700, 2800, 328), (1600, 700, 2600), (260, 8, 2600),
    (1868, 4739, 576), (1113, 6538, 528),       # the last pass's rows, and columns, apart
]


def _operands(M, F, K, dt, seed=0):
    return (randn(M, K, seed=seed, dtype=dt), randn(F, K, seed=seed + 1, dtype=dt, std=K ** -0.5),
            randn(F, K, seed=seed + 2, dtype=dt, std=K ** -0.5))


def _sums(x, W, K):
    """Error bound of an FP32 sum x W^T."""
    return (K + 64) * U * (x.double().abs() @ W.double().abs().t())


def _value_err(g, a, eg, act):
    """Of act(g) from g within eg: |act'| <= 1.13, and the formula's own roundings (the
    exponential's argument and result, the reciprocal, the polynomial)."""
    if act == "relu":
        return eg
    rel = (g.abs() + 4) * 2.0 ** -22 if act == "silu" else 2.0 ** -20 + g * g * 2.0 ** -22
    return 1.13 * eg + rel * a.abs() + 1e-36


def _forward_bound(x, Wg, Wu, g, u, act, out):
    K = x.shape[1]
    eg, eu = _sums(x, Wg, K), _sums(x, Wu, K)
    a = o.gate(g, act)[0]
    ea = _value_err(g, a, eg, act)
    err = ea * u.abs() + (a.abs() + ea) * eu + 2.0 ** -23 * (a * u).abs()
    return rounded(a * u, err, out)


def _backward_bounds(dh, x, Wg, Wu, g, u, act, dt, dx_dt, g_dt):
    K, F, M = x.shape[1], Wg.shape[0], x.shape[0]
    d = dh.double()
    eg, eu = _sums(x, Wg, K), _sums(x, Wu, K)
    a, slope = o.gate(g, act)
    ea = _value_err(g, a, eg, act)
    # |act''| <= 0.8; the slope's own roundings
    es = 0.8 * eg + 2.0 ** -20 * (1 + g.abs())
    if act == "relu":                           # a sum near the corner may fall on its other side
        es = torch.where(g.abs() <= eg, 1.0, 0.0).double()
    dg, du = d * u * slope, d * a
    fine = TINY[dt] * float(d.abs().max()) if dt == FP16 and d.numel() else TINY[dt]
    edg = d.abs() * (u.abs() * es + (slope.abs() + es) * eu) + 2.0 ** -22 * dg.abs()
    edu = d.abs() * ea + 2.0 ** -22 * du.abs()
    edg = edg + half_step(dt) * (dg.abs() + edg) + fine
    edu = edu + half_step(dt) * (du.abs() + edu) + fine
    wg, wu, xa = Wg.double().abs(), Wu.double().abs(), x.double().abs()
    dx_err = edg @ wg + edu @ wu + (2 * F + 64) * U * (dg.abs() @ wg + du.abs() @ wu)
    wg_err = edg.t() @ xa + (M + 64) * U * (dg.abs().t() @ xa)
    wu_err = edu.t() @ xa + (M + 64) * U * (du.abs().t() @ xa)
    return (lambda r: rounded(r, dx_err, dx_dt)), (lambda r: rounded(r, wg_err, g_dt)), (lambda r: rounded(r, wu_err, g_dt))


@pytest.mark.parametrize("M,F,K", SIZES)
@pytest.mark.parametrize("dt,out,act", [(BF16, BF16, "silu"), (FP16, FP32, "gelu"), (BF16, FP16, "relu")])
def test_gated(M, F, K, dt, out, act):
    import dense_gemm_nt_amd as g
    x, Wg, Wu = _operands(M, F, K, dt)
    h = g.gemm_gated(x.to(DEV), Wg.to(DEV), Wu.to(DEV), activation=act, out_dtype=out)
    ref, gs, us = o.gated(x, Wg, Wu, act)
    check(h, ref, _forward_bound(x, Wg, Wu, gs, us, act, out), "h")


@pytest.mark.parametrize("M,F,K", SIZES)
@pytest.mark.parametrize("dt,xdt,gdt,act", [(BF16, BF16, FP32, "silu"), (FP16, FP32, FP16, "gelu"),
                                            (FP16, FP16, FP32, "relu")])
def test_gradients(M, F, K, dt, xdt, gdt, act):
    import dense_gemm_nt_amd as g
    x, Wg, Wu = _operands(M, F, K, dt, seed=5)
    dh = randn(M, F, seed=9, dtype=dt, std=0.1)
    got = g.gemm_gated_backward(dh.to(DEV), x.to(DEV), Wg.to(DEV), Wu.to(DEV), activation=act, grad_dtype=gdt,
                                dx_dtype=xdt)
    ref = o.gated_backward(dh, x, Wg, Wu, act)
    _, gs, us = o.gated(x, Wg, Wu, act)
    bounds = _backward_bounds(dh, x, Wg, Wu, gs, us, act, dt, xdt, gdt)
    for name, y, r, b in zip(("dx", "dWg", "dWu"), got, ref, bounds):
        check(y, r, b(r), name)


@pytest.mark.parametrize("M,F,K", SIZES)
@pytest.mark.parametrize("dt", [BF16, FP16])
def test_small_integers_are_exact(M, F, K, dt):
    """With ReLU, x and the weights in -1 .. 1 and mostly zero, and dh in -2 .. 2, every
    product, sum and rounding is exact: the bits have to be the formula's, so a row or column
    taken twice, left out or exchanged shows whatever its size."""
    import dense_gemm_nt_amd as g
    gen = torch.Generator().manual_seed(M + F + K)

    def ints(*shape, keep):
        v = torch.randint(-1, 2, shape, generator=gen) * (torch.rand(*shape, generator=gen) < keep)
        return v.to(dt)
    keep = min(0.5, (40.0 / K) ** 0.5)
    x, Wg, Wu = ints(M, K, keep=keep), ints(F, K, keep=keep), ints(F, K, keep=keep)
    dh = torch.randint(-2, 3, (M, F), generator=gen).to(dt)
    dev = [t.to(DEV) for t in (dh, x, Wg, Wu)]
    ref, gs, us = o.gated(x, Wg, Wu, "relu")
    assert float(gs.abs().max()) <= 64 and float(us.abs().max()) <= 64       # 2 * 64 fits 8 bits
    h = g.gemm_gated(*dev[1:], activation="relu", out_dtype=FP32)
    assert torch.equal(h.cpu().double(), ref)
    grads = g.gemm_gated_backward(*dev, activation="relu", grad_dtype=FP32, dx_dtype=FP32)
    for name, y, r in zip(("dx", "dWg", "dWu"), grads, o.gated_backward(dh, x, Wg, Wu, "relu")):
        assert float(r.abs().max() if r.numel() else 0.0) < 2 ** 24
        assert torch.equal(y.cpu().double(), r), name
