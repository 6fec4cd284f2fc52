"""The layer products at the ends of their ranges."""
import math

import pytest
import torch

from oracle import layer as o
from tests.rows_util import U, check, half_step, randn, rounded
from tests.test_layer_gated_gpu import SIZES, _operands, _sums, _value_err
from tests.test_layer_int8_gpu import SIZES as INT8_SIZES
from tests.test_layer_int8_gpu import _codes, _scales

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF16, FP16, FP32 = torch.bfloat16, torch.float16, torch.float32


# ------------------------------------------------------------------ FP16 gradients

def _bounds(dh, x, Wg, Wu, act):
    """Bounds of FP32 (dx, dWg, dWu) of FP16 operands, and the results.  dg and du are rounded to
    FP16 twice, in units of their row for dx and of their column for the weights' gradients: a unit
    brings the largest magnitude of the row's (column's) dh times B below 2^15 and above 2^13
    (both rounded up to powers of two), B = 1.15 max ||x|| max ||W|| at least any |u act'(g)| or
    |act(g)|; so an absolute 2^-25 of FP16's is at most 2^-38 of that product."""
    K, F, M = x.shape[1], Wg.shape[0], x.shape[0]
    d = dh.double()
    _, g, u = o.gated(x, Wg, Wu, act)
    eg, eu = _sums(x, Wg, K), _sums(x, Wu, K)
    a, slope = o.gate(g, act)
    ea = _value_err(g, a, eg, act)
    es = 0.8 * eg + 2.0 ** -20 * (1 + g.abs())          # |act''| <= 0.8; the slope's own roundings
    if act == "relu":                                   # a sum near the corner may fall on its other side
        es = torch.where(g.abs() <= eg, 1.0, 0.0).double()
    dg, du = d * u * slope, d * a
    edg = d.abs() * (u.abs() * es + (slope.abs() + es) * eu) + 2.0 ** -22 * dg.abs()
    edu = d.abs() * ea + 2.0 ** -22 * du.abs()
    B = 1.15 * float(x.double().norm(dim=1).max()) * float(torch.cat([Wg, Wu]).double().norm(dim=1).max())

    def held(e, v, most):
        return e + half_step(FP16) * (v.abs() + e) + 2.0 ** -38 * B * most
    row, col = d.abs().amax(1, keepdim=True), d.abs().amax(0, keepdim=True)
    wg, wu, xa = Wg.double().abs(), Wu.double().abs(), x.double().abs()
    dx_err = held(edg, dg, row) @ wg + held(edu, du, row) @ wu + (2 * F + 64) * U * (dg.abs() @ wg + du.abs() @ wu)
    wg_err = held(edg, dg, col).t() @ xa + (M + 64) * U * (dg.abs().t() @ xa)
    wu_err = held(edu, du, col).t() @ xa + (M + 64) * U * (du.abs().t() @ xa)
    ref = o.gated_backward(dh, x, Wg, Wu, act)[:3]
    return ref, [rounded(r, e, FP32) for r, e in zip(ref, (dx_err, wg_err, wu_err))]


def _check_gradients(dh, x, Wg, Wu, act, what):
    import dense_gemm_nt_amd as g
    got = g.gemm_gated_backward(*(t.to(DEV) for t in (dh, x, Wg, Wu)), activation=act, grad_dtype=FP32, dx_dtype=FP32)
    ref, bounds = _bounds(dh, x, Wg, Wu, act)
    for name, y, r, b in zip(("dx", "dWg", "dWu"), got, ref, bounds):
        check(y, r, b, "%s, %s" % (name, what))


@pytest.mark.parametrize("act", ["silu", "gelu", "relu"])
@pytest.mark.parametrize("M,F,K", [(20, 77, 136), (130, 264, 136), (300, 520, 2056)])
def test_fp16_gradients_of_large_sums(M, F, K, act):
    """Sums past 2^15 beside a dh of 1e-6: no gradient is near FP16's end."""
    x, Wg, Wu = randn(M, K, seed=1, std=200.0, dtype=FP16), randn(F, K, seed=2, std=K ** -0.5 / 200, dtype=FP16), \
        randn(F, K, seed=3, std=350 * K ** -0.5, dtype=FP16)
    dh = randn(M, F, seed=4, std=1e-6, dtype=FP16)
    assert float(o.gated(x, Wg, Wu, act)[2].abs().max()) > 1e5
    _check_gradients(dh, x, Wg, Wu, act, "large up values")
    Wg, Wu = Wu, Wg
    _check_gradients(dh, x, Wg, Wu, act, "large gates")


@pytest.mark.parametrize("M,F,K", SIZES)
def test_fp16_gradients_beside_a_large_entry(M, F, K):
    """One entry of dh at 30000 leaves the other rows and columns their own 1e-3."""
    x, Wg, Wu = _operands(M, F, K, FP16, seed=5)
    dh = randn(M, F, seed=9, dtype=FP16, std=1e-3)
    dh[M // 2, F // 3] = 30000.0
    _check_gradients(dh, x, Wg, Wu, "silu", "one entry")


@pytest.mark.parametrize("M,F,K", [(16, 520, 64), (40, 100, 72), (130, 264, 136), (260, 1030, 520)])
@pytest.mark.parametrize("small", [1e-6, 1e-3])
def test_fp16_gradients_beside_a_large_row(M, F, K, small):
    x, Wg, Wu = _operands(M, F, K, FP16, seed=5)
    dh = randn(M, F, seed=9, std=small)
    dh[M // 2] = randn(F, seed=10, std=2e4).clamp(-6e4, 6e4)
    _check_gradients(dh.to(FP16), x, Wg, Wu, "gelu", "one row")
    dh = randn(M, F, seed=9, std=small)
    dh[:, F // 2] = randn(M, seed=10, std=2e4).clamp(-6e4, 6e4)
    _check_gradients(dh.to(FP16), x, Wg, Wu, "gelu", "one column")


@pytest.mark.parametrize("std", [1e-6, 1.0, 1e4])
@pytest.mark.parametrize("value", [math.nan, math.inf, -math.inf])
def test_fp16_gradients_beside_a_value_that_is_not_finite(std, value):
    """A NaN or infinity in dh reaches its own row of dx and its own column's weights, and leaves
    every other bit as it was."""
    import dense_gemm_nt_amd as g
    M, F, K = 70, 136, 72
    x, Wg, Wu = _operands(M, F, K, FP16)
    dh = randn(M, F, seed=4, std=std).clamp(-4 * std, 4 * std).to(FP16)
    bad = dh.clone()
    bad[5, 20] = value
    plain = dh.clone()
    plain[5, 20] = 0.0
    kw = dict(activation="silu", grad_dtype=FP32, dx_dtype=FP32)
    dx, a, b = (t.cpu() for t in g.gemm_gated_backward(*(t.to(DEV) for t in (plain, x, Wg, Wu)), **kw))
    bx, ba, bb = (t.cpu() for t in g.gemm_gated_backward(*(t.to(DEV) for t in (bad, x, Wg, Wu)), **kw))
    rows, cols = [m for m in range(M) if m != 5], [f for f in range(F) if f != 20]
    assert torch.equal(bx[rows], dx[rows]) and not bool(torch.isfinite(bx[5]).any())
    assert torch.equal(ba[cols], a[cols]) and torch.equal(bb[cols], b[cols])
    assert not bool(torch.isfinite(ba[20]).any()) and not bool(torch.isfinite(bb[20]).any())
    _check_gradients(plain, x, Wg, Wu, "silu", "beside it")


# ------------------------------------------------------------ the integer product

def _exact(A, B, sa, sb):
    """The definition: the exact sum to FP32, times scale_a, times scale_b."""
    s = A.double() @ B.double().t()                      # (below 2^31: exact)
    return s.float() * sa[:, None] * sb


@pytest.mark.parametrize("M,N,K", INT8_SIZES)
def test_int8_is_the_exact_sum_whatever_the_splits(M, N, K):
    import dense_gemm_nt_amd as g
    A, B, sa, sb = _codes(M, K, seed=1), _codes(N, K, seed=2), _scales(M, 3), _scales(N, 4)
    y = g.gemm_int8(A.to(DEV), B.to(DEV), sa.to(DEV), sb.to(DEV), out_dtype=FP32)
    assert torch.equal(y.cpu(), _exact(A, B, sa, sb))


@pytest.mark.parametrize("M", [1, 3, 70, 200, 300])
def test_int8_splits_of_a_sum_that_cancels(M):
    """The halves of K cancel up to a few codes; with scales of 1e29 either half is past FP32's end."""
    import dense_gemm_nt_amd as g
    N, K = 300, 16384
    A = torch.full((M, K), 127, dtype=torch.int8)
    B = torch.full((N, K), 127, dtype=torch.int8)
    B[:, K // 2:] = -127
    B[:, 5] = _codes(N, seed=1)
    sa, sb = torch.full((M,), 1e29), torch.full((N,), 100.0)
    y = g.gemm_int8(A.to(DEV), B.to(DEV), sa.to(DEV), sb.to(DEV), out_dtype=FP32)
    assert bool(torch.isfinite(y).all()) and torch.equal(y.cpu(), _exact(A, B, sa, sb))
    y = g.gemm_int8(A.to(DEV), B.to(DEV), torch.full((1,), math.inf, device=DEV), sb.to(DEV), out_dtype=FP32)
    assert torch.equal(y.cpu().nan_to_num(nan=0.5), _exact(A, B, torch.full((M,), math.inf), sb).nan_to_num(nan=0.5))


# ------------------------------------------------------------------- the update

@pytest.mark.parametrize("steps", [0, 1, 2, 5])
@pytest.mark.parametrize("value", [math.nan, math.inf, -math.inf])
def test_an_update_of_what_is_not_finite(steps, value):
    """The whole matrix is NaN after any number of steps, and its neighbours in the stack are not."""
    import dense_gemm_nt_amd as g
    for shape in ((3, 70, 130), (3, 200, 40)):
        S = randn(*shape, seed=1)
        want = g.orthogonalize(S.to(DEV), steps=steps, out_dtype=FP32).cpu()
        S[1, 3, 4] = value
        got = g.orthogonalize(S.to(DEV), steps=steps, out_dtype=FP32).cpu()
        assert bool(got[1].isnan().all())
        assert torch.equal(got[0], want[0]) and torch.equal(got[2], want[2])


# ------------------------------------------------- more values than a launch has threads

@pytest.mark.parametrize("M,K", [((1 << 26) + 3, 8), ((1 << 22) + 5, 24), ((1 << 20) + 5, 2056)])
def test_quantize_rows_of_more_than_a_launch(M, K):
    """Past 2^32 threads at a thread a value or so, and past the blocks of one launch."""
    import dense_gemm_nt_amd as g
    rows = randn(257, K, seed=1, dtype=BF16).to(DEV)
    x = rows.repeat(-(-M // 257), 1)[:M]
    codes, scale = g.quantize_int8(x)
    rc, rs = o.quantize(rows.cpu())
    rc, rs = rc.to(DEV), rs.to(DEV)
    whole = M // 257 * 257
    assert bool((codes[:whole].view(-1, 257, K) == rc).all()) and bool((scale[:whole].view(-1, 257) == rs).all())
    assert torch.equal(codes[whole:], rc[:M - whole]) and torch.equal(scale[whole:], rs[:M - whole])


def test_update_of_more_values_than_a_launch():
    """No steps: the scaled matrix itself, 2^32 values and some."""
    import dense_gemm_nt_amd as g
    m, n = 4097, 1 << 20
    G = torch.zeros(m, n, dtype=BF16, device=DEV)
    G[0, 0], G[m - 1, n - 1], G[2048, 77], G[m - 1, 0] = 1.0, -2.0, 2.0, 4.0      # of norm 5
    U = g.orthogonalize(G, steps=0, eps=0.0, out_dtype=FP32)
    want = {(0, 0): 0.2, (m - 1, n - 1): -0.4, (2048, 77): 0.4, (m - 1, 0): 0.8}
    for at, v in want.items():
        assert abs(float(U[at]) - v) <= 2.0 ** -21 * abs(v), at
        U[at] = 0.0
    for i in range(0, m, 512):
        assert not bool(U[i:i + 512].any())


# ------------------------------------------------------------- pieces and largest sizes

@pytest.mark.parametrize("M,N,K", [(1868, 9480, 144), (1113, 13080, 144)])
def test_int8_pieces_have_their_own_bias_and_prior_rows(M, N, K):
    """The rows, and columns, of a last pass apart: scales, biases and C_old from where they begin."""
    import dense_gemm_nt_amd as g
    A, B = _codes(M, K, seed=5, lo=-4, hi=5).to(DEV), _codes(N, K, seed=6, lo=-4, hi=5).to(DEV)
    sa, sb = 2.0 ** (torch.arange(M, device=DEV) % 5 - 2).float(), 2.0 ** (torch.arange(N, device=DEV) % 7 - 3).float()
    bn, bm = torch.arange(N, device=DEV) % 64 / 8.0, torch.arange(M, device=DEV) % 128 / 4.0
    old = (torch.arange(M, device=DEV)[:, None] * 3 + torch.arange(N, device=DEV)) % 256 / 4.0
    y = (A.float() @ B.float().t()) * sa[:, None] * sb          # (of few bits: exact)
    for bias, along, add in ((bn, "n", bn), (bm, "m", bm[:, None])):
        out = old.clone()
        g.gemm_int8(A, B, sa, sb, out=out, alpha=0.5, beta=2.0, bias=bias, bias_along=along)
        assert torch.equal(out, 0.5 * y + 2.0 * old + add)


@pytest.mark.parametrize("dt", [BF16, FP16])
def test_the_largest_block(dt):
    """F one below its limit: dg and du in rows of 2^22 values.  Of small integers, so exact."""
    import dense_gemm_nt_amd as g
    M, F, K = 300, (1 << 21) - 1, 16
    gen = torch.Generator(device=DEV).manual_seed(1)

    def ints(*shape):
        return torch.randint(-1, 2, shape, generator=gen, device=DEV).to(dt)
    x, Wg, Wu, dh = ints(M, K), ints(F, K), ints(F, K), ints(M, F)
    h = g.gemm_gated(x, Wg, Wu, activation="relu")
    dx, a, b = g.gemm_gated_backward(dh, x, Wg, Wu, activation="relu", grad_dtype=FP32, dx_dtype=FP32)
    want = torch.zeros(M, K, dtype=torch.float64, device=DEV)
    for f in range(0, F, 1 << 18):
        c = slice(f, min(F, f + (1 << 18)))
        gate, up, d = x.float() @ Wg[c].float().t(), x.float() @ Wu[c].float().t(), dh[:, c].float()
        assert torch.equal(h[:, c].float(), gate.clamp(min=0) * up)
        dg, du = d * up * (gate > 0), d * gate.clamp(min=0)
        assert torch.equal(a[c], dg.t().contiguous() @ x.float()) and torch.equal(b[c], du.t().contiguous() @ x.float())
        want += (dg @ Wg[c].float() + du @ Wu[c].float()).double()
    assert float(want.abs().max()) < 2 ** 24 and torch.equal(dx.double(), want)
