"""The layer products' calls where they are easiest to get wrong: strides and given
results, values that are not finite, empty sizes, other streams, captured graphs,
offsets past 32 bits; and a whole feed-forward layer, trained, updated and served."""
import math

import pytest
import torch

from oracle import layer as o
from tests.rows_util import TINY, U, check, half_step, randn, rounded
from tests.test_layer_gated_gpu import _backward_bounds, _forward_bound, _operands
from tests.test_layer_int8_gpu import _codes, _scales

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF16, FP16, FP32 = torch.bfloat16, torch.float16, torch.float32
ABC = (3.4445, -4.7750, 2.0315)


def _wide(t, extra, lead=0, fill=math.nan):
    """The same values as a view of rows `extra` longer, `lead` from their start, the rest `fill`."""
    w = torch.full((t.shape[0], t.shape[1] + extra), fill, dtype=t.dtype, device=DEV) if t.is_floating_point() else \
        torch.full((t.shape[0], t.shape[1] + extra), 77, dtype=t.dtype, device=DEV)
    w[:, lead:lead + t.shape[1]] = t.to(DEV)
    return w[:, lead:lead + t.shape[1]]


# ------------------------------------------------- strides, results given by the caller

@pytest.mark.parametrize("M,F,K", [(3, 77, 136), (130, 515, 264), (600, 1300, 72)])
def test_gated_takes_views(M, F, K):
    import dense_gemm_nt_amd as g
    x, Wg, Wu = _operands(M, F, K, BF16)
    dh = randn(M, F, seed=3, dtype=BF16)
    d = [t.to(DEV) for t in (x, Wg, Wu)]
    v = [_wide(x, 24, 8), _wide(Wg, 8), _wide(Wu, 40, 16)]          # leading dimensions of their own
    for out_dt in (BF16, FP32):
        want = g.gemm_gated(*d, out_dtype=out_dt)
        assert torch.equal(g.gemm_gated(*v, out_dtype=out_dt), want)
        for lead, extra in ((1, 6), (8, 16)):                       # rows at any alignment
            big = torch.full((M + 2, F + extra), 5.0, dtype=out_dt, device=DEV)
            out = big[1:M + 1, lead:lead + F]
            assert g.gemm_gated(*v, out=out) is out
            assert torch.equal(out, want)
            big[1:M + 1, lead:lead + F] = 5.0
            assert bool((big == 5.0).all())                         # nothing beside it is touched
    want = g.gemm_gated_backward(dh.to(DEV), *d)
    for lead, extra in ((0, 0), (1, 3), (8, 8)):
        got = g.gemm_gated_backward(_wide(dh, extra, lead), *v)
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert g.gemm_gated_backward(dh.to(DEV), *d, need_dx=False)[0] is None
    only = g.gemm_gated_backward(dh.to(DEV), *d, need_weights=False)
    assert only[1] is None and only[2] is None and torch.equal(only[0], want[0])
    assert torch.equal(g.gemm_gated_backward(dh.to(DEV), *d, need_dx=False)[2], want[2])


def test_one_row_at_any_stride():
    import dense_gemm_nt_amd as g
    K, F = 72, 136
    Wg, Wu = randn(F, K, seed=1, dtype=BF16).to(DEV), randn(F, K, seed=2, dtype=BF16).to(DEV)
    B, sb = _codes(F, 80, seed=3).to(DEV), _scales(F, 4).to(DEV)
    for step in ((1 << 22) + 8, K + 3, 0):
        def row(cols, seed, dt):
            wide = torch.zeros(step + cols, dtype=dt, device=DEV)
            wide[:cols] = (randn(cols, seed=seed) * 30).to(dt).to(DEV)
            return wide.as_strided((1, cols), (step, 1)), wide[:cols].clone().view(1, cols)
        (x, x1), (dh, dh1), (q, q1) = row(K, 5, BF16), row(F, 6, BF16), row(80, 7, torch.int8)
        assert torch.equal(g.gemm_gated(x, Wg, Wu), g.gemm_gated(x1, Wg, Wu))
        for a, b in zip(g.gemm_gated_backward(dh, x, Wg, Wu), g.gemm_gated_backward(dh1, x1, Wg, Wu)):
            assert torch.equal(a, b)
        for a, b in zip(g.quantize_int8(x), g.quantize_int8(x1)):
            assert torch.equal(a, b)
        one = torch.ones(1, device=DEV)
        assert torch.equal(g.gemm_int8(q, B, one, sb), g.gemm_int8(q1, B, one, sb))
        assert torch.equal(g.orthogonalize(x), g.orthogonalize(x1))


@pytest.mark.parametrize("M,N,K", [(1, 1030, 4096), (2, 77, 2064), (3, 130, 272), (130, 515, 528), (600, 2600, 144)])
def test_int8_takes_views_and_epilogues(M, N, K):
    import dense_gemm_nt_amd as g
    A, B, sa, sb = _codes(M, K, seed=1), _codes(N, K, seed=2), _scales(M, 3), _scales(N, 4)
    a, b = _wide(A, 32, 16), _wide(B, 16)
    ref, s = o.int8(A, B, sa, sb)
    bound = 20 * U * s
    plain = g.gemm_int8(A.to(DEV), B.to(DEV), sa.to(DEV), sb.to(DEV), out_dtype=FP32)
    assert torch.equal(g.gemm_int8(a, b, sa.to(DEV), sb.to(DEV), out_dtype=FP32), plain)
    for lead, extra in ((1, 6), (8, 16)):
        big = torch.full((M + 2, N + extra), 5.0, device=DEV)
        out = big[1:M + 1, lead:lead + N]
        g.gemm_int8(a, b, sa.to(DEV), sb.to(DEV), out=out)
        assert torch.equal(out, plain)
        out.fill_(5.0)
        assert bool((big == 5.0).all())
    # one scale for all rows, or columns
    one = torch.full((1,), 0.5, device=DEV)
    assert torch.equal(g.gemm_int8(a, b, one, sb.to(DEV), out_dtype=FP32),
                       g.gemm_int8(a, b, one.expand(M).contiguous(), sb.to(DEV), out_dtype=FP32))
    assert torch.equal(g.gemm_int8(a, b, sa.to(DEV), one, out_dtype=FP32),
                       g.gemm_int8(a, b, sa.to(DEV), one.expand(N).contiguous(), out_dtype=FP32))
    # alpha y + beta C_old + bias, activation
    bn, bm, old = randn(N, seed=5), randn(M, seed=6), randn(M, N, seed=7)
    for bias, along, act, beta in ((bn, "n", "none", 0.0), (bm, "m", "relu", 0.5), (None, "n", "gelu", -1.5)):
        out = old.to(DEV)
        g.gemm_int8(a, b, sa.to(DEV), sb.to(DEV), out=out, alpha=0.75, beta=beta, bias=None if bias is None else bias.to(DEV),
                    bias_along=along, activation=act)
        add = 0 if bias is None else bias.double()[:, None] if along == "m" else bias.double()
        v = 0.75 * ref + beta * old.double() + add
        err = 0.75 * bound + 4 * U * (0.75 * s + (beta * old.double()).abs() + (abs(add) if bias is not None else 0))
        r = torch.clamp(v, min=0) if act == "relu" else o.gate(v, "gelu")[0] if act == "gelu" else v
        # |act'| <= 1.13, and the library's GELU is within 2^-22 |v| of the exact one
        check(out, r, rounded(r, 1.13 * err + (2.0 ** -21 * v.abs() if act == "gelu" else 0), FP32), "epilogue %s" % act)


def test_quantize_takes_views():
    import dense_gemm_nt_amd as g
    for dt in (BF16, FP16, FP32):
        for M, K in ((5, 77), (3, 2100), (4, 4096)):
            x = randn(M, K, seed=K, dtype=dt)
            want = [t.cpu() for t in g.quantize_int8(x.to(DEV))]
            for lead, extra in ((1, 3), (8, 24)):
                got = g.quantize_int8(_wide(x, extra, lead))
                assert all(torch.equal(a.cpu(), b) for a, b in zip(got, want))


def test_orthogonalize_takes_views_and_itself():
    import dense_gemm_nt_amd as g
    G = randn(100, 260, seed=1)
    want = g.orthogonalize(G.to(DEV), out_dtype=FP32)
    assert torch.equal(g.orthogonalize(_wide(G, 3, 1), out_dtype=FP32), want)
    big = torch.full((102, 267), 5.0, device=DEV)
    out = big[1:101, 3:263]
    g.orthogonalize(G.to(DEV), out=out)
    assert torch.equal(out, want)
    out.fill_(5.0)
    assert bool((big == 5.0).all())
    self = G.to(DEV)
    assert g.orthogonalize(self, out=self) is self and torch.equal(self, want)
    # tall, transposed on its way in and out
    T = G.t().contiguous().to(DEV)
    tall = g.orthogonalize(T, out_dtype=FP32)
    assert torch.equal(tall.t(), want)
    big = torch.full((262, 107), 5.0, dtype=BF16, device=DEV)
    g.orthogonalize(T, out=big[1:261, 5:105])
    assert torch.equal(big[1:261, 5:105], g.orthogonalize(T))
    # a stack whose matrices' rows alternate
    S = randn(3, 40, 72, seed=2).to(DEV)
    out = torch.zeros(40, 3, 72, device=DEV).transpose(0, 1)
    g.orthogonalize(S.transpose(0, 1).contiguous().transpose(0, 1), out=out)
    assert torch.equal(out, g.orthogonalize(S, out_dtype=FP32))
    with pytest.raises(ValueError):
        g.orthogonalize(S, out=torch.zeros(1, 40, 72, device=DEV).expand(3, 40, 72))
    with pytest.raises(ValueError):
        g.orthogonalize(G.t().to(DEV).t()[:, ::2])


# ------------------------------------------------------------- values and empty sizes

@pytest.mark.parametrize("act", ["silu", "gelu", "relu"])
def test_values_that_are_not_finite(act):
    import dense_gemm_nt_amd as g
    M, F, K = 40, 100, 72
    for dt in (BF16, FP16):
        x, Wg, Wu = _operands(M, F, K, dt)
        dh = randn(M, F, seed=4, dtype=dt)
        x[3, 5], x[7, 0], x[9, 1], x[9, 2] = math.inf, math.nan, -math.inf, math.inf
        Wg[11, 7], Wu[12, 8], Wu[13, 9] = math.inf, -math.inf, math.nan
        h = g.gemm_gated(x.to(DEV), Wg.to(DEV), Wu.to(DEV), activation=act, out_dtype=FP32).cpu().double()
        ref, gs, us = o.gated(x, Wg, Wu, act)
        assert torch.equal(h.isnan(), ref.isnan()) and torch.equal(h[ref.isinf()], ref[ref.isinf()])
        fine = torch.isfinite(ref)
        clean = [torch.nan_to_num(t, nan=0.0, posinf=0.0, neginf=0.0) for t in (x, Wg, Wu)]
        r2, g2, u2 = o.gated(*clean, act)
        rows = [m for m in range(M) if m not in (3, 7, 9)]
        cols = [f for f in range(F) if f not in (11, 12, 13)]
        bound = _forward_bound(*clean, g2, u2, act, FP32)
        check(h[rows][:, cols], r2[rows][:, cols], bound[rows][:, cols], "the rest")
        assert bool(fine[rows][:, cols].all())
        # dh: its rows' dx, and every weight's gradient that has them
        dx, dWg, dWu = g.gemm_gated_backward(dh.to(DEV), *(t.to(DEV) for t in clean), activation=act, dx_dtype=FP32)
        bad = dh.clone()
        bad[5, 20] = math.nan
        bx, bg, bu = g.gemm_gated_backward(bad.to(DEV), *(t.to(DEV) for t in clean), activation=act, dx_dtype=FP32)
        keep = [m for m in range(M) if m != 5]
        if dt == BF16:                                   # (FP16: a dh without a largest value is not scaled)
            assert torch.equal(bx[keep], dx[keep])
        assert bool(bx[5].isnan().all())
        nan_g = o.gated_backward(bad, *clean, act)[1].isnan()
        assert torch.equal(bg.cpu().isnan(), nan_g)


def test_large_and_small_gates():
    """act over its whole range: one-hot x and a weight of chosen values make the gate any number."""
    import dense_gemm_nt_amd as g
    v = torch.cat([torch.linspace(-30, 30, 481), torch.tensor([-1e4, -200.0, -104.0, -88.0, 88.0, 200.0, 1e4, 1e-6, -1e-6, 0.0, 3e38])])
    v = v.to(BF16)
    F = v.numel()
    x = torch.zeros(1, 8, dtype=BF16)
    x[0, 0] = 1.0
    Wg, Wu = torch.zeros(F, 8, dtype=BF16), torch.zeros(F, 8, dtype=BF16)
    Wg[:, 0], Wu[:, 0] = v, 1.0
    dh = torch.ones(1, F, dtype=BF16)
    for act in ("silu", "gelu", "relu"):
        h = g.gemm_gated(x.to(DEV), Wg.to(DEV), Wu.to(DEV), activation=act, out_dtype=FP32)[0].cpu().double()
        a, slope = o.gate(v.double(), act)
        rel = 2.0 ** -20 + v.double() ** 2 * 2.0 ** -22 if act == "gelu" else (v.double().abs() + 4) * 2.0 ** -22
        # (exp(88.8) is infinite in FP32: silu is zero where it is below 1e-36)
        assert bool(((h - a).abs() <= rel * a.abs() + 1e-36).all()), act
        # the same through the gradients: dWg[f, 0] = dh u act'(v), dWu[f, 0] = dh act(v)
        _, dWg, dWu = g.gemm_gated_backward(dh.to(DEV), x.to(DEV), Wg.to(DEV), Wu.to(DEV), activation=act, grad_dtype=FP32)
        for got, want in ((dWg[:, 0].cpu().double(), slope), (dWu[:, 0].cpu().double(), a)):
            err = 2.0 ** -20 * (1 + v.double().abs().clamp(max=64)) if got is not None and want is slope else rel * a.abs() + 1e-36
            fine = want.abs() < 3e38
            b = rounded(want, err + half_step(BF16) * (want.abs() + err) + TINY[BF16], FP32)
            assert bool(((got - want).abs() <= b)[fine].all()), act


@pytest.mark.parametrize("scale", [2.0 ** -24, 1e-6, 1e-3, 1.0, 3e4])
def test_fp16_gradients_of_any_scale(scale):
    """Gradients of 1e-6 lose nothing: they are taken in units of dh's largest value."""
    import dense_gemm_nt_amd as g
    M, F, K = 130, 264, 136
    x, Wg, Wu = _operands(M, F, K, FP16)
    dh = (randn(M, F, seed=8).clamp(-2, 2) * scale).to(FP16)
    got = g.gemm_gated_backward(dh.to(DEV), x.to(DEV), Wg.to(DEV), Wu.to(DEV), activation="silu", grad_dtype=FP32, dx_dtype=FP32)
    ref = o.gated_backward(dh, x, Wg, Wu, "silu")
    _, gs, us = o.gated(x, Wg, Wu, "silu")
    for name, y, r, b in zip(("dx", "dWg", "dWu"), got, ref, _backward_bounds(dh, x, Wg, Wu, gs, us, "silu", FP16, FP32, FP32)):
        check(y, r, b(r), "%s at %g" % (name, scale))


def test_quantize_specials():
    import dense_gemm_nt_amd as g
    for dt in (BF16, FP16, FP32):
        x = randn(9, 2056, seed=1, dtype=dt)
        x[1] = 0
        x[2, 7], x[3, 2055], x[4, 0] = math.inf, -math.inf, math.nan
        x[5] = torch.finfo(dt).tiny * torch.sign(randn(2056, seed=2)).to(dt)
        x[6] = torch.finfo(dt).max
        x[7] = (torch.arange(2056) % 255 - 127).to(dt) / 2            # every tie
        x[8] = torch.finfo(dt).smallest_normal / 64 * (torch.arange(2056) % 3 - 1)
        codes, scale = (t.cpu() for t in g.quantize_int8(x.to(DEV)))
        rc, rs = o.quantize(x)
        assert torch.equal(scale.isnan(), rs.isnan()) and torch.equal(scale[~rs.isnan()], rs[~rs.isnan()])
        assert torch.equal(codes, rc)
    # what is not finite reaches its own rows' products only
    x = randn(4, 2048, seed=3)
    x[2, 9] = math.nan
    codes, scale = g.quantize_int8(x.to(DEV))
    B = _codes(70, 2048, seed=4).to(DEV)
    y = g.gemm_int8(codes, B, scale, torch.ones(70, device=DEV), out_dtype=FP32)
    assert bool(y[2].isnan().all()) and not bool(y[[0, 1, 3]].isnan().any())


def test_int8_at_its_largest():
    import dense_gemm_nt_amd as g
    K = (1 << 17) - 16
    for M in (1, 3, 200):
        A, B = torch.full((M, K), -128, dtype=torch.int8), torch.full((5, K), -128, dtype=torch.int8)
        B[1] = 127
        y = g.gemm_int8(A.to(DEV), B.to(DEV), torch.ones(1, device=DEV), torch.ones(1, device=DEV), out_dtype=FP32).cpu()
        # (each split's sum is rounded to 24 bits, and so are the splits' sums)
        want = torch.tensor([K * 16384.0, -K * 16256.0, K * 16384.0, K * 16384.0, K * 16384.0], dtype=torch.float64)
        assert bool(((y.double() - want).abs() <= 32 * 2.0 ** -24 * want.abs()).all())


def test_updates_that_are_not_finite_or_zero():
    import dense_gemm_nt_amd as g
    S = torch.stack([randn(70, 130, seed=i) for i in range(4)])
    S[1] = 0
    S[2, 3, 4] = math.nan
    S[3] *= 1e30
    u = g.orthogonalize(S.to(DEV), out_dtype=FP32).cpu()
    assert bool((u[1] == 0).all()) and bool(u[2].isnan().all())
    assert torch.equal(u[0], g.orthogonalize(S[0].to(DEV), out_dtype=FP32).cpu())
    assert torch.allclose(u[3], g.orthogonalize((S[3] * 1e-30).to(DEV), out_dtype=FP32).cpu(), rtol=0, atol=5e-3)
    S[2, 3, 4] = math.inf
    assert bool(g.orthogonalize(S[2].to(DEV)).isnan().all())
    # eps keeps a gradient that is next to nothing small
    tiny = g.orthogonalize((S[0] * 1e-12).to(DEV), steps=0, out_dtype=FP32).cpu().double()
    want = o.orthogonalize(S[0] * 1e-12, 0, ABC, 1e-7)
    # (X is kept to 22 bits of its largest values' units)
    assert bool(((tiny - want).abs() <= 2.0 ** -21 * want.abs() + 2.0 ** -25).all())


def test_empty_sizes():
    import dense_gemm_nt_amd as g

    def z(*s, dt=BF16):
        return torch.ones(*s, dtype=dt, device=DEV)
    assert g.gemm_gated(z(0, 16), z(8, 16), z(8, 16)).shape == (0, 8)
    assert g.gemm_gated(z(3, 16), z(0, 16), z(0, 16)).shape == (3, 0)
    assert bool((g.gemm_gated(z(3, 0), z(8, 0), z(8, 0)) == 0).all())
    dx, a, b = g.gemm_gated_backward(z(0, 8), z(0, 16), z(8, 16), z(8, 16))
    assert dx.shape == (0, 16) and bool((a == 0).all()) and bool((b == 0).all())
    dx, a, b = g.gemm_gated_backward(z(3, 0), z(3, 16), z(0, 16), z(0, 16))
    assert bool((dx == 0).all()) and a.shape == (0, 16)
    dx, a, b = g.gemm_gated_backward(z(0, 8, dt=FP16), z(0, 16, dt=FP16), z(8, 16, dt=FP16), z(8, 16, dt=FP16))
    assert bool((a == 0).all())
    dx, a, b = g.gemm_gated_backward(z(3, 0, dt=FP16), z(3, 16, dt=FP16), z(0, 16, dt=FP16), z(0, 16, dt=FP16))
    assert bool((dx == 0).all())
    assert [t.shape for t in g.gemm_gated_backward(z(3, 8), z(3, 0), z(8, 0), z(8, 0))] == [(3, 0), (8, 0), (8, 0)]
    q, s = g.quantize_int8(z(0, 16))
    assert q.shape == (0, 16) and s.shape == (0,)
    q, s = g.quantize_int8(z(3, 0))
    assert q.shape == (3, 0) and bool((s == 0).all())
    i8 = torch.int8
    assert g.gemm_int8(z(0, 16, dt=i8), z(8, 16, dt=i8), z(0, dt=FP32), z(8, dt=FP32)).shape == (0, 8)
    assert g.gemm_int8(z(3, 16, dt=i8), z(0, 16, dt=i8), z(3, dt=FP32), z(0, dt=FP32)).shape == (3, 0)
    assert bool((g.gemm_int8(z(3, 0, dt=i8), z(8, 0, dt=i8), z(3, dt=FP32), z(8, dt=FP32)) == 0).all())
    for shape in ((0, 5), (5, 0), (0, 3, 4), (2, 0, 4), (2, 3, 0)):
        assert g.orthogonalize(z(*shape)).shape == shape


# --------------------------------------------------- streams, graphs, repeats, offsets

def _calls(seed):
    """Every call on inputs of a seed: {name: (function of the inputs, inputs)}."""
    import dense_gemm_nt_amd as g
    M, F, K = 136, 520, 2056                    # K splits summed in the kernel; counters
    x, Wg, Wu = _operands(M, F, K, FP16, seed=seed)
    dh = randn(M, F, seed=seed + 3, dtype=FP16)
    few = _codes(2, 2064, seed=seed + 4)
    A, B = _codes(70, 4112, seed=seed + 5), _codes(515, 4112, seed=seed + 6)
    sa, sb = _scales(70, seed + 7), _scales(515, seed + 8)
    G = torch.stack([randn(100, 520, seed=seed + 9), randn(100, 520, seed=seed + 10)])
    return {
        "gated": (lambda x, a, b: (g.gemm_gated(x, a, b),), (x, Wg, Wu)),
        "backward": (lambda d, x, a, b: g.gemm_gated_backward(d, x, a, b, activation="gelu"), (dh, x, Wg, Wu)),
        "quantize": (lambda x: g.quantize_int8(x), (x,)),
        "int8": (lambda A, B, sa, sb: (g.gemm_int8(A, B, sa, sb),), (A, B, sa, sb)),
        "few": (lambda A, B, sa, sb: (g.gemm_int8(A, B, sa, sb),), (few, B[:, :2064].contiguous(), sa[:2].clone(), sb)),
        "ortho": (lambda G: (g.orthogonalize(G),), (G,)),
    }


def test_same_bits_again_and_on_another_stream():
    for name, (fn, args) in _calls(1).items():
        d = [t.to(DEV) for t in args]
        torch.cuda.synchronize()
        want = [t.clone() for t in fn(*d)]
        s, s2 = torch.cuda.Stream(), torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        s2.wait_stream(torch.cuda.current_stream())
        outs = []
        for _ in range(4):                       # calls that may run at once, with memory of their own
            for st in (s, s2):
                with torch.cuda.stream(st):
                    outs.append(fn(*d))
        torch.cuda.synchronize()
        for out in outs:
            assert all(torch.equal(a, b) for a, b in zip(out, want)), name


def test_captured_calls_replay():
    """Two graphs of each call, replayed in turn and at once with new inputs in the same buffers,
    beside the program's own eager calls."""
    for name, (fn, args) in _calls(1).items():
        buf = [t.to(DEV) for t in args]
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        graphs, outs = [], []
        with torch.cuda.stream(s):
            fn(*buf)
            s.synchronize()
            for _ in range(2):
                gr = torch.cuda.CUDAGraph()
                with torch.cuda.graph(gr, stream=s):
                    outs.append(fn(*buf))
                graphs.append(gr)
        for seed in (100, 200, 300):
            for b, t in zip(buf, _calls(seed)[name][1]):
                b.copy_(t)
            torch.cuda.synchronize()
            want = [t.clone() for t in fn(*buf)]
            torch.cuda.synchronize()
            other = torch.cuda.Stream()
            graphs[0].replay()
            with torch.cuda.stream(other):
                graphs[1].replay()
            eager = fn(*buf)
            torch.cuda.synchronize()
            for out in (outs[0], outs[1], eager):
                assert all(torch.equal(a, b) for a, b in zip(out, want)), (name, seed)


def test_offsets_past_32_bits():
    import dense_gemm_nt_amd as g
    # results of more than 2^31 values: the last rows against a call of their own
    M, F, K = 80011, 27000, 16
    x, Wg, Wu = randn(M, K, seed=1, dtype=BF16).to(DEV), randn(F, K, seed=2, dtype=BF16).to(DEV), randn(F, K, seed=3, dtype=BF16).to(DEV)
    h = g.gemm_gated(x, Wg, Wu)
    assert h.numel() > 1 << 31
    want = g.gemm_gated(x[-300:], Wg, Wu)
    # (another tile walks K in the same order: one slab)
    assert torch.equal(h[-300:], want)
    q, s = g.quantize_int8(h)
    q1, s1 = g.quantize_int8(h[-5:].contiguous())
    assert torch.equal(q[-5:], q1) and torch.equal(s[-5:], s1)
    one = torch.ones(1, device=DEV)
    y = g.gemm_int8(q[:, :16].contiguous(), q[:F, :16].contiguous(), one, one)
    assert torch.equal(y[-9:], g.gemm_int8(q[-9:, :16].contiguous(), q[:F, :16].contiguous(), one, one))
    del y, q, want
    dx, a, b = g.gemm_gated_backward(h, x, Wg, Wu)
    dx1, _, _ = g.gemm_gated_backward(h[-300:], x[-300:], Wg, Wu)
    ref = o.gated_backward(h[-300:].cpu(), x[-300:].cpu(), Wg.cpu(), Wu.cpu(), "silu")
    _, gs, us = o.gated(x[-300:].cpu(), Wg.cpu(), Wu.cpu(), "silu")
    bound = _backward_bounds(h[-300:].cpu(), x[-300:].cpu(), Wg.cpu(), Wu.cpu(), gs, us, "silu", BF16, BF16, BF16)[0]
    check(dx[-300:], ref[0], bound(ref[0]), "dx of the last rows")
    check(dx1, ref[0], bound(ref[0]), "dx of them alone")
    # the weights' gradients are sums over rows: of the first and the rest
    parts = [g.gemm_gated_backward(h[r], x[r], Wg, Wu, need_dx=False, grad_dtype=FP32) for r in (slice(0, 40000), slice(40000, M))]
    for i, got in ((1, a), (2, b)):
        both = parts[0][i].double() + parts[1][i].double()
        assert float((got.double() - both).norm() / both.norm()) <= half_step(BF16) + 1e-4
    del h, parts
    # rows far apart
    ld = (1 << 21) + 64
    far = torch.empty(1100, ld, dtype=BF16, device=DEV)[:, :72].copy_(randn(1100, 72, seed=5, dtype=BF16))
    Wg, Wu = randn(136, 72, seed=6, dtype=BF16).to(DEV), randn(136, 72, seed=7, dtype=BF16).to(DEV)
    near = far.contiguous()
    assert torch.equal(g.gemm_gated(far, Wg, Wu), g.gemm_gated(near, Wg, Wu))
    dh = torch.empty(1100, ld, dtype=BF16, device=DEV)[:, :136].copy_(randn(1100, 136, seed=8, dtype=BF16))
    for p, q in zip(g.gemm_gated_backward(dh, far, Wg, Wu), g.gemm_gated_backward(dh.contiguous(), near, Wg, Wu)):
        assert torch.equal(p, q)
    for p, q in zip(g.quantize_int8(far), g.quantize_int8(near)):
        assert torch.equal(p, q)
    assert torch.equal(g.orthogonalize(far), g.orthogonalize(near))
    codes = torch.empty(1100, 2 * ld, dtype=torch.int8, device=DEV)[:, :80].copy_(_codes(1100, 80, seed=9))
    assert torch.equal(g.gemm_int8(codes, codes, one, one), g.gemm_int8(codes.contiguous(), codes.contiguous(), one, one))


# ---------------------------------------------------------------- a layer's whole life

@pytest.mark.parametrize("dt", [BF16, FP16])
@pytest.mark.parametrize("captured", [False, True])
def test_a_layer_is_trained_updated_and_served(dt, captured):
    """One step of a feed-forward layer: forward, gradients, updates of the two weights by their
    orthogonalized gradients; then its up projection in 8-bit integers.  Each operator is checked
    on what it was really given."""
    import dense_gemm_nt_amd as g
    M, D, F = 200, 136, 520
    mk = dict(x=lambda s: randn(M, D, seed=s, dtype=dt), dy=lambda s: randn(M, D, seed=s + 1, dtype=dt, std=0.1),
              Wg=lambda s: randn(F, D, seed=s + 2, dtype=dt, std=D ** -0.5), Wu=lambda s: randn(F, D, seed=s + 3, dtype=dt, std=D ** -0.5),
              Wd=lambda s: randn(D, F, seed=s + 4, dtype=dt, std=F ** -0.5))
    buf = {n: f(0).to(DEV) for n, f in mk.items()}

    def step():
        x, dy, Wg, Wu, Wd = (buf[n] for n in ("x", "dy", "Wg", "Wu", "Wd"))
        h = g.gemm_gated(x, Wg, Wu)
        y = g.gemm_nt(h, Wd)
        dh = g.gemm_nt(dy, Wd.t())
        dx, dWg, dWu = g.gemm_gated_backward(dh, x, Wg, Wu)
        G = torch.stack([dWg, dWu])
        U = g.orthogonalize(G)
        new = (torch.stack([Wg, Wu]).float() - 0.02 * U.float()).to(dt)
        codes, scale = g.quantize_int8(x)
        Wq, ws = g.quantize_int8(new[1])
        up = g.gemm_int8(codes[:, :128].contiguous(), Wq[:, :128].contiguous(), scale, ws, out_dtype=dt)
        return dict(h=h, y=y, dh=dh, dx=dx, dWg=dWg, dWu=dWu, G=G, U=U, new=new, codes=codes, scale=scale, Wq=Wq, ws=ws, up=up)

    res = graph = None
    if captured:
        s = torch.cuda.Stream()
        with torch.cuda.stream(s):
            step()
            s.synchronize()
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph, stream=s):
                res = step()
    for seed in (100, 200, 300):
        for n, f in mk.items():
            buf[n].copy_(f(seed))
        if captured:
            graph.replay()
        else:
            res = step()
        torch.cuda.synchronize()
        c, q = {n: v.cpu() for n, v in buf.items()}, {n: v.cpu() for n, v in res.items()}
        ref, gs, us = o.gated(c["x"], c["Wg"], c["Wu"], "silu")
        check(q["h"], ref, _forward_bound(c["x"], c["Wg"], c["Wu"], gs, us, "silu", dt), "h")
        y = q["h"].double() @ c["Wd"].double().t()
        s = q["h"].double().abs() @ c["Wd"].double().abs().t()
        check(q["y"], y, rounded(y, (F + 64) * U * s, dt), "y")
        grads = o.gated_backward(q["dh"], c["x"], c["Wg"], c["Wu"], "silu")
        bounds = _backward_bounds(q["dh"], c["x"], c["Wg"], c["Wu"], gs, us, "silu", dt, dt, dt)
        for n, r, b in zip(("dx", "dWg", "dWu"), grads, bounds):
            check(q[n], r, b(r), n)
        U_ref = o.orthogonalize(q["G"], 5, ABC, 1e-7)
        for i in range(2):
            rel = float((q["U"][i].double() - U_ref[i]).norm() / U_ref[i].norm())
            assert rel < 5e-3, rel                # 1e-3 of the iteration, and BF16's half step
        rc, rs = o.quantize(c["x"])
        assert torch.equal(q["codes"], rc) and torch.equal(q["scale"], rs)
        rc, rs = o.quantize(q["new"][1])
        assert torch.equal(q["Wq"], rc) and torch.equal(q["ws"], rs)
        up, s = o.int8(q["codes"][:, :128], q["Wq"][:, :128], q["scale"], q["ws"])
        check(q["up"], up, rounded(up, 20 * U * s, dt), "up")
