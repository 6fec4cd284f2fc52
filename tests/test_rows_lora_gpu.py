"""The adapted projection and its gradients against the plain 64-bit forms."""
import itertools

import pytest
import torch

from oracle import rows as o
from tests.rows_util import check, lora_bound, randn

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF16, FP16, FP32 = torch.bfloat16, torch.float16, torch.float32


def _ids(M, L, kind, seed):
    g = torch.Generator().manual_seed(seed)
    if kind == "none":
        return torch.full((M,), -1, dtype=torch.int32)
    if kind == "runs":
        return (torch.arange(M) * L // max(M, 1)).to(torch.int32)
    if kind == "one":
        return torch.full((M,), L - 1, dtype=torch.int32)
    ids = torch.randint(-1, L, (M,), generator=g).to(torch.int32)
    if kind == "wild":          # ids that name no adapter, of every kind
        bad = torch.tensor([-1, L, -5, 2 ** 31 - 1, -2 ** 31, L + 7], dtype=torch.int64).to(torch.int32)
        ids[::3] = bad[torch.arange(len(ids[::3])) % len(bad)]
    return ids


def _case(M, N, K, R, L, kind, dt, seed=0):
    s = 10 * seed
    return dict(x=randn(M, K, seed=s + 1, dtype=dt), W=randn(N, K, seed=s + 2, dtype=dt, std=0.05),
                A=randn(L, R, K, seed=s + 3, dtype=dt, std=max(K, 1) ** -0.5),
                B=randn(L, N, R, seed=s + 4, dtype=dt, std=0.1), ids=_ids(M, L, kind, s + 5),
                scale=randn(L, seed=s + 6) + 1.5)


def _dev(c):
    return {k: v.to(DEV) for k, v in c.items()}


def _tiny(c, dt):
    # fp16's second part below its normal range: half a step of 2^-24 per rank
    return 2.0 ** -25 * c["A"].shape[1] * float(c["B"].abs().max()) if dt == FP16 and c["B"].numel() else 0.0


def _check_forward(c, got, dt, out, what):
    K, R = c["x"].shape[1], c["A"].shape[1]
    y, sb, sl = o.lora(**c)
    check(got, y, lora_bound(y, sb, sl, K, K, R, dt, out, _tiny(c, dt)), what)


# one of each tile and K-split form of the projection's plan
SHAPES = [
    # M, N, K, R, L, ids
    (1, 128, 64, 8, 1, "one"), (1, 4097, 4096, 16, 3, "one"), (2, 1, 8, 8, 2, "mixed"),
    (33, 200, 136, 24, 5, "wild"), (64, 1000, 512, 16, 64, "mixed"), (40, 28672, 64, 16, 7, "mixed"),
    (100, 1000, 512, 32, 40, "mixed"), (192, 4096, 1024, 16, 100, "mixed"), (1500, 3200, 128, 40, 3, "runs"),
    (256, 2048, 8192, 16, 200, "mixed"), (250, 1032, 8192, 128, 3, "wild"), (2048, 4096, 64, 16, 4, "runs"),
    (2050, 4100, 72, 64, 9, "mixed"), (1024, 4096, 2560, 8, 2, "runs"), (130, 300, 264, 120, 2, "mixed"),
    (300, 77, 40, 16, 5, "none"), (256, 8192, 8192, 16, 30, "mixed"),
    (2100, 264, 1000, 128, 3, "mixed"), (2100, 136, 328, 16, 70, "wild"), (2049, 77, 4096, 24, 5, "runs"),
    (2400, 8192, 2560, 16, 3, "wild"),       # full passes of the machine, and the rest with K splits
]


@pytest.mark.parametrize("M,N,K,R,L,kind", SHAPES)
@pytest.mark.parametrize("dt", [BF16, FP16])
def test_forward(M, N, K, R, L, kind, dt):
    import dense_gemm_nt_amd as g
    c = _case(M, N, K, R, L, kind, dt)
    for out in (dt, FP32):
        got = g.gemm_lora(**_dev(c), out_dtype=out)
        _check_forward(c, got, dt, out, "lora %s %s" % ((M, N, K, R, L, kind), out))


@pytest.mark.parametrize("M", [5, 70, 150, 1100])
@pytest.mark.parametrize("beta,act", [(0.0, "gelu"), (0.5, "none"), (0.0, "relu")])
def test_forward_epilogue(M, beta, act):
    import dense_gemm_nt_amd as g
    N, K, R, L, dt = 520, 1032, 16, 4, BF16
    c = _case(M, N, K, R, L, "mixed", dt)
    bias, old = randn(N, seed=7), randn(M, N, seed=8, dtype=FP32)
    out = old.to(DEV).clone()
    got = g.gemm_lora(**_dev(c), out=out, alpha=0.75, beta=beta, bias=bias.to(DEV), activation=act)
    assert got is out
    y, sb, sl = o.lora(**c)
    z = 0.75 * y + beta * old.double() + bias.double()
    ref = {"none": z, "relu": z.clamp(min=0), "gelu": z * 0.5 * (1 + torch.erf(z / 2 ** 0.5))}[act]
    # slope of the activations at most 1.13; the epilogue's own operations at
    # 2^-20 of their magnitudes (its GELU is within 2^-22 of |x|)
    err = lora_bound(torch.zeros_like(y), sb, sl, K, K, R, dt, FP32) * 1.13
    err = err + 2.0 ** -20 * (sb + sl + old.double().abs() + bias.double().abs())
    check(got, ref, err, "epilogue %s" % act)


def test_epilogue_along_rows_in_two_pieces():
    import dense_gemm_nt_amd as g
    M, N, K, R, L, dt = 2400, 8192, 2560, 8, 2, BF16
    c = _case(M, N, K, R, L, "mixed", dt)
    bias = randn(M, seed=7)
    got = g.gemm_lora(**_dev(c), bias=bias.to(DEV), bias_along="m", out_dtype=FP32)
    y, sb, sl = o.lora(**c)
    err = lora_bound(torch.zeros_like(y), sb, sl, K, K, R, dt, FP32) + 2.0 ** -20 * (sb + sl + bias.double().abs()[:, None])
    check(got, y + bias.double()[:, None], err, "row bias")


def test_forward_strides_and_untouched_columns():
    import dense_gemm_nt_amd as g
    M, N, K, R, L, dt = 75, 333, 200, 16, 3, FP16
    c = _case(M, N, K, R, L, "mixed", dt)
    d = _dev(c)
    for name, pad in (("x", 8), ("W", 24), ("A", 16), ("B", 8)):
        wide = torch.full((*d[name].shape[:-1], d[name].shape[-1] + pad), float("nan"), dtype=dt, device=DEV)
        wide[..., :d[name].shape[-1]] = d[name]
        d[name] = wide[..., :d[name].shape[-1]]
    d["B"] = torch.stack([d["B"], d["B"] * 0], 1)[:, 0]        # adapters not next to each other
    wide = torch.full((M, N + 5), float("nan"), dtype=FP32, device=DEV)
    got = g.gemm_lora(**d, out=wide[:, :N])
    _check_forward(c, got, dt, FP32, "strided")
    assert bool(wide[:, N:].isnan().all())


def test_empty_sums_and_no_adapters():
    import dense_gemm_nt_amd as g
    c = _case(9, 24, 0, 8, 2, "mixed", BF16)
    assert bool((g.gemm_lora(**_dev(c)) == 0).all())
    for M, N in ((0, 24), (9, 0)):
        c = _case(M, N, 16, 8, 2, "mixed", BF16)
        assert tuple(g.gemm_lora(**_dev(c)).shape) == (M, N)
    for R, L in ((8, 0), (0, 3)):
        for M in (9, 512):
            c = _case(M, 264, 1024, R, max(L, 1), "none", BF16)
            if L == 0:
                c.update(A=c["A"][:0], B=c["B"][:0], scale=c["scale"][:0])
            _check_forward(c, g.gemm_lora(**_dev(c)), BF16, BF16, "no adapters")


@pytest.mark.parametrize("M", [40, 120, 256, 2048])
@pytest.mark.parametrize("dt", [BF16, FP16])
def test_broken_adapters_reach_their_own_rows_only(M, dt):
    """Infinities and NaNs in an adapter, or in a row, stay with that adapter's
    rows, or that row: exactly where the formula has them."""
    import dense_gemm_nt_amd as g
    N, K, R, L = {40: (256, 64), 120: (256, 64), 256: (2048, 8192), 2048: (4096, 64)}[M] + (16, 5)
    c = _case(M, N, K, R, L, "mixed", dt)
    c["B"][1, 3, 2], c["B"][1, 7, 5], c["B"][1, 7, 6] = float("nan"), float("inf"), float("-inf")
    c["B"][1, 9, 1], c["B"][1, 130, 0] = float("-inf"), float("inf")
    c["B"][2] = float("nan")
    c["ids"][c["ids"] == 2] = 3                       # an adapter of NaNs that no row uses
    c["A"][4, 3] = 0                                   # low-rank values of zero ...
    c["B"][4, 11, 3] = float("inf")                    # ... times infinity
    c["x"][5, 1] = float("nan")
    c["x"][6, 2] = float("inf")
    c["ids"][5], c["ids"][6] = 0, -1
    y, sb, sl = o.lora(**c)
    s = torch.where(torch.isfinite(sb + sl), sb, torch.zeros_like(sb))
    got = g.gemm_lora(**_dev(c), out_dtype=FP32)
    check(got, y, lora_bound(y, s, torch.where(torch.isfinite(sl), sl, torch.zeros_like(sl)), K, K, R, dt, FP32,
                             2.0 ** -25 * R), "broken adapters")
    clean = (c["ids"] != 1) & (c["ids"] != 4)
    clean[5] = clean[6] = False
    assert bool(torch.isfinite(y[clean]).all()) and not bool(torch.isfinite(y).all())


def _check_backward(c, dy, got, dt, dx_dt, g_dt, what):
    M, K = c["x"].shape
    N, R = c["W"].shape[0], c["A"].shape[1]
    ref = o.lora_backward(dy, **c)
    for name, x, terms, inner, out in zip(("dx", "dA", "dB"), got, (N, 0, 0), (N, N, K), (dx_dt, g_dt, g_dt)):
        if x is None:
            continue
        r, sb, sl = ref[name]
        rank = R if name == "dx" else M        # the sum over the low-rank values' products
        far = max(float(c["A"].abs().max()), float(c["x"].abs().max()), float(dy.abs().max())) if c["A"].numel() else 0
        tiny = 2.0 ** -25 * rank * far if dt == FP16 else 0.0
        check(x, r, lora_bound(r, sb, sl, terms, inner, rank, dt, out, tiny), "%s %s" % (what, name))


@pytest.mark.parametrize("M,N,K,R,L,kind", [
    (1, 8, 8, 8, 1, "one"), (3, 136, 64, 16, 2, "mixed"), (65, 264, 520, 24, 7, "wild"),
    (129, 1000, 72, 8, 3, "runs"), (300, 256, 512, 40, 70, "mixed"), (700, 512, 1032, 128, 2, "mixed"),
    (1000, 4096, 64, 64, 3, "runs"), (2500, 136, 4096, 16, 1, "one"), (777, 4096, 2048, 8, 3, "mixed"),
    (64, 64, 64, 16, 4, "none"), (2100, 264, 1000, 128, 3, "mixed"), (2100, 136, 328, 16, 70, "wild"),
    (1024, 136, 72, 48, 1, "one"), (1025, 136, 72, 48, 2, "runs"), (1024, 264, 136, 72, 2, "one"), (1023, 8, 264, 32, 1000, "wild"),
    (1024, 136, 72, 16, 1, "one"), (512, 136, 328, 24, 1, "one"), (128, 136, 264, 128, 1, "one"), (256, 264, 136, 64, 2, "mixed"),
])
@pytest.mark.parametrize("dt", [BF16, FP16])
def test_backward(M, N, K, R, L, kind, dt):
    import dense_gemm_nt_amd as g
    c = _case(M, N, K, R, L, kind, dt)
    dy = randn(M, N, seed=9, dtype=dt)
    got = g.gemm_lora_backward(dy.to(DEV), **_dev(c))
    _check_backward(c, dy, got, dt, dt, FP32, "lora grad %s" % ((M, N, K, R, L, kind),))


@pytest.mark.parametrize("M", [200, 1100])          # few rows and many have kernels of their own
def test_backward_types_parts_and_strides(M):
    import dense_gemm_nt_amd as g
    N, K, R, L, dt = 264, 328, 16, 3, BF16
    c = _case(M, N, K, R, L, "mixed", dt)
    dy = randn(M, N, seed=9, dtype=dt)
    d = _dev(c)
    for name, pad in (("x", 8), ("W", 24), ("A", 16), ("B", 8)):
        wide = torch.full((*d[name].shape[:-1], d[name].shape[-1] + pad), float("nan"), dtype=dt, device=DEV)
        wide[..., :d[name].shape[-1]] = d[name]
        d[name] = wide[..., :d[name].shape[-1]]
    dyw = torch.full((M, N + 8), float("nan"), dtype=dt, device=DEV)
    dyw[:, :N] = dy.to(DEV)
    for g_dt, dx_dt in itertools.product((BF16, FP16, FP32), (BF16, FP32)):
        got = g.gemm_lora_backward(dyw[:, :N], **d, grad_dtype=g_dt, dx_dtype=dx_dt)
        _check_backward(c, dy, got, dt, dx_dt, g_dt, "strided %s %s" % (g_dt, dx_dt))
    whole = g.gemm_lora_backward(dy.to(DEV), **d)
    dx, dA, dB = g.gemm_lora_backward(dy.to(DEV), **d, need_adapters=False)
    assert dA is None and dB is None and torch.equal(dx, whole[0])
    dx, dA, dB = g.gemm_lora_backward(dy.to(DEV), **d, need_dx=False)
    assert dx is None and torch.equal(dA, whole[1]) and torch.equal(dB, whole[2])


@pytest.mark.parametrize("M,N,K,R,L", [(0, 16, 24, 8, 2), (9, 0, 24, 8, 2), (9, 16, 0, 8, 2), (9, 16, 24, 0, 2),
                                       (9, 16, 24, 8, 0), (0, 0, 0, 0, 0)])
def test_backward_of_nothing(M, N, K, R, L):
    import dense_gemm_nt_amd as g
    c = _case(M, N, K, R, max(L, 1), "mixed", BF16)
    if L == 0:
        c.update(A=c["A"][:0], B=c["B"][:0], scale=c["scale"][:0])
    dy = randn(M, N, seed=9, dtype=BF16)
    dx, dA, dB = g.gemm_lora_backward(dy.to(DEV), **_dev(c))
    ref = o.lora_backward(dy, **c)
    assert tuple(dA.shape) == (L, R, K) and tuple(dB.shape) == (L, N, R)
    assert bool((dA == 0).all()) and bool((dB == 0).all())
    check(dx, ref["dx"][0], ref["dx"][0].abs() * 0.05 + 0.1, "dx of little")


@pytest.mark.parametrize("M", [4, 1100])
@pytest.mark.parametrize("dt", [BF16, FP16])
def test_gradients_keep_the_low_rank_values(M, dt):
    """Low-rank values of 21 bits, exact in FP32, meet one row of dy and x each: dA and
    dB are single products, a few FP32 roundings off (2^-24 each)."""
    import dense_gemm_nt_amd as g
    N, K, R = 136, 64, 16
    x, dy = torch.zeros(M, K, dtype=dt), torch.zeros(M, N, dtype=dt)
    parts = torch.tensor([1.0, 2.0 ** -10, 2.0 ** -20])
    x[1, :3], dy[1, :3] = parts.to(dt), parts.to(dt)
    dy[1, 3:] = randn(N - 3, seed=3).to(dt)
    x[1, 3:] = randn(K - 3, seed=4).to(dt)
    A, B = torch.zeros(1, R, K, dtype=dt), torch.zeros(1, N, R, dtype=dt)
    A[0, :, :3] = 1.0
    B[0, :3, :] = 1.0
    c = dict(x=x, W=torch.zeros(N, K, dtype=dt), A=A, B=B, ids=torch.zeros(M, dtype=torch.int32),
             scale=torch.ones(1))
    _, dA, dB = g.gemm_lora_backward(dy.to(DEV), **_dev(c))
    ref = o.lora_backward(dy, **c)
    check(dA, ref["dA"][0], ref["dA"][0].abs() * 2.0 ** -22, "dA")
    check(dB, ref["dB"][0], ref["dB"][0].abs() * 2.0 ** -22, "dB")


@pytest.mark.parametrize("M", [150, 1100])
def test_backward_keeps_broken_rows_apart(M):
    import dense_gemm_nt_amd as g
    N, K, R, L, dt = 264, 328, 16, 4, BF16
    c = _case(M, N, K, R, L, "mixed", dt)
    dy = randn(M, N, seed=9, dtype=dt)
    c["ids"][:4] = torch.tensor([0, 1, 2, 3], dtype=torch.int32)
    c["x"][1, 5] = float("nan")             # adapter 1's gradients, and no others'
    dy[2, 7] = float("inf")
    c["A"][3, 2, 9] = float("nan")
    got = g.gemm_lora_backward(dy.to(DEV), **_dev(c), dx_dtype=FP32)
    ref = o.lora_backward(dy, **c)
    for name, x in zip(("dx", "dA", "dB"), got):
        assert torch.equal(torch.isfinite(x.cpu()), torch.isfinite(ref[name][0])), name
    assert bool(torch.isfinite(ref["dA"][0][0]).all()) and bool(torch.isfinite(ref["dB"][0][0]).all())


@pytest.mark.parametrize("M,R", [(150, 16), (150, 8), (700, 64), (1100, 24), (1500, 64)])
@pytest.mark.parametrize("dt", [BF16, FP16])
def test_backward_infinities_are_the_formulas(M, R, dt):
    """An infinity gives infinities of the formula's signs, not NaNs."""
    import dense_gemm_nt_amd as g
    N, K, L = 264, 328, 4
    c = _case(M, N, K, R, L, "mixed", dt)
    dy = randn(M, N, seed=9, dtype=dt)
    c["ids"][:4] = torch.tensor([0, 1, 2, 3], dtype=torch.int32)
    inf = float("inf")
    c["x"][1, 5], dy[2, 7] = -inf, inf
    c["x"][0, 9], dy[0, 11] = inf, float("nan")
    got = g.gemm_lora_backward(dy.to(DEV), **_dev(c), dx_dtype=FP32)
    ref = o.lora_backward(dy, **c)
    for name, x in zip(("dx", "dA", "dB"), got):
        r, x = ref[name][0], x.cpu()
        assert torch.equal(x.isnan(), r.isnan()), name
        assert torch.equal(x == inf, r == inf) and torch.equal(x == -inf, r == -inf), name
    assert bool(ref["dB"][0][2].isinf().any()) and not bool(ref["dB"][0][2].isnan().any())
    assert bool(ref["dA"][0][1].isinf().any()) and not bool(ref["dA"][0][1].isnan().any())


def test_forward_infinity_times_infinity():
    """An infinite row meets an infinite adapter: the formula's infinities."""
    import dense_gemm_nt_amd as g
    M, N, K, R, L = 40, 136, 64, 8, 2
    c = _case(M, N, K, R, L, "mixed", BF16)
    c["ids"][:2] = torch.tensor([1, 1], dtype=torch.int32)
    c["x"][0, 3] = float("inf")
    c["A"][1, 1:] = 0.0
    c["A"][1, 1:, 3] = 1.0                 # all low-rank values of row 0 infinite
    c["A"][1, 0, 3] = 1.0
    c["B"][1].abs_().add_(0.01)
    c["W"].abs_().add_(0.01)
    c["B"][1, 5, 0] = float("inf")
    c["scale"].abs_().add_(0.1)
    y = o.lora(**c)[0]
    got = g.gemm_lora(**_dev(c), out_dtype=FP32).cpu()
    assert torch.equal(got.isnan(), y.isnan()) and torch.equal(got.isinf(), y.isinf())


def test_same_bits_and_other_streams():
    import dense_gemm_nt_amd as g
    c = _dev(_case(300, 520, 1032, 16, 5, "mixed", BF16))
    dy = randn(300, 520, seed=9, dtype=BF16).to(DEV)
    first = (g.gemm_lora(**c), *g.gemm_lora_backward(dy, **c))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(3)]
    results = []
    for s in streams:
        with torch.cuda.stream(s):
            for _ in range(3):
                results.append((g.gemm_lora(**c), *g.gemm_lora_backward(dy, **c)))
    torch.cuda.synchronize()
    for r in results:
        assert all(torch.equal(a, b) for a, b in zip(r, first))


@pytest.mark.parametrize("M", [8, 520, 1100])
def test_captured_and_replayed(M):
    """Two graphs with memory of their own, replayed after each other with other
    inputs (ids included) in the same tensors; eager work in between."""
    import dense_gemm_nt_amd as g
    N, K, R, L, dt = 264, 2048, 16, 4, BF16
    cases = [_case(M, N, K, R, L, "mixed", dt, seed) for seed in range(3)]
    dys = [randn(M, N, seed=90 + s, dtype=dt) for s in range(3)]
    bufs = [_dev(cases[0]) for _ in range(2)]
    dyb = [dys[0].to(DEV) for _ in range(2)]
    s = torch.cuda.Stream()
    graphs, outs = [], []
    with torch.cuda.stream(s):
        g.gemm_lora(**bufs[0])
        g.gemm_lora_backward(dyb[0], **bufs[0])
        s.synchronize()
        for b, dy in zip(bufs, dyb):
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph, stream=s):
                outs.append((g.gemm_lora(**b), *g.gemm_lora_backward(dy, **b)))
            graphs.append(graph)
    torch.cuda.synchronize()
    for turn in range(3):
        for i in range(2):
            src = (turn + i) % 3
            for k, v in cases[src].items():
                bufs[i][k].copy_(v)
            dyb[i].copy_(dys[src])
        for graph in graphs:
            graph.replay()
        torch.cuda.synchronize()
        for i in range(2):
            want = (g.gemm_lora(**bufs[i]), *g.gemm_lora_backward(dyb[i], **bufs[i]))
            assert all(torch.equal(a, b) for a, b in zip(outs[i], want)), (turn, i)


def test_python_refusals():
    import dense_gemm_nt_amd as g
    c = _dev(_case(9, 24, 16, 8, 2, "mixed", BF16))

    def bad(exc, **kw):
        with pytest.raises(exc):
            g.gemm_lora(**{**c, **kw})
    bad(TypeError, W=c["W"].half())
    bad(TypeError, A=c["A"].half())
    bad(ValueError, ids=c["ids"].long())
    bad(ValueError, ids=c["ids"][:5])
    bad(ValueError, scale=c["scale"].double())
    bad(ValueError, A=c["A"][:1])
    bad(ValueError, x=c["x"].t())
    bad(ValueError, beta=1.0)
    bad(ValueError, W=c["W"].cpu())
    bad(ValueError, out=torch.empty(9, 25, device=DEV))
    bad(g.GemmError, x=c["x"][:, :12].contiguous(), W=c["W"][:, :12].contiguous(), A=c["A"][:, :, :12].contiguous())
    with pytest.raises(TypeError):
        g.gemm_lora_backward(torch.zeros(9, 24, device=DEV), **c)
    with pytest.raises(ValueError):
        g.gemm_lora_backward(torch.zeros(9, 23, dtype=BF16, device=DEV), **c)


# ---- low-rank values of any size ----

def _parts(rows, n, dt, seed):
    """[rows, n] of dt whose rows begin with +-1, +-2^-9 and +-2^-18 and are zero behind: their
    sum takes 19 bits, which no two bf16 values and, scaled down, no two fp16 ones hold."""
    v = torch.zeros(rows, n)
    sign = torch.randint(0, 2, (rows, 3), generator=torch.Generator().manual_seed(seed)) * 2.0 - 1.0
    v[:, :3] = sign * torch.tensor([1.0, 2.0 ** -9, 2.0 ** -18])
    return v.to(dt)


def _signs(*shape, seed, dt):
    return (torch.randint(0, 2, shape, generator=torch.Generator().manual_seed(seed)) * 2.0 - 1.0).to(dt)


SCALES = [2.0 ** -40, 2.0 ** -24, 1.0, 2.0 ** 18, 2.0 ** 40]


@pytest.mark.parametrize("M,R", [(4, 16), (200, 8), (300, 40), (250, 64), (1100, 16), (700, 64), (2300, 24), (1500, 128)])
@pytest.mark.parametrize("dt", [BF16, FP16])
def test_gradients_keep_low_rank_values_of_any_size(M, R, dt):
    """Every adapter has one row that is not zero: its dA and dB are single products of low-rank
    values of 19 bits, as above."""
    import dense_gemm_nt_amd as g
    N, K, L = 264, 328, 3
    x, dy = torch.zeros(M, K, dtype=dt), torch.zeros(M, N, dtype=dt)
    ids = torch.arange(M, dtype=torch.int32) % (L + 1) - 1
    at = torch.tensor([int((ids == a).nonzero()[-1]) for a in range(L)])
    x[at], dy[at] = _parts(L, K, dt, 1), _parts(L, N, dt, 2)
    x[at, 3:], dy[at, 3:] = randn(L, K - 3, seed=3, dtype=dt), randn(L, N - 3, seed=4, dtype=dt)
    c = dict(x=x, W=torch.zeros(N, K, dtype=dt), A=torch.zeros(L, R, K, dtype=dt),
             B=torch.zeros(L, N, R, dtype=dt), ids=ids, scale=torch.ones(L))
    c["A"][:, :, :3], c["B"][:, :3] = _signs(L, R, 3, seed=5, dt=dt), _signs(L, 3, R, seed=6, dt=dt)
    ref = o.lora_backward(dy, **c)
    for s in SCALES:
        got = g.gemm_lora_backward(dy.to(DEV), **_dev({**c, "scale": torch.full((L,), s)}), need_dx=False)
        for name, v in zip(("dA", "dB"), got[1:]):
            want = ref[name][0] * s
            check(v, want, want.abs() * 2.0 ** -20, "%s times %g" % (name, s))


@pytest.mark.parametrize("M,R", [(300, 16), (1100, 32)])
@pytest.mark.parametrize("std_dy,std_B", [(1e-4, 1e-4), (1e-3, 1e-4), (1e-2, 1e-3), (300.0, 30.0)])
def test_fp16_gradients_of_a_beginning_adapter(M, R, std_dy, std_B):
    """Adapters begin at B = 0: dA and dB against 64 bits in the 2-norm.  A rounding to FP32
    is 2^-24 off; of the 1024 of a sum sqrt(1024) add up at random, and the bound is four
    times that, 2^-17."""
    import dense_gemm_nt_amd as g
    N, K, L, dt = 1024, 512, 2, FP16
    c = _case(M, N, K, R, L, "mixed", dt)
    c["B"] = randn(L, N, R, seed=4, dtype=dt, std=std_B)
    dy = randn(M, N, seed=9, dtype=dt, std=std_dy)
    _, dA, dB = g.gemm_lora_backward(dy.to(DEV), **_dev(c), need_dx=False)
    ref = o.lora_backward(dy, **c)
    for name, v in (("dA", dA), ("dB", dB)):
        r = ref[name][0]
        off = float((v.cpu().double() - r).norm() / r.norm())
        print("%s dy %g B %g: off %.3g" % (name, std_dy, std_B, off), flush=True)
        assert off <= 2.0 ** -17


@pytest.mark.parametrize("M,N,K,R,L", [(1, 136, 64, 16, 1), (40, 264, 72, 8, 3), (64, 1000, 512, 16, 9),
                                       (100, 1000, 512, 32, 7), (256, 2048, 8192, 16, 20), (256, 8192, 8192, 24, 5),
                                       (1500, 3200, 128, 40, 3), (2048, 4096, 64, 16, 4), (2050, 4100, 72, 64, 5)])
@pytest.mark.parametrize("dt", [BF16, FP16])
def test_forward_keeps_low_rank_values_of_any_size(M, N, K, R, L, dt):
    """W is zero and every output one product s t[r] B[n, r] of a low-rank value t of 19 bits: in
    FP32 it is off by the roundings of its parts' products as they are added (2^-23
    each, at most six, and the conversions of the parts are exact)."""
    import dense_gemm_nt_amd as g
    c = dict(x=_parts(M, K, dt, 1), W=torch.zeros(N, K, dtype=dt), A=torch.zeros(L, R, K, dtype=dt),
             B=torch.zeros(L, N, R, dtype=dt), ids=_ids(M, L, "mixed", 3), scale=torch.ones(L))
    c["A"][:, :, :3] = _signs(L, R, 3, seed=2, dt=dt)
    n = torch.arange(N)
    c["B"][:, n, n % R] = randn(L, N, seed=4, dtype=dt)
    y = o.lora(**c)[0]
    for s in SCALES:
        got = g.gemm_lora(**_dev({**c, "scale": torch.full((L,), s)}), out_dtype=FP32)
        check(got, y * s, (y * s).abs() * 2.0 ** -20, "low-rank values times %g" % s)


@pytest.mark.parametrize("M,N,K,R,L", [(3, 136, 64, 16, 2), (300, 256, 512, 40, 7), (777, 4096, 2048, 8, 3),
                                       (1100, 264, 328, 24, 3), (2100, 512, 2048, 16, 2)])
@pytest.mark.parametrize("dt", [BF16, FP16])
def test_input_gradient_keeps_low_rank_values_of_any_size(M, N, K, R, L, dt):
    import dense_gemm_nt_amd as g
    c = dict(x=torch.zeros(M, K, dtype=dt), W=torch.zeros(N, K, dtype=dt), A=torch.zeros(L, R, K, dtype=dt),
             B=torch.zeros(L, N, R, dtype=dt), ids=_ids(M, L, "mixed", 3), scale=torch.ones(L))
    c["B"][:, :3] = _signs(L, 3, R, seed=2, dt=dt)
    k = torch.arange(K)
    c["A"][:, k % R, k] = randn(L, K, seed=4, dtype=dt)
    dy = _parts(M, N, dt, 1)
    dx = o.lora_backward(dy, **c)["dx"][0]
    for s in SCALES:
        got = g.gemm_lora_backward(dy.to(DEV), **_dev({**c, "scale": torch.full((L,), s)}), dx_dtype=FP32,
                                   need_adapters=False)[0]
        check(got, dx * s, (dx * s).abs() * 2.0 ** -20, "input gradient times %g" % s)


@pytest.mark.parametrize("M", [40, 120, 256, 2048])
@pytest.mark.parametrize("s", [2.0 ** -30, 2.0 ** 20])
def test_broken_adapters_meet_rows_of_other_units(M, s):
    """Infinities and NaNs in an adapter where FP16 low-rank values are small or large, in both
    directions: where the formula has them, and the other values as near as ever."""
    import dense_gemm_nt_amd as g
    N, K, R, L = {40: (256, 64), 120: (256, 64), 256: (2048, 8192), 2048: (4096, 64)}[M] + (16, 5)
    c = _case(M, N, K, R, L, "mixed", FP16)
    c["W"].zero_()
    c["scale"].fill_(s)
    c["B"][1, 3, 2], c["B"][1, 7, 5], c["B"][1, 7, 6] = float("nan"), float("inf"), float("-inf")
    c["B"][1, 9, 1], c["B"][1, 130, 0] = float("-inf"), float("inf")
    c["A"][4, 3] = 0
    c["B"][4, 11, 3] = float("inf")                    # zero times infinity
    y, sb, sl = o.lora(**c)
    zero = torch.zeros_like(sb)
    got = g.gemm_lora(**_dev(c), out_dtype=FP32)
    check(got, y, lora_bound(y, zero, torch.where(torch.isfinite(sl), sl, zero), K, K, R, FP16, FP32), "units")
    assert not bool(torch.isfinite(y).all())
    d = _case(M, N, K, R, L, "mixed", FP16)
    d["W"].zero_()
    d["scale"].fill_(s)
    d["A"][1, 3, 5], d["A"][1, 7, 9] = float("nan"), float("inf")
    dy = randn(M, N, seed=9, dtype=FP16)
    got = g.gemm_lora_backward(dy.to(DEV), **_dev(d), dx_dtype=FP32, need_adapters=False)[0]
    r, sb, sl = o.lora_backward(dy, **d)["dx"]
    zero = torch.zeros_like(sb)
    check(got, r, lora_bound(r, zero, torch.where(torch.isfinite(sl), sl, zero), N, N, R, FP16, FP32), "units dx")
