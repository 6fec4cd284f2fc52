"""The top-k router, its balance loss and its gradient against the plain 64-bit
forms."""
import pytest
import torch

from oracle import rows as o
from tests.rows_util import half_step, randn

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF16, FP16, FP32 = torch.bfloat16, torch.float16, torch.float32


def _logits(T, E, dt, seed=0, closed=0.02):
    x = randn(T, E, seed=seed, std=2.0)
    g = torch.Generator().manual_seed(seed + 1)
    x[torch.rand(T, E, generator=g) < closed] = float("-inf")
    return x.to(dt)


# p: exp's argument is a rounded difference (|x - max| 2^-24) and a rounded
# product with log2 e (as much again, relative to |x - max| in the exponent), the
# hardware exponential is within 2^-22, the sum of E terms within E 2^-24, the
# division and product within 2^-22
def _p_rel(x, E):
    top = x.double().masked_fill(x.isinf(), -1e30).max(1, keepdim=True).values.clamp(min=-1e30)
    span = (top - x.double().masked_fill(x.isinf() | x.isnan(), 0)).abs().clamp(max=100).max()
    return float(span) * 2.0 ** -22 + E * 2.0 ** -24 + 2.0 ** -20


def _check_route(x, k, mask, renorm, r, what):
    E = x.shape[1]
    ref = o.route(x, k, mask, renorm)
    for name in ("ids", "counts", "offsets", "order"):
        got = getattr(r, name).cpu().long()
        assert torch.equal(got, ref[name]), (what, name)
    assert int(r.tokens) == ref["tokens"]
    rel = _p_rel(x, E)
    w = r.weights.cpu().double()
    # renormalized, numerator and denominator each carry p's error
    assert bool(((w - ref["weights"]).abs() <= (3 * rel) * ref["weights"] + 1e-37).all()), what
    T = x.shape[0]
    # sums of p over the tokens (at most T + 200 additions) and of E terms
    bound = (rel + (T + E + 200) * 2.0 ** -24 + 2.0 ** -20) * abs(float(ref["loss"]))
    assert abs(float(r.loss) - float(ref["loss"])) <= bound, (what, float(r.loss), float(ref["loss"]))
    return ref


def _check_backward(x, ref, renorm, gw, gl, got, what):
    d = o.route_backward(x, ref, renorm, gw, gl)
    T, E = x.shape
    rel = _p_rel(x, E)
    # |dlogit| <= p (|dp| + sum p |dp|); every factor carries p's relative error
    # (that of h twice: weights and 1 / total), the dot product E additions
    n, k = max(ref["tokens"], 1), ref["ids"].shape[1]
    dp = torch.zeros(T, E, dtype=torch.float64)
    if gl is not None:
        dp += abs(float(gl)) * E * ref["counts"].double() / (n * k) / n
    if gw is not None:
        g = gw.double().abs()
        total = torch.zeros(T, dtype=torch.float64)
        for j in range(k):
            e = ref["ids"][:, j].clamp(min=0)
            total += torch.where(ref["ids"][:, j] >= 0, ref["p"].gather(1, e[:, None])[:, 0], 0.0)
        total = torch.where(total > 0, total, 1.0)
        mean = (g * ref["weights"]).sum(1)
        for j in range(k):
            h = (g[:, j] + mean) / total if renorm else g[:, j]
            dp.scatter_add_(1, ref["ids"][:, j:j + 1].clamp(min=0),
                            torch.where(ref["ids"][:, j] >= 0, h, torch.zeros_like(h))[:, None])
    mag = ref["p"] * (dp + (ref["p"] * dp).sum(1, keepdim=True))
    bound = (6 * rel + (E + 2 * k + 32) * 2.0 ** -23) * mag
    if got.dtype != FP32:
        bound = bound + half_step(got.dtype) * (d.abs() + bound) + 2.0 ** -25
    err = (got.cpu().double() - d).abs()
    assert bool((err <= bound + 1e-37).all()), (what, float((err / (bound + 1e-37)).max()))


@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (1, 8, 2), (3, 3, 3), (16, 16, 1), (64, 64, 8), (65, 17, 4),
                                   (200, 60, 6), (130, 65, 8), (100, 256, 8), (77, 257, 5), (40, 512, 64),
                                   (33, 513, 2), (70, 1000, 10), (20, 1024, 64), (1000, 5, 2), (9000, 12, 2)])
@pytest.mark.parametrize("dt", [FP32, BF16, FP16])
@pytest.mark.parametrize("renorm", [True, False])
def test_route(T, E, k, dt, renorm):
    import dense_gemm_nt_amd as g
    x = _logits(T, E, dt, seed=T + E)
    mask = torch.rand(T, generator=torch.Generator().manual_seed(5)) < 0.9
    r = g.route_topk(x.to(DEV), k, mask=mask.to(DEV), renormalize=renorm)
    ref = _check_route(x, k, mask, renorm, r, "route %s" % ((T, E, k, dt),))
    gw, gl = randn(T, k, seed=6), torch.tensor(0.01 * T)
    for a, b in ((gw, gl), (gw, None), (None, gl), (None, None)):
        got = g.route_topk_backward(x.to(DEV), r, a.to(DEV) if a is not None else None,
                                    b.to(DEV) if b is not None else None)
        _check_backward(x, ref, renorm, a, b, got, "route grad %s" % ((T, E, k, dt),))


def test_no_mask_and_every_kind_of_row():
    import dense_gemm_nt_amd as g
    inf, nan = float("inf"), float("nan")
    low = torch.finfo(FP32).min
    x = torch.tensor([[1.0, 3.0, 3.0, 0.0, 3.0], [-inf, 2.0, -inf, -inf, -inf], [-inf] * 5, [low] * 5,
                      [low, 0.0, low, low, -inf], [0.0, -0.0, 0.0, -0.0, 0.0], [80.0, -80.0, 90.0, 0.0, -90.0]])
    for k in (1, 3, 5):
        r = g.route_topk(x.to(DEV), k)
        ref = _check_route(x, k, None, True, r, "rows")
        got = g.route_topk_backward(x.to(DEV), r, randn(7, k, seed=1).to(DEV), torch.ones((), device=DEV))
        _check_backward(x, ref, True, randn(7, k, seed=1), torch.ones(()), got, "rows")
        assert bool((got[2] == 0).all()) and bool(torch.isfinite(got).all())
    # a NaN or an infinity spoils its own token's weights, and the loss
    x[0, 3], x[1, 1] = nan, inf
    r = g.route_topk(x.to(DEV), 5)
    assert r.ids[0].tolist() == [1, 2, 4, 0, 3] and r.ids[1].tolist() == [1, -1, -1, -1, -1]
    assert bool(r.weights[0].isnan().all()) and bool(r.weights[1, 0].isnan()) and bool(r.loss.isnan())
    assert bool(torch.isfinite(r.weights[2:]).all())
    assert torch.equal(r.order.cpu().sort().values, torch.arange(35, dtype=torch.int32))


def test_nothing_routed():
    import dense_gemm_nt_amd as g
    for T in (0, 5, 200):
        x = randn(T, 12, seed=1)
        r = g.route_topk(x.to(DEV), 3, mask=torch.zeros(T, dtype=torch.uint8, device=DEV))
        assert int(r.tokens) == 0 and float(r.loss) == 0.0 and r.counts.tolist() == [0] * 12
        assert r.offsets.tolist() == [0] * 13 and bool((r.ids == -1).all()) and bool((r.weights == 0).all())
        assert r.order.tolist() == list(range(3 * T))
        d = g.route_topk_backward(x.to(DEV), r, randn(T, 3, seed=2).to(DEV), torch.ones((), device=DEV))
        assert tuple(d.shape) == (T, 12) and bool((d == 0).all())


@pytest.mark.parametrize("dt", [FP32, BF16])
def test_strided_rows(dt):
    import dense_gemm_nt_amd as g
    for pad in (1, 3, 4):
        wide = torch.full((50, 30 + pad), float("nan"), dtype=dt, device=DEV)
        x = _logits(50, 30, dt, seed=3)
        wide[:, :30] = x.to(DEV)
        view = wide[:, :30]
        r = g.route_topk(view, 4)
        ref = _check_route(x, 4, None, True, r, "strided")
        out = torch.full((50, 30 + pad), 7.0, dtype=dt, device=DEV)
        gw = randn(50, 4, seed=2)
        g.route_topk_backward(view, r, gw.to(DEV), out=out[:, :30])
        _check_backward(x, ref, True, gw, None, out[:, :30], "strided")
        assert bool((out[:, 30:] == 7.0).all())
    odd = torch.zeros(50 * 30 + 1, dtype=dt, device=DEV)[1:].view(50, 30)
    odd.copy_(x)
    _check_route(x, 4, None, True, g.route_topk(odd, 4), "misaligned base")


def test_gradient_by_differences():
    """The kernel's gradient along a direction against differences of the kernel's
    own loss and weights, in steps that change no choice."""
    import dense_gemm_nt_amd as g
    T, E, k, h = 64, 16, 2, 2.0 ** -7
    x, d = randn(T, E, seed=1), randn(T, E, seed=2)
    gw, gl = randn(T, k, seed=3), 3.0
    r = g.route_topk(x.to(DEV), k)
    keep = torch.ones(T, dtype=torch.bool)
    sides = []
    for s in (h, -h):
        q = g.route_topk((x + s * d).to(DEV), k)
        keep &= (q.ids == r.ids).all(1).cpu()
        sides.append((x + s * d))
    assert int(keep.sum()) > T // 2
    counts = r.counts.cpu().double()

    def value(v):
        q = g.route_topk(v.to(DEV), k)
        p = torch.softmax(v.double(), 1)
        return (q.weights.cpu().double() * gw.double())[keep].sum() + \
            gl * E * (counts / (T * k) * p[keep].sum(0) / T).sum()
    got = g.route_topk_backward(x.to(DEV), r, gw.to(DEV), torch.tensor(gl, device=DEV)).cpu().double()
    along = (got * d.double())[keep].sum()
    diff = (value(sides[0]) - value(sides[1])) / (2 * h)
    # third-order term: h^2 / 6 times the third derivative, below sum |d|^3 (|g| + loss)
    cube = (d.abs().max(1).values.double() ** 3 * (gw.abs().double().sum(1) + gl * E / T))[keep].sum()
    # and FP32 rounding of the weights over 2 h
    bound = h * h * cube + 2.0 ** -20 * gw.abs().double()[keep].sum() / h
    assert abs(float(along - diff)) <= float(bound)
    assert float(bound) < 0.2 * float((got.abs() * d.abs()).sum())       # and the bound says something


def test_captured_and_replayed():
    import dense_gemm_nt_amd as g
    for T, E, k in ((20, 24, 2), (5000, 24, 2)):
        x = _logits(T, E, FP32, seed=1).to(DEV)
        gw, gl = randn(T, k, seed=2).to(DEV), torch.ones((), device=DEV)
        s = torch.cuda.Stream()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.stream(s):
            g.route_topk_backward(x, g.route_topk(x, k), gw, gl)
            s.synchronize()
            with torch.cuda.graph(graph, stream=s):
                r = g.route_topk(x, k)
                d = g.route_topk_backward(x, r, gw, gl)
        for seed in range(4):
            x.copy_(_logits(T, E, FP32, seed=10 + seed))
            graph.replay()
            torch.cuda.synchronize()
            want = g.route_topk(x, k)
            assert all(torch.equal(a, b) for a, b in zip(r[:7], want[:7]))
            assert torch.equal(d, g.route_topk_backward(x, want, gw, gl))


def test_python_refusals():
    import dense_gemm_nt_amd as g
    x = randn(6, 8, seed=1).to(DEV)
    for bad in (lambda: g.route_topk(x.double(), 2), lambda: g.route_topk(x[0], 2), lambda: g.route_topk(x.t(), 2),
                lambda: g.route_topk(x, 9), lambda: g.route_topk(x, 0),
                lambda: g.route_topk(x, 2, mask=torch.ones(5, dtype=torch.bool, device=DEV)),
                lambda: g.route_topk(x, 2, mask=torch.ones(6, device=DEV)),
                lambda: g.route_topk_backward(x[:5], g.route_topk(x, 2)),
                lambda: g.route_topk_backward(x, g.route_topk(x, 2), grad_weights=torch.ones(6, 3, device=DEV)),
                lambda: g.route_topk_backward(x, g.route_topk(x, 2), grad_loss=torch.ones(2, device=DEV))):
        with pytest.raises((ValueError, TypeError, g.GemmError)):
            bad()


def test_backward_refuses_a_routing_of_other_making():
    import dense_gemm_nt_amd as g
    x = torch.randn(6, 9, device=DEV)
    r = g.route_topk(x, 2)
    for name in ("ids", "counts", "tokens"):
        with pytest.raises(ValueError):
            g.route_topk_backward(x, r._replace(**{name: getattr(r, name).long()}))
    with pytest.raises(ValueError):
        g.route_topk_backward(x, r._replace(weights=r.weights.t().contiguous().t()))
    with pytest.raises(ValueError):
        g.route_topk_backward(x, r._replace(weights=r.weights[:5]))
    with pytest.raises(ValueError):
        g.route_topk_backward(x, r._replace(counts=r.counts.cpu()))


@pytest.mark.parametrize("T,E,k", [(5, 8, 1), (70, 40, 1), (130, 256, 1), (40, 600, 1), (300, 12, 2), (90, 60, 3),
                                   (77, 200, 2), (50, 500, 4), (20, 1000, 3)])
@pytest.mark.parametrize("dt", [FP32, BF16])
def test_weights_that_sum_to_one_cancel_exactly(T, E, k, dt):
    """Renormalized weights sum to 1, so with one choice they are 1 and have no gradient,
    and with one choice far ahead theirs is small: near the formula's relative to
    itself, not to grad_weights."""
    import dense_gemm_nt_amd as g
    x = randn(T, E, seed=T + E)
    if k > 1:
        x[torch.arange(T), torch.arange(T) % E] += 12.0                # far ahead of the others
    x = x.to(dt)
    r = g.route_topk(x.to(DEV), k)
    ref = o.route(x, k, None, True)
    gw, gl = randn(T, k, seed=1), torch.tensor(0.5)
    got = g.route_topk_backward(x.to(DEV), r, gw.to(DEV))
    if k == 1:
        assert bool((r.weights == 1.0).all())
        assert bool((got == 0).all())
        both = g.route_topk_backward(x.to(DEV), r, gw.to(DEV), gl.to(DEV))
        assert torch.equal(both, g.route_topk_backward(x.to(DEV), r, None, gl.to(DEV)))
        return
    d = o.route_backward(x, ref, True, gw, None)
    w = ref["weights"]
    total = ref["p"].gather(1, ref["ids"]).sum(1, keepdim=True)
    # h_j = (d_j - sum_i d_i w_i) / S with d_j = g_j - g_0, the terms' errors being the
    # weights' and S's (three and one of p's) and the roundings of k + 3 operations
    far = (gw - gw[:, :1]).double().abs()
    h = (far + (far * w).sum(1, keepdim=True)) / total
    dp = torch.zeros(T, E, dtype=torch.float64).scatter_(1, ref["ids"], h)
    mag = ref["p"] * (dp + (ref["p"] * dp).sum(1, keepdim=True))
    bound = (8 * _p_rel(x, E) + (E + 4 * k + 32) * 2.0 ** -23) * mag
    if dt != FP32:
        bound = bound + half_step(dt) * (d.abs() + bound) + 2.0 ** -133
    err = (got.cpu().double() - d).abs()
    assert bool((err <= bound + 1e-37).all()), float((err / (bound + 1e-37)).max())


@pytest.mark.parametrize("E", [8, 20, 100, 256])
def test_small_probabilities_keep_their_bits(E):
    """Logits a multiple of 1/8, so that their differences are exact: a probability is
    off by its own exponential and those in the sum (2^-22 each), the sum (ten additions
    deep) and four more roundings, however far it is below the largest."""
    import dense_gemm_nt_amd as g
    T, k = 64, 8
    x = (torch.randint(-320, 321, (T, E), generator=torch.Generator().manual_seed(E)) / 8.0)
    ref = o.route(x, k, None, False)
    rel = 2 * 2.0 ** -22 + 14 * 2.0 ** -24
    r = g.route_topk(x.to(DEV), k, renormalize=False)
    err = (r.weights.cpu().double() - ref["weights"]).abs()
    assert bool((err <= rel * ref["weights"] + 1e-37).all()), float((err / ref["weights"]).max())
    # dlogits of one choice's weight with the other weights' gradients zero
    gw = torch.zeros(T, k)
    gw[:, k - 1] = 1.0
    d = o.route_backward(x, ref, False, gw, None)
    got = g.route_topk_backward(x.to(DEV), r, gw.to(DEV)).cpu().double()
    # p_e (delta - p_j): p's error twice, two roundings
    assert bool(((got - d).abs() <= (2 * rel + 3 * 2.0 ** -24) * d.abs() + 1e-37).all())


def test_results_are_apart():
    """A result changed in place leaves the others, and what autograd saved of them, alone."""
    import dense_gemm_nt_amd as g
    for T in (10, 20000):
        r = g.route_topk(randn(T, 24, seed=1).to(DEV), 3)
        p = torch.ones(T, 3, device=DEV, requires_grad=True)
        y = (p * r.weights).sum()                              # saves weights
        r.counts.zero_()
        r.ids.clamp_(min=0)
        y.backward()
        assert torch.equal(p.grad, r.weights)
        # what lives as long as one result does: the results of its size, and 64 KB
        for t in (r.counts, r.offsets, r.tokens, r.loss):
            assert t.untyped_storage().nbytes() <= 65536
        for t in (r.ids, r.weights, r.order):
            assert t.untyped_storage().nbytes() <= 3 * 3 * T * 4 + 65536
