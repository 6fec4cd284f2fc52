"""The experts' products over sorted rows, and a whole expert layer step of the
row-indexed operators together, against the plain 64-bit forms."""
import pytest
import torch

from oracle import rows as o
from tests.rows_util import check, randn, sum_bound

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF16, FP16, FP32 = torch.bfloat16, torch.float16, torch.float32


def _offsets(S, E, kind, seed=0):
    g = torch.Generator().manual_seed(seed)
    if kind == "skew":              # uneven, some experts empty, rows behind the last
        cut = (torch.rand(E, generator=g) ** 3).cumsum(0)
        ends = (cut / cut[-1] * (S - S // 10)).floor()
        return torch.cat([torch.zeros(1), ends]).to(torch.int32)
    if kind == "one":               # everything to the last expert
        return torch.tensor([0] * E + [S], dtype=torch.int32)
    if kind == "late":              # rows before the first, too
        return torch.linspace(S // 5, S - S // 7, E + 1).to(torch.int32)
    wild = torch.randint(-S, 2 * S + 2, (E + 1,), generator=g)
    return wild.to(torch.int32)     # in no order and outside the rows


CASES = [
    # S, E, N, K, offsets: rows per expert for each tile height
    (1, 1, 1, 8, "one"), (1, 5, 130, 72, "one"), (40, 8, 300, 136, "skew"), (512, 64, 264, 200, "skew"),
    (600, 9, 1000, 64, "skew"), (700, 7, 129, 328, "wild"), (3000, 16, 520, 264, "skew"), (2000, 4, 700, 1032, "late"),
    (1500, 3, 256, 512, "one"), (900, 130, 136, 64, "skew"), (64, 1024, 40, 16, "skew"), (333, 2, 77, 40, "wild"),
    (1500, 3, 8200, 264, "one"), (2500, 3, 8300, 72, "skew"), (2500, 3, 8204, 136, "late"), (2500, 4, 8200, 40, "wild"),
]


@pytest.mark.parametrize("S,E,N,K,kind", CASES)
@pytest.mark.parametrize("dt,out", [(BF16, BF16), (FP16, FP32)])
@pytest.mark.parametrize("mn", [False, True])
def test_routed(S, E, N, K, kind, dt, out, mn):
    import dense_gemm_nt_amd as g
    if mn:
        N = -(-N // 8) * 8
    x, W = randn(S, K, seed=1, dtype=dt), randn(E, N, K, seed=2, dtype=dt)
    off = _offsets(S, E, kind)
    Wd = W.transpose(1, 2).contiguous().to(DEV).transpose(1, 2) if mn else W.to(DEV)
    ref, s = o.routed(x, W, off)
    seg, end = o.segments(off.tolist(), S)
    mine = torch.zeros(S, dtype=torch.bool)
    for a, b in seg:
        mine[a:b] = True
    got = g.gemm_routed(x.to(DEV), Wd, off.to(DEV), out_dtype=out)
    check(got[mine], ref[mine], sum_bound(ref, s, K, out)[mine], "routed %s" % ((S, E, N, K, kind),))
    assert bool((got[end:] == 0).all())
    # into a given tensor: the rows of no expert and the columns past N as they were
    wide = torch.full((S, N + 3), 5.0, dtype=out, device=DEV)
    g.gemm_routed(x.to(DEV), Wd, off.to(DEV), out=wide[:, :N])
    assert torch.equal(wide[:, :N].cpu()[mine], got.cpu()[mine])
    assert bool((wide[:, :N].cpu()[~mine] == 5.0).all()) and bool((wide[:, N:] == 5.0).all())


@pytest.mark.parametrize("S,E,N,K,kind", CASES)
@pytest.mark.parametrize("dt,out", [(BF16, FP32), (FP16, FP16)])
def test_wgrad(S, E, N, K, kind, dt, out):
    import dense_gemm_nt_amd as g
    N = -(-N // 8) * 8
    dy, x = randn(S, N, seed=1, dtype=dt, std=0.3), randn(S, K, seed=2, dtype=dt, std=0.3)
    off = _offsets(S, E, kind)
    dW, s = o.routed_wgrad(dy, x, off)
    got = g.gemm_routed_wgrad(dy.to(DEV), x.to(DEV), off.to(DEV), out_dtype=out)
    check(got, dW, sum_bound(dW, s, S, out), "wgrad %s" % ((S, E, N, K, kind),))


def test_strides_and_broken_rows():
    import dense_gemm_nt_amd as g
    S, E, N, K, dt = 300, 4, 264, 136, BF16
    off = torch.tensor([0, 100, 130, 130, 280], dtype=torch.int32)
    xw = torch.full((S, K + 8), float("nan"), dtype=dt)
    dw = torch.full((S, N + 16), float("nan"), dtype=dt)
    W2 = torch.full((E, 2, N, K + 8), float("nan"), dtype=dt)
    xw[:, :K], dw[:, :N], W2[:, 0, :, :K] = randn(S, K, seed=1), randn(S, N, seed=2), randn(E, N, K, seed=3)
    xw[105, 3], dw[105, 9] = float("nan"), float("inf")      # expert 1's, and rows of none
    xw[285:, :] = float("nan")
    dw[285:, :] = float("nan")
    xd, dd, Wd = xw.to(DEV)[:, :K], dw.to(DEV)[:, :N], W2.to(DEV)[:, 0, :, :K]
    x, dy, W = xw[:, :K], dw[:, :N], W2[:, 0, :, :K]
    ref, s = o.routed(x, W, off)
    got = g.gemm_routed(xd, Wd, off.to(DEV), out_dtype=FP32)
    check(got[:280], ref[:280], sum_bound(ref, s, K, FP32)[:280], "strided")
    dx = g.gemm_routed(dd, Wd.transpose(1, 2), off.to(DEV), out_dtype=FP32)
    ref, s = o.routed(dy, W.transpose(1, 2), off)
    check(dx[:280], ref[:280], sum_bound(ref, s, N, FP32)[:280], "strided dx")
    dW = g.gemm_routed_wgrad(dd, xd, off.to(DEV), out_dtype=FP32)
    ref, s = o.routed_wgrad(dy, x, off)
    clean = [0, 2, 3]
    check(dW[clean], ref[clean], sum_bound(ref, s, 150, FP32)[clean], "strided dW")
    assert torch.equal(torch.isfinite(dW[1].cpu()), torch.isfinite(ref[1]))


def test_empty():
    import dense_gemm_nt_amd as g
    off = torch.zeros(4, dtype=torch.int32, device=DEV)
    z = lambda *s: torch.zeros(*s, dtype=BF16, device=DEV)   # noqa: E731
    assert tuple(g.gemm_routed(z(0, 16), z(3, 8, 16), off).shape) == (0, 8)
    assert tuple(g.gemm_routed(z(5, 16), z(3, 0, 16), off).shape) == (5, 0)
    assert bool((g.gemm_routed(z(5, 16) + 1, z(3, 8, 16) + 1, off) == 0).all())
    assert bool((g.gemm_routed(z(5, 0), z(3, 8, 0), off) == 0).all())
    assert bool((g.gemm_routed(z(5, 16), z(0, 8, 16), off[:1]) == 0).all())
    assert bool((g.gemm_routed_wgrad(z(0, 8), z(0, 16), off) == 0).all())
    assert bool((g.gemm_routed_wgrad(z(5, 8) + 1, z(5, 16) + 1, off) == 0).all())
    assert tuple(g.gemm_routed_wgrad(z(5, 8), z(5, 16), off[:1]).shape) == (0, 8, 16)


def test_python_refusals():
    import dense_gemm_nt_amd as g
    x, W = randn(6, 16, seed=1, dtype=BF16).to(DEV), randn(3, 8, 16, seed=2, dtype=BF16).to(DEV)
    off = torch.tensor([0, 2, 4, 6], dtype=torch.int32, device=DEV)
    for bad in (lambda: g.gemm_routed(x.half(), W, off), lambda: g.gemm_routed(x, W, off.long()),
                lambda: g.gemm_routed(x, W, off[:3]), lambda: g.gemm_routed(x[:, :8], W, off),
                lambda: g.gemm_routed(x, W, off.cpu()), lambda: g.gemm_routed(x, W[:, ::2, ::2], off),
                lambda: g.gemm_routed(x.float(), W.float(), off),
                lambda: g.gemm_routed(x[:, :12].contiguous(), W[:, :, :12].contiguous(), off),
                lambda: g.gemm_routed_wgrad(x[:5], x, off),
                lambda: g.gemm_routed_wgrad(x[:, :4].contiguous(), x, off)):
        with pytest.raises((ValueError, TypeError, g.GemmError)):
            bad()


@pytest.mark.parametrize("captured", [False, True])
def test_expert_layer_together(captured):
    """A training step of an expert layer with an adapted shared projection before
    it: gemm_lora -> route_topk -> the experts' product on the gathered rows ->
    weighted sum, then all the gradients; nothing is read back in between, so the
    whole step is captured and replayed with other data."""
    import dense_gemm_nt_amd as g
    T, D, E, k, N, L, R, dt = 150, 64, 6, 2, 72, 3, 8, BF16
    mk = dict(x=lambda s: randn(T, D, seed=s, dtype=dt), W=lambda s: randn(D, D, seed=s + 1, dtype=dt, std=D ** -0.5),
              A=lambda s: randn(L, R, D, seed=s + 2, dtype=dt, std=D ** -0.5),
              B=lambda s: randn(L, D, R, seed=s + 3, dtype=dt, std=0.3),
              ids=lambda s: torch.randint(-1, L, (T,), generator=torch.Generator().manual_seed(s)).to(torch.int32),
              scale=lambda s: randn(L, seed=s + 4) + 1.5)
    buf = {n: f(0).to(DEV) for n, f in mk.items()}
    router, We = randn(E, D, seed=50, dtype=dt).to(DEV), randn(E, N, D, seed=51, dtype=dt, std=D ** -0.5).to(DEV)
    dout = randn(T, N, seed=52, dtype=dt).to(DEV)
    gl = torch.ones((), device=DEV)

    def step():
        h = g.gemm_lora(**buf)
        logits = g.gemm_nt(h, router, out_dtype=FP32)
        r = g.route_topk(logits, k)
        token = (r.order // k).long()
        xs = h.index_select(0, token)
        ys = g.gemm_routed(xs, We, r.offsets)
        y = torch.empty_like(ys)
        y.index_copy_(0, r.order.long(), ys)                 # back to pair order
        out = (y.view(T, k, N).float() * r.weights.unsqueeze(2)).sum(1)
        # backward
        dw = (y.view(T, k, N).float() * dout.float().unsqueeze(1)).sum(2)
        dys = (dout.float().index_select(0, token) *
               r.weights.view(-1).index_select(0, r.order.long()).unsqueeze(1)).to(dt)
        dWe = g.gemm_routed_wgrad(dys, xs, r.offsets, out_dtype=FP32)
        dxs = g.gemm_routed(dys, We.transpose(1, 2), r.offsets, out_dtype=FP32)
        dlog = g.route_topk_backward(logits, r, dw, gl)
        dpair = torch.empty_like(dxs)
        dpair.index_copy_(0, r.order.long(), dxs)
        dh = (dpair.view(T, k, D).sum(1) + dlog @ router.float()).to(dt)
        dx, dA, dB = g.gemm_lora_backward(dh, **buf)
        return dict(h=h, logits=logits, ids=r.ids, loss=r.loss, out=out, dWe=dWe, dlog=dlog, dh=dh, dx=dx, dA=dA,
                    dB=dB, xs=xs, dys=dys, weights=r.weights, offsets=r.offsets, dw=dw)

    res = None
    graph = None
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
        c = {n: v.cpu() for n, v in buf.items()}
        q = {n: v.cpu() for n, v in res.items()}
        # each operator on what it was really given
        from tests.rows_util import lora_bound
        y, sb, sl = o.lora(**c)
        check(q["h"], y, lora_bound(y, sb, sl, D, D, R, dt, dt), "h")
        ref = o.route(q["logits"], k)
        assert torch.equal(q["ids"].long(), ref["ids"]) and torch.equal(q["offsets"].long(), ref["offsets"])
        assert abs(float(q["loss"]) - float(ref["loss"])) < 1e-5 * float(ref["loss"])
        dlog = o.route_backward(q["logits"], ref, True, q["dw"], 1.0)
        assert torch.allclose(q["dlog"].double(), dlog, rtol=1e-4, atol=1e-5 * float(dlog.abs().max()))
        dW, sW = o.routed_wgrad(q["dys"], q["xs"], q["offsets"])
        check(q["dWe"], dW, sum_bound(dW, sW, T * k, FP32), "dWe")
        back = o.lora_backward(q["dh"], **c)
        for name, terms, inner, rank, out in (("dx", D, D, R, dt), ("dA", 0, D, T, FP32), ("dB", 0, D, T, FP32)):
            r0, b0, l0 = back[name]
            check(q[name], r0, lora_bound(r0, b0, l0, terms, inner, rank, dt, out), name)


def _far(t, ld):
    """The same values in rows `ld` elements apart: offsets past 32 bits."""
    wide = torch.empty(t.shape[0], ld, dtype=t.dtype, device=DEV)[:, :t.shape[1]]
    return wide.copy_(t)


def test_rows_more_than_32_bits_apart():
    import dense_gemm_nt_amd as g
    M, N, K, R, L, ld = 1100, 136, 72, 16, 3, (1 << 21) + 64
    x, dy = randn(M, K, seed=1, dtype=BF16).to(DEV), randn(M, N, seed=2, dtype=BF16).to(DEV)
    W, We = randn(N, K, seed=3, dtype=BF16).to(DEV), randn(2, N, K, seed=4, dtype=BF16).to(DEV)
    A, B = randn(L, R, K, seed=5, dtype=BF16).to(DEV), randn(L, N, R, seed=6, dtype=BF16).to(DEV)
    ids = (torch.arange(M, device=DEV) % (L + 1)).to(torch.int32) - 1
    scale, off = torch.ones(L, device=DEV), torch.tensor([0, 300, M - 7], dtype=torch.int32, device=DEV)
    fx, fdy = _far(x, ld), _far(dy, ld)
    out = torch.zeros(M, ld, dtype=BF16, device=DEV)[:, :N]
    assert torch.equal(g.gemm_lora(fx, W, A, B, ids, scale, out=out), g.gemm_lora(x, W, A, B, ids, scale))
    for a, b in zip(g.gemm_lora_backward(fdy, fx, W, A, B, ids, scale), g.gemm_lora_backward(dy, x, W, A, B, ids, scale)):
        assert torch.equal(a, b)
    out.zero_()
    assert torch.equal(g.gemm_routed(fx, We, off, out=out), g.gemm_routed(x, We, off))
    out = out[:, :K].zero_()
    assert torch.equal(g.gemm_routed(fdy, We.transpose(1, 2), off, out=out), g.gemm_routed(dy, We.transpose(1, 2), off))
    assert torch.equal(g.gemm_routed_wgrad(fdy, fx, off), g.gemm_routed_wgrad(dy, x, off))
    r, f = g.route_topk(dy, 4), g.route_topk(fdy, 4)
    for a, b in zip(r, f):
        assert a is b or torch.equal(a, b)
    gw = torch.ones_like(r.weights)
    assert torch.equal(g.route_topk_backward(fdy, f, gw), g.route_topk_backward(dy, r, gw))


@pytest.mark.parametrize("S,E,N,K,mn", [(40, 8, 300, 136, False), (700, 7, 264, 328, False), (2000, 4, 700, 1032, False),
                                        (2500, 3, 8300, 72, False), (700, 7, 264, 328, True), (2500, 3, 8304, 136, True),
                                        (9, 70, 40, 16, False), (300, 64, 136, 64, False)])
def test_rows_of_no_expert_are_zero_in_a_new_result(S, E, N, K, mn):
    """A slice of a router's offsets (the experts held here) begins behind row 0: the rows before it
    belong to no expert, as those behind the last do."""
    import dense_gemm_nt_amd as g
    x, W = randn(S, K, seed=1, dtype=BF16).to(DEV), randn(E, N, K, seed=2, dtype=BF16).to(DEV)
    Wd = W.transpose(1, 2).contiguous().transpose(1, 2) if mn else W
    for off in (_offsets(S, E, "late"), torch.full((E + 1,), S, dtype=torch.int32), _offsets(S, E, "wild", 3),
                torch.full((E + 1,), 2 ** 31 - 1, dtype=torch.int32), torch.full((E + 1,), -7, dtype=torch.int32)):
        ref, s = o.routed(x.cpu(), W.cpu(), off)
        mine = torch.zeros(S, dtype=torch.bool)
        for a, b in o.segments(off.tolist(), S)[0]:
            mine[a:b] = True
        stale = torch.full((S, N), 7.0, dtype=FP32, device=DEV)      # what the allocator gives next
        del stale
        got = g.gemm_routed(x, Wd, off.to(DEV), out_dtype=FP32).cpu()
        assert bool((got[~mine] == 0).all())
        check(got[mine], ref[mine], sum_bound(ref, s, K, FP32)[mine], "late offsets")
        out = torch.full((S, N), 5.0, dtype=FP32, device=DEV)
        g.gemm_routed(x, Wd, off.to(DEV), out=out)
        assert torch.equal(out.cpu()[mine], got[mine]) and bool((out.cpu()[~mine] == 5.0).all())


def test_one_row_at_any_stride():
    """A single row's stride is never used: the last token of a long prompt is such a row."""
    import dense_gemm_nt_amd as g
    K, N, E, R, L, dt = 72, 136, 3, 8, 2, BF16
    W, We = randn(N, K, seed=1, dtype=dt).to(DEV), randn(E, N, K, seed=2, dtype=dt).to(DEV)
    A, B = randn(L, R, K, seed=3, dtype=dt).to(DEV), randn(L, N, R, seed=4, dtype=dt).to(DEV)
    ids, scale = torch.ones(1, dtype=torch.int32, device=DEV), torch.ones(L, device=DEV)
    off = torch.tensor([0, 0, 1, 1], dtype=torch.int32, device=DEV)
    for step in ((1 << 22) + 8, K + 3, 0):
        def row(cols, seed):
            wide = torch.zeros(step + cols, dtype=dt, device=DEV)
            wide[:cols] = randn(cols, seed=seed, dtype=dt).to(DEV)
            return wide.as_strided((1, cols), (step, 1)), wide[:cols].clone().view(1, cols)
        (x, x1), (dy, dy1) = row(K, 5), row(N, 6)
        out = torch.zeros(N + step, dtype=dt, device=DEV).as_strided((1, N), (step, 1))
        assert torch.equal(g.gemm_lora(x, W, A, B, ids, scale, out=out), g.gemm_lora(x1, W, A, B, ids, scale))
        for a, b in zip(g.gemm_lora_backward(dy, x, W, A, B, ids, scale),
                        g.gemm_lora_backward(dy1, x1, W, A, B, ids, scale)):
            assert torch.equal(a, b)
        assert torch.equal(g.gemm_routed(x, We, off), g.gemm_routed(x1, We, off))
        assert torch.equal(g.gemm_routed_wgrad(dy, x, off), g.gemm_routed_wgrad(dy1, x1, off))
        r, r1 = g.route_topk(dy, 4), g.route_topk(dy1, 4)
        assert all(torch.equal(a, b) for a, b in zip(r[:7], r1[:7]))
        assert torch.equal(g.route_topk_backward(dy, r, r.weights), g.route_topk_backward(dy1, r1, r1.weights))
