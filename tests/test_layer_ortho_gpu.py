"""The orthogonalized update against its iteration in 64 bits."""
import pytest
import torch

from oracle import layer as o
from tests.rows_util import half_step, randn

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF16, FP16, FP32 = torch.bfloat16, torch.float16, torch.float32
ABC = (3.4445, -4.7750, 2.0315)


def _predict(G, steps, coefficients):
    """(most, likely): the relative error of the update, as norms.  Each step rounds three
    matrices to FP16: X's copy, A' = X X^T - sigma I and B' (sigma 1 from the third step on),
    each by N with |N_ij| <= 2^-11 of the entry.  To first order in N, in X's singular basis:
      copy   DP[N] - a' N          A'   (b' N + c (A' N + N A')) X          B'   N X
    and what X is off itself goes through DP, the derivative of the step P, which
    multiplies symmetric and antisymmetric parts of entry (i, j) by the divided differences
    (p(si) -+ p(sj)) / (si -+ sj), and columns past X's rows by p(si) / si.  `most` takes the
    largest factor and every rounding at its largest; `likely` independent roundings,
    evenly spread (1 / sqrt 3 of the largest), hence mean squares, where there are many entries."""
    r, k = min(G.shape), max(G.shape)
    X = G.double() if G.shape[0] <= G.shape[1] else G.double().t()
    s = torch.linalg.svdvals(X)
    s = s / s.norm()
    step = 2.0 ** -11
    most = likely = 0.0
    for i in range(steps):
        a, b, c = coefficients[i] if hasattr(coefficients[0], "__len__") else coefficients
        sigma = 1.0 if i >= 2 else 0.0
        a1, b1 = a + sigma * (b + c), b + 2 * c * sigma

        def p(v):
            return a * v + b * v ** 3 + c * v ** 5
        x, y = s[:, None], s[None, :]
        # the divided differences as polynomials (no quotient of nearly equal values)
        minus = a + b * (x * x + x * y + y * y) + c * (x ** 4 + x ** 3 * y + x * x * y * y + x * y ** 3 + y ** 4)
        plus = a + b * (x * x - x * y + y * y) + c * (x ** 4 - x ** 3 * y + x * x * y * y - x * y ** 3 + y ** 4)
        wide = a + b * s ** 2 + c * s ** 4
        al = s ** 2 - sigma
        be = b1 * al + c * al ** 2
        fa = (b1 + c * (al[:, None] + al[None, :])).abs() * y

        def mean(f):
            v = (f(minus) ** 2 + f(plus) ** 2).sum() / 2 + (k - r) * (f(wide) ** 2).sum()
            return float((v / (r * k)).sqrt())

        def top(f):
            return float(max(f(minus).abs().max(), f(plus).abs().max(), f(wide).abs().max()))
        nx, na, nb = float(s.norm()), float(al.norm()), float(be.norm())
        most = most * top(lambda d: d) + step * (nx * top(lambda d: d - a1) + na * float(fa.max()) + nb * float(s.max()))
        likely = ((likely * mean(lambda d: d)) ** 2 + step ** 2 / 3 * (
            (nx * mean(lambda d: d - a1)) ** 2 + (na * float((fa ** 2).mean().sqrt())) ** 2 +
            (nb * float((s ** 2).mean().sqrt())) ** 2)) ** 0.5
        s = p(s).abs()
    return most / float(s.norm()), likely / float(s.norm())


def _spectrum(m, n, kind, seed):
    G = randn(m, n, seed=seed)
    if kind == "flat":
        return G
    U, _, V = torch.linalg.svd(G.double(), full_matrices=False)
    s = torch.arange(1, min(m, n) + 1).double() ** -1.0
    if kind == "rank":
        s[min(m, n) // 2:] = 0
    return ((U * s) @ V).float()


def check(got, ref, dtype, G, steps=5, coefficients=ABC, what=""):
    got = got.cpu().double()
    assert got.shape == ref.shape
    for i in range(ref.shape[0]) if ref.dim() == 3 else [...]:
        y, r, A = got[i], ref[i], G[i]
        most, likely = _predict(A, steps, coefficients)
        rel = float((y - r).norm() / r.norm())
        # (the result's rounding: at most half a step of every entry; sums, the norm and what is
        # of second order: 5% more)
        assert rel <= 1.05 * most + half_step(dtype) + 1e-6, (what, i, rel, most)
        if min(A.shape) >= 64:
            assert rel <= 2 * (likely ** 2 + half_step(dtype) ** 2 / 3) ** 0.5 + 1e-6, (what, i, rel, likely)
        print("%s: %.3g of the norm, likely %.3g, most %.3g" % (what, rel, likely, most), flush=True)


@pytest.mark.parametrize("m,n", [(1, 1), (1, 9), (7, 3), (64, 64), (65, 130), (128, 1000), (300, 257), (1000, 2047), (2048, 768),
                                 (520, 4100)])
@pytest.mark.parametrize("kind", ["flat", "steep"])
@pytest.mark.parametrize("dt,out", [(FP32, BF16), (BF16, FP32)])
def test_update(m, n, kind, dt, out):
    import dense_gemm_nt_amd as g
    G = _spectrum(m, n, kind, m + n).to(dt)
    U = g.orthogonalize(G.to(DEV), out_dtype=out)
    check(U, o.orthogonalize(G, 5, ABC, 1e-7), out, G, what="%dx%d" % (m, n))


@pytest.mark.parametrize("B,m,n", [(3, 40, 70), (12, 200, 72), (2, 1100, 300), (5, 300, 1100), (40, 64, 64)])
def test_stack(B, m, n):
    import dense_gemm_nt_amd as g
    G = torch.stack([_spectrum(m, n, ("flat", "steep", "rank")[i % 3], i) * 10.0 ** (i % 7 - 3) for i in range(B)])
    U = g.orthogonalize(G.to(DEV), out_dtype=FP16)
    check(U, o.orthogonalize(G, 5, ABC, 1e-7), FP16, G, what="stack")
    one = g.orthogonalize(G[1].contiguous().to(DEV), out_dtype=FP32)
    check(one, o.orthogonalize(G[1], 5, ABC, 1e-7), FP32, G[1], what="one of it")


@pytest.mark.parametrize("steps", [0, 1, 2, 3, 8])
def test_steps_and_coefficients(steps):
    import dense_gemm_nt_amd as g
    G = randn(96, 200, seed=1)
    for abc in ((1.5, -0.5, 0.0), (1.875, -1.25, 0.375)):
        check(g.orthogonalize(G.to(DEV), steps=steps, coefficients=abc, out_dtype=FP32),
              o.orthogonalize(G, steps, abc, 1e-7), FP32, G, steps, abc, "steps %d" % steps)


def test_coefficients_of_each_step():
    import dense_gemm_nt_amd as g
    G = randn(150, 90, seed=2)
    each = [ABC, ABC, (1.875, -1.25, 0.375), (1.5, -0.5, 0.0)]
    X = o.orthogonalize(G, 1, ABC, 1e-7)
    for abc in each[1:]:
        n = X.norm()
        X = o.orthogonalize(X * (1 + 0.0), 1, tuple(c * n ** p for c, p in zip(abc, (1, 3, 5))), 0.0)
    check(g.orthogonalize(G.to(DEV), steps=4, coefficients=each, out_dtype=FP32), X, FP32, G, 4, each, "each")


@pytest.mark.parametrize("B,m,n", [(1, 16, 16), (1, 64, 1000), (1, 1024, 256), (3, 256, 1024), (1, 1024, 1024), (1, 1500, 1024),
                                   (2, 1024, 4100), (20, 256, 264), (1, 4096, 4096), (1, 4096, 5000), (1, 5003, 4096),
                                   (9, 1030, 1024)])
def test_signed_permutations_are_exact(B, m, n):
    """r orthogonal rows with one entry of +-1 each, r a power of four: the norm is a power of two, and
    two steps of (1.5, -0.5, 0) take the one singular value 1 / sqrt r to numbers of few bits
    (three of a sixteenth's are exact too), so a value out of place anywhere, or any rounding
    that the formula does not have, shows."""
    import dense_gemm_nt_amd as g
    r, k = min(m, n), max(m, n)
    gen = torch.Generator().manual_seed(m + n)
    G = torch.zeros(B, r, k)
    for b in range(B):
        at = torch.randperm(k, generator=gen)[:r]
        G[b, torch.arange(r), at] = torch.randint(0, 2, (r,), generator=gen).float() * 2 - 1
    G = G if m <= n else G.transpose(1, 2).contiguous()
    G = G[0] if B == 1 else G
    out = g.orthogonalize(G.to(DEV), steps=1, coefficients=(1.5, -0.5, 0.25), eps=0.0, out_dtype=FP32)
    s = 1.0 / r ** 0.5
    assert (r & (r - 1)) == 0
    want = 1.5 * s - 0.5 * s ** 3 + 0.25 * s ** 5
    assert torch.equal(out.cpu(), (G.double() * want).float())
    # three steps of the identity map, so that every product and the turns of the copies are used
    out = g.orthogonalize(G.to(DEV), steps=4, coefficients=[(1.0, 0.0, 0.0), (2.0, 0.0, 0.0), (1.0, 0.0, 0.0), (0.5, 0.0, 0.0)],
                          eps=0.0, out_dtype=BF16)
    assert torch.equal(out.cpu().float(), G * s)


@pytest.mark.parametrize("B,m,n", [(4, 1024, 1024), (3, 1024, 4096), (2, 4096, 4096), (2, 6000, 4096)])
def test_tiles_of_larger_updates_are_exact(B, m, n):
    """The same on 128 x 128 tiles, whole and split, and on 256 x 256 ones with the last pass's in quarters."""
    test_signed_permutations_are_exact(B, m, n)
