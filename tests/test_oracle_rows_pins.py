"""The plain 64-bit forms of the row-indexed products (oracle/rows.py) against
closed cases and, for the gradients, central differences of the forward forms."""
import pytest
import torch

from oracle import rows as o

F64 = torch.float64


def _rand(*shape, seed=0):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed), dtype=F64)


def _difference(f, x, d, h=1e-5):
    return (f(x + h * d) - f(x - h * d)) / (2 * h)


def test_lora_is_a_dense_product_per_adapter():
    x, W, A, B = _rand(7, 16, seed=1), _rand(9, 16, seed=2), _rand(3, 8, 16, seed=3), _rand(3, 9, 8, seed=4)
    ids, scale = torch.tensor([0, -1, 2, 2, 5, 1, 0]), torch.tensor([0.5, 2.0, -1.0], dtype=F64)
    y, base, low = o.lora(x, W, A, B, ids, scale)
    for m, a in enumerate(ids.tolist()):
        Wm = W + (scale[a] * (B[a] @ A[a]) if 0 <= a < 3 else 0)
        assert torch.allclose(y[m], Wm @ x[m], rtol=1e-12, atol=1e-12)
    assert bool((y.abs() <= base + low + 1e-12).all()) and bool((low[[1, 4]] == 0).all())


def test_lora_gradients_are_differences():
    x, W, A, B = _rand(7, 16, seed=1), _rand(8, 16, seed=2), _rand(3, 8, 16, seed=3), _rand(3, 8, 8, seed=4)
    ids, scale, dy = torch.tensor([0, -1, 2, 2, 5, 0, 0]), torch.tensor([0.5, 2.0, -1.0], dtype=F64), _rand(7, 8, seed=5)
    g = o.lora_backward(dy, x, W, A, B, ids, scale)
    for name, arg in (("dx", x), ("dA", A), ("dB", B)):
        d = _rand(*arg.shape, seed=6)

        def loss(v, name=name):
            a = {"dx": (v, W, A, B), "dA": (x, W, v, B), "dB": (x, W, A, v)}[name]
            return (o.lora(*a, ids, scale)[0] * dy).sum()
        # the loss is quadratic at most: the central difference is exact but for rounding
        assert torch.allclose((g[name][0] * d).sum(), _difference(loss, arg, d), rtol=1e-7, atol=1e-7)
    assert bool((g["dA"][0][1] == 0).all()) and bool((g["dB"][0][1] == 0).all())


def test_route_closed_cases():
    inf = float("inf")
    x = torch.tensor([[1.0, 3.0, 3.0, 0.0], [-inf, 2.0, -inf, -inf], [-inf] * 4, [5.0, 1.0, 2.0, 4.0],
                      [0.0, 0.0, 0.0, 0.0]])
    r = o.route(x, 2, mask=torch.tensor([1, 1, 1, 0, 1]))
    assert r["ids"].tolist() == [[1, 2], [1, -1], [-1, -1], [-1, -1], [0, 1]]
    assert r["weights"].tolist() == [[0.5, 0.5], [1.0, 0.0], [0, 0], [0, 0], [0.5, 0.5]]
    assert r["counts"].tolist() == [1, 3, 1, 0] and r["offsets"].tolist() == [0, 1, 4, 5, 5]
    assert r["order"].tolist() == [8, 0, 2, 9, 1, 3, 4, 5, 6, 7] and r["tokens"] == 3
    # an even routing has loss 1, one expert for everything E
    even = torch.eye(4) * 1e3
    assert o.route(even, 1)["loss"] == pytest.approx(1.0)
    assert o.route(torch.tensor([[9e9, 0, 0, 0]] * 3), 1)["loss"] == pytest.approx(4.0)
    assert o.route(x[2:3], 2)["loss"] == 0.0
    nan = o.route(torch.tensor([[float("nan"), 1.0, -inf]]), 3)
    assert nan["ids"].tolist() == [[1, 0, -1]] and bool(nan["loss"].isnan())


@pytest.mark.parametrize("renormalize", [False, True])
def test_route_gradients_are_differences(renormalize):
    T, E, k = 6, 5, 2
    x = _rand(T, E, seed=7)
    x[1, 3] = float("-inf")
    mask = torch.tensor([1, 1, 0, 1, 1, 1])
    r = o.route(x, k, mask, renormalize)
    gw, gl = _rand(T, k, seed=8), 0.7
    got = o.route_backward(x, r, renormalize, gw, gl)
    d = _rand(T, E, seed=9)
    d[1, 3] = 0
    counts = r["counts"].to(F64)

    def loss(v):
        s = o.route(v, k, mask, renormalize)
        assert torch.equal(s["ids"], r["ids"])          # the step changes no choice
        n = s["tokens"]
        balance = E * (counts / (n * k) * s["p"].sum(0) / n).sum()   # counts held fixed
        return (s["weights"] * gw).sum() + gl * balance
    # third-order term below h^2 |d|^3 times the softmax's third derivative (< 1)
    assert torch.allclose((got * d).sum(), _difference(loss, x, d), rtol=1e-6, atol=1e-8)
    assert bool((got[2] == 0).all()) and got[1, 3] == 0


def test_routed_reads_any_offsets():
    assert o.segments([0, 2, 2, 5], 5) == ([(0, 2), (2, 2), (2, 5)], 5)
    assert o.segments([1, 4, 2, 9], 6) == ([(1, 4), (4, 4), (4, 6)], 6)
    assert o.segments([-3, 2], 4) == ([(0, 2)], 2)
    x, W, dy = _rand(5, 8, seed=1), _rand(3, 4, 8, seed=2), _rand(5, 4, seed=3)
    off = torch.tensor([0, 2, 2, 4])
    C, S = o.routed(x, W, off)
    assert torch.allclose(C[3], W[2] @ x[3]) and bool(C[4].isnan().all()) and bool((S[4] == 0).all())
    dW, _ = o.routed_wgrad(dy, x, off)
    assert torch.allclose(dW[0], torch.outer(dy[0], x[0]) + torch.outer(dy[1], x[1])) and bool((dW[1] == 0).all())
