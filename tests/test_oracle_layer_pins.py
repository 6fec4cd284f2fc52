"""The plain 64-bit forms of a feed-forward layer's products (oracle/layer.py) against
closed cases and, for the gradients, central differences of the forward form."""
import math

import pytest
import torch

from oracle import layer as o

F64 = torch.float64


def _rand(*shape, seed=0):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed), dtype=F64)


def test_gates():
    v = torch.tensor([-3.0, -1.0, 0.0, 0.5, 2.0], dtype=F64)
    assert o.gate(v, "relu")[0].tolist() == [0.0, 0.0, 0.0, 0.5, 2.0]
    assert o.gate(v, "relu")[1].tolist() == [0.0, 0.0, 0.0, 1.0, 1.0]
    for x, s in zip(v.tolist(), o.gate(v, "silu")[0].tolist()):
        assert math.isclose(s, x / (1 + math.exp(-x)), rel_tol=1e-14, abs_tol=1e-300)
    for x, s in zip(v.tolist(), o.gate(v, "gelu")[0].tolist()):
        assert math.isclose(s, x * 0.5 * math.erfc(-x / math.sqrt(2)), rel_tol=1e-14, abs_tol=1e-300)
    # far out in the tail the value keeps its digits: Phi(-8) = 6.22096e-16
    assert math.isclose(float(o.gate(torch.tensor([-8.0], dtype=F64), "gelu")[0]), -8 * 6.220960574271785e-16, rel_tol=1e-12)


@pytest.mark.parametrize("act", ["silu", "gelu", "relu"])
def test_block_and_its_gradients(act):
    x, Wg, Wu, dh = _rand(5, 16, seed=1), _rand(7, 16, seed=2), _rand(7, 16, seed=3), _rand(5, 7, seed=4)
    h, g, u = o.gated(x, Wg, Wu, act)
    for m in range(5):
        for f in range(7):
            gate, up = float(Wg[f] @ x[m]), float(Wu[f] @ x[m])
            a = max(0.0, gate) if act == "relu" else gate / (1 + math.exp(-gate)) if act == "silu" else \
                gate * 0.5 * math.erfc(-gate / math.sqrt(2))
            assert math.isclose(float(h[m, f]), a * up, rel_tol=1e-11, abs_tol=1e-13)
    grads = o.gated_backward(dh, x, Wg, Wu, act)
    for i, arg in enumerate((x, Wg, Wu)):
        d = _rand(*arg.shape, seed=6 + i)

        def loss(v, i=i):
            a = [x, Wg, Wu]
            a[i] = v
            return (o.gated(*a, act)[0] * dh).sum()
        step = 1e-6
        diff = (loss(arg + step * d) - loss(arg - step * d)) / (2 * step)
        assert torch.allclose((grads[i] * d).sum(), diff, rtol=1e-6, atol=1e-6)
    # the two sums' gradients are what the three are made of
    assert torch.allclose(grads[3] @ Wg + grads[4] @ Wu, grads[0])


def test_quantize():
    x = torch.tensor([[127.0, -63.5, 0.5, 1.5], [0.0, 0.0, 0.0, 0.0], [1.0, math.inf, 2.0, 0.0], [1.0, math.nan, 2.0, 0.0],
                      [-2.0, 1.0, -1.0, 0.25]])
    q, s = o.quantize(x)
    assert q[0].tolist() == [127, -64, 0, 2] and float(s[0]) == 1.0           # ties to even
    assert q[1].tolist() == [0] * 4 and float(s[1]) == 0.0
    assert math.isnan(float(s[2])) and math.isnan(float(s[3])) and not bool(q[2:4].any())
    # 1 / fl32(2 / 127): the FP32 quotient decides on which side of 63.5 it falls
    scale = torch.tensor(2.0) / 127
    assert float(s[4]) == float(scale)
    want = torch.round(x[4] / scale)
    assert q[4].tolist() == want.to(torch.int8).tolist()


def test_int8_is_a_product_of_what_the_codes_stand_for():
    A = torch.randint(-128, 128, (4, 32), generator=torch.Generator().manual_seed(1)).to(torch.int8)
    B = torch.randint(-128, 128, (6, 32), generator=torch.Generator().manual_seed(2)).to(torch.int8)
    sa, sb = _rand(4, seed=3).abs(), _rand(6, seed=4).abs()
    y, s = o.int8(A, B, sa, sb)
    assert torch.allclose(y, (A.double() * sa[:, None]) @ (B.double() * sb[:, None]).t(), rtol=1e-13)
    assert bool((y.abs() <= s * (1 + 1e-12)).all())
    assert torch.equal(o.int8(A, B, torch.ones(1), torch.ones(1))[0], (A.long() @ B.long().t()).double())


@pytest.mark.parametrize("m,n", [(5, 9), (9, 5), (4, 4)])
def test_orthogonalize_maps_singular_values(m, n):
    G = _rand(m, n, seed=m)
    abc = (3.4445, -4.7750, 2.0315)
    U, s, V = torch.linalg.svd(G, full_matrices=False)
    s = s / (s.norm() + 1e-7)
    for _ in range(5):
        s = abc[0] * s + abc[1] * s ** 3 + abc[2] * s ** 5
    assert torch.allclose(o.orthogonalize(G, 5, abc, 1e-7), (U * s) @ V, rtol=1e-9, atol=1e-10)
    # enough steps of (1.5, -0.5, 0) leave U V^T
    X = o.orthogonalize(torch.stack([G, 3 * G]), 40, (1.5, -0.5, 0.0), 0.0)
    assert torch.allclose(X[0], U @ V, atol=1e-9) and torch.allclose(X[1], U @ V, atol=1e-9)
    # (a sum of squares in another order: within its terms' number of 2^-53)
    assert torch.allclose(o.orthogonalize(G, 0, abc, 0.0), G / G.norm(), rtol=m * n * 2.0 ** -52, atol=0.0)
