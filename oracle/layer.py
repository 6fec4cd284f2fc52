"""The products of a feed-forward layer in 64 bits, from their formulas: the gated block and
its gradients, quantization and the product in 8-bit integers, the orthogonalized
update.  Torch tensors on the CPU; nothing here is shared with the HIP side."""
from __future__ import annotations

import math

import torch

F64 = torch.float64


def gate(v, activation):
    """act(v), act'(v) (0 at ReLU's corner)."""
    if activation == "relu":
        return torch.clamp(v, min=0), (v > 0).to(F64)
    if activation == "silu":
        s = torch.sigmoid(v)
        return v * s, s * (1 + v * torch.sigmoid(-v))
    assert activation == "gelu"
    cdf = 0.5 * torch.special.erfc(-v * math.sqrt(0.5))
    return v * cdf, cdf + v * torch.exp(-0.5 * v * v) / math.sqrt(2 * math.pi)


def gated(x, Wg, Wu, activation):
    """(h, g, u)."""
    x = x.to(F64)
    g, u = x @ Wg.to(F64).t(), x @ Wu.to(F64).t()
    return gate(g, activation)[0] * u, g, u


def gated_backward(dh, x, Wg, Wu, activation):
    """(dx, dWg, dWu, dg, du)."""
    _, g, u = gated(x, Wg, Wu, activation)
    a, slope = gate(g, activation)
    dh, x = dh.to(F64), x.to(F64)
    dg, du = dh * u * slope, dh * a
    return dg @ Wg.to(F64) + du @ Wu.to(F64), dg.t() @ x, du.t() @ x, dg, du


def quantize(x):
    """(codes, scale) of the rows: scale and the quotients are FP32 numbers by definition
    (a 64-bit quotient of two FP32 numbers rounds to FP32 as the exact one does)."""
    x = x.to(F64)
    top = x.abs().amax(1) if x.shape[1] else x.new_zeros(x.shape[0])
    fine = torch.isfinite(top)
    scale = (top / 127).to(torch.float32)
    some = fine & (scale > 0)
    s = torch.where(some, scale.to(F64), torch.ones_like(top))
    q = torch.round((torch.where(some[:, None], x, torch.zeros_like(x)) / s[:, None]).to(torch.float32).to(F64))
    scale = torch.where(fine, scale, torch.full_like(scale, math.nan))
    return q.clamp(-127, 127).to(torch.int8), scale


def int8(A, B, scale_a, scale_b):
    """(y, sum |terms|)."""
    a, b = A.to(F64), B.to(F64)
    s = scale_a.to(F64).reshape(-1, 1) * scale_b.to(F64).reshape(1, -1)
    return (a @ b.t()) * s, (a.abs() @ b.abs().t()) * s.abs()


def orthogonalize(G, steps, coefficients, eps):
    """X <- a X + b (X X^T) X + c (X X^T)^2 X, `steps` times from G / (||G|| + eps): the odd
    polynomial a s + b s^3 + c s^5 of every singular value s."""
    a, b, c = coefficients
    X = G.to(F64)
    flip = X.shape[-2] > X.shape[-1]
    X = X.transpose(-1, -2) if flip else X
    X = X / (torch.sqrt((X * X).sum((-1, -2), keepdim=True)) + eps)
    for _ in range(steps):
        S = X @ X.transpose(-1, -2)
        X = a * X + (b * S + c * (S @ S)) @ X
    return X.transpose(-1, -2) if flip else X
