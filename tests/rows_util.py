"""Tolerances and inputs of the row-indexed products' GPU tests."""
from __future__ import annotations

import torch

U = 2.0 ** -23           # an FP32 addition, were it to truncate (rounding is half of it)
# what is left of a value held as the sum of two 16-bit ones: half a step of each
SPLIT = {torch.bfloat16: 2.0 ** -16, torch.float16: 2.0 ** -22}
TINY = {torch.bfloat16: 2.0 ** -134, torch.float16: 2.0 ** -25, torch.float32: 2.0 ** -150}


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def randn(*shape, seed, dtype=torch.float32, std=1.0):
    return (torch.randn(*shape, generator=torch.Generator().manual_seed(seed)) * std).to(dtype)


def rounded(ref, err, dtype):
    """Bound of a result that is within `err` of `ref` before its rounding to dtype."""
    return err + half_step(dtype) * (ref.abs() + err) + TINY[dtype]


def sum_bound(ref, s, terms, dtype):
    """Bound of an FP32 sum of `terms` exact products with absolute sum s, in any
    order, rounded to dtype once."""
    return rounded(ref, (terms + 64) * U * s, dtype)


def lora_bound(ref, s_base, s_low, terms, inner, rank, in_dtype, out_dtype, tiny=0.0):
    """Bound of a projection's sum (`terms` products) plus its adapters' (rank
    products of low-rank values that are FP32 sums of `inner` products, scaled
    and split into two 16-bit values, of which an absolute `tiny` may be lost)."""
    err = (terms + rank + 64) * U * s_base + ((inner + 2 * rank + 128) * U + SPLIT[in_dtype]) * s_low + tiny
    return rounded(ref, err, out_dtype)


def check(got, ref, bound, what=""):
    got = got.detach().to("cpu", torch.float64)
    assert got.shape == ref.shape, (what, got.shape, ref.shape)
    assert torch.equal(got.isnan(), ref.isnan()), what + ": NaNs in other places"
    inf = ref.isinf()
    assert torch.equal(got[inf], ref[inf]), what + ": other infinities"
    fine = torch.isfinite(ref)
    err = (got - ref).abs()[fine]
    over = err > bound[fine]
    assert not bool(over.any()), "%s: %d of %d over the bound, worst %.3g of it" % (
        what, int(over.sum()), err.numel(), float((err / bound[fine]).max()))
    worst = float((err / bound[fine]).max()) if err.numel() else 0.0
    print("%s: worst/bound %.3g" % (what, worst), flush=True)
