"""The layer products at the ends of their ranges."""
import math

import pytest
import torch

from tests.rows_util import randn

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF16, FP16, FP32 = torch.bfloat16, torch.float16, torch.float32


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
