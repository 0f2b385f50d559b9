"""The key/value cache calls where magnitudes lie far apart or at the ends of their types."""
import numpy as np
import pytest
import torch

from tests import kv_reference as R
from tests import test_gpu_kv as T

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------------ append
@pytest.mark.parametrize("fmt", [R.INT8, R.E4M3])
@pytest.mark.parametrize("top", [2e9, 1e20, 3e38])
def test_append_quotients_that_underflow(fmt, top):
    """x / s below the smallest subnormal is a zero with x's sign, whatever its sign, and no NaN."""
    page, dim, heads = 16, 64, 1
    x = torch.zeros(2, 5, dim)
    x[:, :, 0] = top
    tiny = torch.tensor([1e-40, 9.2e-41, 1.2e-38, 1e-36, 1e-30, 1e-20, 1e-10])
    for t in range(5):
        x[0, t, 1 + t:8 + t], x[1, t, 1 + t:8 + t] = tiny, -tiny
        x[0, t, 20 + t:27 + t], x[1, t, 20 + t:27 + t] = -tiny, tiny
    codes, scales = T.make_cache(9, fmt, 2, heads, page, dim)
    T.check_append(fmt, 1, page, dim, heads, codes, scales, x.bfloat16(), np.arange(5))
