"""qnt_kv_attn's tcgen05 kernel: its own tests."""
import math

import pytest
import torch

from tests import kv_reference as R
from tests import test_gpu_kv as T

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dim", [64, 128, 256])
def test_non_finite_queries_stay_in_their_row(dim):
    c = T.make_attn(82, R.INT8, 0, 16, 1, 8, dim, [270, 150], [40, 30])
    y0 = T.call_attn(c)
    c["q"][20, 2, 5], c["q"][60, 7, 0] = math.nan, math.inf
    y1 = T.call_attn(c)
    same = torch.ones(c["tokens"], 8, dtype=torch.bool)
    same[20, 2] = same[60, 7] = False
    assert torch.equal(y0[same], y1[same]) and y1[20, 2].isnan().all()


@pytest.mark.parametrize("fmt,xdt,dim", [(R.INT8, 0, 128), (R.E4M3, 1, 64), (R.INT8, 1, 256), (R.E4M3, 0, 128)])
def test_mixed_batches(fmt, xdt, dim):
    """Requests on both sides of the border in one call, of few and of many jobs, full, partial and empty warps of rows."""
    T.check_attn(T.make_attn(dim, fmt, xdt, 16, 1, 1, dim, [400, 50, 300, 0, 97, 1, 260], [97, 1, 200, 0, 97, 1, 129]))
    c = T.make_attn(dim + 1, fmt, xdt, 32, 8, 1, dim, [40] * 13 + [130, 97, 33], [1] * 8 + [32, 33, 31, 34, 40, 97, 96, 33])
    T.check_attn(c)
    T.check_attn(c, max_new=1)
