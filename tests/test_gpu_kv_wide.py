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
