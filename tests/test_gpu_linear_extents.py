"""The linear layer's operators at the ends of their documented extents."""
from __future__ import annotations

import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF16 = torch.bfloat16
MOST = 2 ** 31 - 1025   # the largest extent


@pytest.fixture(scope="module")
def pts():
    import persistent_tile_scheduling_amd as mod
    return mod


def test_bias_gradient_of_the_most_rows(pts):
    """The last workgroup's rows end past 2^31 when they are rounded up."""
    dy = torch.zeros((MOST, 8), device=DEV, dtype=BF16)     # 34 GB
    dy[:100] = 1
    dy[-9_000_000:] = 1                                     # more than a workgroup's rows
    x, w = torch.empty((MOST, 0), device=DEV, dtype=BF16), torch.empty((8, 0), device=DEV, dtype=BF16)
    got = pts.linear_backward(dy, x, w, need_dx=False, need_dw=False).dbias
    assert (got == 9_000_100).all(), got
