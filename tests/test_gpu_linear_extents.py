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


def test_bias_gradient_alone_takes_no_room_for_dz(pts):
    """dz of these rows would be 256 GB."""
    dy = torch.zeros((MOST, 8), device=DEV, dtype=BF16)     # 34 GB, and z too
    dy[:100] = 1
    dy[-9_000_000:] = 1
    got = pts.linear_backward(dy, None, None, dy, activation="relu", need_dx=False, need_dw=False).dbias
    assert (got == 9_000_100).all(), got


@pytest.mark.parametrize("m", [3, 256, 257, 3000])
def test_bias_gradient_alone_in_the_workspace_that_it_needs(pts, m):
    n = 1000
    dy, z = torch.randn((m, n), device=DEV).bfloat16(), torch.randn((m, n), device=DEV).bfloat16()
    want = pts.linear_backward(dy, dy, torch.randn((n, n), device=DEV).bfloat16(), z, activation="gelu").dbias
    need = pts.pts_linear_backward_workspace(m, n, 0, pts.PTS_ACTIVATION_NONE)
    work = torch.full((need + 64,), 77, device=DEV, dtype=torch.uint8)
    db = torch.empty(n, device=DEV)
    pts.pts_linear_backward(dy, n, z, n, pts.PTS_ACTIVATION_GELU, None, 0, None, 0, None, 0, None, 0, 0, db, m, n, 0, work, need)
    assert torch.equal(db, want) and (work[need:] == 77).all()
