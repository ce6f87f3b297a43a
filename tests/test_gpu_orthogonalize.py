"""Newton-Schulz steps on the GPU against 64-bit references."""
from __future__ import annotations

import pytest
import torch

from tests import linear_reference as R

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.fixture(scope="module")
def pts():
    import persistent_tile_scheduling_amd as mod
    return mod


def matrix(shape, seed, dtype, rank=None):
    g = torch.Generator(device=DEV).manual_seed(seed)
    x = torch.randn(shape, generator=g, device=DEV)
    if rank is not None:
        u = torch.randn((*shape[:-1], rank), generator=g, device=DEV)
        x = torch.matmul(u, torch.randn((*shape[:-2], rank, shape[-1]), generator=g, device=DEV))
    return (1e-3 * x).to(dtype)


def check(got, x, **how):
    """Within a bf16 rounding of every element of what the stated roundings give (a sum's order turns a few of them the
    other way), and as near to the exact result as those allow."""
    exact, rounded = R.orthogonalize(x, **how), R.orthogonalize(x, rounded=True, **how)
    size = exact.norm()
    assert torch.isfinite(got).all()
    assert (got.double() - rounded).norm() <= 2 * R.HALF[torch.bfloat16] * size
    assert (got.double() - exact).norm() <= (rounded - exact).norm() + 2 * R.HALF[torch.bfloat16] * size


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("shape", [(1, 1), (1, 9), (7, 1), (16, 16), (64, 65), (130, 63), (200, 1000), (1025, 257),
                                   (3, 100, 60), (2, 260, 384), (5, 17, 64), (4, 64, 17), (33, 5000), (5000, 64),
                                   (2, 9, 20000), (65, 65), (3, 66, 130)])
def test_orthogonalize(pts, shape, dtype):
    x = matrix(shape, 1, dtype)
    check(pts.orthogonalize(x), x)
