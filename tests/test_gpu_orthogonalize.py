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


@pytest.mark.parametrize("rank", [1, 5, 30])
@pytest.mark.parametrize("shape", [(70, 900), (300, 200), (40, 400)])
def test_low_rank(pts, shape, rank):
    """Directions that x does not have stay as small as the matrix's sixteen-odd bits leave them."""
    x = matrix(shape, 3, torch.float32, rank=rank)
    check(pts.orthogonalize(x), x)


@pytest.mark.parametrize("coefficients", [(1.5, -0.5, 0.0), (1.875, -1.25, 0.375), (2.0, -1.5, 0.5), (1.0, 0.0, 0.0)])
@pytest.mark.parametrize("steps", [1, 2, 9])
def test_other_steps(pts, steps, coefficients):
    for shape in ((90, 130), (20, 300)):
        x = matrix(shape, 4, torch.bfloat16)
        check(pts.orthogonalize(x, steps, coefficients), x, steps=steps, coefficients=coefficients)


@pytest.mark.parametrize("scale", [1e33, 1e-3, 1e-28])
@pytest.mark.parametrize("shape", [(80, 100), (30, 100)])
def test_any_scale(pts, shape, scale):
    """The norm is of 64 bits: a matrix whose squares no float holds comes out the same."""
    x = matrix(shape, 5, torch.float32) * 1e3
    eps = 1e-7 * scale
    check(pts.orthogonalize(x * scale, eps=eps), x * scale, eps=eps)


def test_eps_shrinks_small_matrices(pts):
    for shape in ((80, 100), (30, 100)):
        x = matrix(shape, 6, torch.float32) * 1e-9
        check(pts.orthogonalize(x), x)


def test_zeros_stay_and_infinities_keep_to_their_matrix(pts):
    for shape in ((4, 70, 90), (4, 20, 90)):
        x = matrix(shape, 7, torch.bfloat16)
        clean = pts.orthogonalize(x)
        x[0] = 0
        x[1, 3, 5] = float("inf")
        x[2, 3, 5] = float("nan")
        y = pts.orthogonalize(x)
        assert not y[0].any() and torch.isnan(y[1:3]).all() and torch.equal(y[3], clean[3])


@pytest.mark.parametrize("shape", [(70, 200), (200, 70), (30, 200), (3, 90, 101), (3, 20, 101)])
def test_strides(pts, shape):
    """Rows that start anywhere, transposes, stacks apart from each other; results in place, nothing else written."""
    for dtype in (torch.bfloat16, torch.float32):
        x = matrix(shape, 8, dtype)
        want = pts.orthogonalize(x)
        wide = torch.full((*shape[:-2], shape[-2] + 3, shape[-1] + 7), float("nan"), device=DEV, dtype=dtype)
        inside = wide[..., 2:2 + shape[-2], 3:3 + shape[-1]]
        inside.copy_(x)
        assert torch.equal(pts.orthogonalize(inside), want)
        out = torch.full_like(wide, float("nan"), dtype=torch.bfloat16)
        place = out[..., 1:1 + shape[-2], 5:5 + shape[-1]]
        assert pts.orthogonalize(inside, out=place) is place and torch.equal(place, want)
        untouched = torch.ones_like(out, dtype=torch.bool)
        untouched[..., 1:1 + shape[-2], 5:5 + shape[-1]] = False
        assert torch.isnan(out[untouched]).all()
        t = x.transpose(-1, -2).contiguous().transpose(-1, -2)      # the columns are contiguous
        check(pts.orthogonalize(t), x)
        turned = torch.full((*shape[:-2], shape[-1], shape[-2]), 0.0, device=DEV, dtype=torch.bfloat16).transpose(-1, -2)
        assert pts.orthogonalize(t, out=turned) is turned and torch.equal(turned, pts.orthogonalize(t))


def test_empty(pts):
    for shape in ((0, 8), (8, 0), (0, 4, 4), (3, 0, 5)):
        assert pts.orthogonalize(torch.empty(shape, device=DEV)).shape == shape


@pytest.mark.parametrize("shape", [(1100, 1100), (2300, 700), (5, 520, 1000), (600, 6000), (8, 1024, 2048), (4100, 1500),
                                   (1500, 4100), (2304, 2304)])
def test_larger_tiles(pts, shape):
    x = matrix(shape, 9, torch.bfloat16)
    check(pts.orthogonalize(x), x)


def test_stack_past_32_bits(pts):
    """5 GB of matrices, all different: the last ones against the same matrices by themselves and the definition."""
    count, side = 620, 1450
    g = torch.Generator(device=DEV).manual_seed(1)
    x = torch.randn((count, side, side), generator=g, device=DEV)
    y = pts.orthogonalize(x)
    for i in (0, 409, 410, count - 1):
        check(y[i], x[i])


def test_same_call_same_bits(pts):
    for shape in ((300, 500), (40, 3000), (2, 500, 300)):
        x = matrix(shape, 10, torch.bfloat16)
        first = pts.orthogonalize(x)
        assert all(torch.equal(first, pts.orthogonalize(x)) for _ in range(3))
