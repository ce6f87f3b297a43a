"""Newton-Schulz steps of short sides on the GPU, for any number of steps and matrices of any rank."""
from __future__ import annotations

import pytest
import torch

from tests import steps_reference as S

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pts():
    import persistent_tile_scheduling_amd as mod
    return mod


@pytest.mark.parametrize("steps", [5, 8, 9, 10, 20, 64])
@pytest.mark.parametrize("kind", S.MATRICES)
@pytest.mark.parametrize("coefficients", [S.QUINTIC, S.CUBIC])
def test_many_steps(pts, kind, coefficients, steps):
    x = S.matrix(kind)
    y = pts.orthogonalize(x.cuda(), steps, coefficients)
    S.check(x, y if x.shape[0] <= x.shape[1] else y.t(), steps, coefficients, S.HALF_BF16)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("shape", [(3, 20, 301), (3, 301, 20), (2, 64, 64), (300, 7, 9), (1, 4999)])
def test_stacks_and_strides_between_chains(pts, shape, dtype):
    """Twenty steps write X between chains: each matrix of a stack as by itself, from rows that start anywhere into such."""
    g = torch.Generator().manual_seed(2)
    x = torch.randn(shape, generator=g).to(dtype)
    wide = torch.full((*shape[:-2], shape[-2] + 3, shape[-1] + 7), float("nan"), dtype=dtype, device="cuda")
    inside = wide[..., 2:2 + shape[-2], 3:3 + shape[-1]]
    inside.copy_(x)
    out = torch.full_like(wide, float("nan"), dtype=torch.bfloat16)
    place = out[..., 1:1 + shape[-2], 5:5 + shape[-1]]
    pts.orthogonalize(inside, 20, out=place)
    outside = torch.ones_like(out, dtype=torch.bool)
    outside[..., 1:1 + shape[-2], 5:5 + shape[-1]] = False
    assert torch.isnan(out[outside]).all()
    for i, (one, y) in enumerate(zip(x, place) if len(shape) == 3 else [(x, place)]):
        assert torch.equal(pts.orthogonalize(one.cuda(), 20), y)
        if i < 3:
            S.check(one, y if one.shape[0] <= one.shape[1] else y.t(), 20, S.QUINTIC, S.HALF_BF16)


def test_infinities_and_zeros_after_many_steps(pts):
    x = torch.randn((4, 20, 90), generator=torch.Generator().manual_seed(3)).cuda()
    clean = pts.orthogonalize(x, 20)
    x[0] = 0
    x[1, 3, 5] = float("inf")
    x[2, 3, 5] = float("nan")
    y = pts.orthogonalize(x, 20)
    assert not y[0].any() and torch.isnan(y[1:3]).all() and torch.equal(y[3], clean[3])


def test_captured(pts):
    x = torch.randn((40, 333), generator=torch.Generator().manual_seed(4)).cuda()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        pts.orthogonalize(x, 20)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = pts.orthogonalize(x, 20)
    for seed in range(3):
        x.copy_(torch.randn((40, 333), generator=torch.Generator().manual_seed(seed)))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, pts.orthogonalize(x, 20))


@pytest.mark.parametrize("eps", [5e-324, 1e-310, 1e-7])
@pytest.mark.parametrize("shape", [(20, 30), (80, 90)])
def test_zeros_stay_zero_with_any_eps(pts, shape, eps):
    x = torch.zeros((2, *shape), device="cuda")
    x[1] = torch.randn(shape, generator=torch.Generator().manual_seed(5)).cuda()
    y = pts.orthogonalize(x, eps=eps)
    assert not y[0].any() and torch.isfinite(y[1]).all() and y[1].any()


@pytest.mark.parametrize("coefficients,steps,top", [
    (S.QUINTIC, 64, 1.22), (S.CUBIC, 64, 1.01), ((2.0, -1.5, 0.5), 64, 1.01), ((3.0, -3.2, 1.2), 64, 1.23), ((2.6, -1.0, 0.0), 64, 1.63),
    ((5.0, -20.0, 16.0), 2, 2.1), ((3.0, -1.0, 0.0), 4, 6.8), ((3.0, -4 / 49, 0.0), 4, 7.7)])
@pytest.mark.parametrize("shape", [(40, 90), (80, 90), (90, 80), (200, 500)])
def test_accepted_coefficients_stay_within_reach(pts, shape, coefficients, steps, top):
    """Singular values at the end of the range (rank 1), inside it, and directions that x does not have."""
    g = torch.Generator().manual_seed(6)
    for rank in (1, 3, min(shape)):
        x = torch.randn((shape[0], rank), generator=g) @ torch.randn((rank, shape[1]), generator=g)
        y = pts.orthogonalize(x.cuda(), steps, coefficients).double().cpu()
        assert torch.isfinite(y).all()
        assert torch.linalg.matrix_norm(y, ord=2) <= top * (1 + S.HALF_BF16), (rank, torch.linalg.matrix_norm(y, ord=2))
