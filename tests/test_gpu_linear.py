"""The linear layer's operators on the GPU against 64-bit references."""
from __future__ import annotations

import pytest
import torch

from tests import linear_reference as R

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def pts():
    import persistent_tile_scheduling_amd as mod
    return mod


def padded(m, n, seed, dtype=BF16, scale=1.0, integers=0, pad=None):
    """An m x n matrix whose rows start at whole 16 bytes and are followed by other values, NaN if `pad` says so."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    ld = 8 * ((n + 7) // 8)
    if integers:
        t = torch.randint(-integers, integers + 1, (m, ld), generator=g, device=DEV).to(dtype)
    else:
        t = (torch.randn((m, ld), generator=g, device=DEV) * scale).to(dtype)
    if pad is not None:
        t[:, n:] = pad
    return t[:, :n]


# Sizes at and around the edges of tiles, k tiles, strips of few rows and 16-byte pieces.
SHAPES = [(1, 1, 1), (1, 16, 8), (3, 17, 9), (16, 64, 64), (17, 33, 65), (32, 130, 200), (33, 8, 64), (64, 64, 63),
          (65, 65, 129), (129, 127, 192), (200, 72, 1000), (257, 300, 136), (300, 257, 321), (128, 128, 4096)]


@pytest.mark.parametrize("m,n,k", SHAPES)
def test_linear_is_exact_on_integers(pts, m, n, k):
    x, w = padded(m, k, 1, integers=3, pad=float("nan")), padded(n, k, 2, integers=3, pad=float("nan"))
    got = pts.linear(x, w, out_dtype=F32)
    want = x.double() @ w.double().t()
    assert torch.equal(got.double(), want)


@pytest.mark.parametrize("m,n,k", SHAPES)
def test_gradients_are_exact_on_integers(pts, m, n, k):
    dy, x, w = (padded(m, n, 1, integers=2, pad=float("nan")), padded(m, k, 2, integers=2, pad=float("nan")),
                padded(n, k, 3, integers=2, pad=float("nan")))
    dx, dw, db = pts.linear_backward(dy, x, w, dw_dtype=F32)
    assert torch.equal(dw.double(), dy.double().t() @ x.double())
    assert torch.equal(db.double(), dy.double().sum(0))
    want = dy.double() @ w.double()
    R.check(dx, want, torch.zeros_like(want), "dx")


# One size in each kind of tile: 256 x 256, 128 x 128, and split contractions of both.
@pytest.mark.parametrize("m,n,k", [(3000, 3100, 200), (2300, 2100, 136), (1000, 1100, 4160), (300, 500, 9000)])
def test_large_tiles_are_exact_on_integers(pts, m, n, k):
    x, w = padded(m, k, 1, integers=2, pad=float("nan")), padded(n, k, 2, integers=2, pad=float("nan"))
    assert torch.equal(pts.linear(x, w, out_dtype=F32), x.float() @ w.float().t())
    dy = padded(m, n, 3, integers=1, pad=float("nan"))
    dx, dw, db = pts.linear_backward(dy, x, w, dw_dtype=F32)
    assert torch.equal(dw, dy.float().t() @ x.float())
    assert torch.equal(dx, (dy.float() @ w.float()).bfloat16())
    assert torch.equal(db, dy.float().sum(0))
