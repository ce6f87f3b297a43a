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


# Each kernel of few rows: strips of 16 and 32 columns, split and not; their last k blocks whole and ragged.
@pytest.mark.parametrize("m,n,k", [(1, 4100, 520), (5, 40, 2500), (16, 4200, 64), (16, 1000, 8200), (2, 8200, 1000),
                                   (1, 4096, 2049), (31, 1000, 4104), (24, 8300, 65), (32, 33, 7), (17, 70, 9000)])
def test_few_rows_are_exact_on_integers(pts, m, n, k):
    x, w = padded(m, k, 1, integers=2, pad=float("nan")), padded(n, k, 2, integers=2, pad=float("nan"))
    assert torch.equal(pts.linear(x, w, out_dtype=F32), x.float() @ w.float().t())


def test_zero_sizes(pts):
    for m, n, k in ((0, 8, 8), (8, 0, 8), (8, 8, 0), (0, 0, 0), (40, 300, 0)):
        x, w = padded(m, k, 1), padded(n, k, 2)
        bias = torch.randn(n, device=DEV)
        y, z = pts.linear(x, w, bias, activation="silu", out_dtype=F32, preactivation=True)
        want = bias.double().expand(m, n)
        R.check(y, R.activation(want, "silu"), 32 * R.HALF[F32] * want.abs(), "y")
        R.check(z, want, torch.zeros_like(want), "z")
        dy = padded(m, n, 3)
        dx, dw, db = pts.linear_backward(dy, x, w, z, activation="silu")
        assert dx.shape == (m, k) and dw.shape == (n, k) and db.shape == (n,)
        if m == 0 or n == 0:
            assert not dx.any() and not dw.any() and not db.any()


@pytest.mark.parametrize("act", R.ACTIVATIONS)
def test_activation_of_every_value(pts, act):
    """k = 1 and w = 1: the result is the activation of x, for every finite bf16."""
    bits = torch.arange(65536, device=DEV, dtype=torch.int32).to(torch.int16)
    v = bits.view(BF16)
    v = v[torch.isfinite(v)]
    x = torch.zeros((v.numel(), 8), device=DEV, dtype=BF16)
    x[:, 0] = v
    one = torch.ones((1, 8), device=DEV, dtype=BF16)
    got = pts.linear(x[:, :1], one[:, :1], activation=act, out_dtype=F32)[:, 0]
    want, _, bound, _ = R.linear(x[:, :1], one[:, :1], act=act)
    R.check(got, want[:, 0], bound[:, 0], str(act))


@pytest.mark.parametrize("act", R.ACTIVATIONS[1:])
def test_slope_of_every_value(pts, act):
    """m = 1 and dy = 1: dbias is the slope at z, dw its rounding, for every finite bf16."""
    v = torch.arange(65536, device=DEV, dtype=torch.int32).to(torch.int16).view(BF16)
    v = v[torch.isfinite(v)]
    z = torch.zeros((1, (v.numel() + 7) // 8 * 8), device=DEV, dtype=BF16)[:, :v.numel()]
    z[0] = v
    dy, x, w = torch.ones_like(z), torch.ones((1, 8), device=DEV, dtype=BF16), torch.ones((v.numel(), 8), device=DEV, dtype=BF16)
    _, dw, db = pts.linear_backward(dy, x, w, z, activation=act, dw_dtype=F32, need_dx=False)
    want, off = R.slope_bound(dy, z, act)
    R.check(db, want[0], off[0] + 2 * R.HALF[F32] * want[0].abs(), act)
    for c in range(8):
        assert torch.equal(dw[:, c], db.bfloat16().float())


# The least work for each choice of tiles (256, 128 by four or eight waves, 64), none, some or all of them shared.
@pytest.mark.parametrize("m,n,k", [(70, 200, 40), (70, 200, 1500), (1777, 2500, 40), (1000, 1300, 8000), (2049, 4100, 2100),
                                   (1000, 2049, 40), (200, 1777, 8000), (1000, 4100, 2100), (2049, 4100, 40),
                                   (1777, 3001, 8000), (4100, 5000, 4000)])
def test_every_choice_of_tiles(pts, m, n, k):
    """The three ways the operands lie, each with the contraction k: exact on integers, edges followed by NaN."""
    def take(a, b, seed):
        return padded(a, b, seed, integers=2, pad=float("nan"))
    x, w = take(m, k, 1), take(n, k, 2)
    assert torch.equal(pts.linear(x, w, out_dtype=F32), x.float() @ w.float().t())
    dy, w, x = take(m, k, 3), take(k, n, 4), take(m, n, 5)
    dx = pts.linear_backward(dy, x, w, need_dw=False, need_dbias=False).dx
    assert torch.equal(dx, (dy.float() @ w.float()).bfloat16())
    dy, x, w = take(k, m, 6), take(k, n, 7), take(m, n, 8)
    dw = pts.linear_backward(dy, x, w, need_dx=False, need_dbias=False, dw_dtype=F32).dw
    assert torch.equal(dw, dy.float().t() @ x.float())
