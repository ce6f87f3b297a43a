"""orthogonalize between matrices whose rows and whose columns are contiguous, in place, in every combination."""
from __future__ import annotations

import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.fixture(scope="module")
def pts():
    import persistent_tile_scheduling_amd as mod
    return mod


def laid(shape, dtype, turned, apart):
    """An empty matrix (a stack) with its rows or its columns contiguous, and others' memory between them if `apart`."""
    *stack, rows, cols = shape
    if turned:
        rows, cols = cols, rows
    wide = torch.full((*stack, rows + 3 * apart, cols + 5 * apart), float("nan"), dtype=dtype, device=DEV)
    inside = wide[..., apart:apart + rows, 2 * apart:2 * apart + cols]
    return (inside.transpose(-1, -2) if turned else inside), wide


@pytest.mark.parametrize("apart", [0, 1])
@pytest.mark.parametrize("x_turned,out_turned", [(False, False), (False, True), (True, False), (True, True)])
@pytest.mark.parametrize("shape", [(90, 130), (130, 90), (3, 70, 81), (20, 33), (3, 33, 20), (1, 40), (40, 1), (3, 1, 40), (1, 1)])
def test_every_layout(pts, shape, x_turned, out_turned, apart):
    g = torch.Generator(device=DEV).manual_seed(1)
    value = torch.randn(shape, generator=g, device=DEV)
    x, _ = laid(shape, torch.float32, x_turned, apart)
    x.copy_(value)
    want = pts.orthogonalize(x)
    out, wide = laid(shape, torch.bfloat16, out_turned, apart)
    assert pts.orthogonalize(x, out=out) is out
    assert torch.equal(out, want)
    assert torch.isnan(wide).sum() == wide.numel() - out.numel()     # nothing else is written


def test_a_row_of_any_stride(pts):
    x = torch.randn((1, 60), device=DEV)
    buf = torch.full((1, 180), float("nan"), device=DEV, dtype=torch.bfloat16)
    want = pts.orthogonalize(x)
    for a in (x, x.repeat_interleave(2, 1)[:, ::2]):
        assert torch.equal(pts.orthogonalize(a, out=buf[:, ::3]), want)
    assert torch.isnan(buf).sum() == 120


def test_overlapping_results_are_refused(pts):
    x = torch.randn((3, 20, 30), device=DEV)
    t = x.transpose(-1, -2).contiguous().transpose(-1, -2)
    buf = torch.zeros(4000, device=DEV, dtype=torch.bfloat16)
    for strides in ((599, 30, 1), (0, 30, 1), (20, 40, 1)):
        for a in (x, t):
            with pytest.raises((ValueError, pts.GemmError), match="overlap"):
                pts.orthogonalize(a, out=buf.as_strided((3, 20, 30), strides))
    for strides in ((599, 1, 20), (0, 1, 20), (20, 1, 40)):
        for a in (x, t):
            with pytest.raises((ValueError, pts.GemmError), match="overlap"):
                pts.orthogonalize(a, out=buf.as_strided((3, 20, 30), strides))
    for strides in ((600, 30, 1), (30, 90, 1), (600, 1, 20), (20, 1, 60)):
        for a in (x, t):
            out = buf.as_strided((3, 20, 30), strides)
            assert torch.equal(pts.orthogonalize(a, out=out), pts.orthogonalize(a))
    with pytest.raises(ValueError, match="unit stride"):
        pts.orthogonalize(t, out=torch.zeros((3, 20, 60), device=DEV, dtype=torch.bfloat16)[..., ::2])
    with pytest.raises(ValueError, match="unit stride"):
        pts.orthogonalize(x, out=torch.zeros((3, 20, 60), device=DEV, dtype=torch.bfloat16)[..., ::2])
