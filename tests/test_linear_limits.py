"""The linear layer's C ABI and binding at their limits, without a GPU: what is refused, and what is not."""
from __future__ import annotations

import re

import numpy as np
import pytest
import torch

P = 4096            # a pointer that passes the alignment checks; nothing here reaches a launch
BIG = 1 << 62
MOST = 2 ** 31 - 1025   # the largest extent


@pytest.fixture(scope="module")
def pts():
    import persistent_tile_scheduling_amd as mod
    return mod


def refused(pts, call, status, fragment):
    with pytest.raises(pts.GemmError) as ei:
        call()
    assert ei.value.status == status and fragment in str(ei.value), str(ei.value)


LINEAR = dict(x=P, ldx=64, w=P, ldw=64, bias=None, dtype_bias=0, act=0, residual=None, ldr=0, y=P, ldy=40, dtype=0, z=None,
              ldz=0, m=33, n=40, k=64, work=P, bytes=BIG)
BACK = dict(dy=P, ld_dy=40, z=P, ldz=40, act=4, x=P, ldx=64, w=P, ldw=64, dx=P, ld_dx=64, dw=P, ld_dw=64, dtype=0, db=P,
            m=33, n=40, k=64, work=P, bytes=BIG)
ORTHO = dict(x=P, dtype=0, ldx=64, xs=0, count=1, rows=40, cols=64, steps=5, a=3.4445, b=-4.775, c=2.0315, eps=1e-7, out=P,
             ldo=64, os=0, work=P, bytes=BIG)


def test_the_largest_extents(pts):
    """Extents are below 2^31 - 1024: one less passes their check (and is refused for its pointer here)."""
    for most, fragment in ((MOST, "x: NULL"), (MOST + 1, "m, n and k")):
        refused(pts, lambda: pts.pts_linear(*{**LINEAR, "m": most, "x": None}.values(), stream=0), 1, fragment)
    for most, fragment in ((MOST, "dy: NULL"), (MOST + 1, "m, n and k")):
        refused(pts, lambda: pts.pts_linear_backward(*{**BACK, "m": most, "dy": None}.values(), stream=0), 1, fragment)
    for most, fragment in ((MOST, "x: NULL"), (MOST + 1, "count, rows and cols")):
        refused(pts, lambda: pts.pts_orthogonalize(*{**ORTHO, "rows": most, "x": None}.values(), stream=0), 1, fragment)


def test_workspaces_of_refused_sizes(pts):
    """0, and no overflow on the way, wherever no pointers and strides make the sizes' call pass."""
    wide = 2 ** 22 - 8      # the widest operand
    assert pts.pts_linear_workspace(40, 300, wide) > 0 and pts.pts_linear_workspace(40, 300, wide + 1) == 0
    assert pts.pts_linear_workspace(4, 300, wide) > 0 and pts.pts_linear_workspace(4, 300, wide + 1) == 0
    assert pts.pts_linear_workspace(MOST, MOST, 8) == 0
    for act in range(5):
        assert pts.pts_linear_backward_workspace(MOST, MOST, MOST, act) == 0
        assert pts.pts_linear_backward_workspace(300, wide, 40, act) > 0
        assert pts.pts_linear_backward_workspace(300, wide + 1, 40, act) == 0
        assert pts.pts_linear_backward_workspace(300, wide, MOST, act) > 0     # a call for the bias alone does not look at k
    assert pts.pts_linear_backward_workspace(MOST, 300, 40, 1) > 2 * MOST * 300
    assert pts.pts_linear_backward_workspace(64, 72, 64, 4) == 64 * 128 * 2     # dz has rows of whole cache lines
    ortho = pts.pts_orthogonalize_workspace
    assert ortho(65535, 64, 64, 5) > 0 and ortho(65536, 64, 64, 5) == 0 and ortho(65536, 80, 80, 5) == 0
    assert ortho(1, 64, 2 ** 22 - 64, 5) > 0 and ortho(1, 64, 2 ** 22 - 63, 5) == 0
    assert ortho(1, 70, 2 ** 22 - 64, 5) > 0 and ortho(1, 70, 2 ** 22 - 63, 5) == 0 and ortho(1, 2 ** 22 - 63, 70, 5) > 0
    assert ortho(65535, 64, 2 ** 15, 5) == 0      # too large for one launch
    assert ortho(MOST, MOST, MOST, 64) == 0 and ortho(1, MOST, 64, 64) == 0 and ortho(1, 2 ** 29, 64, 64) > 0


@pytest.mark.parametrize("change,fragment", [
    (dict(x=None), "x must be"), (dict(w=None), "w must be"), (dict(w=None, need_dw=False), "w must be"),
    (dict(x=None, need_dx=False), "x must be"), (dict(x=torch.zeros(5, 8).bfloat16()), "(5, 8)"),
    (dict(x=torch.zeros(5, 8).bfloat16(), need_dx=False), "w None do not fit"),
    (dict(w=torch.zeros(9, 8).bfloat16(), need_dw=False), "x None and w (9, 8) do not fit"),
    (dict(w=torch.zeros(8, 16).bfloat16()), "do not fit"),
])
def test_operands_that_are_needed(pts, change, fragment):
    given = dict(dy=torch.zeros(4, 8).bfloat16(), x=torch.zeros(4, 8).bfloat16(), w=torch.zeros(8, 8).bfloat16())
    with pytest.raises(ValueError, match=re.escape(fragment)):
        pts.linear_backward(**{**given, **change})


@pytest.mark.parametrize("change,fragment", [
    (dict(residual=3.0), "residual must be bfloat16 of shape (4, 8), not float"), (dict(out=[1]), "out must be"),
    (dict(residual=torch.zeros(4, 8)), "residual must be bfloat16"), (dict(residual=torch.zeros(4, 9).bfloat16()), "residual must be"),
    (dict(out=torch.zeros(4, 8).half()), "out must be"), (dict(out=torch.zeros(4, 8), residual=torch.zeros(4, 8).bfloat16()), "residual must be float32"),
    (dict(bias=1.0), "bias must be"),
])
def test_what_is_no_fitting_tensor(pts, change, fragment):
    with pytest.raises(ValueError, match=re.escape(fragment)):
        pts.linear(torch.zeros(4, 8).bfloat16(), torch.zeros(8, 8).bfloat16(), **change)


@pytest.mark.parametrize("steps", [5.7, 0, 65, 2 ** 32 + 5, -1, "5", None])
def test_steps_are_a_whole_number_within_the_range(pts, steps, monkeypatch):
    """Nothing is cut off or wrapped to a number of steps that is in the range."""
    from persistent_tile_scheduling_amd import experts
    monkeypatch.setattr(experts, "_current", lambda: 0)
    with pytest.raises(ValueError, match="steps must be a whole number"):
        pts.orthogonalize(torch.zeros(4, 4), steps)


@pytest.mark.parametrize("steps", [5, 5.0, np.int64(64), np.float32(1), torch.tensor(5)])
def test_whole_numbers_of_any_type_are_steps(pts, steps):
    with pytest.raises(ValueError, match="not on the current GPU"):     # the next thing that is checked
        pts.orthogonalize(torch.zeros(4, 4), steps)


@pytest.mark.parametrize("rows,coefficients,steps", [
    # p maps [0, 1] (0 to 2, to 7) onto itself and grows 25-fold (9-fold) beyond: roundings leave it in some steps
    (80, (5.0, -20.0, 16.0), 3), (40, (5.0, -20.0, 16.0), 5), (80, (3.0, -1.0, 0.0), 5), (40, (3.0, -1.0, 0.0), 7),
    (80, (3.0, -4 / 49, 0.0), 5), (80, (5.0, -20.0, 16.0), 64), (40, (5.0, -20.0, 16.0), 64),
])
def test_coefficients_that_roundings_carry_away(pts, rows, coefficients, steps):
    a, b, c = coefficients
    given = {**ORTHO, "rows": rows, "cols": 100, "ldx": 100, "ldo": 100, "a": a, "b": b, "c": c}
    refused(pts, lambda: pts.pts_orthogonalize(*{**given, "steps": steps}.values(), stream=0), 1, "fp16's reach")
    # one step fewer is taken (and refused for its pointer here)
    fewer = steps - 1 if steps < 10 else 2
    refused(pts, lambda: pts.pts_orthogonalize(*{**given, "steps": fewer, "x": None}.values(), stream=0), 1, "x: NULL")


@pytest.mark.parametrize("rows", [40, 80])
@pytest.mark.parametrize("coefficients", [(3.4445, -4.775, 2.0315), (1.5, -0.5, 0.0), (1.875, -1.25, 0.375), (2.0, -1.5, 0.5),
                                          (3.0, -3.2, 1.2), (1.0, 0.0, 0.0), (0.1, 0.0, 0.0), (2.6, -1.0, 0.0)])
def test_coefficients_that_stay(pts, rows, coefficients):
    a, b, c = coefficients
    given = {**ORTHO, "rows": rows, "cols": 100, "ldx": 100, "ldo": 100, "a": a, "b": b, "c": c, "steps": 64, "x": None}
    refused(pts, lambda: pts.pts_orthogonalize(*given.values(), stream=0), 1, "x: NULL")
