"""The linear layer's C ABI and binding without a GPU: exported names, constants, and every refusal that precedes a launch."""
from __future__ import annotations

import math
import os
import re

import pytest
import torch

from tests import linear_reference as R

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "pts_linear.h")
P = 4096  # a pointer that passes the alignment checks; nothing here reaches a launch


@pytest.fixture(scope="module")
def pts():
    import persistent_tile_scheduling_amd as mod
    return mod


def test_every_declared_function_is_exported_and_bound(pts):
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = sorted(set(re.findall(r"^\s*(?:gemm_status|int64_t)\s+([a-z_0-9]+)\s*\(", text, flags=re.M)))
    assert len(names) == 6
    for n in names:
        assert hasattr(pts._lib, n) and callable(getattr(pts, n)), n


def test_constants_match(pts):
    found = re.findall(r"(PTS_ACTIVATION_[A-Z_]+) = (\d+)", open(HEADER).read())
    assert len(found) == 5
    for name, value in found:
        assert getattr(pts, name) == int(value), name


def _refused(pts, call, status, fragment):
    with pytest.raises(pts.GemmError) as ei:
        call()
    assert ei.value.status == status and fragment in str(ei.value), str(ei.value)


BIG = 1 << 40
LINEAR = dict(x=P, ldx=64, w=P, ldw=64, bias=None, dtype_bias=0, act=0, residual=None, ldr=0, y=P, ldy=40, dtype=0, z=None,
              ldz=0, m=33, n=40, k=64, work=P, bytes=BIG)


@pytest.mark.parametrize("change,status,fragment", [
    (dict(dtype=2), 2, "fp32 or bf16"), (dict(bias=P, dtype_bias=3), 2, "fp32 or bf16"), (dict(act=5), 1, "activation"),
    (dict(act=-1), 1, "activation"), (dict(m=-1), 1, "m, n and k"), (dict(n=2 ** 31), 1, "m, n and k"),
    (dict(k=2 ** 31 - 1024, ldx=2 ** 31, ldw=2 ** 31), 1, "m, n and k"), (dict(ldx=56), 1, "x: leading"),
    (dict(ldw=60, k=60), 1, "w: leading"), (dict(ldx=68), 1, "multiple of 8"), (dict(ldw=1 << 22), 2, "32-bit"),
    (dict(x=P + 8), 1, "x must be 16-byte"), (dict(w=P + 2), 1, "w must be 16-byte"), (dict(x=None), 1, "x: NULL"),
    (dict(y=None), 1, "y: NULL"), (dict(ldy=39), 1, "y: leading"), (dict(ldy=2 ** 62), 1, "y: leading"),
    (dict(y=P + 1), 1, "y must be element"), (dict(dtype=1, y=P + 2), 1, "y must be element"),
    (dict(residual=P, ldr=39), 1, "residual: leading"), (dict(residual=P + 1, ldr=40), 1, "residual must be"),
    (dict(z=P, ldz=8), 1, "z_out: leading"), (dict(z=P + 1, ldz=40), 1, "z_out must be"), (dict(bias=P + 1), 1, "bias must be"),
    (dict(bias=P + 2, dtype_bias=1), 1, "bias must be"), (dict(work=P + 8), 1, "workspace must be 16-byte"),
    (dict(m=1, n=16, k=8192, ldx=8192, ldw=8192, work=None), 1, "workspace of 0 bytes"),
    (dict(m=1, n=16, k=8192, ldx=8192, ldw=8192, bytes=16), 1, "workspace of 16 bytes"),
])
def test_linear_refusals(pts, change, status, fragment):
    _refused(pts, lambda: pts.pts_linear(*{**LINEAR, **change}.values(), stream=0), status, fragment)


BACK = dict(dy=P, ld_dy=40, z=P, ldz=40, act=4, x=P, ldx=64, w=P, ldw=64, dx=P, ld_dx=64, dw=P, ld_dw=64, dtype=0, db=P,
            m=33, n=40, k=64, work=P, bytes=BIG)


@pytest.mark.parametrize("change,status,fragment", [
    (dict(dtype=2), 2, "fp32 or bf16"), (dict(act=9), 1, "activation"), (dict(m=-1), 1, "m, n and k"),
    (dict(ld_dy=36), 1, "dy: leading"), (dict(ld_dy=44), 1, "dy: leading"), (dict(z=None), 1, "z: NULL"),
    (dict(z=P + 4), 1, "z must be 16-byte"), (dict(ldx=60), 1, "x: leading"), (dict(w=None), 1, "w: NULL"),
    (dict(x=None), 1, "x: NULL"), (dict(ld_dx=63), 1, "dx: leading"), (dict(ld_dw=63), 1, "dw: leading"),
    (dict(dw=P + 2, dtype=1), 1, "dw must be element"), (dict(m=2 ** 31 - 2048, k=300, ldx=304, ldw=304, ld_dx=304, ld_dw=304), 2, "too large"), (dict(db=P + 2), 1, "dbias"), (dict(bytes=0), 1, "workspace"),
])
def test_backward_refusals(pts, change, status, fragment):
    _refused(pts, lambda: pts.pts_linear_backward(*{**BACK, **change}.values(), stream=0), status, fragment)


ORTHO = dict(x=P, dtype=0, ldx=64, xs=0, count=1, rows=40, cols=64, steps=5, a=3.4445, b=-4.775, c=2.0315, eps=1e-7, out=P,
             ldo=64, os=0, work=P, bytes=BIG)


@pytest.mark.parametrize("change,status,fragment", [
    (dict(dtype=2), 2, "fp32 or bf16"), (dict(count=-1), 1, "count"), (dict(rows=2 ** 31 - 1024), 1, "count"),
    (dict(rows=2 ** 30, cols=2 ** 22, ldx=2 ** 22, ldo=2 ** 22), 1, "2^48"), (dict(count=65536), 2, "65535"),
    (dict(cols=(1 << 22) - 63, ldx=1 << 22, ldo=1 << 22), 2, "32-bit"), (dict(steps=0), 1, "steps"), (dict(steps=65), 1, "steps"),
    (dict(eps=0.0), 1, "eps"), (dict(eps=float("nan")), 1, "eps"), (dict(a=9.0), 1, "fp16's reach"),
    (dict(a=2.0, b=2.0, c=2.0), 1, "fp16's reach"), (dict(a=float("nan")), 1, "fp16's reach"),
    (dict(a=1.0, b=-200.0, c=200.0), 1, "fp16's reach"), (dict(ldx=63), 1, "x: leading"), (dict(ldo=63), 1, "out: leading"),
    (dict(x=None), 1, "x: NULL"), (dict(out=P + 1), 1, "out must be"), (dict(dtype=1, x=P + 2), 1, "x must be"),
    (dict(count=2, os=63), 1, "overlap"), (dict(count=2, ldo=100, os=64), 1, "overlap"),
    (dict(count=65535, rows=64, cols=1 << 15, ldx=1 << 15, ldo=1 << 15, os=1 << 21), 2, "too large"),
    (dict(xs=-1), 1, "strides"), (dict(count=2, os=2 ** 62), 1, "strides"), (dict(bytes=64), 1, "workspace"),
])
def test_orthogonalize_refusals(pts, change, status, fragment):
    _refused(pts, lambda: pts.pts_orthogonalize(*{**ORTHO, **change}.values(), stream=0), status, fragment)


def test_workspaces(pts):
    assert pts.pts_linear_workspace(0, 8, 8) == 0 and pts.pts_linear_workspace(-1, 8, 8) == 0
    assert pts.pts_linear_workspace(1, 4096, 4096) == 0                    # a workgroup for each strip
    assert pts.pts_linear_workspace(1, 1000, 8192) == 4 * 1000 * 4         # four to a strip
    assert pts.pts_linear_workspace(8192, 8192, 8192) == 0                 # four whole rounds of tiles
    assert pts.pts_linear_workspace(5000, 7000, 3000) == 48 * 4 * 256 * 256 * 4  # the last 48 of 560 tiles, four to a tile
    assert pts.pts_linear_backward_workspace(64, 64, 64, 0) == 0
    assert pts.pts_linear_backward_workspace(64, 60, 64, 4) == 64 * 64 * 2  # dz, rows of whole 16 bytes
    assert pts.pts_orthogonalize_workspace(0, 64, 64, 5) == 0 and pts.pts_orthogonalize_workspace(1, 64, 64, 0) == 0
    assert pts.pts_orthogonalize_workspace(1, 65, 65, 5) > 65 * 72 * 2 * 4


def test_empty_calls_launch_nothing(pts):
    pts.pts_linear(*{**LINEAR, "m": 0}.values(), stream=0)
    pts.pts_linear(*{**LINEAR, "n": 0}.values(), stream=0)
    pts.pts_linear_backward(*{**BACK, "dx": None, "dw": None, "db": None}.values(), stream=0)
    pts.pts_orthogonalize(*{**ORTHO, "count": 0}.values(), stream=0)
    pts.pts_orthogonalize(*{**ORTHO, "rows": 0}.values(), stream=0)


def _bf16(*shape):
    return torch.zeros(shape, dtype=torch.bfloat16)


@pytest.mark.parametrize("call,fragment", [
    (lambda p: p.linear(torch.zeros(4, 8), _bf16(8, 8)), "x must be bfloat16"),
    (lambda p: p.linear(_bf16(4, 8), _bf16(8, 16)), "8 and 16 columns"),
    (lambda p: p.linear(_bf16(4, 12)[:, :9], _bf16(8, 9)), "multiple of 8"),
    (lambda p: p.linear(_bf16(4, 8).t(), _bf16(8, 4)), "unit stride"),
    (lambda p: p.linear(_bf16(4, 16)[:, 4:12], _bf16(8, 8)), "16-byte aligned"),
    (lambda p: p.linear(_bf16(4, 8), _bf16(8, 8), activation="tanh"), "activation must be"),
    (lambda p: p.linear(_bf16(4, 8), _bf16(8, 8), torch.zeros(7)), "bias must be"),
    (lambda p: p.linear(_bf16(4, 8), _bf16(8, 8), torch.zeros(16)[::2]), "bias must be contiguous"),
    (lambda p: p.linear(_bf16(4, 8), _bf16(8, 8)), "not on the current GPU"),
    (lambda p: p.linear_backward(_bf16(4, 8), _bf16(5, 8), _bf16(8, 8)), "do not fit"),
    (lambda p: p.linear_backward(_bf16(4, 8), _bf16(4, 8), _bf16(8, 8), None, "silu"), "z must be bfloat16"),
    (lambda p: p.linear_backward(_bf16(4, 8), _bf16(4, 8), _bf16(8, 8), _bf16(4, 16), "silu"), "z must be bfloat16"),
    (lambda p: p.linear_backward(_bf16(4, 8), _bf16(4, 8), _bf16(8, 8), dw_dtype=torch.float16), "dw_dtype"),
    (lambda p: p.orthogonalize(torch.zeros(4, 4, dtype=torch.float16)), "x must be"),
    (lambda p: p.orthogonalize(torch.zeros(4)), "x must be"),
    (lambda p: p.orthogonalize(torch.zeros(4, 4)), "not on the current GPU"),
    (lambda p: p.orthogonalize(torch.zeros(4, 4), out=torch.zeros(4, 4)), "out must be bfloat16"),
])
def test_binding_refusals(pts, call, fragment, monkeypatch):
    from persistent_tile_scheduling_amd import experts
    monkeypatch.setattr(experts, "_current", lambda: 0)     # what the binding asks of a GPU before it refuses
    with pytest.raises(ValueError, match=re.escape(fragment)):
        call(pts)


@pytest.mark.parametrize("act", R.ACTIVATIONS)
def test_reference_slopes_are_the_activations_differences(act):
    z = torch.linspace(-9, 9, 4001, dtype=torch.float64)
    z = z[z.abs() > 1e-3]
    h = 1e-5
    by_difference = (R.activation(z + h, act) - R.activation(z - h, act)) / (2 * h)
    # the third derivative is below 3 for each: h^2 / 6 of it, and the rounding of values up to 9 over h
    assert (R.slope(z, act) - by_difference).abs().max() < 0.5 * h * h * 3 + 9 * 2.0 ** -52 / h


def test_reference_steps_map_the_singular_values():
    g = torch.Generator().manual_seed(1)
    x = torch.randn((40, 70), generator=g, dtype=torch.float64)
    u, s, v = torch.linalg.svd(x, full_matrices=False)
    s = s / (s.square().sum().sqrt() + 1e-7)
    for _ in range(5):
        s = 3.4445 * s - 4.7750 * s ** 3 + 2.0315 * s ** 5
    assert torch.allclose(R.orthogonalize(x), (u * s) @ v, atol=1e-11)
    assert math.isclose(s.max().item(), 1.0, abs_tol=0.3)
