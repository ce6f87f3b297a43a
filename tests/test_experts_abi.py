"""The routed-experts C ABI without a GPU: exported names, constants, and every refusal that precedes a launch."""
from __future__ import annotations

import os
import re

import numpy as np
import pytest
import torch

from tests import experts_reference as R

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "pts_experts.h")
P = 4096  # a pointer that passes the alignment checks; nothing here reaches a launch


@pytest.fixture(scope="module")
def pts():
    import persistent_tile_scheduling_amd as mod
    return mod


def _declared():
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    return sorted(set(re.findall(r"^\s*(?:gemm_status|int64_t)\s+([a-z_0-9]+)\s*\(", text, flags=re.M)))


def test_every_declared_function_is_exported_and_bound(pts):
    names = _declared()
    assert len(names) == 8
    for n in names:
        assert hasattr(pts._lib, n) and callable(getattr(pts, n)), n


def test_constants_match(pts):
    text = open(HEADER).read()
    for name, value in re.findall(r"#define (PTS_[A-Z0-9_]+) (\d+)", text) + re.findall(r"(PTS_SCORE_[A-Z]+) = (\d+)", text):
        assert getattr(pts, name) == int(value), name


def _refused(pts, call, status, fragment):
    with pytest.raises(pts.GemmError) as ei:
        call()
    assert ei.value.status == status and fragment in str(ei.value), str(ei.value)


QUANTIZE = dict(x=P, dtype=0, layout=0, m=4, k=128, ldx=128, block=1, swiglu=0, q=P, ldq=128, scale=P, sm=1, sk=4)


@pytest.mark.parametrize("change,status,fragment", [
    (dict(dtype=2), 2, "bf16 or fp32"), (dict(layout=2), 2, "row-major"), (dict(block=64), 2, "blocks"),
    (dict(swiglu=1, block=128, ldx=256), 2, "gated"), (dict(swiglu=1, layout=1, ldx=256), 2, "gated"),
    (dict(swiglu=1), 1, "leading"), (dict(m=-1), 1, "m and k"), (dict(k=2 ** 31), 1, "m and k"),
    (dict(ldx=127), 1, "leading"), (dict(layout=1, ldx=3), 1, "leading"), (dict(ldq=112), 1, "leading"),
    (dict(ldq=136), 1, "multiple of 16"), (dict(sm=0), 1, "strides"), (dict(x=None), 1, "NULL"),
    (dict(q=P + 8), 1, "aligned"), (dict(x=P + 1), 1, "aligned"), (dict(scale=P + 2), 1, "aligned"),
])
def test_quantize_refusals(pts, change, status, fragment):
    _refused(pts, lambda: pts.pts_quantize_fp8(*{**QUANTIZE, **change}.values(), stream=0), status, fragment)


PRODUCT = dict(a=P, lda=128, sa=P, sam=1, sak=4, b=P, ldb=128, sb=P, sbn=1, sbk=1, block=128, d=P, ldd=8, dtype=1, m=4,
               n=8, k=128)


@pytest.mark.parametrize("change,status,fragment", [
    (dict(dtype=2), 2, "fp32 or bf16"), (dict(block=64), 2, "per row or per 128"), (dict(m=-1), 1, "[0, 2^31)"),
    (dict(k=2 ** 31, lda=2 ** 31, ldb=2 ** 31), 1, "[0, 2^31)"), (dict(lda=112), 1, "leading"), (dict(ldd=7), 1, "leading"),
    (dict(lda=136), 1, "multiples of 16"), (dict(ldb=136), 1, "multiples of 16"), (dict(sam=-1), 1, "strides"),
    (dict(lda=2 ** 23), 2, "32-bit"), (dict(sak=2 ** 30), 2, "32-bit"), (dict(sbn=2 ** 30), 2, "32-bit"),
    (dict(sam=2 ** 62), 2, "32-bit"), (dict(sbk=2 ** 62), 2, "32-bit"),
    (dict(n=2 ** 31 - 1, ldd=2 ** 31, sbn=2 ** 30 - 1, block=1), 2, "32-bit"),
    (dict(a=None), 1, "NULL"), (dict(sb=None), 1, "NULL"), (dict(d=None), 1, "NULL"), (dict(a=P + 8), 1, "16-byte"),
    (dict(sa=P + 2), 1, "4-byte"), (dict(d=P + 2), 1, "element aligned"),
])
def test_product_refusals(pts, change, status, fragment):
    _refused(pts, lambda: pts.pts_gemm_fp8(*{**PRODUCT, **change}.values(), stream=0), status, fragment)


EXPERTS = dict(a=P, a_rows=4, lda=128, sa=P, sam=1, sak=4, b=P, ldb=128, bse=1024, sb=P, sbe=1, sbn=1, sbk=1, experts=2,
               offsets=P, rows=None, d=P, ldd=8, dtype=1, m=4, n=8, k=128)


@pytest.mark.parametrize("change,status,fragment", [
    (dict(experts=0), 2, "experts must be"), (dict(experts=1025), 2, "experts must be"), (dict(bse=1000), 1, "multiple of 16"),
    (dict(offsets=None), 1, "offsets"), (dict(offsets=P + 2), 1, "4-byte"), (dict(a_rows=3), 1, "too few"),
    (dict(a_rows=0, rows=P), 1, "too few"), (dict(a_rows=2 ** 25, rows=P), 2, "32-bit"), (dict(dtype=5), 2, "fp32 or bf16"),
    (dict(lda=136), 1, "multiples of 16"),
])
def test_experts_refusals(pts, change, status, fragment):
    _refused(pts, lambda: pts.pts_gemm_fp8_experts(*{**EXPERTS, **change}.values(), stream=0), status, fragment)


ROUTE = dict(x=P, dtype=1, ld=8, bias=None, m=4, experts=8, top=2, score=0, groups=1, keep=1, pair=0, renorm=1, scale=1.0,
             ids=P, w=P, offsets=P, rows=P, positions=P, work=None, bytes=0)


@pytest.mark.parametrize("change,status,fragment", [
    (dict(dtype=7), 2, "bf16 or fp32"), (dict(experts=1025, ld=1025), 2, "top <="), (dict(top=9), 2, "top <="),
    (dict(top=33, experts=64, ld=64), 2, "top <="), (dict(top=0), 2, "top <="), (dict(score=2), 1, "score"),
    (dict(groups=3), 1, "groups"), (dict(groups=2, keep=3), 1, "groups"), (dict(groups=8, keep=1), 1, "fewer than top"),
    (dict(m=-1), 1, "m * top"), (dict(m=2 ** 30), 1, "m * top"), (dict(ld=7), 1, "leading"), (dict(rows=None), 1, "order"),
    (dict(m=10000), 1, "workspace"), (dict(ids=None), 1, "NULL"), (dict(x=P + 2), 1, "aligned"),
])
def test_route_refusals(pts, change, status, fragment):
    _refused(pts, lambda: pts.pts_moe_route(*{**ROUTE, **change}.values(), stream=0), status, fragment)


def test_route_workspace(pts):
    assert pts.pts_moe_route_workspace(0, 8, 2) == 0 and pts.pts_moe_route_workspace(16, 8, 2) == 0
    assert pts.pts_moe_route_workspace(10000, 8, 2) == 10 * 9 * 4         # ten chunks of 2048 slots
    assert pts.pts_moe_route_workspace(1 << 26, 64, 8) == 256 * 65 * 4    # never more than 256


BACK = dict(dw=P, x=P, dtype=1, ld=8, ids=P, m=4, experts=8, top=2, score=0, renorm=1, scale=1.0, out=P, ldd=8)


@pytest.mark.parametrize("change,status,fragment", [
    (dict(dtype=7), 2, "bf16 or fp32"), (dict(experts=0), 2, "experts"), (dict(score=-1), 1, "score"), (dict(m=-4), 1, "m * top"),
    (dict(ld=4), 1, "leading"), (dict(ldd=4), 1, "leading"), (dict(dw=None), 1, "NULL"), (dict(out=P + 1), 1, "aligned"),
])
def test_route_backward_refusals(pts, change, status, fragment):
    _refused(pts, lambda: pts.pts_moe_route_backward(*{**BACK, **change}.values(), stream=0), status, fragment)


COMBINE = dict(y=P, dtype=0, ldy=64, rows=8, w=P, pos=P, m=4, n=64, top=2, out=P, ldo=64)


@pytest.mark.parametrize("change,status,fragment", [
    (dict(dtype=3), 2, "bf16 or fp32"), (dict(top=33), 2, "top"), (dict(m=1 << 24), 1, "2^24"), (dict(n=-1), 1, "2^26"),
    (dict(ldy=63), 1, "leading"), (dict(ldo=63), 1, "leading"), (dict(w=None), 1, "NULL"), (dict(y=None), 1, "NULL"),
    (dict(out=P + 1), 1, "aligned"),
])
def test_combine_refusals(pts, change, status, fragment):
    _refused(pts, lambda: pts.pts_moe_combine(*{**COMBINE, **change}.values(), stream=0), status, fragment)


GRAD = dict(dout=P, ldd=64, y=P, dtype=0, ldy=64, rows=8, w=P, pos=P, m=4, n=64, top=2, dy=P, ldo=64, dw=P)


@pytest.mark.parametrize("change,status,fragment", [
    (dict(dtype=3), 2, "bf16 or fp32"), (dict(ldd=63), 1, "leading"), (dict(dw=None), 1, "NULL"), (dict(dout=None), 1, "NULL"),
    (dict(dw=P + 2), 1, "aligned"), (dict(rows=-1), 1, "rows"),
])
def test_combine_backward_refusals(pts, change, status, fragment):
    _refused(pts, lambda: pts.pts_moe_combine_backward(*{**GRAD, **change}.values(), stream=0), status, fragment)


def test_empty_calls_do_nothing(pts):
    pts.pts_quantize_fp8(*{**QUANTIZE, "m": 0, "x": None}.values(), stream=0)
    pts.pts_gemm_fp8(*{**PRODUCT, "n": 0, "b": None}.values(), stream=0)
    pts.pts_gemm_fp8_experts(*{**EXPERTS, "m": 0, "a_rows": 0, "offsets": None}.values(), stream=0)
    pts.pts_moe_route_backward(*{**BACK, "m": 0, "x": None}.values(), stream=0)
    pts.pts_moe_combine(*{**COMBINE, "m": 0, "y": None}.values(), stream=0)
    pts.pts_moe_combine_backward(*{**GRAD, "m": 0, "y": None}.values(), stream=0)


def test_tensor_checks_come_before_the_device(pts):
    x = torch.zeros((4, 256), dtype=torch.bfloat16)
    q, s = torch.zeros((4, 256), dtype=torch.float8_e4m3fn), torch.zeros((4, 2))
    i = torch.zeros((4, 2), dtype=torch.int32)
    for call in (
            lambda: pts.quantize_fp8(x.half()), lambda: pts.quantize_fp8(x[0]), lambda: pts.quantize_fp8(x, block=(64, 64)),
            lambda: pts.quantize_fp8(x),                                                # not on a GPU
            lambda: pts.gemm_fp8(x, s, q, s), lambda: pts.gemm_fp8(q, s[:, :1], q, s),
            lambda: pts.gemm_fp8(q, s, q, s.double()), lambda: pts.gemm_fp8(q, s, q, torch.zeros((3, 2))),
            lambda: pts.gemm_fp8(q, s, q, s),
            lambda: pts.gemm_fp8_experts(q, s, q, s, i), lambda: pts.gemm_fp8_experts(q, s, q[None], s[None, :1], i[0].long()),
            lambda: pts.moe_route(x, 0), lambda: pts.moe_route(x.half(), 2), lambda: pts.moe_route(x, 2, score="relu"),
            lambda: pts.moe_route(x, 2, bias=torch.zeros(3)), lambda: pts.moe_route(x, 2),
            lambda: pts.moe_route_backward(s, x, i.long()), lambda: pts.moe_combine(x, s, i.long()),
            lambda: pts.moe_combine_backward(s, x, s, i)):
        with pytest.raises(ValueError):
            call()


@pytest.mark.parametrize("extent", [2 ** 31 - 1, 2 ** 31 - 1023])
def test_extents_that_do_not_round_up_are_refused(pts, extent):
    for change in (dict(m=extent, n=1, ldd=1), dict(n=extent, ldd=2 ** 31, block=128)):
        _refused(pts, lambda: pts.pts_gemm_fp8(*{**PRODUCT, **change}.values(), stream=0), 2, "2^31 - 1024")
    for change in (dict(m=extent), dict(k=extent, ldx=2 ** 31, ldq=2 ** 31)):
        _refused(pts, lambda: pts.pts_quantize_fp8(*{**QUANTIZE, **change}.values(), stream=0), 1, "m and k")


def test_slot_counts_past_64_bits_are_refused(pts):
    m = 2 ** 62 + 1  # times 4 is 4 again in 64 bits
    assert pts.pts_moe_route_workspace(m, 8, 4) == 0
    _refused(pts, lambda: pts.pts_moe_route(*{**ROUTE, "m": m, "top": 4}.values(), stream=0), 1, "m * top")
    _refused(pts, lambda: pts.pts_moe_route_backward(*{**BACK, "m": m, "top": 4}.values(), stream=0), 1, "m * top")
    _refused(pts, lambda: pts.pts_moe_combine(*{**COMBINE, "m": m, "top": 4}.values(), stream=0), 1, "m * top")


def test_combined_rows_past_the_grid_are_refused(pts):
    n = 2 ** 26 - 1023
    _refused(pts, lambda: pts.pts_moe_combine(*{**COMBINE, "n": n, "ldy": n, "ldo": n}.values(), stream=0), 1, "2^26")


def test_layer_needs_logits_of_every_token(pts):
    x = torch.zeros((4, 256), dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="logits"):
        pts.moe_fp8(x, torch.zeros((5, 8)), 2, None, None, None, None)


def test_reference_rounding_matches_an_exhaustive_search():
    # the tests' own rounding: against the nearest of all codes, on values around every midpoint
    grid = R.E4M3[:127]
    mid = (grid[1:] + grid[:-1]) / 2
    v = np.concatenate([grid, mid, np.nextafter(mid, 0), np.nextafter(mid, 500), -mid])
    got = R.nearest_e4m3(v)
    d = np.abs(np.abs(v)[:, None] - grid[None, :])
    assert np.array_equal(np.abs(np.abs(v) - np.abs(got)), d.min(1))
    ties = np.abs(R.nearest_e4m3(mid))
    assert np.all(np.isin(ties, grid[::2]))


def test_more_than_one_launch_holds_is_refused(pts):
    m, k = 2 ** 31 - 2048, 2 ** 17                      # 2^34 blocks of 128 x 128
    change = dict(m=m, k=k, ldx=k, ldq=k, block=128)
    _refused(pts, lambda: pts.pts_quantize_fp8(*{**QUANTIZE, **change}.values(), stream=0), 2, "too large")
