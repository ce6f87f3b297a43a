"""GPU tests of the routed-experts operators against 64-bit references (tests/experts_reference.py).

Tolerances are stated where they are used, from the number of roundings: one is
off by at most half a step (2^-24 relative in fp32, 2^-8 in bf16, 2^-4 in e4m3).
"""
from __future__ import annotations

import numpy as np
import pytest
import torch

from tests import experts_reference as R
from tests import gpu_util as U

pytestmark = pytest.mark.gpu
DEV = U.DEV
BF16, F32, E4M3 = torch.bfloat16, torch.float32, torch.float8_e4m3fn


@pytest.fixture(scope="module")
def pts():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import persistent_tile_scheduling_amd as mod
    return mod



def _f64(t):
    return t.detach().float().cpu().double().numpy()


def _same(x, y):
    return np.array_equal(x, y, equal_nan=True)


# ---- quantisation --------------------------------------------------------------

def _values(m, k, dtype, seed):
    """Normal values of mixed magnitude, with a zero block, tiny blocks and exact midpoints."""
    rng = np.random.default_rng(seed)
    x = rng.standard_normal((m, k)) * np.exp(3 * rng.standard_normal((1, k)))
    x[0, :128] = 0
    if m > 2:
        x[1, :128] = rng.standard_normal(min(128, k)) * 1e-38
        x[2, :min(128, k)] = rng.integers(-448 * 2, 448 * 2 + 1, min(128, k)) / 2.0
        x[2, 0] = 448                                  # scale 1 exactly: halves of integers are midpoints
    return torch.from_numpy(x).to(dtype)


@pytest.mark.parametrize("m,k", [(1, 1), (1, 128), (3, 4096), (130, 129), (257, 1000), (64, 7), (300, 640)])
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("block,across", [(1, False), (1, True), (128, False), (128, True)])
def test_quantize_equals_the_definition(pts, m, k, dtype, block, across):
    U.log(f"quantize {m}x{k} {dtype} block {block} across {across}")
    x = _values(m, k, dtype, m * 7 + k)
    dev = x.t().contiguous().to(DEV).t() if across else x.to(DEV)
    q, s = pts.quantize_fp8(dev, block=(block, 128))
    assert q.shape == (m, k) and q.stride(0) % 16 == 0 and s.dtype == F32
    want_q, want_s = R.quantize(x.float().numpy(), block)
    assert _same(s.cpu().numpy(), want_s)
    assert _same(R.decode(q), want_q)


def test_quantize_views_and_padding(pts):
    """Unaligned and strided views; the codes' padding is zero; nothing else is written."""
    x = _values(70, 300, BF16, 5).to(DEV)
    for view in (x[:, 1:200], x[3:, 8:299], x[::2, :130], x.t()[5:, :33], x[:1, 3:100]):
        q, s = pts.quantize_fp8(view)
        want_q, want_s = R.quantize(view.float().cpu().numpy(), 1)
        assert _same(s.cpu().numpy(), want_s) and _same(R.decode(q), want_q)
    m, k, ldq = 5, 20, 48
    q = torch.full((m, ldq), 0x55, dtype=torch.uint8, device=DEV)
    s = torch.full((m, 3), 7.0, device=DEV)
    pts.pts_quantize_fp8(x, 0, 0, m, k, 300, 1, 0, q, ldq, s, 3, 1)
    torch.cuda.synchronize()
    assert torch.all(q[:, 20:32] == 0) and torch.all(q[:, 32:] == 0x55) and torch.all(s[:, 1:] == 7.0)


@pytest.mark.parametrize("across,block", [(False, 1), (True, 1), (False, 128)])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_quantize_marks_blocks_that_are_not_finite(pts, across, block, bad):
    x = _values(130, 300, F32, 3)
    x[129, 130] = bad
    q, s = pts.quantize_fp8(x.t().contiguous().to(DEV).t() if across else x.to(DEV), block=(block, 128))
    want_q, want_s = R.quantize(x.numpy(), block)
    assert np.isnan(want_s).sum() == 1 and _same(s.cpu().numpy(), want_s) and _same(R.decode(q), want_q)


@pytest.mark.parametrize("m,k,dtype", [(1, 1, BF16), (5, 128, F32), (33, 1000, BF16), (130, 264, BF16), (17, 4097, F32)])
def test_quantize_gated(pts, m, k, dtype):
    x = (torch.randn((m, 2 * k), generator=torch.Generator().manual_seed(k)) * 3).to(dtype)
    q, s = pts.quantize_fp8(x.to(DEV), swiglu=True)
    g, u = _f64(x)[:, :k], _f64(x)[:, k:]
    h = g / (1 + np.exp(-g)) * u
    # exp's argument is rounded twice (|g| 2^-23 in the result), exp and the reciprocal are good to 2 steps, sum and
    # three products round: |g| + 8 steps of 2^-23 at most
    rel = (np.abs(g).max() + 8) * 2.0 ** -23
    kb = -(-k // 128)
    most = np.stack([np.abs(h[:, b * 128:(b + 1) * 128]).max(1) for b in range(kb)], 1)
    scale = _f64(s)
    assert np.all(np.abs(scale - most / 448) <= most / 448 * (rel + 2.0 ** -23))
    step = np.maximum(np.abs(h) * 2.0 ** -4, R.expand(s.cpu().numpy(), m, k) * 2.0 ** -10)
    assert np.all(np.abs(R.decode(q) * R.expand(s.cpu().numpy(), m, k) - h) <= step * (1 + 2.0 ** -20) + np.abs(h) * rel * 2)


@pytest.mark.parametrize("k", [1000, 1003])
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("gated", [False, True])
def test_quantize_many_rows_equals_few(pts, k, dtype, gated):
    """Workgroups of eight rows, the last one short, against slices that take four."""
    m = 4101
    x = _values(m, 2 * k if gated else k, dtype, k).to(DEV)
    q, s = pts.quantize_fp8(x, swiglu=gated)
    for lo, hi in ((0, 70), (2047, 2050), (m - 9, m)):
        qs, ss = pts.quantize_fp8(x[lo:hi], swiglu=gated)
        assert torch.equal(q[lo:hi].contiguous().view(torch.uint8), qs.contiguous().view(torch.uint8)), (lo, hi)
        assert torch.equal(s[lo:hi], ss), (lo, hi)


def test_quantize_every_e4m3_value_and_midpoint(pts):
    grid = R.E4M3[:127]
    mid = (grid[1:] + grid[:-1]) / 2
    v = np.concatenate([grid, -grid, mid, -mid, np.nextafter(mid.astype(np.float32), np.float32(500)),
                        np.nextafter(mid.astype(np.float32), np.float32(0))]).astype(np.float32)
    for factor in (1.0, 3.0, 0.1, 2.0 ** -100, 2.0 ** 100, 2.0 ** -133):
        x = np.zeros((-(-len(v) // 127), 128), dtype=np.float32)
        for i in range(0, len(v), 127):
            part = v[i:i + 127] * np.float32(factor)
            x[i // 127, :len(part)] = part
            x[i // 127, 127] = np.float32(448) * np.float32(factor)
        q, s = pts.quantize_fp8(torch.from_numpy(x).to(DEV))
        want_q, want_s = R.quantize(x, 1)
        assert _same(s.cpu().numpy(), want_s), factor
        assert _same(R.decode(q), want_q), factor


# ---- products ------------------------------------------------------------------

def _operand(m, k, seed, poison=True):
    """Codes over the whole range of e4m3, in rows padded with NaN codes."""
    rng = np.random.default_rng(seed)
    wide = 16 * (-(-k // 16)) + 16 * (seed % 3)
    codes = rng.integers(0, 256, (m, wide)).astype(np.uint8)
    codes[(codes & 0x7F) == 0x7F] = 0
    if poison:
        codes[:, k:] = 0x7F
    return torch.from_numpy(codes).to(DEV).view(E4M3)[:, :k]


def _scale(m, kb, seed, by_column=True):
    s = np.random.default_rng(seed).uniform(0.5, 2.0, (m, kb)).astype(np.float32) * 2.0 ** -8
    t = torch.from_numpy(s).to(DEV)
    return t.t().contiguous().t() if by_column else t


def _check_product(d, a, sa, b, sb, what):
    want, mag, largest = R.product(R.decode(a), sa.cpu().numpy(), R.decode(b), sb.cpu().numpy())
    err = np.abs(_f64(d) - want)
    bound = R.product_bound(mag, largest, want, a.shape[1], d.dtype)
    worst = float((err / np.maximum(bound, 1e-300)).max()) if err.size else 0.0
    U.log(f"{what}: worst error / bound = {worst:.3f}")
    good = bool(np.all(np.isfinite(_f64(d)))) and worst <= 1
    assert good, what


SHAPES = [(1, 1, 1), (1, 64, 128), (3, 40, 100), (8, 4096, 512), (16, 17, 1000), (17, 100, 128), (33, 130, 257),
          (64, 200, 2048), (65, 300, 384), (100, 127, 129), (130, 260, 130), (255, 257, 640), (300, 520, 1023),
          (128, 128, 64), (1000, 777, 333)]


@pytest.mark.parametrize("m,n,k", SHAPES)
@pytest.mark.parametrize("rows", [False, True])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_product(pts, m, n, k, rows, dtype):
    U.log(f"product {m}x{n}x{k} rows {rows} {dtype}")
    kb = -(-k // 128)
    a, b = _operand(m, k, 1 + m), _operand(n, k, 2 + n)
    sa, sb = _scale(m, kb, 3), _scale(n if rows else -(-n // 128), kb, 4, rows)
    back = torch.full((m + 1, n + 3), 9.0, dtype=dtype, device=DEV)
    _check_product(pts.gemm_fp8(a, sa, b, sb, out=back[:m, :n]), a, sa, b, sb, "strided out")
    assert torch.all(back[m:] == 9.0) and torch.all(back[:, n:] == 9.0)
    d = pts.gemm_fp8(a, sa, b, sb, dtype)
    assert torch.equal(d, back[:m, :n])


@pytest.mark.parametrize("m,n,k,rows", [(2200, 2310, 700, False), (2000, 2100, 1100, True), (2560, 2304, 1024, False)])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_product_large_tiles(pts, m, n, k, rows, dtype):
    """Sizes that take the 256 x 256 tiles, several per compute unit at the ragged ones."""
    U.log(f"product {m}x{n}x{k} rows {rows} {dtype}")
    kb = -(-k // 128)
    a, b = _operand(m, k, 1), _operand(n, k, 2)
    sa, sb = _scale(m, kb, 3, False), _scale(n if rows else -(-n // 128), kb, 4, rows)
    _check_product(pts.gemm_fp8(a, sa, b, sb, dtype), a, sa, b, sb, "large")


@pytest.mark.parametrize("m,n,k,rows", [(3200, 3400, 700, False), (3330, 3102, 384, True), (3328, 3200, 1024, False),
                                        (3000, 3405, 130, False)])
def test_product_of_many_large_tiles(pts, m, n, k, rows):
    """More than half the compute units' worth of 256 x 256 tiles; D's rows at whole lines, whole 16 bytes and anywhere."""
    U.log(f"product {m}x{n}x{k} rows {rows} bf16")
    kb = -(-k // 128)
    a, b = _operand(m, k, 1 + m), _operand(n, k, 2 + n)
    sa, sb = _scale(m, kb, 3), _scale(n if rows else -(-n // 128), kb, 4, by_column=rows)
    d = torch.full((m, n + 8), 7.0, dtype=BF16, device=DEV)
    out = pts.gemm_fp8(a, sa, b, sb, out=d[:, :n])
    _check_product(out, a, sa, b, sb, f"{m}x{n}x{k}")
    assert torch.all(d[:, n:] == 7.0)
    # a slice of the same: its rows start elsewhere, its values are those
    wide = torch.empty((m, n + 72), dtype=BF16, device=DEV)
    assert torch.equal(pts.gemm_fp8(a, sa, b, sb, out=wide[:, 8:8 + n]), out)


@pytest.mark.parametrize("m,n,k,rows", [(1, 70000, 300, False), (8, 66001, 128, True), (20, 65560, 200, False),
                                        (50, 66008, 128, True)])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_product_of_few_rows_and_many_columns(pts, m, n, k, rows, dtype):
    """Columns enough for two 16-column tiles per workgroup, the last one alone or ragged."""
    U.log(f"product {m}x{n}x{k} rows {rows} {dtype}")
    kb = -(-k // 128)
    a, b = _operand(m, k, 1 + m), _operand(n, k, 2)
    sa, sb = _scale(m, kb, 3), _scale(n if rows else -(-n // 128), kb, 4)
    _check_product(pts.gemm_fp8(a, sa, b, sb, dtype), a, sa, b, sb, f"{m}x{n}x{k}")


@pytest.mark.parametrize("n", [2000, 2003])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_experts_of_few_rows_and_many_columns(pts, n, dtype):
    sizes = [i % 4 for i in range(64)] + [17, 0, 40]
    U.log(f"67 experts of few rows, n {n} {dtype}")
    a, sa, b, sb, offsets, rows, m = _expert_inputs(sizes, n, 384, 5, behind=3, gather=True)
    out = torch.full((m, n), 9.0, dtype=dtype, device=DEV)
    pts.gemm_fp8_experts(a, sa, b, sb, offsets, rows, out=out)
    o = offsets.cpu().tolist()
    for e in [i for i in range(len(sizes)) if sizes[i]]:
        pick = rows[o[e]:o[e + 1]].long()
        _check_product(out[o[e]:o[e + 1]], a.view(torch.uint8)[pick].view(E4M3), sa[pick], b[e], sb[e], f"expert {e}")
    assert torch.all(out[o[-1]:] == 9.0)


def test_product_of_nothing(pts):
    a, b = _operand(5, 128, 1), _operand(7, 128, 2)
    s = _scale(5, 1, 1)
    assert torch.all(pts.gemm_fp8(a[:, :0], s[:, :0], b[:, :0], s[:1, :0]) == 0)
    assert pts.gemm_fp8(a[:0], s[:0], b, s[:1]).shape == (0, 7)
    assert pts.gemm_fp8(a, s, b[:0], s[:0]).shape == (5, 0)
    big = torch.zeros((300, 0), dtype=E4M3, device=DEV)
    assert torch.all(pts.gemm_fp8(big, torch.zeros((300, 0), device=DEV), big, torch.zeros((3, 0), device=DEV)) == 0)


@pytest.mark.parametrize("m", [4, 40, 200])
def test_product_carries_nan_and_nothing_else(pts, m):
    """A NaN code reaches its row (or column) only; a NaN scale its blocks' rows."""
    n, k = 150, 300
    a, b = _operand(m, k, 1).clone(), _operand(n, k, 2)
    a = torch.nn.functional.pad(a.view(torch.uint8), (0, 4)).contiguous().view(E4M3)[:, :k]
    a.view(torch.uint8)[2, 299] = 0x7F
    sa, sb = _scale(m, 3, 3), _scale(2, 3, 4, False)
    d = pts.gemm_fp8(a, sa, b, sb)
    assert torch.all(torch.isnan(d[2])) and not torch.any(torch.isnan(torch.cat([d[:2], d[3:]])))
    sb[1, 0] = float("nan")
    d = pts.gemm_fp8(a, sa, b, sb)
    assert torch.all(torch.isnan(d[:, 128:])) and not torch.any(torch.isnan(d[0, :128]))


@pytest.mark.parametrize("m,n,k", [(7, 48, 256), (100, 130, 384), (2100, 2150, 256)])
def test_product_gradients_are_products(pts, m, n, k):
    """dA = dD . B and dB = dD^T . A from the quantiser's transposed forms, against the formula on the quantised values."""
    g = torch.Generator().manual_seed(m)
    x, w, dd = (torch.randn(s, generator=g).to(DEV) for s in ((m, k), (n, k), (m, n)))
    da = pts.gemm_fp8(*(qd := pts.quantize_fp8(dd)), *(qw := pts.quantize_fp8(w.t(), (128, 128))))
    _check_product(da, *qd, *qw, "dA")
    dw = pts.gemm_fp8(*(qt := pts.quantize_fp8(dd.t())), *(qx := pts.quantize_fp8(x.t())))
    _check_product(dw, *qt, *qx, "dB")
    # and against the unquantised formula: each factor is off by at most 2^-4 of its value (or 2^-10 of its scale),
    # so a sum of products by (2 2^-4 + 2^-8) of the magnitudes, and below that where values underflow
    want = _f64(dd).T @ _f64(x)
    mag = np.abs(_f64(dd)).T @ np.abs(_f64(x)) + 2.0 ** -6 * np.sqrt(np.outer((_f64(dd) ** 2).sum(0), (_f64(x) ** 2).sum(0)))
    assert np.all(np.abs(_f64(dw) - want) <= (2 * 2.0 ** -4 + 2.0 ** -8) * mag)


# ---- experts -------------------------------------------------------------------

def _expert_inputs(sizes, n, k, seed, behind=0, gather=False, before=0):
    e, m = len(sizes), before + sum(sizes) + behind
    kb, nb = -(-k // 128), -(-n // 128)
    have = max(1, m // 3) if gather else m
    a, sa = _operand(have, k, seed + 1), _scale(have, kb, seed + 2)
    b = torch.stack([_operand(n, k, 3 * (seed + 10 + i)).contiguous() for i in range(e)]) if k % 16 == 0 else None
    if b is None:
        wide = 16 * (-(-k // 16))
        b = torch.full((e, n, wide), 0x7F, dtype=torch.uint8, device=DEV).view(E4M3)[:, :, :k]
        for i in range(e):
            b.view(torch.uint8)[i] = _operand(n, k, seed + 10 + i).view(torch.uint8)
    sb = torch.stack([_scale(nb, kb, seed + 50 + i, False) for i in range(e)])
    offsets = torch.tensor(np.concatenate([[before], before + np.cumsum(sizes)]), dtype=torch.int32, device=DEV)
    rows = None
    if gather:
        rows = torch.from_numpy(np.random.default_rng(seed).integers(0, have, m).astype(np.int32)).to(DEV)
    return a, sa, b, sb, offsets, rows, m


EXPERTS = [
    ([1], 16, 128), ([0, 3, 0, 1, 16, 17, 0], 100, 300), ([5] * 9, 64, 1024), ([20, 0, 31, 40], 130, 200),
    ([60, 10, 0, 0, 64, 65], 200, 256), ([100, 70, 129, 0, 128], 140, 400), ([300, 255, 256, 1], 300, 384),
    ([2000, 0, 900, 257], 520, 256), ([0, 0, 0], 32, 128), ([1] * 70, 48, 144),
]


@pytest.mark.parametrize("sizes,n,k", EXPERTS)
@pytest.mark.parametrize("gather", [False, True])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_experts(pts, sizes, n, k, gather, dtype):
    U.log(f"experts {sizes[:8]} n {n} k {k} gather {gather} {dtype}")
    a, sa, b, sb, offsets, rows, m = _expert_inputs(sizes, n, k, len(sizes), behind=5, gather=gather, before=2)
    out = torch.full((m, n), 9.0, dtype=dtype, device=DEV)
    assert pts.gemm_fp8_experts(a, sa, b, sb, offsets, rows, out=out) is out
    at = offsets.tolist()
    assert torch.all(out[:at[0]] == 9.0) and torch.all(out[at[-1]:] == 9.0)
    for e in range(len(sizes)):
        if sizes[e]:
            pick = rows[at[e]:at[e + 1]].long() if gather else torch.arange(at[e], at[e + 1], device=DEV)
            ae = a.contiguous().view(torch.uint8)[pick].view(E4M3)
            _check_product(out[at[e]:at[e + 1]], ae, sa[pick], b[e], sb[e], f"expert {e}")


@pytest.mark.parametrize("gather", [False, True])
@pytest.mark.parametrize("n", [3400, 3200])
def test_experts_in_large_tiles(pts, n, gather):
    """256 x 256 tiles: experts of less than a tile, exactly one, several and a part, and none."""
    sizes, k = [600, 0, 300, 900, 257, 256, 255, 0, 100], 300
    U.log(f"experts {sizes} n {n} k {k} gather {gather}")
    a, sa, b, sb, offsets, rows, m = _expert_inputs(sizes, n, k, 31, behind=5, gather=gather, before=2)
    out = torch.full((m, n), 9.0, dtype=BF16, device=DEV)
    pts.gemm_fp8_experts(a, sa, b, sb, offsets, rows, out=out)
    o = offsets.cpu().tolist()
    for e in range(len(sizes)):
        if sizes[e]:
            pick = (rows[o[e]:o[e + 1]] if gather else torch.arange(o[e], o[e + 1], device=DEV)).long()
            ae = a.view(torch.uint8)[pick].view(E4M3)
            _check_product(out[o[e]:o[e + 1]], ae, sa[pick], b[e], sb[e], f"expert {e}")
    assert torch.all(out[:o[0]] == 9.0) and torch.all(out[o[-1]:] == 9.0)


@pytest.mark.parametrize("per", [2, 100, 300])
def test_experts_equal_the_dense_product_on_one_expert(pts, per):
    a, sa, b, sb, offsets, _, _ = _expert_inputs([per], 260, 512, 3)
    assert torch.equal(pts.gemm_fp8_experts(a, sa, b, sb, offsets, out_dtype=F32), pts.gemm_fp8(a, sa, b[0], sb[0]))


@pytest.mark.parametrize("per", [3, 80, 400])
def test_experts_with_a_bad_table_stay_inside(pts, per):
    """Offsets that go back or leave the range, and row numbers outside A: values are some row's, nothing outside is written."""
    sizes = [per] * 4
    a, sa, b, sb, offsets, rows, m = _expert_inputs(sizes, 70, 256, 9, gather=True)
    back = torch.full((m + 300, 70), 9.0, dtype=F32, device=DEV)
    rows = torch.where(torch.arange(m, device=DEV) % 3 == 0, rows + 10 ** 6, rows).int()
    rows[1] = -5
    for bad in ([-7, per, m + 10 ** 6, 0, m], [0, m, 0, m, 5], [m + 9] * 5, [-1] * 5):
        pts.gemm_fp8_experts(a, sa, b, sb, torch.tensor(bad, dtype=torch.int32, device=DEV), rows, out=back[:m])
        torch.cuda.synchronize()
        assert torch.all(back[m:] == 9.0) and torch.all(torch.isfinite(back))
    d = pts.gemm_fp8_experts(a, sa, b, sb, offsets, rows, F32)
    near = pts.gemm_fp8_experts(a, sa, b, sb, offsets, rows.clamp(0, a.shape[0] - 1), F32)
    assert torch.equal(d, near)


def test_many_experts_of_few_rows(pts):
    """1024 experts (16 scans of 64), most without rows; a row of A named by several."""
    n, k, e = 40, 144, 1024
    rng = np.random.default_rng(8)
    sizes = (rng.random(e) < 0.2) * rng.integers(1, 40, e)
    sizes[-1] = 3
    b = torch.full((e, n, 144), 0, dtype=torch.uint8, device=DEV)
    b.copy_(_operand(e * n, k, 3)[:, :144].contiguous().view(torch.uint8).view(e, n, k))
    b = b.view(E4M3)
    m = int(sizes.sum())
    a, sa = _operand(7, k, 4), _scale(7, 2, 5)
    sb = _scale(e, 2, 6, False).view(e, 1, 2)
    offsets = torch.from_numpy(np.concatenate([[0], np.cumsum(sizes)]).astype(np.int32)).to(DEV)
    rows = torch.from_numpy(rng.integers(0, 7, m).astype(np.int32)).to(DEV)
    for dtype in (BF16, F32):
        d = pts.gemm_fp8_experts(a, sa, b, sb, offsets, rows, dtype)
        at = offsets.tolist()
        for x in np.flatnonzero(sizes):
            pick = rows[at[x]:at[x + 1]].long()
            _check_product(d[at[x]:at[x + 1]], a.contiguous().view(torch.uint8)[pick].view(E4M3), sa[pick], b[x], sb[x],
                           f"expert {x}")


# ---- sizes past 32 bits ----------------------------------------------------------

def test_operands_past_four_gigabytes(pts):
    """The last rows (or the last expert) of operands and results of more than 2^32 bytes equal the same rows on their own."""
    if torch.cuda.mem_get_info()[0] < 60 << 30:
        pytest.skip("needs 60 GB")
    k, m = 4096, (1 << 20) + (1 << 17) + 5
    part = torch.randn((8192, k), device=DEV).to(BF16)
    x = part.repeat(m // 8192 + 1, 1)[:m]               # 9.7 GB
    U.log(f"quantise {m} x {k}")
    q, s = pts.quantize_fp8(x)
    qp, sp = pts.quantize_fp8(x[m - 100:])
    assert torch.equal(q[m - 100:].view(torch.uint8), qp.view(torch.uint8)) and torch.equal(s[m - 100:], sp)
    qt, st = pts.quantize_fp8(x.t())                    # codes of 4096 x m, scales along m
    qs, ss = pts.quantize_fp8(x[m - 5:].t())            # the last, partial block: m % 128 = 5
    assert torch.equal(qt[:, m - 5:].contiguous().view(torch.uint8), qs.contiguous().view(torch.uint8))
    assert torch.equal(st[:, -1:], ss)
    U.log("product with an A of 4.8 GB, and an output of 4.8 GB")
    w, ws = pts.quantize_fp8(torch.randn((2048, k), device=DEV), (128, 128))
    d = pts.gemm_fp8(q, s, w, ws, BF16)
    assert torch.equal(d[m - 300:], pts.gemm_fp8(q, s, w, ws, BF16)[m - 300:])
    small = pts.gemm_fp8(qp, sp, w, ws, F32)            # the same rows on their own, fp32
    # both are within product_bound of the exact value; bf16's rounding is the larger part
    assert torch.all((d[m - 100:].float() - small).abs() <= small.abs() * 2.0 ** -7 + small.abs().max() * 2.0 ** -9)
    out = pts.moe_combine(d, torch.ones((4, 2), device=DEV),
                          torch.tensor([[m - 1, -1], [m - 7, -1], [0, -1], [m - 300, 5]], dtype=torch.int32, device=DEV))
    assert torch.equal(out[:3], d[[m - 1, m - 7, 0]])
    del x, qt, d, out
    U.log("experts whose weights span 5 GB")
    e, n = 80, 8192
    b = w.repeat(4, 2).view(torch.uint8).repeat(e, 1).view(e, n, 2 * k).view(E4M3)
    sb = ws.repeat(4, 2).repeat(e, 1).view(e, n // 128, 2 * k // 128)
    a, sa = pts.quantize_fp8(torch.randn((e, 2 * k), device=DEV))
    offsets = torch.arange(e + 1, dtype=torch.int32, device=DEV)
    d = pts.gemm_fp8_experts(a, sa, b, sb, offsets)
    for x in (0, e - 1):
        assert torch.equal(d[x:x + 1], pts.gemm_fp8(a[x:x + 1], sa[x:x + 1], b[x], sb[x], BF16)), x


# ---- routing -------------------------------------------------------------------

def _logits(m, e, dtype, seed, closed=0.0, ties=False):
    rng = np.random.default_rng(seed)
    x = rng.standard_normal((m, e)) * 2
    if ties:
        x = np.round(x)                                # many equal logits
    x[rng.random((m, e)) < closed] = -np.inf
    return torch.from_numpy(x).to(dtype)


ROUTES = [  # m, experts, k, groups, keep
    (1, 1, 1, 1, 1), (1, 256, 8, 8, 4), (3, 7, 7, 1, 1), (5, 64, 6, 4, 2), (16, 60, 4, 1, 1), (17, 128, 8, 1, 1), (100, 96, 2, 8, 3),
    (33, 512, 16, 16, 5), (20, 1024, 32, 64, 10), (40, 300, 5, 3, 1), (700, 160, 6, 8, 3), (4500, 64, 8, 1, 1), (4200, 130, 3, 2, 1),
    (4100, 256, 8, 8, 4),
]


@pytest.mark.parametrize("m,experts,k,groups,keep", ROUTES)
@pytest.mark.parametrize("score,bias,pair,renorm,dtype,closed,ties", [
    ("softmax", False, False, True, F32, 0.0, False), ("sigmoid", True, True, True, F32, 0.1, False),
    ("softmax", True, False, False, BF16, 0.0, True), ("sigmoid", False, True, False, BF16, 0.3, True),
    ("softmax", False, True, True, BF16, 0.9, True)])
def test_route(pts, m, experts, k, groups, keep, score, bias, pair, renorm, dtype, closed, ties):
    U.log(f"route {m}x{experts} k {k} groups {groups}/{keep} {score} bias {bias} pair {pair} {dtype} closed {closed}")
    x = _logits(m, experts, dtype, m + experts, closed, ties)
    if closed:
        x[m // 2] = float("-inf")                      # a token with no expert at all
    b = torch.from_numpy(np.round(np.random.default_rng(1).standard_normal(experts), 1).astype(np.float32)) if bias else None
    r = pts.moe_route(x.to(DEV), k, score=score, bias=None if b is None else b.to(DEV), groups=groups, topk_groups=keep,
                      group_score="top2_sum" if pair else "max", renormalize=renorm, scale=1.5)
    ids, w, offsets, rows, positions = R.route(_f64(x), k, score, None if b is None else _f64(b), groups, keep, pair, renorm, 1.5)
    assert np.array_equal(r.ids.cpu().numpy(), ids)
    assert np.array_equal(r.offsets.cpu().numpy(), offsets)
    assert np.array_equal(r.rows.cpu().numpy(), rows)
    assert np.array_equal(r.positions.cpu().numpy(), positions)
    # x - max is rounded once (its size in steps), exp is good to 2 steps, up to 1024 terms are added in chains of at
    # most 16 per lane and 6 across, a few products and divisions: span + 32 steps, twice (numerator and denominator)
    span = float(x[torch.isfinite(x)].float().abs().max()) * 2 if torch.isfinite(x).any() else 0.0
    assert np.all(np.abs(_f64(r.weights) - w) <= np.abs(w) * 2 * (span + 32) * 2.0 ** -24)


@pytest.mark.parametrize("m,experts,k", [(2049, 3, 1), (65536, 9, 8), (65537, 9, 8), (70001, 200, 8), (300007, 33, 4)])
def test_order_of_many_slots(pts, m, experts, k):
    """Chunks of the order on both sides of 2048 slots each, and of the count that needs no launch of its own."""
    U.log(f"order {m}x{experts} k {k}")
    x = _logits(m, experts, F32, m, 0.2, True)
    x[m // 3:m // 3 + 100] = float("-inf")
    r = pts.moe_route(x.to(DEV), k)
    ids = r.ids.cpu().numpy().reshape(-1)
    assert ids.min() == -1 and ids.max() == experts - 1
    expert = np.where(ids < 0, experts, ids)
    order = np.argsort(expert, kind="stable")
    assert np.array_equal(r.offsets.cpu().numpy(), np.searchsorted(expert[order], np.arange(experts + 1)))
    assert np.array_equal(r.rows.cpu().numpy(), order // k)
    position = np.empty_like(order)
    position[order] = np.arange(len(order))
    assert np.array_equal(r.positions.cpu().numpy().reshape(-1), np.where(ids < 0, -2 - position, position))


def test_route_of_no_tokens_and_strided_logits(pts):
    x = _logits(6, 40, F32, 1).to(DEV)
    r = pts.moe_route(x[:0], 2)
    assert r.ids.shape == (0, 2) and torch.all(r.offsets == 0)
    v = pts.moe_route(x[:, 3:35], 4)
    assert all(torch.equal(p, q) for p, q in zip(v, pts.moe_route(x[:, 3:35].contiguous(), 4)))


def test_route_with_logits_that_are_not_numbers(pts):
    x = _logits(4, 32, F32, 2)
    x[0, 5], x[1, 6], x[2, 7] = float("nan"), float("inf"), -float("inf")
    for score in ("softmax", "sigmoid"):
        for bias in (None, torch.zeros(32, device=DEV)):
            r = pts.moe_route(x.to(DEV), 3, score=score, bias=bias)
            ids, w, *_ = R.route(_f64(x), 3, score, None if bias is None else np.zeros(32))
            assert np.array_equal(r.ids.cpu().numpy(), ids), (score, bias is None)
            got = r.weights.cpu().numpy()
            assert np.array_equal(np.isnan(got), np.isnan(w)), (score, bias is None)
            assert not np.isnan(got[2:]).any() and 5 not in ids[0] and ids[1][0] == 6
    assert torch.isnan(pts.moe_route(x.to(DEV), 3).weights[0]).all()


def test_route_choice_is_not_rounded(pts):
    """Scores that differ by less than fp32 shows: 1 - sigmoid(x) near 2^-27, and biases that cancel the scores' gap."""
    x = torch.tensor([[18.0, 18.5, 19.0, 18.25]], device=DEV)
    r = pts.moe_route(x, 4, score="sigmoid", bias=torch.zeros(4, device=DEV))
    assert r.ids.tolist() == [[2, 1, 3, 0]]
    x = torch.tensor([[0.0, 2.0 ** -20, 2.0 ** -19, 0.0]], device=DEV)
    r = pts.moe_route(x, 4, score="sigmoid", bias=torch.full((4,), 4.0, device=DEV))
    assert r.ids.tolist() == [[2, 1, 0, 3]]


@pytest.mark.parametrize("m,experts,k", [(1, 8, 2), (5, 100, 32), (70, 256, 8), (30, 700, 6), (9, 1024, 17), (4200, 40, 4),
                                          (4100, 128, 8), (4097, 200, 5)])
@pytest.mark.parametrize("score,renorm,dtype", [("softmax", True, F32), ("softmax", False, BF16), ("sigmoid", True, BF16),
                                                 ("sigmoid", False, F32)])
def test_route_backward(pts, m, experts, k, score, renorm, dtype):
    U.log(f"route backward {m}x{experts} k {k} {score} {renorm} {dtype}")
    x = _logits(m, experts, dtype, m + k)
    if m > 4:
        x[3] = float("-inf")
        x[4, ::2] = float("-inf")
    ids = pts.moe_route(x.to(DEV), k, score=score, renormalize=renorm, scale=2.5).ids
    dw = torch.randn((m, k), generator=torch.Generator().manual_seed(k))
    dx = pts.moe_route_backward(dw.to(DEV), x.to(DEV), ids, score=score, renormalize=renorm, scale=2.5)
    i = ids.cpu().numpy()
    want = R.route_backward(_f64(dw), _f64(x), i, score, renorm, 2.5)
    # every term of the formula carries the scores' relative error (as in test_route, span 20) and a few roundings of
    # its own; the terms of one element are at most 2 scale (sum |dw|) in size for each p it is multiplied by
    p = np.stack([R.scores(row, score) for row in _f64(x)])
    got = np.where(i >= 0, np.take_along_axis(p, np.maximum(i, 0), 1), 0)
    size = 2.5 * np.abs(_f64(dw)).sum(1, keepdims=True) * (2 / (got.sum(1, keepdims=True) + 1e-20) if renorm else 1)
    bound = 8 * (20 + 32 + k) * 2.0 ** -24 * size * p * (1 + size * 0)
    if dtype == BF16:
        bound = bound + (np.abs(want) + bound) * 2.0 ** -8
    assert dx.dtype == dtype and np.all(np.abs(_f64(dx) - want) <= bound)
    if m <= 70:                                        # and against differences of the weights in 64 bits
        z, h = _f64(x), 1e-6
        for t, e in [(0, int(i[0, 0])), (0, experts - 1), (m // 2, int(max(i[m // 2, -1], 0)))]:
            if not np.isfinite(z[t, e]):
                continue
            up, dn = z[t:t + 1].copy(), z[t:t + 1].copy()
            up[0, e] += h
            dn[0, e] -= h
            diff = (_f64(dw)[t] * (R.weights_of(up, i[t:t + 1], score, renorm, 2.5) -
                                   R.weights_of(dn, i[t:t + 1], score, renorm, 2.5))).sum() / (2 * h)
            assert abs(want[t, e] - diff) <= 1e-6 * (1 + abs(diff))


@pytest.mark.parametrize("shift", [-300.0, 300.0, -3e38, 2e38])
@pytest.mark.parametrize("m,experts", [(3, 40), (5, 300), (4200, 64)])
def test_route_far_from_zero(pts, shift, m, experts):
    """The softmax and its gradient do not depend on where the logits lie."""
    base = torch.randint(-8, 9, (m, experts), generator=torch.Generator().manual_seed(m)).float()
    x = base + shift if abs(shift) < 1e6 else torch.where(base > 0, torch.tensor(shift), torch.tensor(shift) * 1.1)
    if shift == -300.0:
        x[0] = base[0] - 5000.0
    r = pts.moe_route(x.to(DEV), 4)
    ids, w, *_ = R.route(_f64(x), 4)
    assert np.array_equal(r.ids.cpu().numpy(), ids)
    assert np.all(np.abs(_f64(r.weights) - w) <= np.abs(w) * 2 * (20 + 32) * 2.0 ** -24)      # the spans are at most 16
    dw = torch.randn((m, 4), generator=torch.Generator().manual_seed(1))
    for renorm in (True, False):
        dx = pts.moe_route_backward(dw.to(DEV), x.to(DEV), r.ids, renormalize=renorm)
        want = R.route_backward(_f64(dw), _f64(x), ids, "softmax", renorm, 1.0)
        size = np.abs(_f64(dw)).sum(1, keepdims=True) * (2 / w.sum(1, keepdims=True) if renorm else 1)
        p = np.stack([R.scores(row, "softmax") for row in _f64(x)])
        got = np.take_along_axis(p, ids, 1).sum(1, keepdims=True)
        bound = 8 * (20 + 32 + 4) * 2.0 ** -24 * size * p / np.minimum(got, 1)
        assert np.all(np.abs(_f64(dx) - want) <= bound)


def test_route_backward_ids_twice_and_outside(pts):
    x = _logits(3, 20, F32, 4)
    ids = torch.tensor([[1, 1, 2], [-1, 25, 7], [-1, -1, 1 << 30]], dtype=torch.int32)
    dw = torch.randn((3, 3), generator=torch.Generator().manual_seed(1))
    for renorm in (True, False):
        for score in ("softmax", "sigmoid"):
            dx = pts.moe_route_backward(dw.to(DEV), x.to(DEV), ids.to(DEV), score=score, renormalize=renorm)
            i = np.where((ids.numpy() >= 0) & (ids.numpy() < 20), ids.numpy(), -1)
            want = R.route_backward(_f64(dw), _f64(x), i, score, renorm, 1.0)
            assert np.allclose(_f64(dx), want, rtol=1e-5, atol=1e-5 * np.abs(want).max()) and torch.all(dx[2] == 0)


# ---- combination ---------------------------------------------------------------

def _combine_inputs(m, n, k, dtype, seed, dropped=0.0, extra=0):
    rng = np.random.default_rng(seed)
    rows = m * k + extra
    pos = rng.permutation(m * k).reshape(m, k)
    pos = np.where(rng.random((m, k)) < dropped, -2 - pos, pos).astype(np.int32)
    y = torch.from_numpy(rng.standard_normal((rows, n))).to(dtype)
    w = torch.from_numpy(rng.random((m, k)).astype(np.float32))
    d = torch.from_numpy(rng.standard_normal((m, n))).to(dtype)
    return y, w, torch.from_numpy(pos), d


@pytest.mark.parametrize("m,n,k", [(1, 1, 1), (1, 4096, 8), (3, 100, 2), (7, 2056, 9), (50, 515, 5), (20, 64, 32), (300, 1000, 3)])
@pytest.mark.parametrize("dtype,dropped", [(BF16, 0.0), (F32, 0.3), (BF16, 0.5)])
def test_combine_and_gradients(pts, m, n, k, dtype, dropped):
    U.log(f"combine {m}x{n} k {k} {dtype} dropped {dropped}")
    y, w, pos, d = _combine_inputs(m, n, k, dtype, m + n, dropped)
    out = pts.moe_combine(y.to(DEV), w.to(DEV), pos.to(DEV))
    dy, dw = pts.moe_combine_backward(d.to(DEV), y.to(DEV), w.to(DEV), pos.to(DEV))
    p = pos.numpy()
    have = (p >= 0)[..., None]
    terms = np.where(have, _f64(w)[..., None] * _f64(y)[np.maximum(p, 0)], 0.0)
    want, mag = terms.sum(1), np.abs(terms).sum(1)
    half = 2.0 ** -8 if dtype == BF16 else 0.0
    tol = (k + 1) * 2.0 ** -24 * mag                    # k multiply-adds
    assert np.all(np.abs(_f64(out) - want) <= tol + half * (np.abs(want) + tol))
    want_dy = np.zeros((m * k, n))
    want_dy[np.where(p >= 0, p, -2 - p).reshape(-1)] = np.where(have, _f64(w)[..., None] * _f64(d)[:, None], 0.0).reshape(-1, n)
    assert np.all(np.abs(_f64(dy) - want_dy) <= np.abs(want_dy) * (half or 2.0 ** -24) * (1 + 2.0 ** -20))
    prod = np.where(have, _f64(y)[np.maximum(p, 0)] * _f64(d)[:, None], 0.0)
    # each thread adds at most ceil(n / 256) + 8 products in a chain, then 8 levels
    assert np.all(np.abs(_f64(dw) - prod.sum(2)) <= (n / 256 + 8 + 8) * 2.0 ** -24 * np.abs(prod).sum(2))


def test_combine_positions_outside_and_rows_unnamed(pts):
    y, w, pos, d = _combine_inputs(4, 40, 3, F32, 2, extra=5)
    pos[0, 0], pos[1, 1], pos[2, 2], pos[3, 0] = -1, 17, 1 << 30, -(1 << 31)
    w[0, 0] = float("nan")                              # the weight of no row is not looked at
    out = pts.moe_combine(y.to(DEV), w.to(DEV), pos.to(DEV))
    p = np.where((pos.numpy() >= 0) & (pos.numpy() < 17), pos.numpy(), -1)
    want = np.where(p[..., None] >= 0, np.nan_to_num(_f64(w))[..., None] * _f64(y)[np.maximum(p, 0)], 0).sum(1)
    assert np.allclose(_f64(out), want, rtol=1e-5, atol=1e-5)
    dy = torch.full((17, 40), 9.0, device=DEV)
    dw = torch.empty((4, 3), device=DEV)
    pts.pts_moe_combine_backward(d.to(DEV), 40, y.to(DEV), 1, 40, 17, w.to(DEV), pos.to(DEV), 4, 40, 3, dy, 40, dw)
    torch.cuda.synchronize()
    named = set(p[p >= 0].tolist())
    for r in range(17):
        assert bool(torch.all(dy[r] == 9.0)) == (r not in named), r
    assert torch.all(dw.cpu()[torch.from_numpy(p < 0)] == 0)
    empty = pts.moe_combine(y[:0].to(DEV), w.to(DEV), pos.to(DEV))
    assert torch.all(empty == 0)


def test_combine_strided(pts):
    y, w, pos, d = _combine_inputs(9, 64, 4, BF16, 6)
    wide = torch.nn.functional.pad(y, (1, 6)).to(DEV)[:, 1:65]   # unaligned rows
    assert torch.equal(pts.moe_combine(wide, w.to(DEV), pos.to(DEV)), pts.moe_combine(y.to(DEV), w.to(DEV), pos.to(DEV)))
    p = pts.moe_combine_backward(torch.nn.functional.pad(d, (3, 2)).to(DEV)[:, 3:67], wide, w.to(DEV), pos.to(DEV))
    q = pts.moe_combine_backward(d.to(DEV), y.to(DEV), w.to(DEV), pos.to(DEV))
    assert torch.equal(p[0], q[0]) and torch.allclose(p[1], q[1], rtol=1e-5, atol=1e-4)


# ---- together ------------------------------------------------------------------

def _layer(tokens, hidden, inner, experts, seed, pts):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((tokens, hidden), generator=g).to(DEV).to(BF16)
    logits = torch.randn((tokens, experts), generator=g).to(DEV)
    gu = torch.randn((experts, 2 * inner, hidden), generator=g).to(DEV).to(BF16) * hidden ** -0.5
    dn = torch.randn((experts, hidden, inner), generator=g).to(DEV).to(BF16) * inner ** -0.5
    pack = lambda w: tuple(torch.stack(t) for t in zip(*(pts.quantize_fp8(e, (128, 128)) for e in w)))  # noqa: E731
    return x, logits, *pack(gu), *pack(dn)


@pytest.mark.parametrize("tokens,hidden,inner,experts,k", [(1, 256, 128, 8, 2), (30, 512, 256, 16, 4), (500, 256, 384, 8, 3)])
def test_layer_of_experts(pts, tokens, hidden, inner, experts, k):
    """Routing, both products, the gate and the combination in a row, each stage from the one before."""
    U.log(f"layer {tokens} tokens {hidden}/{inner} {experts} experts")
    x, logits, gu, gus, dn, dns = _layer(tokens, hidden, inner, experts, 11, pts)
    if tokens > 4:
        logits[tokens - 3:] = float("-inf")             # a padded batch
    out = pts.moe_fp8(x, logits, k, gu, gus, dn, dns, scale=2.0)
    ids, w, offsets, rows, positions = R.route(_f64(logits), k, scale=2.0)
    xq, xs = R.quantize(x.float().cpu().numpy(), 1)
    xv = xq * R.expand(xs, tokens, hidden)
    want, mag = np.zeros((tokens, hidden)), np.zeros((tokens, hidden))
    for t in range(tokens):
        for j in range(k):
            e = ids[t, j]
            if e < 0:
                continue
            h = R.decode(gu[e]) * R.expand(gus[e].cpu().numpy(), 2 * inner, hidden) @ xv[t]
            act = h[:inner] / (1 + np.exp(-h[:inner])) * h[inner:]
            v = R.decode(dn[e]) * R.expand(dns[e].cpu().numpy(), hidden, inner)
            want[t] += w[t, j] * (v @ act)
            mag[t] += w[t, j] * (np.abs(v) @ (np.abs(act) + np.abs(act).max() * 2.0 ** -9))
    # per row of y: the activation's two bf16 inputs (|g| + 2 half steps of 2^-8 of them), its e4m3 code (2^-4, or 2^-10
    # of the block's scale, which the magnitude's floor covers), y's rounding; fp32 sums are far below these
    tol = (2.0 ** -4 + 8 * 2.0 ** -8 + 2.0 ** -8) * mag
    err = np.abs(_f64(out) - want)
    U.log(f"layer: worst error / bound {float((err / np.maximum(tol + np.abs(want) * 2.0 ** -8, 1e-30)).max()):.3f}")
    assert np.all(err <= tol + np.abs(want) * 2.0 ** -8)
    if tokens > 4:
        assert torch.all(out[tokens - 3:] == 0)


def test_every_operator_replays_from_a_graph(pts):
    tokens, k = 200, 2
    x, logits, gu, gus, dn, dns = _layer(tokens, 256, 128, 8, 5, pts)
    dw = torch.randn((tokens, k), device=DEV)

    def step():
        r = pts.moe_route(logits, k)
        out = pts.moe_fp8(x, logits, k, gu, gus, dn, dns)
        y = pts.gemm_fp8_experts(*pts.quantize_fp8(x), gu, gus, r.offsets, r.rows)
        dy, dwt = pts.moe_combine_backward(y[:tokens], y, r.weights, r.positions)
        dx = pts.moe_route_backward(dwt + dw, logits, r.ids)
        a, sa = pts.quantize_fp8(x.t())
        return [out, y, dy, dwt, dx, pts.gemm_fp8(a, sa, a, sa), *r]

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for i in range(3):
        x.copy_(torch.randn_like(x))
        logits.copy_(torch.randn_like(logits))
        for t in got:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for j, (p, q) in enumerate(zip(got, step())):
            assert torch.equal(p, q), (i, j)


def test_two_graphs_of_the_router_share_nothing(pts):
    """Two captured routings (with workspaces) replayed at once on two streams."""
    xs = [torch.randn((3000 + 500 * i, 64), device=DEV) for i in range(2)]
    pts.moe_route(xs[0], 4)
    torch.cuda.synchronize()
    graphs, got = [], []
    for x in xs:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            got.append(pts.moe_route(x, 4))
        graphs.append(g)
    want = [pts.moe_route(x, 4) for x in xs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in xs]
    for _ in range(4):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        for p, q in zip(got, want):
            assert all(torch.equal(u, v) for u, v in zip(p, q))


def test_calls_on_several_streams_at_once(pts):
    inputs = [_layer(t, 256, 128, 8, 20 + i, pts) for i, t in enumerate((7, 300, 40, 3000))]
    alone = [pts.moe_fp8(*v[:2], 2, *v[2:]) for v in inputs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in inputs]
    got = [[] for _ in inputs]
    for _ in range(3):
        for i, v in enumerate(inputs):
            with torch.cuda.stream(streams[i]):
                got[i].append(pts.moe_fp8(*v[:2], 2, *v[2:]))
    torch.cuda.synchronize()
    for i, want in enumerate(alone):
        assert all(torch.equal(g, want) for g in got[i]), i


def test_one_plan_of_the_bf16_gemm_beside_them(pts):
    """The bf16 GEMM's results do not change beside the new calls."""
    a = U.device_uniform(700, 512, 3, 1)
    b = U.device_uniform(900, 512, 3, 2)
    before = pts.gemm(a, b)
    q, s = pts.quantize_fp8(a)
    w, t = pts.quantize_fp8(b, (128, 128))
    pts.gemm_fp8(q, s, w, t)
    assert torch.equal(before, pts.gemm(a, b))
