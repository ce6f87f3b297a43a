"""GPU tests of the routed-experts operators where they go wrong most easily: scores near their
limits, gates far from zero, blocks that are not finite, workgroups that take a second tile, and
operands past 4 GB whose rows all differ.

The references are 64-bit; those of large products are computed on the device. Tolerances are
stated where they are used, in units u = 2^-24, half a step of fp32 relative to the value.
"""
from __future__ import annotations

import numpy as np
import pytest
import torch

from tests import experts_reference as R
from tests import gpu_util as U
from tests.test_gpu_experts import _expert_inputs, _operand, _scale

pytestmark = pytest.mark.gpu
DEV = U.DEV
BF16, F32, E4M3 = torch.bfloat16, torch.float32, torch.float8_e4m3fn
u = 2.0 ** -24


@pytest.fixture(scope="module")
def pts():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import persistent_tile_scheduling_amd as mod
    return mod


def _f64(t):
    return t.detach().float().cpu().double().numpy()


# ---- the router's gradient ---------------------------------------------------------

def _sigmoid_slope(x):
    """p (1 - p) without the difference: z / (1 + z)^2 with z = exp(-|x|)."""
    z = np.exp(-np.abs(x))
    return z / (1 + z) ** 2


def _sigmoid_gradient(dw, x, ids, renorm, scale):
    """The formula's gradient in 64 bits, and the sum of the magnitudes of its terms (both m x experts)."""
    p, slope = 1 / (1 + np.exp(-x)), _sigmoid_slope(x)
    dx, size = np.zeros_like(x), np.zeros_like(x)
    for t in range(x.shape[0]):
        ok = ids[t] >= 0
        at, d = ids[t][ok], dw[t][ok]
        total = p[t, at].sum() + 1e-20 if renorm else 1.0
        mean, most = ((d * p[t, at]).sum() / total, (np.abs(d) * p[t, at]).sum() / total) if renorm else (0.0, 0.0)
        np.add.at(dx[t], at, scale / total * (d - mean) * slope[t, at])
        np.add.at(size[t], at, scale / total * (np.abs(d) + most) * slope[t, at])
    return dx, size


@pytest.mark.parametrize("m,experts,k", [(5, 40, 4), (3, 300, 6), (2, 700, 3), (4200, 24, 2)])
@pytest.mark.parametrize("low,high", [(10.0, 30.0), (-30.0, -10.0), (60.0, 85.0), (-1.0, 40.0)])
@pytest.mark.parametrize("renorm", [True, False])
def test_sigmoid_gradient_of_scores_near_one(pts, m, experts, k, low, high, renorm):
    """The gradient of a score near one is as exact relative to its size as any other's."""
    U.log(f"sigmoid gradient {m}x{experts} k {k} logits in [{low}, {high}] renormalised {renorm}")
    rng = np.random.default_rng(m + int(abs(high)))
    x = torch.from_numpy(rng.uniform(low, high, (m, experts)).astype(np.float32))
    dw = torch.from_numpy(rng.standard_normal((m, k)).astype(np.float32))
    ids = torch.from_numpy(np.stack([rng.permutation(experts)[:k] for _ in range(m)]).astype(np.int32))
    dx = pts.moe_route_backward(dw.to(DEV), x.to(DEV), ids.to(DEV), score="sigmoid", renormalize=renorm, scale=2.5)
    want, size = _sigmoid_gradient(_f64(dw), _f64(x), ids.numpy(), renorm, 2.5)
    # exp is good to 2 u, so a score to 4 u (exp 2, sum 1, division 1); dw p then to 5 + k u summed, the scores' sum to
    # 5 + k, their quotient to 2 k + 11, less dw 1, times scale / sum k + 7: 3 k + 19 u of the terms' magnitude. The slope
    # is exp (2), two reciprocals of a sum (4 each) and two products: 12 u. Second orders: 1%
    assert np.all(np.abs(_f64(dx) - want) <= 1.01 * (3 * k + 19 + 12) * u * size)
    if renorm and low == 10.0:                         # and against differences of the weights in 64 bits
        z, h = _f64(x)[:1], 1e-2
        for e in ids[0].tolist():
            up, dn = z.copy(), z.copy()
            up[0, e] += h
            dn[0, e] -= h
            diff = (_f64(dw)[0] * (R.weights_of(up, ids[:1].numpy(), "sigmoid", True, 2.5) -
                                   R.weights_of(dn, ids[:1].numpy(), "sigmoid", True, 2.5))).sum() / (2 * h)
            # h^2 / 6 of the third derivative (at most the first, the scores being 1 - exp(-x)), and the weights' own
            # 64-bit rounding over 2 h
            assert abs(want[0, e] - diff) <= 1e-4 * abs(want[0, e]) + 64 * 2.0 ** -53 * 2.5 * np.abs(_f64(dw)[0]).sum() / h


def _gradient_by_differences_of_slots(dw, x, ids, score, renorm, scale):
    """The formula's gradient in 64 bits with every difference taken term by term, and the magnitudes of those terms:
    1 - p as the sum of the other scores, a weight's derivative as sums of p_i (dw_s - dw_i)."""
    dx, size = np.zeros_like(x), np.zeros_like(x)
    for t in range(x.shape[0]):
        if score == "sigmoid":
            p, factor = 1 / (1 + np.exp(-x[t])), _sigmoid_slope(x[t])
        else:
            p = factor = R.scores(x[t], score)
        ok = np.flatnonzero(ids[t] >= 0)
        at, d = ids[t][ok], dw[t][ok].astype(np.float64)
        q = p[at]
        by, most = scale * d, scale * np.abs(d)        # the gradient by each slot's score
        if renorm:
            total = q.sum() + 1e-20
            by = scale / total ** 2 * ((q[None, :] * (d[:, None] - d[None, :])).sum(1) + 1e-20 * d)
            most = scale / total ** 2 * ((q[None, :] * (np.abs(d)[:, None] + np.abs(d)[None, :]) * (1 - np.eye(len(ok)))).sum(1) +
                                         1e-20 * np.abs(d))
        if score == "sigmoid":
            np.add.at(dx[t], at, by * factor[at])
            np.add.at(size[t], at, most * factor[at])
            continue
        if renorm:                                     # sum of by q: the differences cancel in pairs, the 1e-20 stays
            back, back_most = scale / total ** 2 * 1e-20 * (d * q).sum(), scale / total ** 2 * 1e-20 * (np.abs(d) * q).sum()
            dx[t], size[t] = -p * back, p * back_most
            np.add.at(dx[t], at, by * q)
            np.add.at(size[t], at, most * q)
            continue
        for e in range(x.shape[1]):
            mine = at == e
            rest = p.sum() - p[e] if p[e] < 0.5 else np.delete(p, e).sum()
            dx[t, e] = p[e] * (by[mine].sum() * rest - (by * q)[~mine].sum())
            size[t, e] = p[e] * (most[mine].sum() * rest + (most * q)[~mine].sum())
    return dx, size


@pytest.mark.parametrize("m,experts,k", [(5, 40, 4), (3, 300, 6), (2, 700, 32), (6, 30, 1), (4200, 24, 2), (4100, 120, 8),
                                          (4097, 200, 17)])
@pytest.mark.parametrize("lead", [0.0, 8.0, 25.0])
@pytest.mark.parametrize("score,renorm", [("softmax", False), ("softmax", True), ("sigmoid", True)])
@pytest.mark.parametrize("twice", [False, True])
def test_gradient_of_a_score_that_leads(pts, m, experts, k, lead, score, renorm, twice):
    """One expert far ahead of the others: its gradient and theirs are as small as 1 - p, and as exact relative to that."""
    U.log(f"gradient {m}x{experts} k {k} lead {lead} {score} renormalised {renorm} twice {twice}")
    rng = np.random.default_rng(m + k)
    x = rng.standard_normal((m, experts)) - (20 if score == "sigmoid" else 0)
    ids = np.stack([rng.permutation(experts)[:k] for _ in range(m)]).astype(np.int32)
    np.put_along_axis(x, ids[:, :1].astype(np.int64), x.max(1, keepdims=True) + lead, 1)
    if twice:
        ids[:, k // 2] = ids[:, (k - 1) * (m % 2)]      # another slot's, or the leading one's
    ids[1, k - 1] = -1 if k > 1 else ids[1, k - 1]
    x, dw = torch.from_numpy(x.astype(np.float32)), torch.from_numpy(rng.standard_normal((m, k)).astype(np.float32))
    some = np.arange(m) if m < 100 else np.r_[:40, m - 40:m]
    for dtype in (F32, BF16):
        v = x.to(dtype)
        dx = pts.moe_route_backward(dw.to(DEV), v.to(DEV), torch.from_numpy(ids).to(DEV), score=score, renormalize=renorm, scale=2.5)
        z = _f64(v)[some]
        want, size = _gradient_by_differences_of_slots(_f64(dw)[some], z, ids[some], score, renorm, 2.5)
        # a softmax score: x - max rounds (its span in u), exp is good to 2 u, the sum adds 22 roundings, the division 1,
        # numerator and denominator: 2 span + 28 u; a sigmoid's 4 u and its slope 12. Not renormalised: the rest's sum 22
        # more, differences, products and sums 2 k + 10, times a score. Renormalised: three scores' sums, k + 3 each
        one = 12 if score == "sigmoid" else 2 * (z.max() - z.min()) + 28
        bound = 1.01 * (4 * one + 3 * k + 32) * u * size + 2.0 ** -140
        if dtype == BF16:
            bound = bound + (np.abs(want) + bound) * 2.0 ** -8
        assert np.all(np.abs(_f64(dx)[some] - want) <= bound), dtype


@pytest.mark.parametrize("m,experts", [(5, 40), (4200, 100)])
@pytest.mark.parametrize("renorm", [True, False])
def test_sigmoid_gradient_of_experts_that_are_closed(pts, m, experts, renorm):
    """An expert that a NaN closes to a token has no part in its weights: gradient 0, the others' as without it."""
    x = torch.randn((m, experts), generator=torch.Generator().manual_seed(m)) * 2
    x[::2, 3] = float("nan")
    x[1::2, 5] = -float("inf")
    dw = torch.randn((m, 3), generator=torch.Generator().manual_seed(1)).to(DEV)
    r = pts.moe_route(x.to(DEV), 3, score="sigmoid", renormalize=renorm)
    assert not torch.any(torch.isnan(r.weights))
    dx = pts.moe_route_backward(dw, x.to(DEV), r.ids, score="sigmoid", renormalize=renorm)
    same = pts.moe_route_backward(dw, torch.nan_to_num(x, nan=0.0, neginf=-float("inf")).to(DEV), r.ids, score="sigmoid",
                                  renormalize=renorm)
    assert torch.equal(dx, same) and torch.all(dx[::2, 3] == 0) and torch.all(dx[1::2, 5] == 0)


# ---- quantisation ------------------------------------------------------------------

@pytest.mark.parametrize("low,high", [(-4.0, 4.0), (-87.0, -40.0), (40.0, 87.0), (-88.7, -87.3), (-100.0, -88.7)])
@pytest.mark.parametrize("up", [1e3, 3e30])
def test_gate_far_from_zero(pts, low, high, up):
    """The gated value in fp32, seen through the scale of blocks that hold one value each."""
    m, blocks = 40, 9
    rng = np.random.default_rng(int(abs(high)))
    x = np.zeros((m, 2, blocks, 128), dtype=np.float32)
    at = rng.integers(0, 128, (m, blocks))
    rows, cols = np.arange(m)[:, None], np.arange(blocks)[None, :]
    x[rows, 0, cols, at] = g = rng.uniform(low, high, (m, blocks)).astype(np.float32)
    x[rows, 1, cols, at] = v = (up * rng.uniform(1, 2, (m, blocks))).astype(np.float32)
    q, s = pts.quantize_fp8(torch.from_numpy(x.reshape(m, -1)).to(DEV), swiglu=True)
    g, v = g.astype(np.float64), v.astype(np.float64)
    z = np.exp(-np.abs(g))
    h = np.where(g < 0, g * z, g) / (1 + z) * v
    # exp is good to a step: 2 u of z, or 2^-149; then 1 + z (2 u at most, as z <= 1), g z, the division, the product with
    # `up` and the scale's division: 8 u
    tol = (8 * u + np.where(g < 0, np.maximum(2.0 ** -149 / z - 2 * u, 0), 0)) * 1.001
    want = np.abs(h) / 448
    clear = want * (1 - tol) > 2.0 ** -126             # below, the scale is its least value
    assert clear.mean() > (0.9 if up > 1e4 or low > -88 else -1)
    assert np.all(np.abs(_f64(s) - want)[clear] <= (tol * want)[clear])
    codes = R.decode(q).reshape(m, blocks, 128)
    assert np.all(codes[rows, cols, at][clear] == (448 * np.sign(h))[clear])


@pytest.mark.parametrize("k", [300, 129, 7, 256])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("form", ["rows", "gated", "across", "square", "square across"])
def test_padding_is_zero_beside_a_block_that_is_not_finite(pts, k, bad, dtype, form):
    """The codes between k and the next multiple of 16 are written as 0, also where their block's codes are NaN."""
    m, ldq, wide = 130, 320, -(-k // 16) * 16
    x = torch.randn((m, 2 * k if form == "gated" else k), generator=torch.Generator().manual_seed(k)).to(dtype)
    x[m - 1, k - 1] = x[0, k - 1] = bad
    across, square = "across" in form, "square" in form
    dev = x.t().contiguous().to(DEV) if across else x.to(DEV)
    q = torch.full((m, ldq), 0x55, dtype=torch.uint8, device=DEV)
    s = torch.empty((m, 3), device=DEV)
    pts.pts_quantize_fp8(dev, 0 if dtype == BF16 else 1, 1 if across else 0, m, k, dev.shape[1], 128 if square else 1,
                         int(form == "gated"), q, ldq, s, 3, 1)
    torch.cuda.synchronize()
    first = (k - 1) // 128 * 128
    assert torch.all(q[m - 1, first:k] & 0x7F == 0x7F) and torch.all(q[0, first:k] & 0x7F == 0x7F)
    assert torch.all(q[:, k:wide] == 0) and torch.all(q[:, wide:] == 0x55)


# ---- products ------------------------------------------------------------------------

_TABLE = torch.from_numpy(R.E4M3)


def _values64(codes, scale):
    """What codes and block scales stand for, on the device in 64 bits."""
    m, k = codes.shape
    v = _TABLE.to(DEV)[codes.contiguous().view(torch.uint8).int()]
    s = scale.double()
    if s.shape[0] != m:
        s = s.repeat_interleave(128, 0)[:m]
    return v * s.repeat_interleave(128, 1)[:, :k]


def _check(d, a, sa, b, sb, what):
    """|d - A . B| against the bound of tests/experts_reference.py (product_bound), all on the device."""
    x, y = _values64(a, sa), _values64(b, sb)
    k = x.shape[1]
    want, mag = x @ y.t(), x.abs() @ y.abs().t()
    bound = (128 + 2 + -(-k // 128) + 7) * u * mag
    if d.dtype == BF16:
        largest = torch.zeros_like(want)
        xa, ya = x.abs(), y.abs()
        for k0 in range(0, k, 8):
            most = torch.zeros_like(want)
            for i in range(k0, min(k0 + 8, k)):
                most = torch.maximum(most, xa[:, i:i + 1] * ya[:, i])
            largest += most
        bound = bound + 7 * 2.0 ** -13 * largest
        bound = bound + (want.abs() + bound) * 2.0 ** -8
    worst = float(((d.double() - want).abs() / bound.clamp(min=1e-300)).max())
    U.log(f"{what}: worst error / bound = {worst:.3f}")
    assert worst <= 1, what                            # false for a NaN too


@pytest.mark.parametrize("m,n,k,dtype", [
    (3100, 3300, 300, F32),         # 650 tiles of 128 x 128, two of which share a compute unit
    (2810, 3000, 300, BF16),        # 528 of them
    (2816, 3000, 640, BF16),
    (4500, 4400, 300, BF16),        # 324 tiles of 256 x 256
    (4500, 4404, 1024, BF16),
    (4352, 4608, 130, BF16),
])
@pytest.mark.parametrize("rows", [False, True])
def test_workgroups_that_take_a_second_tile(pts, m, n, k, dtype, rows):
    """More tiles than workgroups on 256 compute units, ragged and whole extents and k blocks."""
    U.log(f"product {m}x{n}x{k} rows {rows} {dtype}")
    kb = -(-k // 128)
    a, b = _operand(m, k, 1 + m), _operand(n, k, 2 + n)
    sa, sb = _scale(m, kb, 3), _scale(n if rows else -(-n // 128), kb, 4, rows)
    back = torch.full((m + 1, n + 8), 9.0, dtype=dtype, device=DEV)
    d = pts.gemm_fp8(a, sa, b, sb, out=back[:m, :n])
    _check(d, a, sa, b, sb, f"{m}x{n}x{k}")
    assert torch.all(back[m:] == 9.0) and torch.all(back[:, n:] == 9.0)


@pytest.mark.parametrize("gather", [False, True])
@pytest.mark.parametrize("n,k", [(4400, 300), (4608, 256)])
def test_experts_whose_workgroups_take_a_second_tile(pts, n, k, gather):
    sizes = [600, 0, 300, 900, 257, 256, 255, 0, 100, 1500]     # 20 tile rows of 18
    U.log(f"experts {sizes} n {n} k {k} gather {gather}")
    a, sa, b, sb, offsets, rows, m = _expert_inputs(sizes, n, k, 41, behind=5, gather=gather, before=2)
    out = torch.full((m, n), 9.0, dtype=BF16, device=DEV)
    pts.gemm_fp8_experts(a, sa, b, sb, offsets, rows, out=out)
    o = offsets.cpu().tolist()
    for e in range(len(sizes)):
        if sizes[e]:
            pick = (rows[o[e]:o[e + 1]] if gather else torch.arange(o[e], o[e + 1], device=DEV)).long()
            _check(out[o[e]:o[e + 1]], a.view(torch.uint8)[pick].view(E4M3), sa[pick], b[e], sb[e], f"expert {e}")
    assert torch.all(out[:o[0]] == 9.0) and torch.all(out[o[-1]:] == 9.0)


@pytest.mark.parametrize("m,n,bad", [(4, 150, 2), (40, 150, 17), (200, 150, 127), (2000, 2100, 128),
                                     (4100, 4000, 255)])
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("rows", [False, True])
def test_nan_stays_in_its_row_and_column(pts, m, n, bad, dtype, rows):
    """A NaN code, in the ragged last k block, and a NaN scale reach their own row or columns and nothing else, in every
    kernel of both result types."""
    U.log(f"NaN in {m}x{n} {dtype} rows {rows}")
    k = 300
    a, b = _operand(m, k, 1), _operand(n, k, 2)
    a.view(torch.uint8)[bad, 299] = 0x7F
    sa, sb = _scale(m, 3, 3), _scale(n if rows else -(-n // 128), 3, 4, False)
    d = torch.isnan(pts.gemm_fp8(a, sa, b, sb, dtype))
    assert torch.all(d[bad]) and not torch.any(d[:bad]) and not torch.any(d[bad + 1:])
    sb[1, 0] = float("nan")
    d = torch.isnan(pts.gemm_fp8(a, sa, b, sb, dtype))
    at = torch.zeros(n, dtype=torch.bool, device=DEV)
    at[1:2] = rows
    at[128:256] |= not rows
    assert torch.all(d[:, at]) and torch.all(d[bad])
    assert not torch.any(d[:bad, ~at]) and not torch.any(d[bad + 1:, ~at])


# ---- operands past 4 GB ----------------------------------------------------------------

def test_rows_past_four_gigabytes_are_the_right_ones(pts):
    """Rows that repeat with a period of 8191, so that an offset short of 2^31 or 2^32 bytes or elements names another row:
    the quantiser's two directions, the product, and the combination with its gradients against their definitions."""
    if torch.cuda.mem_get_info()[0] < 60 << 30:
        pytest.skip("needs 60 GB")
    k, n, m = 4096, 2048, (1 << 20) + (1 << 17) + 5
    part = torch.randn((8191, k), generator=torch.Generator(DEV).manual_seed(1), device=DEV).to(BF16)
    x = part[torch.arange(m, device=DEV) % 8191]        # 9.7 GB
    some = torch.cat([torch.arange(at - 4, at + 4) for at in (1 << 18, 1 << 19, 1 << 20, m - 4)]).to(DEV)
    U.log(f"quantise {m} x {k}")
    q, s = pts.quantize_fp8(x)
    want_q, want_s = R.quantize(x[some].float().cpu().numpy(), 1)
    assert np.array_equal(R.decode(q.view(torch.uint8)[some]), want_q)
    assert np.array_equal(s[some].cpu().numpy(), want_s)
    U.log("and its transpose")
    qt, st = pts.quantize_fp8(x.t())
    for at in (1 << 19, 1 << 20, m - 5):                # blocks of 128 rows of x, the last one of 5
        want_q, want_s = R.quantize(x[at:at + 128, :200].t().float().cpu().numpy(), 1)
        assert np.array_equal(R.decode(qt[:200, at:at + 128]), want_q)
        assert np.array_equal(st[:200, at // 128].cpu().numpy(), want_s[:, 0])
    del qt, st, x
    U.log("product with an A and a result of 4.8 GB")
    w, ws = pts.quantize_fp8(torch.randn((n, k), generator=torch.Generator(DEV).manual_seed(2), device=DEV), (128, 128))
    d = pts.gemm_fp8(q, s, w, ws, BF16)
    _check(d[some], q.view(torch.uint8)[some].view(E4M3), s[some], w, ws, "rows on both sides of the limits")
    U.log("combination of rows of 4.8 GB")
    positions = some.flip(0).view(-1, 4).int()
    weights = torch.rand(positions.shape, device=DEV)
    out = pts.moe_combine(d, weights, positions)
    y, wt = d[some.flip(0)].double().view(-1, 4, n), weights.double().unsqueeze(2)
    tol = 5 * u * (wt * y).abs().sum(1)
    want = (wt * y).sum(1)
    assert torch.all((out.double() - want).abs() <= tol + (want.abs() + tol) * 2.0 ** -8)
    dout = torch.randn(out.shape, device=DEV).to(BF16)
    dy, dweights = pts.moe_combine_backward(dout, d, weights, positions)
    want = (wt * dout.double().unsqueeze(1)).view(-1, n)
    assert torch.all((dy[some.flip(0)].double() - want).abs() <= want.abs() * (2.0 ** -8 * (1 + 2.0 ** -10)))
    prod = y * dout.double().unsqueeze(1)
    assert torch.all((dweights.double() - prod.sum(2)).abs() <= (n / 256 + 16) * u * prod.abs().sum(2))


def test_experts_past_four_gigabytes_are_the_right_ones(pts):
    """80 experts of 64 MB, all different: the first, the ones on both sides of 2^30, 2^31 and 2^32 bytes, and the last."""
    if torch.cuda.mem_get_info()[0] < 40 << 30:
        pytest.skip("needs 40 GB")
    e, n, k = 80, 8192, 8192
    g = torch.Generator(DEV).manual_seed(3)
    b = torch.empty((e, n, k), dtype=torch.uint8, device=DEV)
    for i in range(e):
        v = torch.randint(0, 256, (n, k), generator=g, dtype=torch.uint8, device=DEV)
        b[i] = torch.where(v & 0x7F == 0x7F, 0, v)
    b = b.view(E4M3)
    sb = torch.rand((e, n // 128, k // 128), generator=g, device=DEV) + 0.5
    a, sa = pts.quantize_fp8(torch.randn((e, k), generator=g, device=DEV))
    offsets = torch.arange(e + 1, dtype=torch.int32, device=DEV)
    for dtype in (BF16, F32):
        d = pts.gemm_fp8_experts(a, sa, b, sb, offsets, out_dtype=dtype)
        for i in (0, 15, 16, 31, 32, 63, 64, 79):
            _check(d[i:i + 1], a[i:i + 1], sa[i:i + 1], b[i], sb[i], f"expert {i} {dtype}")
