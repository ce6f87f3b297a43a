"""GPU tests of the routed-experts operators where they go wrong most easily: scores near their
limits.

The references are 64-bit. Tolerances are stated where they are used, in units u = 2^-24, half a
step of fp32 relative to the value.
"""
from __future__ import annotations

import numpy as np
import pytest
import torch

from tests import experts_reference as R
from tests import gpu_util as U

pytestmark = pytest.mark.gpu
DEV = U.DEV
BF16, F32 = torch.bfloat16, torch.float32
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
