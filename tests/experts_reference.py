"""The routed-experts operators in 64 bits, for the tests: plain loops over
blocks, experts and tokens, from the definitions in ``include/pts_experts.h``."""
from __future__ import annotations

import numpy as np
import torch

E4M3_CODES = np.arange(256, dtype=np.uint8)


def e4m3_values() -> np.ndarray:
    """The value of each of the 256 codes: sign, 4 exponent bits (bias 7), 3 fraction bits; 0x7F and 0xFF are NaN."""
    sign = np.where(E4M3_CODES & 0x80, -1.0, 1.0)
    exp, frac = (E4M3_CODES >> 3) & 15, (E4M3_CODES & 7).astype(np.float64)
    v = np.where(exp == 0, frac / 8 * 2.0 ** -6, (1 + frac / 8) * 2.0 ** (exp.astype(np.float64) - 7))
    v[(E4M3_CODES & 0x7F) == 0x7F] = np.nan
    return sign * v


E4M3 = e4m3_values()


def decode(codes: torch.Tensor) -> np.ndarray:
    return E4M3[codes.detach().contiguous().view(torch.uint8).cpu().numpy()]


def nearest_e4m3(v: np.ndarray) -> np.ndarray:
    """Values rounded to the nearest e4m3 value, ties to the code with an even fraction."""
    grid = E4M3[:127]                                  # 0 .. 448
    a = np.abs(np.nan_to_num(v, nan=0.0))
    hi = np.clip(np.searchsorted(grid, a), 1, 126)
    lo = hi - 1
    down = (a - grid[lo] < grid[hi] - a) | ((a - grid[lo] == grid[hi] - a) & (lo % 2 == 0))
    r = np.where(a >= grid[126], grid[126], np.where(down, grid[lo], grid[hi]))
    return np.where(np.isnan(v), np.nan, np.copysign(r, v))


def quantize(x: np.ndarray, tall: int):
    """(codes' values, scales) of float32-valued x for blocks of `tall` x 128, by float32 divisions."""
    x = np.asarray(x, dtype=np.float32)
    m, k = x.shape
    mb, kb = -(-m // tall), -(-k // 128)
    scale = np.empty((mb, kb), dtype=np.float32)
    q = np.empty((m, k))
    for i in range(mb):
        for j in range(kb):
            at = np.s_[i * tall:(i + 1) * tall, j * 128:(j + 1) * 128]
            most = np.float32(np.abs(x[at]).max())
            s = np.maximum(most / np.float32(448), np.float32(2.0 ** -126)) if np.isfinite(most) else np.float32(np.nan)
            scale[i, j] = s
            with np.errstate(invalid="ignore"):
                q[at] = nearest_e4m3((x[at] / s).astype(np.float64))
    return q, scale


def expand(scale: np.ndarray, m: int, k: int) -> np.ndarray:
    """Block scales (one per row or per 128 rows) at every element."""
    s = scale.astype(np.float64)
    if s.shape[0] != m:
        s = np.repeat(s, 128, axis=0)[:m]
    return np.repeat(s, 128, axis=1)[:, :k]


def product(a, sa, b, sb):
    """(A . B^T, sum of the terms' magnitudes, sum over groups of 8 consecutive k of the largest term) from values and
    block scales."""
    x = a * expand(sa, *a.shape)
    y = b * expand(sb, *b.shape)
    k = a.shape[1]
    largest = np.zeros((a.shape[0], b.shape[0]))
    for k0 in range(0, k, 8):
        u, v = np.abs(x[:, k0:k0 + 8]), np.abs(y[:, k0:k0 + 8])
        most = np.zeros_like(largest)
        for i in range(u.shape[1]):
            np.maximum(most, np.outer(u[:, i], v[:, i]), out=most)
        largest += most
    return x @ y.T, np.abs(x) @ np.abs(y).T, largest


def product_bound(magnitude, largest, exact, k: int, dtype) -> np.ndarray:
    """How far a result may be off. Each of a block's 128 products is exact; summing them in
    fp32 rounds at most 128 times, the scale product and the multiply-add twice, and each of the ceil(k / 128) (+ 7
    partial sums) additions once, each by 2^-24 of a partial result that is at most the sum of magnitudes.

    bf16 results come from the matrix unit's e4m3 products, of which it drops, in each group of 8 consecutive k, what
    lies 14 binary places below the largest product's exponent: at most 7 products lose less than 2^-13 of the largest
    each. They round once more, by 2^-8."""
    bound = (128 + 2 + -(-k // 128) + 7) * 2.0 ** -24 * magnitude
    if dtype == torch.bfloat16:
        bound = bound + 7 * 2.0 ** -13 * largest
        bound = bound + (np.abs(exact) + bound) * 2.0 ** -8
    return bound


def route(x, k, score="softmax", bias=None, groups=1, keep=1, pair=False, renorm=True, scale=1.0):
    """ids, weights, offsets, rows, positions of logits x (float64)."""
    m, e = x.shape
    ids = np.full((m, k), -1, dtype=np.int64)
    w = np.zeros((m, k))
    for t in range(m):
        row = x[t]
        p = scores(row, score)
        c = p + (0 if bias is None else bias)
        broken = score == "softmax" and np.isnan(p).any()
        by = row if bias is None or broken else c
        shown = row if broken else c
        open_ = (row > -np.inf) & (by > -np.inf)
        pool = np.flatnonzero(open_)
        if groups > 1:
            size = e // groups
            rank = []
            for g in range(groups):
                mine = [i for i in pool if i // size == g]
                if pair:
                    best = sorted((shown[i] for i in mine), reverse=True)[:2]
                    rank.append(sum(best) if best else -np.inf)
                else:
                    rank.append(max((by[i] for i in mine), default=-np.inf))
            stay = sorted(range(groups), key=lambda g: (-rank[g], g))[:keep]
            pool = np.array([i for i in pool if i // size in stay], dtype=np.int64)
        best = sorted(pool, key=lambda i: (-by[i], i))[:k]
        ids[t, :len(best)] = best
        got = p[best]
        total = got.sum() + 1e-20
        w[t, :len(best)] = scale * got / total if renorm else scale * got
    flat = np.where(ids < 0, e, ids).reshape(-1)
    order = np.argsort(flat, kind="stable")
    offsets = np.searchsorted(flat[order], np.arange(e + 1))
    positions = np.empty(m * k, dtype=np.int64)
    positions[order] = np.arange(m * k)
    positions = np.where(flat == e, -2 - positions, positions).reshape(m, k)
    return ids, w, offsets, order // k, positions


def scores(row, score):
    if score == "sigmoid":
        with np.errstate(over="ignore"):
            return 1.0 / (1.0 + np.exp(-row))
    top = np.max(np.where(np.isnan(row), -np.inf, row))
    if top == -np.inf:
        return np.zeros_like(row)
    with np.errstate(invalid="ignore"):
        p = np.exp(row - top)
        return p / p.sum()


def weights_of(x, ids, score, renorm, scale):
    """The weights as a function of the logits for a fixed choice (for differences)."""
    w = np.zeros(ids.shape)
    for t in range(x.shape[0]):
        p = scores(x[t], score)
        ok = (ids[t] >= 0) & (ids[t] < x.shape[1])
        got = np.where(ok, p[np.where(ok, ids[t], 0)], 0.0)
        w[t] = scale * got / (got.sum() + 1e-20) if renorm else scale * got
    return w


def route_backward(dw, x, ids, score, renorm, scale):
    dx = np.zeros_like(x)
    for t in range(x.shape[0]):
        p = scores(x[t], score)
        dp = np.zeros(x.shape[1])
        ok = (ids[t] >= 0) & (ids[t] < x.shape[1])
        got, d = p[ids[t][ok]], dw[t][ok]
        if renorm:
            total = got.sum() + 1e-20
            d = scale / total * (d - (d * got).sum() / total)
        else:
            d = scale * d
        np.add.at(dp, ids[t][ok], d)
        dx[t] = p * (dp - (dp * p).sum()) if score == "softmax" else dp * p * (1 - p)
    return dx
