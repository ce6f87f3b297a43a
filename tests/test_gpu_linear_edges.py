"""The linear layer's operators where they can go wrong: epilogues of every kind of tile, strides, masks of the edges,
infinities, offsets past 32 bits, streams, graphs, and a layer's training step run together."""
from __future__ import annotations

import pytest
import torch

from tests import linear_reference as R

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF16, F32 = torch.bfloat16, torch.float32
NAN = float("nan")


@pytest.fixture(scope="module")
def pts():
    import persistent_tile_scheduling_amd as mod
    return mod


def padded(m, n, seed, dtype=BF16, scale=1.0):
    """An m x n matrix whose rows start at whole 16 bytes and are followed by NaN."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    t = torch.full((m, 8 * ((n + 7) // 8)), NAN, device=DEV, dtype=dtype)
    t[:, :n] = (torch.randn((m, n), generator=g, device=DEV) * scale).to(dtype)
    return t[:, :n]


def island(m, n, dtype, ld, offset):
    """An m x n result inside a buffer of NaN, and the buffer."""
    buf = torch.full((m + 2, ld), NAN, device=DEV, dtype=dtype)
    return buf[1:m + 1, offset:offset + n], buf


# One size for each kernel: few rows (one and two row blocks, split), tiles of 64, 128 and 256, and split ones.
KINDS = [(1, 300, 520), (3, 40, 4200), (30, 200, 1100), (40, 90, 72), (100, 70, 2200), (700, 2100, 200), (1030, 1030, 2100),
         (4000, 4200, 130)]


@pytest.mark.parametrize("act", R.ACTIVATIONS)
@pytest.mark.parametrize("m,n,k", KINDS)
def test_epilogue(pts, m, n, k, act):
    x, w = padded(m, k, 1), padded(n, k, 2, scale=1.5 * k ** -0.5)
    bias = padded(1, n, 3)[0]
    for out_dtype, b in ((BF16, bias), (F32, bias.float())):
        residual = padded(m, n, 4, dtype=out_dtype)
        y, z = pts.linear(x, w, b, activation=act, residual=residual, out_dtype=out_dtype, preactivation=True)
        want_y, want_z, bound_y, bound_z = R.linear(x, w, b, act, residual)
        R.check(y, want_y, bound_y, f"{out_dtype} y")
        R.check(z, want_z, bound_z, f"{out_dtype} z")


@pytest.mark.parametrize("act", R.ACTIVATIONS)
@pytest.mark.parametrize("m,n,k", [(1, 300, 520), (40, 90, 72), (300, 70, 2200), (700, 2100, 200), (257, 1030, 2100),
                                   (4000, 130, 4200)])
def test_gradients(pts, m, n, k, act):
    dy, x, w = padded(m, n, 1), padded(m, k, 2), padded(n, k, 3)
    z = None if act is None else padded(m, n, 4, scale=1.5)
    dx, dw, db, bound_dx, bound_dw, bound_db = R.gradients(dy, x, w, z, act)
    for dtype in (BF16, F32):
        got = pts.linear_backward(dy, x, w, z, activation=act, dw_dtype=dtype)
        R.check(got.dx, dx, bound_dx, "dx")
        R.check(got.dw, dw, bound_dw, "dw")
        R.check(got.dbias, db, bound_db, "dbias")
    for need in ((True, False, False), (False, True, False), (False, False, True), (False, False, False)):
        part = pts.linear_backward(dy, x, w, z, activation=act, need_dx=need[0], need_dw=need[1], need_dbias=need[2])
        for one, whole, wanted in zip(part, pts.linear_backward(dy, x, w, z, activation=act), need):
            assert (one is None) != wanted and (not wanted or torch.equal(one, whole))


@pytest.mark.parametrize("act", ["gelu", "gelu_tanh", "silu"])
def test_bias_gradient_by_differences(pts, act):
    """x = 0, so that z is the bias, exact in bf16. y is good to 2^-20 |y|, |y| < 4, and the second difference's rest is
    below h^2 / 6 of a third derivative below 3: for 40 rows of |dy| <= 1."""
    m, n, h = 40, 500, 2.0 ** -5
    dy = padded(m, n, 1).clamp_(-1, 1)
    x, w = torch.zeros((m, 8), device=DEV, dtype=BF16), torch.zeros((n, 8), device=DEV, dtype=BF16)
    bias = torch.linspace(-3.5, 3.5, n, device=DEV).bfloat16()
    z = padded(m, n, 2).copy_(bias.expand(m, n))
    db = pts.linear_backward(dy, x, w, z, activation=act, need_dx=False, need_dw=False).dbias
    y = [pts.linear(x, w, bias.float() + s * h, activation=act, out_dtype=F32).double() for s in (1, -1)]
    by_difference = (dy.double() * (y[0] - y[1]) / (2 * h)).sum(0)
    assert (db.double() - by_difference).abs().max() <= m * (h * h / 6 * 3 + 2 * 4 * 2.0 ** -20 / (2 * h))


@pytest.mark.parametrize("m,n,k", KINDS)
@pytest.mark.parametrize("offset,extra", [(0, 8), (8, 16), (3, 5)])
def test_results_leave_their_surroundings(pts, m, n, k, offset, extra):
    """Rows that start anywhere; nothing outside them is written; the result may be the residual itself."""
    x, w = padded(m, k, 1), padded(n, k, 2, scale=k ** -0.5)
    for dtype in (BF16, F32):
        ld = offset + n + extra
        out, buf = island(m, n, dtype, ld, offset)
        r = padded(m, n, 3, dtype=dtype)
        out.copy_(r)
        assert pts.linear(x, w, residual=out, out=out) is out
        assert torch.equal(out, pts.linear(x, w, residual=r, out_dtype=dtype))
        outside = torch.ones_like(buf, dtype=torch.bool)
        outside[1:m + 1, offset:offset + n] = False
        assert torch.isnan(buf[outside]).all()


@pytest.mark.parametrize("m,n,k", KINDS)
def test_rows_with_infinities_keep_to_themselves(pts, m, n, k):
    x, w = padded(m, k, 1), padded(n, k, 2)
    base = pts.linear(x, w, out_dtype=F32)
    row, col = m // 2, n // 2
    x[row, k - 1] = float("inf")
    w[col, 0] = NAN
    y = pts.linear(x, w, out_dtype=F32)
    fine = torch.ones_like(y, dtype=torch.bool)
    fine[row] = fine[:, col] = False
    assert torch.equal(y[fine], base[fine]) and not torch.isfinite(y[row]).any() and torch.isnan(y[:, col]).all()


def test_infinite_preactivations(pts):
    inf = float("inf")
    one = torch.zeros((1, 8), device=DEV, dtype=BF16)
    for act, at_inf, at_minus in (("relu", inf, 0.0), ("gelu", inf, 0.0), ("gelu_tanh", inf, None), ("silu", inf, None)):
        y = pts.linear(one[:, :1], one.expand(3, 8).contiguous()[:, :1], torch.tensor([inf, -inf, NAN], device=DEV), act, out_dtype=F32)[0]
        assert y[0] == at_inf and torch.isnan(y[2]) and (at_minus is None or y[1] == at_minus), (act, y)


def test_same_call_same_bits(pts):
    for m, n, k in KINDS:
        x, w, dy = padded(m, k, 1), padded(n, k, 2), padded(m, n, 3)
        first = (pts.linear(x, w), *pts.linear_backward(dy, x, w))
        for _ in range(3):
            assert all(torch.equal(a, b) for a, b in zip(first, (pts.linear(x, w), *pts.linear_backward(dy, x, w))))


# 4.9 GB operands and results: offsets past 32 bits in each place an index is multiplied by a row's length.
LONG, WIDE = 300_000, 8192


def test_long_operands(pts):
    g = torch.Generator(device=DEV).manual_seed(1)
    big = torch.randint(-2, 3, (LONG, WIDE), generator=g, device=DEV, dtype=torch.int8).to(BF16)
    small = torch.randint(-2, 3, (24, WIDE), generator=g, device=DEV).to(BF16)
    rows = torch.cat([torch.arange(0, LONG, 997, device=DEV), torch.arange(LONG - 300, LONG, device=DEV)])
    y = pts.linear(big, small, out_dtype=F32)                       # x is long
    assert torch.equal(y[rows], big[rows].float() @ small.float().t())
    y = pts.linear(small, big, out_dtype=F32)                       # w is long, few rows
    assert torch.equal(y[:, rows], small.float() @ big[rows].float().t())
    many = torch.randint(-2, 3, (70, WIDE), generator=g, device=DEV).to(BF16)
    y = pts.linear(many, big, out_dtype=F32)                        # w is long, tiles
    assert torch.equal(y[:, rows], many.float() @ big[rows].float().t())
    thin = torch.randint(-1, 2, (LONG, 16), generator=g, device=DEV).to(BF16)
    narrow = torch.randint(-1, 2, (WIDE, 16), generator=g, device=DEV).to(BF16)
    got = pts.linear_backward(big, thin, narrow, dw_dtype=F32)      # dy is long, its rows are summed over
    assert torch.equal(got.dbias.double(), big.double().sum(0))
    assert torch.equal(got.dx[rows].float(), (big[rows].float() @ narrow.float()).bfloat16().float())
    want = torch.zeros((WIDE, 16), device=DEV, dtype=torch.float64)
    for lo in range(0, LONG, 30_000):
        want += big[lo:lo + 30_000].double().t() @ thin[lo:lo + 30_000].double()
    assert torch.equal(got.dw.double(), want)
    del got, want
    # y, its residual and the preactivation are long
    r = torch.randint(-3, 4, (LONG, WIDE), generator=g, device=DEV, dtype=torch.int8).to(BF16)
    y, z = pts.linear(thin, narrow, activation="relu", residual=r, preactivation=True)
    want = thin[rows].float() @ narrow.float().t()
    assert torch.equal(z[rows].float(), want) and torch.equal(y[rows].float(), want.clamp(min=0) + r[rows].float())
    del y
    # with an activation dz is long too
    got = pts.linear_backward(big, thin, narrow, z, activation="relu", dw_dtype=F32)
    dz = torch.where(z[rows] > 0, big[rows], 0.0)
    assert torch.equal(got.dx[rows].float(), (dz.float() @ narrow.float()).bfloat16().float())
    assert torch.equal(got.dbias.double(), torch.where(z > 0, big, 0.0).double().sum(0))


def test_other_streams(pts):
    m, n, k = 600, 700, 2000
    sets = [(padded(m, k, s), padded(n, k, s + 1), padded(m, n, s + 2)) for s in (1, 11)]
    want = [(pts.linear(x, w, activation="silu"), *pts.linear_backward(dy, x, w)) for x, w, dy in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    got = [[] for _ in sets]
    for _ in range(10):
        for i, (stream, (x, w, dy)) in enumerate(zip(streams, sets)):
            with torch.cuda.stream(stream):
                got[i].append((pts.linear(x, w, activation="silu"), *pts.linear_backward(dy, x, w)))
    torch.cuda.synchronize()
    for i in range(len(sets)):
        assert all(torch.equal(a, b) for r in got[i] for a, b in zip(r, want[i]))


def test_two_graphs_replayed(pts):
    """Each captures a layer's forward and backward pass and its update; replays follow new inputs, eager work between."""
    m, n, k = 500, 260, 2300
    graphs = []
    for s in (1, 21):
        x, w, dy = padded(m, k, s), padded(n, k, s + 1, scale=k ** -0.5), padded(m, n, s + 2)

        def step(x=x, w=w, dy=dy):
            y, z = pts.linear(x, w, activation="gelu", preactivation=True)
            grads = pts.linear_backward(dy, x, w, z, activation="gelu")
            return (y, z, *grads, pts.orthogonalize(grads.dw), pts.orthogonalize(grads.dw[:50]))
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            step()
        torch.cuda.current_stream().wait_stream(side)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = step()
        graphs.append((graph, out, step, (x, w, dy)))
    for again in range(4):
        for i, (graph, out, step, inputs) in enumerate(graphs):
            for j, t in enumerate(inputs):
                t.copy_(padded(*t.shape, 100 * again + 10 * i + j, scale=k ** -0.5 if j == 1 else 1.0))
        for graph, *_ in graphs:
            graph.replay()
        torch.cuda.synchronize()
        for graph, out, step, _ in graphs:
            assert all(torch.equal(a, b) for a, b in zip(out, step()))


def test_a_feed_forward_block_learns_together(pts):
    """Two layers, a residual, their gradients, and the orthogonalised updates of both weights: every result against the
    64-bit formula on the values that the calls before it gave."""
    tokens, hidden, inner = 333, 200, 520
    x = padded(tokens, hidden, 1)
    w1, w2 = padded(inner, hidden, 2, scale=hidden ** -0.5), padded(hidden, inner, 3, scale=inner ** -0.5)
    b1, b2 = torch.randn(inner, device=DEV) * 0.1, torch.randn(hidden, device=DEV) * 0.1
    h, z = pts.linear(x, w1, b1, activation="gelu", preactivation=True)
    y = pts.linear(h, w2, b2, residual=x)
    dy = padded(tokens, hidden, 4)
    dh, dw2, db2 = pts.linear_backward(dy, h, w2)
    dx, dw1, db1 = pts.linear_backward(dh, x, w1, z, activation="gelu")
    dx = dx + dy

    want, _, bound, _ = R.linear(h, w2, b2, None, x)
    R.check(y, want, bound, "y")
    g = R.gradients(dy, h, w2)
    for got, want, bound in zip((dh, dw2, db2), g[:3], g[3:]):
        R.check(got, want, bound)
    g = R.gradients(dh, x, w1, z, "gelu")
    R.check(dw1, g[1], g[4], "dw1")
    R.check(db1, g[2], g[5], "db1")
    # The same gradient of x by one 64-bit pass through the block: h, z, dh and dx are each rounded to bf16 once.
    zz = x.double() @ w1.double().t() + b1.double()
    dz = (dy.double() @ w2.double()) * R.slope(zz, "gelu")
    whole = dz @ w1.double() + dy.double()
    assert (dx.double() - whole).norm() <= 6 * R.HALF[BF16] * whole.norm()
    for w, dw in ((w1, dw1), (w2, dw2)):
        update = pts.orthogonalize(dw)
        exact = R.orthogonalize(dw)
        assert (update.double() - exact).norm() <= 2e-2 * exact.norm()
        s = torch.linalg.svdvals(update.double())
        assert 0.5 < s.median() < 1.3
        w.sub_((0.02 * update.float()).bfloat16())
    assert torch.isfinite(pts.linear(x, w1, b1, activation="gelu")).all()
