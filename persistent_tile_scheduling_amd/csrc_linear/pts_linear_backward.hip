// Host side of pts_linear_backward: argument checks, the choice of a kernel, the
// launches.
#include "linear/checks.h"
#include "linear/gradient.h"
#include "linear/plan.h"

namespace {

using namespace pts;

// Up to this many rows one workgroup of 64 rows at a time sums a strip of 128
// columns, and its sums are the result: a launch less.
constexpr int64_t ONE_BLOCK = 256;

// Rows of dy per workgroup of the column sums: some 2048 workgroups, and at most 256 row blocks.
int64_t block_rows(int64_t m, int64_t n)
{
    if (m <= ONE_BLOCK)
        return ONE_BLOCK;
    const int64_t strips = ceil_div(n, 128), blocks = std::max<int64_t>(1, std::min<int64_t>(256, 2048 / strips));
    return ceil_div(ceil_div(m, blocks), 16) * 16;
}

// Parts of the workspace, in bytes from its start.
struct Layout {
    int64_t sums, part_x, part_w, all; // dz is first
    Split dx, dw;
};
int64_t round16(int64_t v) { return (v + 15) / 16 * 16; }
Layout layout(int64_t m, int64_t n, int64_t k, int32_t activation)
{
    Layout l;
    l.dx = choose_split(m, k, n, 1, false);
    l.dw = choose_split(n, k, m, 1, false);
    l.sums = activation == PTS_ACTIVATION_NONE ? 0 : round16(m * own_pitch(n) * 2);
    l.part_x = l.sums + (m <= ONE_BLOCK ? 0 : round16(ceil_div(m, block_rows(m, n)) * n * 4));
    l.part_w = l.part_x + part_bytes(l.dx);
    l.all = l.part_w + part_bytes(l.dw);
    return l;
}

using TilesX = Tiles64<Bf16, ROWS, COLS>;
using TilesW = Tiles64<Bf16, COLS, COLS>;

} // namespace

extern "C" {

int64_t pts_linear_backward_workspace(int64_t m, int64_t n, int64_t k, int32_t activation)
{
    if (!extent(m) || !extent(n) || !extent(k) || !operand_width(n) || m == 0 || n == 0)
        return 0;
    return layout(m, n, k, activation).all;
}

gemm_status pts_linear_backward(const void *dy, int64_t ld_dy, const void *z, int64_t ldz, int32_t activation,
                                const void *x, int64_t ldx, const void *w, int64_t ldw, void *dx, int64_t ld_dx,
                                void *dw, int64_t ld_dw, int32_t dtype_dw, float *dbias, int64_t m, int64_t n,
                                int64_t k, void *workspace, size_t workspace_bytes, void *stream)
{
    if (dtype_dw != GEMM_DTYPE_F32 && dtype_dw != GEMM_DTYPE_BF16)
        return fail(GEMM_ERR_UNSUPPORTED, "dw must be fp32 or bf16");
    if (activation < PTS_ACTIVATION_NONE || activation > PTS_ACTIVATION_SILU)
        return fail(GEMM_ERR_INVALID_VALUE, "activation %d", activation);
    if (!extent(m) || !extent(n) || !extent(k))
        return fail(GEMM_ERR_INVALID_VALUE, "m, n and k must be in [0, 2^31 - 1024)");
    const bool act = activation != PTS_ACTIVATION_NONE;
    gemm_status st;
    if ((st = check_operand("dy", dy, ld_dy, m, n)) != GEMM_OK || (act && (st = check_operand("z", z, ldz, m, n)) != GEMM_OK) ||
        (dw != nullptr && (st = check_operand("x", x, ldx, m, k)) != GEMM_OK) ||
        (dx != nullptr && (st = check_operand("w", w, ldw, n, k)) != GEMM_OK) ||
        (dx != nullptr && (st = check_rows("dx", dx, ld_dx, m, k, 2)) != GEMM_OK) ||
        (dw != nullptr && (st = check_rows("dw", dw, ld_dw, n, k, dtype_dw == GEMM_DTYPE_F32 ? 4 : 2)) != GEMM_OK))
        return st;
    if (!aligned(dbias, 4))
        return fail(GEMM_ERR_INVALID_VALUE, "dbias must be element aligned");
    const int32_t dz_of = dx != nullptr || dw != nullptr ? activation : PTS_ACTIVATION_NONE; // the bias's gradient keeps no dz
    if ((st = check_workspace(workspace, workspace_bytes, pts_linear_backward_workspace(m, n, k, dz_of))) != GEMM_OK)
        return st;
    if (n == 0 && (dx == nullptr || m == 0 || k == 0))
        return GEMM_OK;

    const Layout l = layout(std::max<int64_t>(m, 1), std::max<int64_t>(n, 1), k, dz_of);
    if ((dx != nullptr && (st = check_launches(l.dx)) != GEMM_OK) || (dw != nullptr && (st = check_launches(l.dw)) != GEMM_OK))
        return st;
    if (ceil_div(n, 128) * ceil_div(std::max<int64_t>(m, 1), block_rows(m, std::max<int64_t>(n, 1))) > (int64_t)UINT32_MAX / 1024)
        return fail(GEMM_ERR_UNSUPPORTED, "n = %lld: too large a problem for one launch", (long long)n);
    uint8_t *const work = (uint8_t *)workspace;
    const uint16_t *dz = (const uint16_t *)dy;
    int64_t ld_dz = ld_dy;
    if (m > 0 && n > 0 && (act || dbias != nullptr)) {
        SlopeArgs s{};
        s.dy = (const uint16_t *)dy;
        s.z = (const uint16_t *)z;
        s.ld_dy = ld_dy;
        s.ldz = ldz;
        s.act = activation;
        if (act && (dx != nullptr || dw != nullptr)) {
            s.dz = (uint16_t *)work;
            s.ld_dz = ld_dz = own_pitch(n);
            dz = s.dz;
        }
        s.sums = dbias == nullptr ? nullptr : m <= ONE_BLOCK ? dbias : (float *)(work + l.sums);
        s.sums_ld = n;
        s.m = (int32_t)m;
        s.n = (int32_t)n;
        s.rows = (int32_t)block_rows(m, n);
        if (s.sums != nullptr || s.dz != nullptr) {
            st = m <= ONE_BLOCK ? launch_grid(&slope_kernel<64>, ceil_div(n, 128), 1, 1024, stream, s)
                                : launch_grid(&slope_kernel<16>, ceil_div(n, 128), ceil_div(m, s.rows), 256, stream, s);
            if (st != GEMM_OK)
                return st;
        }
    }
    if (dbias != nullptr && n > 0 && (m == 0 || m > ONE_BLOCK)) {
        SumArgs s{(const float *)(work + l.sums), dbias, n, (int32_t)n, m > 0 ? (int32_t)ceil_div(m, block_rows(m, n)) : 0};
        if ((st = launch_grid(&sum_kernel, ceil_div(n, 64), 1, 1024, stream, s)) != GEMM_OK)
            return st;
    }
    TileArgs to_x{}, to_w{};
    LinearArgs epi_x{}, epi_w{};
    to_x.a = to_w.a = dz;
    to_x.lda = to_w.lda = ld_dz;
    to_x.part = (float *)(work + l.part_x);
    to_w.part = (float *)(work + l.part_w);
    to_x.batch = to_w.batch = 1;
    to_x.n = to_w.n = (int32_t)k;
    to_x.b = (const uint16_t *)w;
    to_x.ldb = ldw;
    to_x.m = (int32_t)m;
    to_x.k = (int32_t)n;
    epi_x.d = dx;
    epi_x.ldd = ld_dx;
    epi_x.d_whole = whole_rows(dx, ld_dx, 2);
    to_w.b = (const uint16_t *)x;
    to_w.ldb = ldx;
    to_w.m = (int32_t)n;
    to_w.k = (int32_t)m;
    epi_w.d = dw;
    epi_w.ldd = ld_dw;
    epi_w.d_f32 = dtype_dw == GEMM_DTYPE_F32;
    epi_w.d_whole = whole_rows(dw, ld_dw, epi_w.d_f32 ? 4 : 2);
    // Small products, which do not fill the card by themselves, in one launch (2186 x 48 x 4935 29.3 us with two).
    if (dx != nullptr && dw != nullptr && m > 0 && n > 0 && k > 0 && l.dx.edge == 64 && l.dw.edge == 64) {
        int64_t grid_x, grid_w;
        if ((st = plan_tiles<TilesX>(to_x, l.dx, &grid_x)) != GEMM_OK || (st = plan_tiles<TilesW>(to_w, l.dw, &grid_w)) != GEMM_OK)
            return st;
        int blocks = (int)grid_x;
        if ((st = launch_grid(&tile_pair_kernel<TilesX, TilesW, PlainEpilogue>, grid_x + grid_w, 1, TilesX::THREADS, stream, to_x,
                              epi_x, to_w, epi_w, blocks)) != GEMM_OK ||
            (st = launch_join<TilesX, PlainEpilogue>(to_x, epi_x, l.dx, stream)) != GEMM_OK)
            return st;
        return launch_join<TilesW, PlainEpilogue>(to_w, epi_w, l.dw, stream);
    }
    if (dx != nullptr && (st = run_product<Bf16, ROWS, COLS, PlainEpilogue>(to_x, epi_x, l.dx, stream)) != GEMM_OK)
        return st;
    return dw == nullptr ? GEMM_OK : run_product<Bf16, COLS, COLS, PlainEpilogue>(to_w, epi_w, l.dw, stream);
}

} // extern "C"
