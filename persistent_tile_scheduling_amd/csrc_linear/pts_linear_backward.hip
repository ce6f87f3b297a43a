// Host side of pts_linear_backward: argument checks, the choice of a kernel, the
// launches.
#include "linear/checks.h"
#include "linear/gradient.h"
#include "linear/plan.h"

namespace {

using namespace pts;

// Rows of dy per workgroup of the column sums: some 2048 workgroups, and at most 256 row blocks.
int64_t block_rows(int64_t m, int64_t n)
{
    const int64_t strips = ceil_div(n, 128), blocks = std::max<int64_t>(1, std::min<int64_t>(256, 2048 / strips));
    return ceil_div(ceil_div(m, blocks), 16) * 16;
}

// Parts of the workspace, in bytes from its start.
struct Layout {
    int64_t sums, part, all; // dz is first
    Split dx, dw;
};
int64_t round16(int64_t v) { return (v + 15) / 16 * 16; }
Layout layout(int64_t m, int64_t n, int64_t k, int32_t activation)
{
    Layout l;
    l.dx = choose_split(m, k, n, 1, false);
    l.dw = choose_split(n, k, m, 1, false);
    l.sums = activation == PTS_ACTIVATION_NONE ? 0 : round16(m * pitch8(n) * 2);
    l.part = l.sums + round16(ceil_div(m, block_rows(m, n)) * n * 4);
    l.all = l.part + std::max(part_bytes(l.dx), part_bytes(l.dw));
    return l;
}

} // namespace

extern "C" {

int64_t pts_linear_backward_workspace(int64_t m, int64_t n, int64_t k, int32_t activation)
{
    if (!extent(m) || !extent(n) || !extent(k) || m == 0 || n == 0)
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
    if ((st = check_workspace(workspace, workspace_bytes, pts_linear_backward_workspace(m, n, k, activation))) != GEMM_OK)
        return st;
    if (n == 0 && (dx == nullptr || m == 0 || k == 0))
        return GEMM_OK;

    const Layout l = layout(std::max<int64_t>(m, 1), std::max<int64_t>(n, 1), k, activation);
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
            s.ld_dz = ld_dz = pitch8(n);
            dz = s.dz;
        }
        s.sums = dbias != nullptr ? (float *)(work + l.sums) : nullptr;
        s.sums_ld = n;
        s.m = (int32_t)m;
        s.n = (int32_t)n;
        s.rows = (int32_t)block_rows(m, n);
        if (s.sums != nullptr || s.dz != nullptr)
            if ((st = launch_grid(&slope_kernel, ceil_div(n, 128), ceil_div(m, s.rows), 256, stream, s)) != GEMM_OK)
                return st;
    }
    if (dbias != nullptr && n > 0) {
        SumArgs s{(const float *)(work + l.sums), dbias, n, (int32_t)n, m > 0 ? (int32_t)ceil_div(m, block_rows(m, n)) : 0};
        if ((st = launch_grid(&sum_kernel, ceil_div(n, 64), 1, 1024, stream, s)) != GEMM_OK)
            return st;
    }
    TileArgs args{};
    args.a = dz;
    args.lda = ld_dz;
    args.part = (float *)(work + l.part);
    args.batch = 1;
    args.n = (int32_t)k;
    LinearArgs epi{};
    if (dx != nullptr) {
        args.b = (const uint16_t *)w;
        args.ldb = ldw;
        args.m = (int32_t)m;
        args.k = (int32_t)n;
        epi.d = dx;
        epi.ldd = ld_dx;
        epi.d_whole = whole_rows(dx, ld_dx, 2);
        if ((st = run_product<Bf16, ROWS, COLS, PlainEpilogue>(args, epi, l.dx, stream)) != GEMM_OK)
            return st;
    }
    if (dw != nullptr) {
        args.b = (const uint16_t *)x;
        args.ldb = ldx;
        args.m = (int32_t)n;
        args.k = (int32_t)m;
        epi.d = dw;
        epi.ldd = ld_dw;
        epi.d_f32 = dtype_dw == GEMM_DTYPE_F32;
        epi.d_whole = whole_rows(dw, ld_dw, epi.d_f32 ? 4 : 2);
        return run_product<Bf16, COLS, COLS, PlainEpilogue>(args, epi, l.dw, stream);
    }
    return GEMM_OK;
}

} // extern "C"
