// Host side of pts_linear: argument checks, the choice of a kernel, the launches.
#include "linear/checks.h"
#include "linear/epilogue.h"
#include "linear/plan.h"
#include "linear/rows.h"

namespace {

using namespace pts;

// Up to 32 rows go without LDS (rows_kernel).
constexpr int64_t FEW_ROWS = 32;

// Its split: a workgroup has 16 columns; a narrow layer's long rows are shared by more.
struct RowsSplit {
    int splits, per;
};
RowsSplit split_rows(int64_t n, int64_t k)
{
    const int64_t nk = std::max<int64_t>(ceil_div(k, 64), 1), strips = ceil_div(n, 16);
    const int64_t splits = std::max<int64_t>(1, std::min(UNITS / 2 / strips, nk / 64));
    RowsSplit s{1, (int)ceil_div(nk, splits)};
    s.splits = (int)ceil_div(nk, s.per);
    return s;
}

template <int MB, int U> gemm_status run_rows(TileArgs &args, LinearArgs &epi, void *stream)
{
    const RowsSplit s = split_rows(args.n, args.k);
    args.splits = s.splits;
    args.split_k = s.per;
    const gemm_status st = launch_grid(&rows_kernel<MB, U, LinearEpilogue>, ceil_div(args.n, 16), s.splits, 512, stream, args, epi);
    if (st != GEMM_OK || s.splits == 1)
        return st;
    return launch_grid(&rows_join_kernel<LinearEpilogue>, ceil_div((int64_t)args.m * ((args.n + 7) / 8), 256), 1, 256, stream, args, epi);
}

} // namespace

extern "C" {

int64_t pts_linear_workspace(int64_t m, int64_t n, int64_t k)
{
    if (!extent(m) || !extent(n) || !extent(k) || m == 0 || n == 0)
        return 0;
    if (m <= FEW_ROWS) {
        const RowsSplit s = split_rows(n, k);
        return s.splits == 1 ? 0 : s.splits * m * rows_pitch(n) * (int64_t)sizeof(float);
    }
    return part_bytes(choose_split(m, n, k, 1, false));
}

gemm_status pts_linear(const void *x, int64_t ldx, const void *w, int64_t ldw, const void *bias, int32_t dtype_bias,
                       int32_t activation, const void *residual, int64_t ldr, void *y, int64_t ldy, int32_t dtype_y,
                       void *z_out, int64_t ldz, int64_t m, int64_t n, int64_t k, void *workspace,
                       size_t workspace_bytes, void *stream)
{
    if ((dtype_y != GEMM_DTYPE_F32 && dtype_y != GEMM_DTYPE_BF16) ||
        (bias != nullptr && dtype_bias != GEMM_DTYPE_F32 && dtype_bias != GEMM_DTYPE_BF16))
        return fail(GEMM_ERR_UNSUPPORTED, "y and bias must be fp32 or bf16");
    if (activation < PTS_ACTIVATION_NONE || activation > PTS_ACTIVATION_SILU)
        return fail(GEMM_ERR_INVALID_VALUE, "activation %d", activation);
    if (!extent(m) || !extent(n) || !extent(k))
        return fail(GEMM_ERR_INVALID_VALUE, "m, n and k must be in [0, 2^31 - 1024)");
    const int size = dtype_y == GEMM_DTYPE_F32 ? 4 : 2;
    gemm_status st;
    if ((st = check_operand("x", x, ldx, m, k)) != GEMM_OK || (st = check_operand("w", w, ldw, n, k)) != GEMM_OK ||
        (st = check_rows("y", y, ldy, m, n, size)) != GEMM_OK ||
        (residual != nullptr && (st = check_rows("residual", residual, ldr, m, n, size)) != GEMM_OK) ||
        (z_out != nullptr && (st = check_rows("z_out", z_out, ldz, m, n, 2)) != GEMM_OK))
        return st;
    if (!aligned(bias, dtype_bias == GEMM_DTYPE_F32 ? 4 : 2))
        return fail(GEMM_ERR_INVALID_VALUE, "bias must be element aligned");
    if ((st = check_workspace(workspace, workspace_bytes, pts_linear_workspace(m, n, k))) != GEMM_OK)
        return st;
    if (m == 0 || n == 0)
        return GEMM_OK;
    TileArgs args{};
    args.a = (const uint16_t *)x;
    args.b = (const uint16_t *)w;
    args.lda = ldx;
    args.ldb = ldw;
    args.part = (float *)workspace;
    args.m = (int32_t)m;
    args.n = (int32_t)n;
    args.k = (int32_t)k;
    args.batch = 1;
    LinearArgs epi{};
    epi.d = y;
    epi.bias = bias;
    epi.residual = residual;
    epi.z = (uint16_t *)z_out;
    epi.ldd = ldy;
    epi.ldr = ldr;
    epi.ldz = ldz;
    epi.d_f32 = dtype_y == GEMM_DTYPE_F32;
    epi.bias_f32 = dtype_bias == GEMM_DTYPE_F32;
    epi.act = activation;
    epi.d_whole = whole_rows(y, ldy, size);
    epi.r_whole = residual != nullptr && whole_rows(residual, ldr, size);
    epi.z_whole = z_out != nullptr && whole_rows(z_out, ldz, 2);
    if (m <= 16)
        return run_rows<1, 4>(args, epi, stream);
    if (m <= FEW_ROWS)
        return run_rows<2, 4>(args, epi, stream);
    return run_product<Bf16, ROWS, ROWS, LinearEpilogue>(args, epi, choose_split(m, n, k, 1, false), stream);
}

} // extern "C"
