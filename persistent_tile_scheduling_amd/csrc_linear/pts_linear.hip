// Host side of pts_linear: argument checks, the choice of a kernel, the launches.
#include "linear/checks.h"
#include "linear/epilogue.h"
#include "linear/plan.h"
#include "linear/rows.h"

namespace {

using namespace pts;

// Up to 32 rows go without LDS (rows_kernel). A compute unit has some 130 cache
// lines on their way to it, 20 GB/s from memory, so what counts is that all of
// them load: a narrow layer's long rows are split over the workgroups, as far as
// one pass of a workgroup's waves covers a share (24 x 1000 x 8192: 16.2 us in 2
// shares, 11.9 in 8, launches in a row from a graph; 1 x 1000 x 8192 14.6 in one,
// 8.7 in 4).
//
// One row block: strips of 16 columns, sixteen waves (1 x 4096 x 4096 9.3 against
// 10.0 with eight, 8192 x 8192 28.0 against 31.2), eight where they are split; and
// strips of 32 where there are many and the rows are short (1 x 8192 x 1024 6.0
// against 8.9; 8192 x 8192 29.4). The border, in calls with weights from memory,
// 32 against 16: one row of n = 4112 to 14336 at k = 1024 7.3 to 8.7 us against 8.1
// to 14.3, at 1536 level, at 2048 3 to 10% slower, from 4096 on 3 to 36% slower;
// twelve rows at 2048 2 to 7% faster, at 4096 and beyond 12% faster to 2% slower.
// Two row blocks: strips of 32, which halve the loads of x (32 x 8192 x 8192: 37
// against 51 with 16). With 48 rows the tiles are level or better (48 x 4096 x 4096
// 15.7 against 18.0).
constexpr int64_t FEW_ROWS = 32;

struct RowsPlan {
    int wide, waves, ahead; // columns of a strip, waves, k blocks (of 64) a wave loads at once
    int splits, per;        // workgroups that share a strip, and k blocks for each
};
RowsPlan plan_rows(int64_t m, int64_t n, int64_t k)
{
    const int64_t nk = std::max<int64_t>(ceil_div(k, 64), 1);
    RowsPlan p{32, 8, 2, 1, (int)nk};
    if (m <= 16 && !(ceil_div(n, 16) > UNITS && nk <= 32))
        p = ceil_div(n, 16) <= UNITS / 2 ? RowsPlan{16, 8, 4, 1, (int)nk} : RowsPlan{16, 16, 2, 1, (int)nk};
    const int64_t strips = ceil_div(n, p.wide);
    const int64_t splits = std::max<int64_t>(1, std::min(UNITS / strips, ceil_div(nk, p.waves * p.ahead)));
    p.per = (int)ceil_div(nk, splits);
    p.splits = (int)ceil_div(nk, p.per);
    return p;
}

template <int MB, int NB, int U, int WAVES>
gemm_status launch_rows(TileArgs &args, LinearArgs &epi, const RowsPlan &p, void *stream)
{
    args.splits = p.splits;
    args.split_k = p.per;
    const gemm_status st = launch_grid(&rows_kernel<MB, NB, U, WAVES, LinearEpilogue>, ceil_div(args.n, 16 * NB), p.splits, 64 * WAVES,
                                       stream, args, epi);
    if (st != GEMM_OK || p.splits == 1)
        return st;
    return launch_grid(&rows_join_kernel<LinearEpilogue>, ceil_div((int64_t)args.m * ((args.n + 7) / 8), 256), 1, 256, stream, args, epi);
}

gemm_status run_rows(TileArgs &args, LinearArgs &epi, void *stream)
{
    const RowsPlan p = plan_rows(args.m, args.n, args.k);
    if (args.m > 16)
        return launch_rows<2, 2, 2, 8>(args, epi, p, stream);
    if (p.wide == 32)
        return launch_rows<1, 2, 2, 8>(args, epi, p, stream);
    return p.waves == 16 ? launch_rows<1, 1, 2, 16>(args, epi, p, stream) : launch_rows<1, 1, 4, 8>(args, epi, p, stream);
}

} // namespace

extern "C" {

int64_t pts_linear_workspace(int64_t m, int64_t n, int64_t k)
{
    if (!extent(m) || !extent(n) || !extent(k) || !operand_width(k) || m == 0 || n == 0)
        return 0;
    if (m <= FEW_ROWS) {
        const RowsPlan p = plan_rows(m, n, k); // strips that no launch holds are not split
        return p.splits == 1 ? 0 : p.splits * m * rows_pitch(n) * (int64_t)sizeof(float);
    }
    const Split s = choose_split(m, n, k, 1, false);
    return launchable(s) ? part_bytes(s) : 0;
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
    if (m <= FEW_ROWS)
        return run_rows(args, epi, stream);
    return run_product<Bf16, ROWS, ROWS, LinearEpilogue>(args, epi, choose_split(m, n, k, 1, false), stream);
}

} // extern "C"
