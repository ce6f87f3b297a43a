// Host side of pts_orthogonalize: argument checks and the chain of launches.
#include "linear/ortho.h"
#include "linear/ortho_small.h"

#include <cmath>

#include "linear/checks.h"

namespace {

using namespace pts;

// Parts of the workspace, in bytes from its start, and the products' splits.
struct Layout {
    int64_t scale, gram, poly, half[2], rest, part, all; // the squares' sums are first
    int64_t ldx, lds;                                      // pitches of rows x cols and side x side matrices
    int32_t blocks;
    Split gram_split, square_split, update_split;
};
int64_t round16(int64_t v) { return (v + 15) / 16 * 16; }
Layout layout(int64_t count, int64_t rows, int64_t cols)
{
    const int64_t side = std::min(rows, cols), lng = std::max(rows, cols);
    Layout l;
    l.ldx = own_pitch(cols);
    l.lds = own_pitch(side);
    l.gram_split = choose_split(side, side, lng, count, true);
    l.square_split = choose_split(side, side, side, count, true);
    l.update_split = choose_split(rows, cols, side, count, false);
    l.blocks = (int32_t)std::min<int64_t>(256, ceil_div(rows * ceil_div(cols, 8), 1024));
    l.scale = count * l.blocks * 8;
    l.gram = round16(l.scale + count * 8);
    l.poly = l.gram + count * side * l.lds * 2;
    l.half[0] = l.poly + count * side * l.lds * 2;
    l.half[1] = l.half[0] + count * rows * l.ldx * 2;
    l.rest = l.half[1] + count * rows * l.ldx * 2;
    l.part = l.rest + round16(count * rows * l.ldx);
    l.all = l.part + std::max({part_bytes(l.gram_split), part_bytes(l.square_split), part_bytes(l.update_split)});
    return l;
}

// The same for short sides of up to 64: the squares' sums, the chunks' Gram matrices, a chain's polynomials, and, since
// the coefficients decide how many chains the steps take, X between them.
constexpr int32_t CHAIN = 16; // the most steps of a chain
struct SmallLayout {
    int64_t parts, polys, mid, all;
    int32_t blocks, chunks, chunk;
};
SmallLayout small_layout(int64_t count, int64_t rows, int64_t cols, int64_t steps)
{
    const int64_t lng = std::max(rows, cols);
    SmallLayout l;
    l.blocks = (int32_t)std::min<int64_t>(32, ceil_div(rows * ceil_div(cols, 8), 1024));
    l.chunk = (int32_t)(ceil_div(ceil_div(lng, 64), 32) * 64); // at most 32 chunks: one workgroup adds them up
    l.chunks = (int32_t)ceil_div(lng, l.chunk);
    l.parts = round16(count * l.blocks * 8);
    l.polys = l.parts + count * l.chunks * small_blocks((int)std::min(rows, cols)) * 256 * 8;
    l.mid = l.polys + count * std::min<int64_t>(steps, CHAIN) * SMALL_MATRIX * 4;
    l.all = l.mid + (steps > 1 ? round16(count * rows * cols * 4) : 0);
    return l;
}

bool sizes(int64_t count, int64_t rows, int64_t cols)
{
    // the workspace's bytes and every product of the extents stay in 64 bits
    return extent(count) && extent(rows) && extent(cols) && (count == 0 || rows == 0 || cols == 0 || rows * cols <= (INT64_C(1) << 48) / count);
}
bool widths(int64_t rows, int64_t cols) { return cols <= MAX_PITCH - 64 && std::min(rows, cols) <= MAX_PITCH - 64; }
bool small_launchable(int64_t count, int64_t rows, int64_t cols)
{
    return ceil_div(std::max(rows, cols), 64) * count <= (int64_t)UINT32_MAX / 256;
}

// The largest |c0 + c1 t + c2 t^2| on [0, top].
double most(double c0, double c1, double c2, double top)
{
    auto value = [&](double t) { return std::fabs(c0 + t * (c1 + t * c2)); };
    const double t = c2 != 0.0 ? -c1 / (2.0 * c2) : 0.0;
    return std::max({value(0.0), value(top), t > 0.0 && t < top ? value(t) : 0.0});
}

// The largest |a s + b s^3 + c s^5| on [0, top]: at its end or where a + 3 b t + 5 c t^2 = 0, t = s^2.
double reach(double a, double b, double c, double top)
{
    auto p = [&](double s) { return std::fabs(s * (a + s * s * (b + s * s * c))); };
    double most = p(top);
    auto at = [&](double t) {
        if (t > 0.0 && t < top * top)
            most = std::max(most, p(std::sqrt(t)));
    };
    if (c != 0.0) {
        const double d = 9.0 * b * b - 20.0 * a * c;
        if (d >= 0.0) {
            at((-3.0 * b + std::sqrt(d)) / (10.0 * c));
            at((-3.0 * b - std::sqrt(d)) / (10.0 * c));
        }
    } else if (b != 0.0) {
        at(-a / (3.0 * b));
    }
    return most;
}

// A bound on X's singular values after a step from [0, top], its roundings counted: those of X as an operand, of A and of
// B, half a step of eps each, come into X' = a X + B X with |B|, with |dB/dA| |A| three times (A is made from two rounded
// X), and with |B| again. Without them a polynomial that maps [0, top] onto itself but grows beyond would be taken for one
// that stays (5 s - 20 s^3 + 16 s^5 comes to NaN from six steps on in fp16).
constexpr double EPS_F16 = 0x1p-11, EPS_F32 = 0x1p-20; // of fp32 some steps: its sums' too
double bound(double a, double b, double c, double top, double eps)
{
    const double t = top * top;
    return std::max(reach(a, b, c, top) + eps * top * (2.0 * most(0.0, b, c, t) + 3.0 * t * most(b, 2.0 * c, 0.0, t)), 1e-30);
}

// How many of `steps` steps one chain may take (at least one), X's singular values being in [0, top]; top then has the
// bound after them.
//
// A step takes an eigenvalue t = s^2 of A to f(t) = t q(t)^2, q(t) = a + b t + c t^2, so an error of A grows by at most
// the largest |f'| = |q p'|, and comes into X' by the largest |q'| times top: it starts as 2^-50 of A (the rounding of
// its sums in 64 bits) and is kept below 2^-14 of the result, a sixtieth of its rounding to bf16. X's own rounding in
// fp32 grows by at most the largest |q|, and the chain does not see it: its square is missing in A. It starts as 2^-22
// (some steps of fp32) and is kept below 2^-6 of X, so that 2^-12 is missing. By the default coefficients the latter
// ends a chain, after eight steps with 2^-7.
int32_t chain_steps(double a, double b, double c, double &top, int32_t steps)
{
    double error = 0.0, noise = 0.0;
    for (int32_t i = 0;; ++i) {
        const double t = top * top, next = bound(a, b, c, top, EPS_F32);
        const double q = most(a, b, c, t);
        error += 0x1p-50 * t;
        noise = (noise + 0x1p-22 * top) * q;
        if (i > 0 && (i == std::min(steps, CHAIN) || !(error * most(b, 2.0 * c, 0.0, t) * top <= 0x1p-14 * next) || !(noise <= 0x1p-6 * next)))
            return i;
        error *= q * most(a, 3.0 * b, 5.0 * c, t);
        top = next;
    }
}

gemm_status run_small(NormArgs &norm, uint8_t *work, void *out, int64_t ldo, int64_t o_batch, int64_t count, int32_t steps, float a,
                      float b, float c, void *stream)
{
    const SmallLayout l = small_layout(count, norm.rows, norm.cols, steps);
    norm.blocks = l.blocks;
    SmallArgs args{};
    args.norm = norm;
    args.parts = (double *)(work + l.parts);
    args.polys = (float *)(work + l.polys);
    args.out = (uint16_t *)out;
    args.ldo = ldo;
    args.o_batch = o_batch;
    args.a = a;
    args.b = b;
    args.c = c;
    args.tall = norm.rows > norm.cols;
    args.side = std::min(norm.rows, norm.cols);
    args.lng = std::max(norm.rows, norm.cols);
    args.chunks = l.chunks;
    args.chunk = l.chunk;
    gemm_status st;
    if ((st = launch_grid(&norm_kernel, l.blocks, count, 256, stream, norm)) != GEMM_OK)
        return st;
    double top = 1.0;
    for (int32_t left = steps; left > 0; left -= args.steps) {
        args.steps = chain_steps(a, b, c, top, left);
        args.mid = args.steps < left ? (float *)(work + l.mid) : nullptr;
        if ((st = launch_grid(&small_gram_kernel, l.chunks, count, 1024, stream, args)) != GEMM_OK ||
            (st = launch_grid(&small_chain_kernel, count, 1, 64 * small_blocks(args.side), stream, args)) != GEMM_OK ||
            (st = launch_grid(&small_update_kernel, ceil_div(args.lng, 64), count, 256, stream, args)) != GEMM_OK)
            return st;
        args.norm.x = args.mid;
        args.norm.ldx = norm.cols;
        args.norm.x_batch = (int64_t)norm.rows * norm.cols;
        args.norm.f32 = 1;
        args.scaled = 1;
    }
    return GEMM_OK;
}

} // namespace

extern "C" {

int64_t pts_orthogonalize_workspace(int64_t count, int64_t rows, int64_t cols, int32_t steps)
{
    if (!sizes(count, rows, cols) || !widths(rows, cols) || count > 65535 || count == 0 || rows == 0 || cols == 0 || steps < 1 || steps > 64)
        return 0;
    if (std::min(rows, cols) <= SMALL)
        return small_launchable(count, rows, cols) ? small_layout(count, rows, cols, steps).all : 0;
    const Layout l = layout(count, rows, cols);
    return launchable(l.gram_split) && launchable(l.square_split) && launchable(l.update_split) ? l.all : 0;
}

gemm_status pts_orthogonalize(const void *x, int32_t dtype_x, int64_t ldx, int64_t x_stride, int64_t count,
                              int64_t rows, int64_t cols, int32_t steps, float a, float b, float c, double eps,
                              void *out, int64_t ld_out, int64_t out_stride, void *workspace, size_t workspace_bytes,
                              void *stream)
{
    if (dtype_x != GEMM_DTYPE_F32 && dtype_x != GEMM_DTYPE_BF16)
        return fail(GEMM_ERR_UNSUPPORTED, "x must be fp32 or bf16");
    if (!sizes(count, rows, cols))
        return fail(GEMM_ERR_INVALID_VALUE, "count, rows and cols must be in [0, 2^31 - 1024), count * rows * cols at most 2^48");
    if (count > 65535)
        return fail(GEMM_ERR_UNSUPPORTED, "%lld matrices; at most 65535", (long long)count);
    if (!widths(rows, cols))
        return fail(GEMM_ERR_UNSUPPORTED, "a tile's offsets must fit in 32-bit: at most 2^22 - 64 columns");
    if (steps < 1 || steps > 64)
        return fail(GEMM_ERR_INVALID_VALUE, "steps must be in [1, 64], not %d", steps);
    if (!(eps > 0.0))
        return fail(GEMM_ERR_INVALID_VALUE, "eps must be above 0");
    double top = 1.0;
    for (int i = 0; i < steps; ++i) {
        const double poly = most(0.0, b, c, top * top), next = bound(a, b, c, top, std::min(rows, cols) <= SMALL ? EPS_F32 : EPS_F16);
        if (!(poly <= 128.0) || !(next <= 8.0))
            return fail(GEMM_ERR_INVALID_VALUE, "the coefficients take singular values to %g in step %d: beyond fp16's reach",
                        next, i + 1);
        top = next;
    }
    const int size = dtype_x == GEMM_DTYPE_F32 ? 4 : 2;
    if (x_stride < 0 || out_stride < 0 || (count > 1 && (x_stride > INT64_MAX / 16 / count || out_stride > INT64_MAX / 16 / count)))
        return fail(GEMM_ERR_INVALID_VALUE, "bad strides of the stack");
    gemm_status st;
    if ((st = check_rows("x", x, ldx, rows * (count > 0), cols, size)) != GEMM_OK ||
        (st = check_rows("out", out, ld_out, rows * (count > 0), cols, 2)) != GEMM_OK)
        return st;
    if (count > 1 && rows > 0 && cols > 0 && out_stride < (rows - 1) * ld_out + cols &&
        (out_stride < cols || ld_out < (count - 1) * out_stride + cols))
        return fail(GEMM_ERR_INVALID_VALUE, "out's matrices overlap (stride %lld)", (long long)out_stride);
    if ((st = check_workspace(workspace, workspace_bytes, pts_orthogonalize_workspace(count, rows, cols, steps))) != GEMM_OK)
        return st;
    if (count == 0 || rows == 0 || cols == 0)
        return GEMM_OK;
    const bool small = std::min(rows, cols) <= SMALL;
    if (small && !small_launchable(count, rows, cols))
        return fail(GEMM_ERR_UNSUPPORTED, "%lld x %lld x %lld: too large a problem for one launch", (long long)count, (long long)rows,
                    (long long)cols);

    NormArgs norm{};
    norm.x = x;
    norm.sums = (double *)workspace;
    norm.ldx = ldx;
    norm.x_batch = x_stride;
    norm.eps = eps;
    norm.rows = (int32_t)rows;
    norm.cols = (int32_t)cols;
    norm.f32 = dtype_x == GEMM_DTYPE_F32;
    norm.whole = whole_rows(x, ldx, size) && x_stride * size % 16 == 0;
    if (small)
        return run_small(norm, (uint8_t *)workspace, out, ld_out, out_stride, count, steps, a, b, c, stream);
    const Layout l = layout(count, rows, cols);
    for (const Split *s : {&l.gram_split, &l.square_split, &l.update_split})
        if ((st = check_launches(*s)) != GEMM_OK)
            return st;
    uint8_t *const work = (uint8_t *)workspace;
    uint16_t *const gram = (uint16_t *)(work + l.gram), *const poly = (uint16_t *)(work + l.poly);
    uint16_t *const half[2] = {(uint16_t *)(work + l.half[0]), (uint16_t *)(work + l.half[1])};
    uint8_t *const rest = work + l.rest;
    const bool tall = rows > cols;
    const int64_t side = std::min(rows, cols), lng = std::max(rows, cols);

    norm.scale = (double *)(work + l.scale);
    norm.half = half[0];
    norm.ldh = l.ldx;
    norm.h_batch = rows * l.ldx;
    norm.blocks = l.blocks;
    if ((st = launch_grid(&norm_kernel, l.blocks, count, 256, stream, norm)) != GEMM_OK ||
        (st = launch_grid(&start_kernel, std::min<int64_t>(ceil_div(rows * ceil_div(cols, 8), 1024), std::max<int64_t>(1, 65536 / count)), count, 256, stream, norm)) != GEMM_OK)
        return st;

    for (int i = 0; i < steps; ++i) {
        uint16_t *const now = half[i & 1], *const next = half[(i & 1) ^ 1];
        TileArgs args{};
        args.part = (float *)(work + l.part);
        args.batch = (int32_t)count;
        // A = X X^T or X^T X
        args.a = args.b = now;
        args.lda = args.ldb = l.ldx;
        args.a_batch = args.b_batch = rows * l.ldx;
        args.m = args.n = (int32_t)side;
        args.k = (int32_t)lng;
        args.symmetric = 1;
        OrthoArgs epi{};
        epi.half = gram;
        epi.ldh = l.lds;
        epi.h_batch = side * l.lds;
        epi.alpha = 1.f / (ORTHO_SX * ORTHO_SX);
        epi.half_scale = ORTHO_SA;
        st = tall ? run_product<F16, COLS, COLS, OrthoEpilogue>(args, epi, l.gram_split, stream)
                  : run_product<F16, ROWS, ROWS, OrthoEpilogue>(args, epi, l.gram_split, stream);
        if (st != GEMM_OK)
            return st;
        // B = b A + c A A
        args.a = args.b = gram;
        args.lda = args.ldb = l.lds;
        args.a_batch = args.b_batch = side * l.lds;
        args.k = (int32_t)side;
        epi.half = poly;
        epi.alpha = c / (ORTHO_SA * ORTHO_SA);
        epi.beta = b / ORTHO_SA;
        epi.r = gram;
        epi.r_type = R_F16;
        epi.ldr = l.lds;
        epi.r_batch = side * l.lds;
        if ((st = run_product<F16, ROWS, ROWS, OrthoEpilogue>(args, epi, l.square_split, stream)) != GEMM_OK)
            return st;
        // X' = a X + B X or a X + X B (B = B^T)
        args.a = tall ? now : poly;
        args.b = tall ? poly : now;
        args.lda = tall ? l.ldx : l.lds;
        args.ldb = tall ? l.lds : l.ldx;
        args.a_batch = tall ? rows * l.ldx : side * l.lds;
        args.b_batch = tall ? side * l.lds : rows * l.ldx;
        args.m = (int32_t)rows;
        args.n = (int32_t)cols;
        args.symmetric = 0;
        epi = OrthoArgs{};
        epi.alpha = 1.f / (ORTHO_SA * ORTHO_SX);
        if (i == 0) {
            epi.beta = a;
            epi.r = x;
            epi.r_scale = norm.scale;
            epi.r_type = norm.f32 ? R_F32 : R_BF16;
            epi.ldr = ldx;
            epi.r_batch = x_stride;
            epi.r_whole = norm.whole;
        } else {
            epi.beta = a / ORTHO_SX;
            epi.r = now;
            epi.r_rest = i + 1 < steps ? rest : nullptr;
            epi.r_type = R_F16;
            epi.ldr = l.ldx;
            epi.r_batch = rows * l.ldx;
        }
        if (i + 1 < steps) {
            epi.half = next;
            epi.ldh = l.ldx;
            epi.h_batch = rows * l.ldx;
            epi.half_scale = ORTHO_SX;
            epi.rest = i + 2 < steps ? rest : nullptr;
        } else {
            epi.out = (uint16_t *)out;
            epi.ldo = ld_out;
            epi.o_batch = out_stride;
            epi.o_whole = whole_rows(out, ld_out, 2) && out_stride % 8 == 0;
        }
        st = tall ? run_product<F16, ROWS, ROWS, OrthoEpilogue>(args, epi, l.update_split, stream)
                  : run_product<F16, ROWS, COLS, OrthoEpilogue>(args, epi, l.update_split, stream);
        if (st != GEMM_OK)
            return st;
    }
    return GEMM_OK;
}

} // extern "C"
