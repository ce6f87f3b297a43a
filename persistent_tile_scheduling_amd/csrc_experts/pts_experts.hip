// Host side of the C ABI declared in include/pts_experts.h: argument checks,
// the choice of a kernel, and the launches.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <atomic>

#include "host_error.h"
#include "pts_experts.h"

#include "experts/combine.h"
#include "experts/gemm_fp8.h"
#include "experts/quantize.h"
#include "experts/route.h"

namespace {

using pts::fail;
using pts::hip_fail;

static_assert(pts::QBLOCK == PTS_FP8_BLOCK && pts::ROUTE_MAX_EXPERTS == PTS_MOE_MAX_EXPERTS &&
                  pts::ROUTE_MAX_TOP == PTS_MOE_MAX_TOP && pts::ROUTE_MAX_GROUPS == PTS_MOE_MAX_GROUPS,
              "the header's limits are the kernels'");

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// Compute units of the current device, asked for once per device.
gemm_status compute_units(int *out)
{
    static std::atomic<int> known[64];
    int dev = 0;
    hipError_t e = hipGetDevice(&dev);
    if (e != hipSuccess)
        return hip_fail(e, "hipGetDevice");
    const bool keep = dev >= 0 && dev < 64;
    int cus = keep ? known[dev].load(std::memory_order_relaxed) : 0;
    if (cus == 0) {
        e = hipDeviceGetAttribute(&cus, hipDeviceAttributeMultiprocessorCount, dev);
        if (e != hipSuccess)
            return hip_fail(e, "querying the compute unit count");
        if (keep)
            known[dev].store(cus, std::memory_order_relaxed);
    }
    *out = cus;
    return GEMM_OK;
}

template <class Args> gemm_status launch(void (*kernel)(Args), dim3 grid, int threads, Args &args, void *stream)
{
    void *kargs[] = {&args};
    const hipError_t e = hipLaunchKernel((const void *)kernel, grid, dim3(threads), kargs, 0, (hipStream_t)stream);
    return e == hipSuccess ? GEMM_OK : hip_fail(e, "hipLaunchKernel");
}

// A one-dimensional grid; HIP limits it to 2^32 - 1 threads.
template <class Args> gemm_status launch_blocks(void (*kernel)(Args), int64_t blocks, int threads, Args &args, void *stream)
{
    if (blocks * threads > (int64_t)UINT32_MAX)
        return fail(GEMM_ERR_UNSUPPORTED, "%lld workgroups: too large a problem for one launch", (long long)blocks);
    return launch(kernel, dim3((uint32_t)blocks), threads, args, stream);
}

bool aligned(const void *p, size_t to) { return ((uintptr_t)p % to) == 0; }
constexpr int64_t MAX_EXTENT = INT32_MAX - 1024; // kernels round an extent up to whole tiles in 32 bits
bool in_range(int64_t v) { return v >= 0 && v <= INT32_MAX; }

// ---- products ------------------------------------------------------------------

// Tile rows of height bm: exact for one product; for experts the most there can
// be, since each expert with rows adds at most one partial tile.
int64_t tile_rows(const pts::Fp8Args &args, int64_t bm)
{
    if (args.offsets == nullptr)
        return ceil_div(args.m, bm);
    return (args.m + std::min<int64_t>(args.experts, args.m) * (bm - 1)) / bm;
}

// Few rows, 16-column tiles: two per workgroup where there are plenty, and
// fewer loads in flight per wave where several workgroups share a compute unit
// (measured at the kernel).
template <int MB, int U, bool ROWS, bool BF16> gemm_status launch_rows_kernel(pts::Fp8Args &args, int cus, void *stream)
{
    const int64_t tiles_m = tile_rows(args, 16 * MB);
    args.strip = tiles_m * ceil_div(args.n, 16) >= 16 * (int64_t)cus ? 2 : 1;
    args.tiles_n = (int32_t)ceil_div(args.n, 16 * args.strip);
    return launch_blocks(&pts::gemm_fp8_rows_kernel<MB, U, ROWS, BF16>, tiles_m * args.tiles_n, 512, args, stream);
}

template <int MB, bool ROWS, bool BF16> gemm_status launch_rows_typed(pts::Fp8Args &args, int cus, void *stream)
{
    if constexpr (MB == 1)
        if (tile_rows(args, 16) * ceil_div(args.n, 16) <= 2 * (int64_t)cus)
            return launch_rows_kernel<1, 4, ROWS, BF16>(args, cus, stream);
    return launch_rows_kernel<MB, 2, ROWS, BF16>(args, cus, stream);
}

template <int MB> gemm_status launch_rows(pts::Fp8Args &args, bool rows, bool bf16, int cus, void *stream)
{
    if (rows)
        return bf16 ? launch_rows_typed<MB, true, true>(args, cus, stream) : launch_rows_typed<MB, true, false>(args, cus, stream);
    return bf16 ? launch_rows_typed<MB, false, true>(args, cus, stream) : launch_rows_typed<MB, false, false>(args, cus, stream);
}

// Persistent workgroups, dealt to the dies in rounds of what is resident (an
// 8 x 4 block of tiles per die and round). Experts with smaller tiles than 256 x
// 256 have few tiles per weight: there each die gets one stretch of all tiles,
// so that an expert's weights pass through one die's L2, and a workgroup takes
// one tile, since the dies' shares differ (64 experts of 8 rows, 4096 x 4096: 179
// us against 211 in rounds, 64 rows 219 against 233; 256 x 256, 512 rows: 670
// against 662).
template <class C> gemm_status launch_tiles(pts::Fp8Args &args, int cus, void *stream)
{
    args.tiles_n = (int32_t)ceil_div(args.n, C::BN);
    const int64_t tiles = tile_rows(args, C::BM) * args.tiles_n;
    const int64_t resident = (int64_t)cus * (160 * 1024 / (C::STAGES * C::STAGE));
    const int64_t grid = args.offsets != nullptr && C::BM < 256 ? tiles : std::min(tiles, resident);
    args.round = (int32_t)grid;
    return launch_blocks(&pts::gemm_fp8_tile_kernel<C>, grid, C::THREADS, args, stream);
}

// The kernel of a product, by its output type, the rows that share a weight
// (`together`: all of them, or the experts' average) and the number of tiles.
// Times in us on MI355X, m x n x k.
//
// 256 x 256 tiles (bf16 results) once they reach 55% of the compute units:
// 2048 x 8192 x 8192 128 against 141 with 128 x 128; 2048 x 4096 x 4096 (half of
// the units) 41 with 128 x 128. Experts need more than 192 rows each (64
// experts, 4096 x 4096: 224 rows 389 against 425, 160 rows 334 with 128 x 128).
// With both operands scaled per row that kernel takes all 256 registers and keeps
// 24 bytes per lane in scratch; it still is the faster one but at ragged sizes
// (8192^3 515 against 608, 4096^3 70 against 80, 2048 x 8192 x 8192 132 against
// 152, 5000 x 7000 x 3000 150 against 142). The average is all that the host knows
// of the experts' loads: where a few have most of the rows, the tiles fit it and
// not them.
// For fp32 results, whose widened operands keep the vector units busy, 128 x 128
// is as good or better throughout (4096 x 8192 x 8192: 603 against 665 with 256 x
// 128): two independent workgroups per compute unit hide each other's waits.
//
// 64 x 128 tiles while 128 x 128 ones would not outnumber the compute units
// (1024 x 4096 x 4096, 256 tiles: 24 against 31; 768 x 8192 x 8192, 384 tiles: 64
// against 59), and for experts of up to 64 rows.
template <bool ROWS, bool BF16> gemm_status run_tiles(pts::Fp8Args &args, int64_t together, int cus, void *stream)
{
    if constexpr (BF16)
        if (together > 192 && 20 * tile_rows(args, 256) * ceil_div(args.n, 256) >= 11 * (int64_t)cus)
            return launch_tiles<pts::Fp8Config<256, 256, 2, 4, 2, ROWS, true>>(args, cus, stream);
    if (together > 64 && tile_rows(args, 128) * ceil_div(args.n, 128) > cus)
        return launch_tiles<pts::Fp8Config<128, 128, 2, 2, 2, ROWS, BF16>>(args, cus, stream);
    return launch_tiles<pts::Fp8Config<64, 128, 2, 2, 3, ROWS, BF16>>(args, cus, stream);
}

// The kernel without LDS up to 4 rows per expert (64 experts, 4096 x 4096, 2 rows
// each: 159 against 167 with 64 x 128 tiles, 8 rows 235 against 211); for one
// product up to 32 rows (32 x 4096 x 4096: 9.5 against 14.7), or 64 for fp32
// results (64 x 4096 x 4096: 14 against 29; 64 x 8192 x 8192: 44 against 53). With
// 64 rows and bf16 results the tiles lose 1.8 us of 14.9 at the first of these
// sizes and gain 17 of 43 at the second.
gemm_status run_product(pts::Fp8Args &args, bool rows, bool bf16, void *stream)
{
    int cus = 0;
    gemm_status st = compute_units(&cus);
    if (st != GEMM_OK)
        return st;
    const bool one = args.offsets == nullptr;
    const int64_t together = one ? args.m : ceil_div(args.m, args.experts);
    if (tile_rows(args, 16) * ceil_div(args.n, 16) > INT32_MAX)
        return fail(GEMM_ERR_UNSUPPORTED, "more than 2^31 output tiles");
    if (together <= (one ? 16 : 4))
        return launch_rows<1>(args, rows, bf16, cus, stream);
    if (one && together <= 32)
        return launch_rows<2>(args, rows, bf16, cus, stream);
    if (one && together <= 64 && !bf16)
        return rows ? launch_rows_kernel<4, 2, true, false>(args, cus, stream) : launch_rows_kernel<4, 2, false, false>(args, cus, stream);
    if (rows)
        return bf16 ? run_tiles<true, true>(args, together, cus, stream) : run_tiles<true, false>(args, together, cus, stream);
    return bf16 ? run_tiles<false, true>(args, together, cus, stream) : run_tiles<false, false>(args, together, cus, stream);
}

struct ScaleStrides {
    int64_t a_m, a_k, b_n, b_k;
};

gemm_status check_product(const void *a, int64_t a_rows, int64_t lda, const float *a_scale, const void *b, int64_t ldb,
                          const float *b_scale, const ScaleStrides &s, int32_t b_block_n, const void *d, int64_t ldd,
                          int32_t dtype_d, int64_t m, int64_t n, int64_t k, bool gathered)
{
    if (dtype_d != GEMM_DTYPE_F32 && dtype_d != GEMM_DTYPE_BF16)
        return fail(GEMM_ERR_UNSUPPORTED, "D must be fp32 or bf16");
    if (b_block_n != 1 && b_block_n != PTS_FP8_BLOCK)
        return fail(GEMM_ERR_UNSUPPORTED, "B's scales must be per row or per 128 x 128 block (b_block_n %d)", b_block_n);
    if (!in_range(m) || !in_range(n) || !in_range(k) || !in_range(a_rows))
        return fail(GEMM_ERR_INVALID_VALUE, "m, n, k and a_rows must be in [0, 2^31)");
    if (lda < k || ldb < k || ldd < n)
        return fail(GEMM_ERR_INVALID_VALUE, "leading dimension smaller than the packed extent");
    if (lda % 16 != 0 || ldb % 16 != 0)
        return fail(GEMM_ERR_INVALID_VALUE, "lda (%lld) and ldb (%lld) must be multiples of 16 elements", (long long)lda,
                    (long long)ldb);
    if (s.a_m < 0 || s.a_k < 0 || s.b_n < 0 || s.b_k < 0)
        return fail(GEMM_ERR_INVALID_VALUE, "scale strides must be >= 0");
    // offsets inside a tile, and from the first to the last k block's scales, are 32-bit byte offsets
    const int64_t limit = (int64_t)1 << 32, nk = ceil_div(k, PTS_FP8_BLOCK);
    const int64_t a_span = gathered ? a_rows : 256;
    auto spans = [&](int64_t rows, int64_t stride_row, int64_t stride_k) { // a scale's; each factor is below 2^31
        return stride_row >= limit / 4 || stride_k >= limit / 4 || rows * stride_row >= limit / 8 || nk * stride_k >= limit / 8;
    };
    if (lda >= limit / 512 || ldb >= limit / 512 || (gathered && a_span * lda + 128 > limit) || spans(a_span, s.a_m, s.a_k) ||
        spans(ceil_div(n, b_block_n), s.b_n, s.b_k))
        return fail(GEMM_ERR_UNSUPPORTED, "operand or scale strides too large for 32-bit tile offsets");
    if (std::max(m, n) > MAX_EXTENT)
        return fail(GEMM_ERR_UNSUPPORTED, "m and n must be below 2^31 - 1024");
    if (m == 0 || n == 0)
        return GEMM_OK;
    if (d == nullptr || (k > 0 && (a == nullptr || b == nullptr || a_scale == nullptr || b_scale == nullptr)))
        return fail(GEMM_ERR_INVALID_VALUE, "NULL operand pointer");
    if (k > 0 && (!aligned(a, 16) || !aligned(b, 16) || !aligned(a_scale, 4) || !aligned(b_scale, 4)))
        return fail(GEMM_ERR_INVALID_VALUE, "A and B must be 16-byte aligned, their scales 4-byte aligned");
    if (!aligned(d, dtype_d == GEMM_DTYPE_BF16 ? 2 : 4))
        return fail(GEMM_ERR_INVALID_VALUE, "D must be element aligned");
    return GEMM_OK;
}

// Rows that start at whole 16 bytes (1), at whole cache lines (2), anywhere (0).
int32_t vector_rows(const void *d, int64_t ldd, int32_t dtype)
{
    const int64_t pitch = ldd * (dtype == GEMM_DTYPE_BF16 ? 2 : 4);
    return !aligned(d, 16) || pitch % 16 != 0 ? 0 : !aligned(d, 128) || pitch % 128 != 0 ? 1 : 2;
}

// ---- routing -------------------------------------------------------------------

// Slots per workgroup of the order and the number of workgroups: at least 2048
// slots each, at most 256 workgroups (each adds up every chunk's counts).
void order_chunks(int64_t slots, int64_t *chunk, int64_t *chunks)
{
    *chunk = std::max<int64_t>(2048, ceil_div(ceil_div(slots, 256), 512) * 512);
    *chunks = ceil_div(slots, *chunk);
}

template <bool WIDE, bool GROUPED> gemm_status launch_route(pts::RouteArgs &args, int cus, void *stream)
{
    // 16 lanes per token once that gives every SIMD a wave (four tokens each)
    const bool many = args.m >= 16 * (int64_t)cus;
    const int e = args.experts;
    void (*k)(pts::RouteArgs);
    int tokens = 4;
    if (many && e <= 256) {
        tokens = 16;
        k = e <= 64    ? &pts::route_kernel<16, 4, WIDE, GROUPED>
            : e <= 128 ? &pts::route_kernel<16, 8, WIDE, GROUPED>
                       : &pts::route_kernel<16, 16, WIDE, GROUPED>;
    } else {
        k = e <= 256   ? &pts::route_kernel<64, 4, WIDE, GROUPED>
            : e <= 512 ? &pts::route_kernel<64, 8, WIDE, GROUPED>
                       : &pts::route_kernel<64, 16, WIDE, GROUPED>;
    }
    const int64_t blocks = args.fused ? 1 : ceil_div(args.m, tokens);
    return launch_blocks(k, blocks, 256, args, stream);
}

} // namespace

extern "C" {

gemm_status pts_quantize_fp8(const void *x, int32_t dtype_x, int32_t layout_x, int64_t m, int64_t k, int64_t ldx,
                             int32_t block_m, int32_t swiglu, void *q, int64_t ldq, float *scale,
                             int64_t scale_stride_m, int64_t scale_stride_k, void *stream)
{
    if (dtype_x != GEMM_DTYPE_BF16 && dtype_x != GEMM_DTYPE_F32)
        return fail(GEMM_ERR_UNSUPPORTED, "x must be bf16 or fp32");
    if (layout_x != GEMM_ROW_MAJOR && layout_x != GEMM_COL_MAJOR)
        return fail(GEMM_ERR_UNSUPPORTED, "x must be row-major or column-major");
    if (block_m != 1 && block_m != PTS_FP8_BLOCK)
        return fail(GEMM_ERR_UNSUPPORTED, "blocks are 1 x 128 or 128 x 128 (block_m %d)", block_m);
    const bool col = layout_x == GEMM_COL_MAJOR;
    if (swiglu && (col || block_m != 1))
        return fail(GEMM_ERR_UNSUPPORTED, "the gated form takes a row-major x and 1 x 128 blocks");
    if (m < 0 || k < 0 || m > MAX_EXTENT || k > MAX_EXTENT)
        return fail(GEMM_ERR_INVALID_VALUE, "m and k must be in [0, 2^31 - 1024)");
    if (ldx < (col ? m : swiglu ? 2 * k : k) || ldq < k)
        return fail(GEMM_ERR_INVALID_VALUE, "leading dimension smaller than the packed extent");
    if (ldq % 16 != 0)
        return fail(GEMM_ERR_INVALID_VALUE, "ldq (%lld) must be a multiple of 16", (long long)ldq);
    if (scale_stride_m < 1 || scale_stride_k < 1)
        return fail(GEMM_ERR_INVALID_VALUE, "scale strides must be >= 1");
    if (m == 0 || k == 0)
        return GEMM_OK;
    if (x == nullptr || q == nullptr || scale == nullptr)
        return fail(GEMM_ERR_INVALID_VALUE, "NULL pointer");
    const bool bf16 = dtype_x == GEMM_DTYPE_BF16;
    const int es = bf16 ? 2 : 4;
    if (!aligned(q, 16) || !aligned(x, es) || !aligned(scale, 4))
        return fail(GEMM_ERR_INVALID_VALUE, "q must be 16-byte aligned, x and scale element aligned");
    pts::QuantizeArgs args{x, (uint8_t *)q, scale, ldx, ldq, scale_stride_m, scale_stride_k, (int32_t)m, (int32_t)k, 0, 0};
    const bool vec = aligned(x, 16) && ldx * es % 16 == 0 && (!swiglu || k * es % 16 == 0);
    if (!col && block_m == 1) {
        int cus = 0;
        const gemm_status st = compute_units(&cus);
        if (st != GEMM_OK)
            return st;
        // 8 rows per workgroup, 4 (one per wave) while 8 would leave compute units idle
        const int64_t strips = ceil_div(k, 512);
        const int64_t per = ceil_div(m, 8) * strips < 4 * (int64_t)cus ? 4 : 8;
        args.rows_per_group = (int32_t)per;
        args.strips = (int32_t)strips;
        void (*kern)(pts::QuantizeArgs);
        if (bf16)
            kern = swiglu ? (vec ? &pts::quantize_rows_kernel<true, true, true> : &pts::quantize_rows_kernel<true, true, false>)
                          : (vec ? &pts::quantize_rows_kernel<true, false, true> : &pts::quantize_rows_kernel<true, false, false>);
        else
            kern = swiglu ? (vec ? &pts::quantize_rows_kernel<false, true, true> : &pts::quantize_rows_kernel<false, true, false>)
                          : (vec ? &pts::quantize_rows_kernel<false, false, true> : &pts::quantize_rows_kernel<false, false, false>);
        return launch_blocks(kern, strips * ceil_div(m, per), 256, args, stream);
    }
    args.strips = (int32_t)ceil_div(k, 128);
    void (*kern)(pts::QuantizeArgs);
#define PTS_TILE(COL, SQ)                                                                                              \
    (bf16 ? (vec ? &pts::quantize_tile_kernel<true, COL, SQ, true> : &pts::quantize_tile_kernel<true, COL, SQ, false>) \
          : (vec ? &pts::quantize_tile_kernel<false, COL, SQ, true> : &pts::quantize_tile_kernel<false, COL, SQ, false>))
    if (col)
        kern = block_m == 1 ? PTS_TILE(true, false) : PTS_TILE(true, true);
    else
        kern = PTS_TILE(false, true);
#undef PTS_TILE
    return launch_blocks(kern, args.strips * ceil_div(m, 128), 256, args, stream);
}

gemm_status pts_gemm_fp8(const void *a, int64_t lda, const float *a_scale, int64_t a_scale_stride_m,
                         int64_t a_scale_stride_k, const void *b, int64_t ldb, const float *b_scale,
                         int64_t b_scale_stride_n, int64_t b_scale_stride_k, int32_t b_block_n, void *d, int64_t ldd,
                         int32_t dtype_d, int64_t m, int64_t n, int64_t k, void *stream)
{
    const ScaleStrides s{a_scale_stride_m, a_scale_stride_k, b_scale_stride_n, b_scale_stride_k};
    const gemm_status st =
        check_product(a, m, lda, a_scale, b, ldb, b_scale, s, b_block_n, d, ldd, dtype_d, m, n, k, false);
    if (st != GEMM_OK || m == 0 || n == 0)
        return st;
    pts::Fp8Args args{(const uint8_t *)a, (const uint8_t *)b, a_scale, b_scale, d, nullptr, nullptr, lda, ldb, ldd,
                      s.a_m, s.a_k, s.b_n, s.b_k, 0, 0, (int32_t)m, (int32_t)n, (int32_t)k,
                      (int32_t)ceil_div(k, PTS_FP8_BLOCK), 0, 1, (int32_t)m, vector_rows(d, ldd, dtype_d), 1, 1};
    return run_product(args, b_block_n == 1, dtype_d == GEMM_DTYPE_BF16, stream);
}

gemm_status pts_gemm_fp8_experts(const void *a, int64_t a_rows, int64_t lda, const float *a_scale,
                                 int64_t a_scale_stride_m, int64_t a_scale_stride_k, const void *b, int64_t ldb,
                                 int64_t b_stride_expert, const float *b_scale, int64_t b_scale_stride_expert,
                                 int64_t b_scale_stride_n, int64_t b_scale_stride_k, int32_t experts,
                                 const int32_t *offsets, const int32_t *rows, void *d, int64_t ldd, int32_t dtype_d,
                                 int64_t m, int64_t n, int64_t k, void *stream)
{
    const ScaleStrides s{a_scale_stride_m, a_scale_stride_k, b_scale_stride_n, b_scale_stride_k};
    if (experts < 1 || experts > PTS_MOE_MAX_EXPERTS)
        return fail(GEMM_ERR_UNSUPPORTED, "experts must be in [1, %d] (got %d)", PTS_MOE_MAX_EXPERTS, experts);
    if (b_stride_expert < 0 || b_stride_expert % 16 != 0 || b_scale_stride_expert < 0)
        return fail(GEMM_ERR_INVALID_VALUE, "expert strides must be >= 0, B's a multiple of 16 elements");
    const gemm_status st = check_product(a, a_rows, lda, a_scale, b, ldb, b_scale, s, PTS_FP8_BLOCK, d, ldd, dtype_d, m,
                                         n, k, rows != nullptr);
    if (st != GEMM_OK || m == 0 || n == 0)
        return st;
    if (offsets == nullptr || !aligned(offsets, 4) || !aligned(rows, 4))
        return fail(GEMM_ERR_INVALID_VALUE, "offsets must be given, offsets and rows 4-byte aligned");
    if (a_rows < (rows == nullptr ? m : 1))
        return fail(GEMM_ERR_INVALID_VALUE, "A has %lld rows: too few", (long long)a_rows);
    pts::Fp8Args args{(const uint8_t *)a, (const uint8_t *)b, a_scale, b_scale, d, offsets, rows, lda, ldb, ldd,
                      s.a_m, s.a_k, s.b_n, s.b_k, b_stride_expert, b_scale_stride_expert, (int32_t)m, (int32_t)n,
                      (int32_t)k, (int32_t)ceil_div(k, PTS_FP8_BLOCK), 0, experts, (int32_t)a_rows,
                      vector_rows(d, ldd, dtype_d), 1, 1};
    return run_product(args, false, dtype_d == GEMM_DTYPE_BF16, stream);
}

int64_t pts_moe_route_workspace(int64_t m, int32_t experts, int32_t top)
{
    int64_t chunk, chunks;
    if (m <= 0 || experts <= 0 || top <= 0 || m > INT32_MAX / top)
        return 0; // nothing to order, or a call that is refused
    order_chunks(m * top, &chunk, &chunks);
    return chunks <= pts::ORDER_SELF_COUNTED ? 0 : chunks * (experts + 1) * (int64_t)sizeof(int32_t);
}

gemm_status pts_moe_route(const void *logits, int32_t dtype, int64_t ld, const float *bias, int64_t m, int32_t experts,
                          int32_t top, int32_t score, int32_t groups, int32_t topk_groups, int32_t group_top2,
                          int32_t renormalize, float scale, int32_t *ids, float *weights, int32_t *offsets,
                          int32_t *rows, int32_t *positions, void *workspace, size_t workspace_bytes, void *stream)
{
    if (dtype != GEMM_DTYPE_BF16 && dtype != GEMM_DTYPE_F32)
        return fail(GEMM_ERR_UNSUPPORTED, "logits must be bf16 or fp32");
    if (experts < 1 || experts > PTS_MOE_MAX_EXPERTS || top < 1 || top > PTS_MOE_MAX_TOP || top > experts)
        return fail(GEMM_ERR_UNSUPPORTED, "1 <= top <= min(experts, %d), experts <= %d (got %d of %d)", PTS_MOE_MAX_TOP,
                    PTS_MOE_MAX_EXPERTS, top, experts);
    if (score != PTS_SCORE_SOFTMAX && score != PTS_SCORE_SIGMOID)
        return fail(GEMM_ERR_INVALID_VALUE, "score must be softmax (0) or sigmoid (1)");
    if (groups < 1 || groups > PTS_MOE_MAX_GROUPS || experts % groups != 0 || topk_groups < 1 || topk_groups > groups)
        return fail(GEMM_ERR_INVALID_VALUE, "groups (%d) must divide experts and be <= %d, topk_groups (%d) <= groups",
                    groups, PTS_MOE_MAX_GROUPS, topk_groups);
    if (topk_groups * (experts / groups) < top)
        return fail(GEMM_ERR_INVALID_VALUE, "%d groups of %d experts hold fewer than top = %d", topk_groups,
                    experts / groups, top);
    if (m < 0 || m > INT32_MAX / top)
        return fail(GEMM_ERR_INVALID_VALUE, "m * top must be in [0, 2^31)");
    if (ld < experts)
        return fail(GEMM_ERR_INVALID_VALUE, "leading dimension smaller than the packed extent");
    if (offsets != nullptr && (m > 0 && (rows == nullptr || positions == nullptr)))
        return fail(GEMM_ERR_INVALID_VALUE, "the order needs offsets, rows and positions");
    const int64_t need = offsets == nullptr ? 0 : pts_moe_route_workspace(m, experts, top);
    if (need > 0 && (workspace == nullptr || (int64_t)workspace_bytes < need))
        return fail(GEMM_ERR_INVALID_VALUE, "workspace of %zu bytes; %lld needed", workspace_bytes, (long long)need);
    if (m > 0 && (logits == nullptr || ids == nullptr || weights == nullptr))
        return fail(GEMM_ERR_INVALID_VALUE, "NULL pointer");
    if (!aligned(logits, dtype == GEMM_DTYPE_BF16 ? 2 : 4) || !aligned(bias, 4) || !aligned(ids, 4) ||
        !aligned(weights, 4) || !aligned(offsets, 4) || !aligned(rows, 4) || !aligned(positions, 4) ||
        !aligned(workspace, 4))
        return fail(GEMM_ERR_INVALID_VALUE, "every pointer must be element aligned");
    if (m == 0 && offsets == nullptr)
        return GEMM_OK;
    int cus = 0;
    gemm_status st = compute_units(&cus);
    if (st != GEMM_OK)
        return st;
    int64_t chunk, chunks;
    order_chunks(std::max<int64_t>(m * top, 1), &chunk, &chunks);
    pts::RouteArgs args{logits, bias, ids, weights, offsets, rows, positions, (int32_t *)workspace, ld, (int32_t)m,
                        experts, top, groups, topk_groups, dtype == GEMM_DTYPE_BF16, score == PTS_SCORE_SIGMOID,
                        group_top2 != 0, renormalize != 0, 0, (int32_t)chunk, (int32_t)chunks, scale};
    // few tokens: one workgroup routes them all and orders their slots, one launch for both
    args.fused = offsets != nullptr && m <= 16 && m * top <= pts::ROUTE_FUSED_SLOTS;
    if (m > 0 || args.fused) {
        if (groups > 1)
            st = bias != nullptr ? launch_route<true, true>(args, cus, stream) : launch_route<false, true>(args, cus, stream);
        else
            st = bias != nullptr ? launch_route<true, false>(args, cus, stream) : launch_route<false, false>(args, cus, stream);
        if (st != GEMM_OK || offsets == nullptr || args.fused)
            return st;
    }
    if (chunks > pts::ORDER_SELF_COUNTED)
        st = launch(&pts::order_count_kernel, dim3((uint32_t)chunks), pts::ORDER_THREADS, args, stream);
    return st != GEMM_OK ? st
                         : launch(&pts::order_place_kernel, dim3((uint32_t)chunks), pts::ORDER_THREADS, args, stream);
}

gemm_status pts_moe_route_backward(const float *dweights, const void *logits, int32_t dtype, int64_t ld,
                                   const int32_t *ids, int64_t m, int32_t experts, int32_t top, int32_t score,
                                   int32_t renormalize, float scale, void *dlogits, int64_t ld_d, void *stream)
{
    if (dtype != GEMM_DTYPE_BF16 && dtype != GEMM_DTYPE_F32)
        return fail(GEMM_ERR_UNSUPPORTED, "logits must be bf16 or fp32");
    if (experts < 1 || experts > PTS_MOE_MAX_EXPERTS || top < 1 || top > PTS_MOE_MAX_TOP)
        return fail(GEMM_ERR_UNSUPPORTED, "1 <= top <= %d, 1 <= experts <= %d (got %d, %d)", PTS_MOE_MAX_TOP,
                    PTS_MOE_MAX_EXPERTS, top, experts);
    if (score != PTS_SCORE_SOFTMAX && score != PTS_SCORE_SIGMOID)
        return fail(GEMM_ERR_INVALID_VALUE, "score must be softmax (0) or sigmoid (1)");
    if (m < 0 || m > INT32_MAX / top)
        return fail(GEMM_ERR_INVALID_VALUE, "m * top must be in [0, 2^31)");
    if (ld < experts || ld_d < experts)
        return fail(GEMM_ERR_INVALID_VALUE, "leading dimension smaller than the packed extent");
    if (m == 0)
        return GEMM_OK;
    if (dweights == nullptr || logits == nullptr || ids == nullptr || dlogits == nullptr)
        return fail(GEMM_ERR_INVALID_VALUE, "NULL pointer");
    const size_t es = dtype == GEMM_DTYPE_BF16 ? 2 : 4;
    if (!aligned(dweights, 4) || !aligned(ids, 4) || !aligned(logits, es) || !aligned(dlogits, es))
        return fail(GEMM_ERR_INVALID_VALUE, "every pointer must be element aligned");
    int cus = 0;
    const gemm_status st = compute_units(&cus);
    if (st != GEMM_OK)
        return st;
    pts::RouteGradArgs args{logits, dweights, ids, dlogits, ld, ld_d, (int32_t)m, experts, top,
                            dtype == GEMM_DTYPE_BF16, score == PTS_SCORE_SIGMOID, renormalize != 0, scale};
    const bool many = m >= 16 * (int64_t)cus && experts <= 256;
    void (*k)(pts::RouteGradArgs);
    if (many)
        k = experts <= 64    ? &pts::route_backward_kernel<16, 4>
            : experts <= 128 ? &pts::route_backward_kernel<16, 8>
                             : &pts::route_backward_kernel<16, 16>;
    else
        k = experts <= 256   ? &pts::route_backward_kernel<64, 4>
            : experts <= 512 ? &pts::route_backward_kernel<64, 8>
                             : &pts::route_backward_kernel<64, 16>;
    return launch_blocks(k, ceil_div(m, many ? 16 : 4), 256, args, stream);
}

static gemm_status check_combine(int32_t dtype, int64_t ldy, int64_t rows, int64_t m, int64_t n, int32_t top,
                                 int64_t ld_out)
{
    if (dtype != GEMM_DTYPE_BF16 && dtype != GEMM_DTYPE_F32)
        return fail(GEMM_ERR_UNSUPPORTED, "y must be bf16 or fp32");
    if (top < 1 || top > PTS_MOE_MAX_TOP)
        return fail(GEMM_ERR_UNSUPPORTED, "1 <= top <= %d (got %d)", PTS_MOE_MAX_TOP, top);
    // one workgroup per token and 1024 or 2048 columns: the grid's limits
    if (m < 0 || m >= 1 << 24 || m * top > INT32_MAX || !in_range(rows) || n < 0 || n > (1 << 26) - 1024)
        return fail(GEMM_ERR_INVALID_VALUE, "m must be in [0, 2^24), rows and m * top in [0, 2^31), n in [0, 2^26 - 1024]");
    if (ldy < n || ld_out < n)
        return fail(GEMM_ERR_INVALID_VALUE, "leading dimension smaller than the packed extent");
    return GEMM_OK;
}

gemm_status pts_moe_combine(const void *y, int32_t dtype, int64_t ldy, int64_t rows, const float *weights,
                            const int32_t *positions, int64_t m, int64_t n, int32_t top, void *out, int64_t ld_out,
                            void *stream)
{
    const gemm_status st = check_combine(dtype, ldy, rows, m, n, top, ld_out);
    if (st != GEMM_OK || m == 0 || n == 0)
        return st;
    if ((y == nullptr && rows > 0) || weights == nullptr || positions == nullptr || out == nullptr)
        return fail(GEMM_ERR_INVALID_VALUE, "NULL pointer");
    const size_t es = dtype == GEMM_DTYPE_BF16 ? 2 : 4;
    if (!aligned(y, es) || !aligned(out, es) || !aligned(weights, 4) || !aligned(positions, 4))
        return fail(GEMM_ERR_INVALID_VALUE, "every pointer must be element aligned");
    pts::CombineArgs args{y, weights, positions, nullptr, out, nullptr, ldy, ld_out, 0, (int32_t)m, (int32_t)n, top,
                          (int32_t)rows, vector_rows(y, ldy, dtype) && vector_rows(out, ld_out, dtype)};
    const bool bf16 = dtype == GEMM_DTYPE_BF16;
    return launch(bf16 ? &pts::combine_kernel<true> : &pts::combine_kernel<false>,
                  dim3((uint32_t)m, (uint32_t)ceil_div(n, 256 * (bf16 ? 8 : 4))), 256, args, stream);
}

gemm_status pts_moe_combine_backward(const void *dout, int64_t ld_dout, const void *y, int32_t dtype, int64_t ldy,
                                     int64_t rows, const float *weights, const int32_t *positions, int64_t m,
                                     int64_t n, int32_t top, void *dy, int64_t ld_dy, float *dweights, void *stream)
{
    const gemm_status st = check_combine(dtype, ldy, rows, m, n, top, ld_dy);
    if (st != GEMM_OK)
        return st;
    if (ld_dout < n)
        return fail(GEMM_ERR_INVALID_VALUE, "leading dimension smaller than the packed extent");
    if (m == 0)
        return GEMM_OK;
    if (weights == nullptr || positions == nullptr || dweights == nullptr ||
        (n > 0 && (dout == nullptr || (rows > 0 && (y == nullptr || dy == nullptr)))))
        return fail(GEMM_ERR_INVALID_VALUE, "NULL pointer");
    const size_t es = dtype == GEMM_DTYPE_BF16 ? 2 : 4;
    if (!aligned(y, es) || !aligned(dy, es) || !aligned(dout, es) || !aligned(weights, 4) || !aligned(positions, 4) ||
        !aligned(dweights, 4))
        return fail(GEMM_ERR_INVALID_VALUE, "every pointer must be element aligned");
    pts::CombineArgs args{y, weights, positions, dout, dy, dweights, ldy, ld_dy, ld_dout, (int32_t)m, (int32_t)n, top,
                          (int32_t)rows, vector_rows(y, ldy, dtype) && vector_rows(dy, ld_dy, dtype) &&
                              vector_rows(dout, ld_dout, dtype)};
    return launch(dtype == GEMM_DTYPE_BF16 ? &pts::combine_backward_kernel<true> : &pts::combine_backward_kernel<false>,
                  dim3((uint32_t)m), 256, args, stream);
}

} // extern "C"
