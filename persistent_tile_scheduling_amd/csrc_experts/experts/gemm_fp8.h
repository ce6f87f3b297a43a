// Products of e4m3 matrices with an fp32 scale per block of 128:
//
//   D[i][j] = sum_b sa[i][b] sb[j or j / 128][b] sum_{k in block b} A[i][k] B[k][j]
//
// one dense product, or one per expert over rows ordered by expert. The inner
// sum of a block starts from zero in the matrix unit; the outer sum is an fp32
// multiply-add of its result by the block's scale. The blocks are summed in
// ascending order, one accumulator per output, or with few rows one for every
// eighth block, added up in a fixed order: a result does not depend on timing.
//
// On MI355X, by the clock that the card holds: 8192^3 to bf16 430 to 480 us, 2290
// to 2560 TFLOP/s. The matrix unit is busy about 64% of the cycles; each of its
// 32-cycle instructions is followed by four multiply-adds (the scales), and the
// power limit holds the clock at 1.7 to 2.0 of 2.4 GHz, so that cycles saved
// elsewhere come back as a lower clock. 5000 x 7000 x 3000 to fp32, both operands
// scaled per row: 227 to 259 us, 810 to 925 TFLOP/s, bound by the vector
// instructions (two widenings and over two scalings per 16-cycle matrix
// instruction).
#pragma once

#include "device/common.h"
#include "device/scheduler.h"

namespace pts {

typedef int32_t i32x4 __attribute__((ext_vector_type(4)));
typedef int32_t i32x8 __attribute__((ext_vector_type(8)));

struct Fp8Args {
    const uint8_t *a, *b;
    const float *sa, *sb;
    void *d;
    const int32_t *offsets; // experts + 1 row offsets, or null: one dense product
    const int32_t *rows;    // row of A of each row of D, or null: the same row
    int64_t lda, ldb, ldd;  // elements
    int64_t sa_m, sa_k, sb_n, sb_k; // element strides of the scales
    int64_t b_expert, sb_expert;    // element strides from one expert's B to the next
    int32_t m, n, k, nk;
    int32_t tiles_n, experts, a_rows;
    int32_t d_vec; // D's rows start at whole 16 bytes (1), at whole cache lines (2)
    int32_t strip; // few rows: 16-column tiles per workgroup
    int32_t round; // tiles: the width of the dealing to the dies
};

// One row's share of a k block in a lane: lane l has, of row l % 16, the two
// 16-byte chunks l / 16 and l / 16 + 4 (which chunk is which k does not matter
// as long as both operands agree), as e4m3 or widened to bf16.
//
// The matrix unit sums e4m3 products in groups of 8 consecutive k: within a
// group, what lies 14 or more binary places below the largest product's
// exponent is dropped before the fp32 addition (found by adding a single small
// product to a large one; the same for the 16 x 16 x 32 form). On normal data
// that is 1.4e-5 of the result, far below bf16's 2^-8, but not fp32. So bf16
// results are computed from e4m3 products, one v_mfma_f32_16x16x128_f8f6f4 per
// 16 x 16 outputs and k block, at twice bf16's rate; and fp32 results (EXACT)
// from the same codes widened to bf16, whose products the unit sums in fp32,
// four v_mfma_f32_16x16x32_bf16 per block.
template <bool EXACT> struct Fragment;
template <> struct Fragment<false> {
    i32x8 v;
    __device__ __forceinline__ void set(i32x4 lo, i32x4 hi) { v = __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7); }
};
template <> struct Fragment<true> {
    bf16x8 v[4];
    __device__ __forceinline__ void set(i32x4 lo, i32x4 hi)
    {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const i32x4 src = i < 2 ? lo : hi;
#pragma unroll
            for (int w = 0; w < 2; ++w) {
                const uint32_t word = (uint32_t)src[(i & 1) * 2 + w];
                const bf16x2 x = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(word, 1.0f, false);
                const bf16x2 y = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(word, 1.0f, true);
                v[i][4 * w] = x[0];
                v[i][4 * w + 1] = x[1];
                v[i][4 * w + 2] = y[0];
                v[i][4 * w + 3] = y[1];
            }
        }
    }
};

// The sums of one k block for 16 rows of X against 16 rows of Y: lane l gets
// rows 4 (l / 16) .. + 3 of X against row l % 16 of Y.
__device__ __forceinline__ f32x4 block_sums(const Fragment<false> &x, const Fragment<false> &y)
{
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(x.v, y.v, f32x4{0.f, 0.f, 0.f, 0.f}, 0, 0, 0, 0, 0, 0);
}
__device__ __forceinline__ f32x4 block_sums(const Fragment<true> &x, const Fragment<true> &y)
{
    f32x4 c = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int i = 0; i < 4; ++i)
        c = __builtin_amdgcn_mfma_f32_16x16x32_bf16(x.v[i], y.v[i], c, 0, 0, 0);
    return c;
}

// One output tile: rows [row0, row0 + vm) of D and columns [col0, col0 + vn).
struct Fp8Tile {
    int expert, row0, vm, col0, vn;
};

// Position inside one problem: groups of 8 tile rows walked column by column,
// so that 32 consecutive positions (one die's share of a round) are an 8 x 4
// block whose operands its L2 holds.
__device__ __forceinline__ void fp8_raster(int local, int tiles_m, int tiles_n, int &tm, int &tn)
{
    const int first = local / (8 * tiles_n) * 8;
    const int in = local - first * tiles_n;
    const int rows = min(8, tiles_m - first);
    tm = first + in % rows;
    tn = in / rows;
}

// The tile at position t: the expert is found by a scan of the experts' tile
// counts, 64 at a time, one per lane. Offsets are clamped into [0, m] and an
// expert's end to its start, so a bad table cannot lead outside the operands.
// Returns false past the last tile.
__device__ __forceinline__ bool fp8_find_tile(const Fp8Args &args, int bm, int bn, int t, Fp8Tile &tile)
{
    if (args.offsets == nullptr) {
        const int tiles_m = (args.m + bm - 1) / bm;
        if (t >= tiles_m * args.tiles_n)
            return false;
        int tm, tn;
        fp8_raster(t, tiles_m, args.tiles_n, tm, tn);
        tile.expert = 0;
        tile.row0 = tm * bm;
        tile.vm = min(bm, args.m - tile.row0);
        tile.col0 = tn * bn;
        tile.vn = min(bn, args.n - tile.col0);
        return true;
    }
    const int lane = threadIdx.x & 63;
    int before = 0;
    for (int e0 = 0; e0 < args.experts; e0 += 64) {
        const int e = e0 + lane;
        int lo = 0, hi = 0;
        if (e < args.experts) {
            lo = min(max(args.offsets[e], 0), args.m);
            hi = min(max(args.offsets[e + 1], lo), args.m);
        }
        const int tiles = (hi - lo + bm - 1) / bm * args.tiles_n;
        int sum = tiles;
#pragma unroll
        for (int d = 1; d < 64; d *= 2) {
            const int v = __shfl_up(sum, d);
            if (lane >= d)
                sum += v;
        }
        const uint64_t past = __ballot(before + sum > t);
        if (past != 0) {
            const int src = __builtin_ctzll(past);
            const int begin = __builtin_amdgcn_readlane(sum - tiles, src) + before;
            const int elo = __builtin_amdgcn_readlane(lo, src), ehi = __builtin_amdgcn_readlane(hi, src);
            int tm, tn;
            fp8_raster(t - begin, (ehi - elo + bm - 1) / bm, args.tiles_n, tm, tn);
            tile.expert = e0 + src;
            tile.row0 = elo + tm * bm;
            tile.vm = min(bm, ehi - tile.row0);
            tile.col0 = tn * bn;
            tile.vn = min(bn, args.n - tile.col0);
            // a table whose ranges overlap can have more tiles than an int counts: nothing beyond this expert's rows
            return tile.row0 >= elo && tile.vm > 0 && tile.col0 >= 0 && tile.vn > 0;
        }
        before += __builtin_amdgcn_readlane(sum, 63);
    }
    return false;
}

// Upper bound of fp8_find_tile's positions is not known on the host for
// experts: a worker needs the total to deal positions to the dies.
__device__ __forceinline__ int fp8_total_tiles(const Fp8Args &args, int bm)
{
    if (args.offsets == nullptr)
        return (args.m + bm - 1) / bm * args.tiles_n;
    const int lane = threadIdx.x & 63;
    int tiles = 0;
    for (int e = lane; e < args.experts; e += 64) {
        const int lo = min(max(args.offsets[e], 0), args.m);
        const int hi = min(max(args.offsets[e + 1], lo), args.m);
        tiles += (hi - lo + bm - 1) / bm;
    }
#pragma unroll
    for (int d = 32; d > 0; d /= 2)
        tiles += __shfl_xor(tiles, d);
    return uniform(tiles) * args.tiles_n;
}

// Row of A that row p of D reads.
__device__ __forceinline__ int fp8_a_row(const Fp8Args &args, int p)
{
    if (args.rows == nullptr)
        return p;
    return min(max(args.rows[p], 0), args.a_rows - 1);
}

// Four consecutive values of one row of D, of which the first `valid` exist.
template <bool BF16>
__device__ __forceinline__ void fp8_store4(void *d, int64_t at, const float (&v)[4], int valid, bool vec)
{
    if (vec && valid >= 4) {
        if constexpr (BF16)
            *(bf16x4 *)((__bf16 *)d + at) = bf16x4{(__bf16)v[0], (__bf16)v[1], (__bf16)v[2], (__bf16)v[3]};
        else
            *(f32x4 *)((float *)d + at) = f32x4{v[0], v[1], v[2], v[3]};
        return;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
        if (i < valid) {
            if constexpr (BF16)
                ((__bf16 *)d)[at + i] = (__bf16)v[i];
            else
                ((float *)d)[at + i] = v[i];
        }
}

// ---- tiles through LDS -------------------------------------------------------

// WM_ x WN_ waves, each a (BM / WM_) x (BN / WN_) piece; a ring of STAGES_ k
// blocks. ROWS: B's scales are per row of 128 k (as A's), otherwise per 128 x 128.
template <int BM_, int BN_, int WM_, int WN_, int STAGES_, bool ROWS_, bool BF16_>
struct Fp8Config {
    static constexpr int BM = BM_, BN = BN_, WM = WM_, WN = WN_, WAVES = WM * WN, THREADS = 64 * WAVES;
    static constexpr bool ROWS = ROWS_, BF16 = BF16_, EXACT = !BF16_;
    static constexpr int WTM = BM / WM, WTN = BN / WN, MI = WTM / 16, NI = WTN / 16;
    static constexpr int A_BYTES = BM * 128, B_BYTES = BN * 128;
    static constexpr int STAGES = STAGES_;
    static constexpr int S_BYTES = THREADS * 4; // one scale per thread, past BM + BN a copy
    static constexpr int STAGE = A_BYTES + B_BYTES + S_BYTES;
    static constexpr int LOADS_A = A_BYTES / 16 / THREADS, LOADS_B = B_BYTES / 16 / THREADS;
    static constexpr int D_ROW = WTN * (BF16 ? 2 : 4), D_BYTES = WTM * D_ROW; // a wave's piece of D
    static_assert(WAVES * D_BYTES <= STAGES * STAGE, "the ring holds the tile of D");
    static_assert(BM + BN <= THREADS && BM % 64 == 0 && BN % 64 == 0, "one scale per thread and stage");
    static_assert(NI == 4 && 128 % WTN == 0, "a wave's columns share a block scale, 16 per lane");
    static_assert(STAGES >= 2 && STAGES * STAGE <= 160 * 1024 && (STAGES - 2) * (LOADS_A + LOADS_B + 1) <= 63, "ring");
};

template <class C>
struct Fp8Loop {
    // A's rows and B's columns keep their 128 bytes of a k block in eight
    // 16-byte chunks, chunk c at position c ^ swizzle(row), so that a wave-wide
    // fragment read covers every bank once. A fragment holds 16 consecutive
    // rows of A, but of B the columns 16 j + 4 ni + t (j, t = 0..3): a lane
    // then owns 16 consecutive columns of D over its four blocks, whole 16-byte
    // pieces of a row for the store.
    static __device__ __forceinline__ int swizzle_a(int r) { return (r >> 1) & 7; }
    static __device__ __forceinline__ int swizzle_b(int r) { return ((r >> 1) & 1) | ((r >> 3) & 6); }

    u32x4 a_rsrc, b_rsrc, s_rsrc;
    uint32_t a_off[C::LOADS_A], b_off[C::LOADS_B], s_off;
    uint32_t s_step; // bytes from one k block's scales to the next
    int wave;

    __device__ __forceinline__ void setup(const Fp8Args &args, const Fp8Tile &t, int tid)
    {
        const int lane = tid & 63;
        wave = uniform(tid >> 6);
        const int64_t first = args.rows == nullptr ? t.row0 : 0;
        a_rsrc = buffer_rsrc(args.a + first * args.lda);
        b_rsrc = buffer_rsrc(args.b + t.expert * args.b_expert + (int64_t)t.col0 * args.ldb);
#pragma unroll
        for (int i = 0; i < C::LOADS_A; ++i) {
            const int r = (wave * C::LOADS_A + i) * 8 + lane / 8;
            const int row = fp8_a_row(args, t.row0 + min(r, t.vm - 1)) - (int)first;
            a_off[i] = (uint32_t)row * (uint32_t)args.lda + (((lane & 7) ^ swizzle_a(r)) << 4);
        }
#pragma unroll
        for (int i = 0; i < C::LOADS_B; ++i) {
            const int r = (wave * C::LOADS_B + i) * 8 + lane / 8;
            b_off[i] = (uint32_t)min(r, t.vn - 1) * (uint32_t)args.ldb + (((lane & 7) ^ swizzle_b(r)) << 4);
        }
        if (wave * 64 < C::BM) {
            const int row = fp8_a_row(args, t.row0 + min(wave * 64 + lane, t.vm - 1)) - (int)first;
            s_rsrc = buffer_rsrc(args.sa + first * args.sa_m);
            s_off = (uint32_t)row * (uint32_t)args.sa_m * 4u;
            s_step = (uint32_t)args.sa_k * 4u;
        } else {
            const int col = t.col0 + min(wave * 64 + lane - C::BM, t.vn - 1);
            s_rsrc = buffer_rsrc(args.sb + t.expert * args.sb_expert);
            s_off = (uint32_t)(C::ROWS ? col : col >> 7) * (uint32_t)args.sb_n * 4u;
            s_step = (uint32_t)args.sb_k * 4u;
        }
    }

    // Start the loads of k block kb into the stage at LDS address `stage`, all
    // at once. In the last, partial block a chunk past the row's end reads the
    // last chunk instead (cleared before it is used).
    __device__ __forceinline__ void issue(uint32_t stage, int kb, int k)
    {
        const uint32_t at = (uint32_t)kb * 128u;
        const int left = k - kb * 128;
        if (left >= 128) {
#pragma unroll
            for (int i = 0; i < C::LOADS_A; ++i)
                dma_load16_imm(stage + wave * (C::LOADS_A * 1024), i * 1024, a_off[i], a_rsrc, at);
#pragma unroll
            for (int i = 0; i < C::LOADS_B; ++i)
                dma_load16_imm(stage + wave * (C::LOADS_B * 1024), C::A_BYTES + i * 1024, b_off[i], b_rsrc, at);
        } else {
            const uint32_t last = (uint32_t)((left - 1) / 16);
            const uint32_t lane = lane_id();
#pragma unroll
            for (int i = 0; i < C::LOADS_A; ++i) {
                const int r = (wave * C::LOADS_A + i) * 8 + (int)lane / 8;
                const uint32_t c = (lane & 7) ^ swizzle_a(r);
                dma_load16_imm(stage + wave * (C::LOADS_A * 1024), i * 1024,
                               a_off[i] - ((c > last ? c - last : 0u) << 4), a_rsrc, at);
            }
#pragma unroll
            for (int i = 0; i < C::LOADS_B; ++i) {
                const int r = (wave * C::LOADS_B + i) * 8 + (int)lane / 8;
                const uint32_t c = (lane & 7) ^ swizzle_b(r);
                dma_load16_imm(stage + wave * (C::LOADS_B * 1024), C::A_BYTES + i * 1024,
                               b_off[i] - ((c > last ? c - last : 0u) << 4), b_rsrc, at);
            }
        }
        dma_load4(stage + C::A_BYTES + C::B_BYTES + wave * 256, s_off, s_rsrc, (uint32_t)kb * s_step);
    }

    // Load I of the PIECES that `issue` starts, for a whole k block.
    static constexpr int PIECES = C::LOADS_A + C::LOADS_B + 1;
    template <int I> __device__ __forceinline__ void issue_piece(uint32_t stage, int kb)
    {
        const uint32_t at = (uint32_t)kb * 128u;
        if constexpr (I < C::LOADS_A)
            dma_load16_imm(stage + wave * (C::LOADS_A * 1024), I * 1024, a_off[I], a_rsrc, at);
        else if constexpr (I < C::LOADS_A + C::LOADS_B)
            dma_load16_imm(stage + wave * (C::LOADS_B * 1024), C::A_BYTES + (I - C::LOADS_A) * 1024, b_off[I - C::LOADS_A],
                           b_rsrc, at);
        else
            dma_load4(stage + C::A_BYTES + C::B_BYTES + wave * 256, s_off, s_rsrc, (uint32_t)kb * s_step);
    }

    // One wave-wide 4-byte-per-lane global -> LDS load (see dma_load16).
    static __device__ __forceinline__ void dma_load4(uint32_t lds_addr, uint32_t voff, u32x4 rsrc, uint32_t soff)
    {
        asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dword %1, %2, %3 offen lds"
                     :
                     : "s"(lds_addr), "v"(voff), "s"(rsrc), "s"(soff)
                     : "memory");
    }

    // Clear the bytes past the row's end in a partial k block of `left` bytes.
    static __device__ __forceinline__ void clear_tail(uint8_t *stage, int left, int tid)
    {
        const int c0 = left / 16;
        for (int i = tid; i < (C::BM + C::BN) * 8; i += C::THREADS) {
            const int r = i / 8, c = i % 8;
            if (c < c0)
                continue;
            const int swz = r < C::BM ? swizzle_a(r) : swizzle_b(r - C::BM);
            u32x4 *p = (u32x4 *)(stage + r * 128 + ((c ^ swz) << 4));
            u32x4 v = {0u, 0u, 0u, 0u};
            if (c == c0 && left % 16 != 0) {
                v = *p;
#pragma unroll
                for (int w = 0; w < 4; ++w) {
                    const int bytes = min(max(left - c0 * 16 - 4 * w, 0), 4);
                    v[w] = bytes == 4 ? v[w] : v[w] & ((1u << (8 * bytes)) - 1u);
                }
            }
            *p = v;
        }
    }
};

enum : int { LAST = 0, GENERAL = 1, STEADY = 2 }; // kinds of k block

// Fix the order of what stands before and after in the instruction stream.
__device__ __forceinline__ void keep_order() { __builtin_amdgcn_sched_barrier(0); }

// One wave's share of the tile: its fragments of the two operands and scales
// for the k block being computed, and the sums not yet added up.
template <class C> struct Fp8Wave {
    static constexpr int MI = C::MI, NI = C::NI;
    // Blocks of a k block in the order of their matrix instructions, STEP at a
    // time: EXACT interleaves two, whose four instructions each depend on the
    // one before. The scaled sum of a step is added LAG steps later, so that
    // the multiply-adds run under the matrix instructions that follow.
    static constexpr int STEP = C::EXACT ? 2 : 1, STEPS = MI * NI / STEP, LAG = C::EXACT ? 1 : 2, RING = 2 * LAG;
    // The sums in flight from one k block to the next belong to the last LAG steps: their columns' scales (ROWS) stay
    // until those are added, the other columns' are loaded with the next block's fragments.
    static constexpr int EARLY_COL = NI - LAG * STEP;
    f32x4 acc[MI][NI], sums[RING][STEP];
    Fragment<C::EXACT> a[2], b[NI];
    f32x4 col[NI]; // ROWS: the scales of this lane's columns
    float scale[MI], late; // row scales of this k block; the last row's of the one before
    int at_a, at_b, at_sa, at_sb; // this lane's places in stage 0, byte offsets

    __device__ __forceinline__ void init(int wm, int wn, int lane)
    {
        const int l16 = lane & 15, g = lane >> 4;
        const int b_row = wn * C::WTN + (l16 >> 2) * 16 + (l16 & 3);
        at_a = (wm * C::WTM + l16) * 128 + ((g ^ Fp8Loop<C>::swizzle_a(l16)) << 4);
        at_b = C::A_BYTES + b_row * 128 + ((g ^ Fp8Loop<C>::swizzle_b(b_row)) << 4);
        at_sa = C::A_BYTES + C::B_BYTES + (wm * C::WTM + l16) * 4;
        at_sb = C::A_BYTES + C::B_BYTES + (C::BM + wn * C::WTN + (C::ROWS ? g * 16 : 0)) * 4;
    }
    __device__ __forceinline__ void start_tile()
    {
#pragma unroll
        for (int i = 0; i < MI; ++i)
#pragma unroll
            for (int j = 0; j < NI; ++j)
                acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int i = 0; i < RING; ++i)
#pragma unroll
            for (int j = 0; j < STEP; ++j)
                sums[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int j = 0; j < NI; ++j)
            col[j] = f32x4{0.f, 0.f, 0.f, 0.f};
        late = 0.f;
        scale[MI - 1] = 0.f;
    }
    // `stage`: its first byte in LDS.
    __device__ __forceinline__ void load_a(int which, int i, const uint8_t *stage)
    {
        a[which].set(*(const i32x4 *)(stage + at_a + i * 2048), *(const i32x4 *)(stage + (at_a ^ 64) + i * 2048));
    }
    __device__ __forceinline__ void load_b(int j, const uint8_t *stage)
    {
        b[j].set(*(const i32x4 *)(stage + at_b + j * 512), *(const i32x4 *)(stage + (at_b ^ 64) + j * 512));
    }
    // The new row scales; the old last row's stays for the sums in flight.
    __device__ __forceinline__ void load_scales(const uint8_t *stage)
    {
        late = scale[MI - 1];
        const float block = C::ROWS ? 1.f : *(const float *)(stage + at_sb);
#pragma unroll
        for (int i = 0; i < MI; ++i)
            scale[i] = *(const float *)(stage + at_sa + i * 64) * block;
    }
    __device__ __forceinline__ void load_col(int j, const uint8_t *stage)
    {
        if constexpr (C::ROWS)
            col[j] = *(const f32x4 *)(stage + at_sb + j * 16);
    }
    // Matrix instructions of step n of the k block.
    template <int N> __device__ __forceinline__ void multiply()
    {
        constexpr int I = N * STEP / NI, J = N * STEP % NI;
        if constexpr (C::EXACT) {
            f32x4 c[STEP];
#pragma unroll
            for (int u = 0; u < STEP; ++u)
                c[u] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int q = 0; q < 4; ++q)
#pragma unroll
                for (int u = 0; u < STEP; ++u)
                    c[u] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(b[J + u].v[q], a[I & 1].v[q], c[u], 0, 0, 0);
#pragma unroll
            for (int u = 0; u < STEP; ++u)
                sums[N % RING][u] = c[u];
        } else {
            sums[N % RING][0] = block_sums(b[J], a[I & 1]);
        }
    }
    // Add the scaled sums of step n; n < 0 counts from the end of the k block before.
    template <int N> __device__ __forceinline__ void add()
    {
        constexpr int M = (N + STEPS) % STEPS, I = M * STEP / NI, J = M * STEP % NI;
        const float s = N < 0 ? late : scale[I];
#pragma unroll
        for (int u = 0; u < STEP; ++u)
#pragma unroll
            for (int r = 0; r < 4; ++r)
                acc[I][J + u][r] = fmaf(sums[M % RING][u][r], C::ROWS ? s * col[J + u][r] : s, acc[I][J + u][r]);
        // Used next a whole k block later, the sums would be moved down there, out from under the matrix instructions.
#pragma unroll
        for (int u = 0; u < STEP; ++u)
            asm volatile("" : "+v"(acc[I][J + u]));
    }
    // Write the wave's piece of D, through its part `out` of LDS, so that an
    // instruction writes whole rows of the piece (128 or 256 bytes): straight
    // from the registers, where a lane holds 16 columns, every instruction
    // touched each line for a part of it (8192 x 8192 from k = 512: fp32 490 us,
    // bf16 124). A row's 16-byte chunks are exchanged by the row's number, which
    // spreads them over the banks. D streams past the caches, but for bf16 rows
    // that start inside a line: there two waves write each line, and the L2 joins
    // them (5000 x 7000 x 3000: 131 us against 141; whole lines and fp32 lose 1 to 3%).
    __device__ __forceinline__ void store(const Fp8Args &args, const Fp8Tile &tile, uint8_t *out, int row0, int col0)
    {
        const int lane = (int)lane_id(); // computed here, so that nothing built on it is kept through the k loop
        constexpr int ES = C::BF16 ? 2 : 4, CHUNKS = C::D_ROW / 16, W = 16 / ES, ROWS_AT_ONCE = 64 / CHUNKS;
        const int vm = min(C::WTM, tile.vm - row0), vn = min(C::WTN, tile.vn - col0);
        if (vm <= 0 || vn <= 0)
            return;
        auto place = [](int r, int c) { return r * C::D_ROW + ((c ^ ((C::BF16 ? r >> 1 : r) & (CHUNKS - 1))) << 4); };
        const int l16 = lane & 15, g = lane >> 4;
#pragma unroll
        for (int i = 0; i < MI; ++i) {
            const int r = i * 16 + l16;
            if constexpr (C::BF16) {
#pragma unroll
                for (int j = 0; j < NI; j += 2) {
                    u32x4 v;
#pragma unroll
                    for (int h = 0; h < 4; ++h) {
                        const f32x4 &s = acc[i][j + h / 2];
                        const bf16x2 p = {(__bf16)s[2 * (h & 1)], (__bf16)s[2 * (h & 1) + 1]};
                        v[h] = __builtin_bit_cast(uint32_t, p);
                    }
                    *(u32x4 *)(out + place(r, g * 2 + j / 2)) = v;
                }
            } else {
#pragma unroll
                for (int j = 0; j < NI; ++j)
                    *(f32x4 *)(out + place(r, g * 4 + j)) = acc[i][j];
            }
        }
        wave_lds_exchange();
        uint8_t *const d = (uint8_t *)args.d + ((int64_t)(tile.row0 + row0) * args.ldd + tile.col0 + col0) * ES;
        const int64_t pitch = args.ldd * ES;
        if (args.d_vec) {
            auto rows = [&](auto stream) {
                const int c = lane % CHUNKS;
#pragma unroll 4
                for (int r = lane / CHUNKS; r < C::WTM; r += ROWS_AT_ONCE) {
                    const u32x4 v = *(const u32x4 *)(out + place(r, c));
                    uint8_t *const p = d + r * pitch + c * 16;
                    if (r < vm && (c + 1) * W <= vn) {
                        if constexpr (stream.value)
                            __builtin_nontemporal_store(v, (u32x4 *)p);
                        else
                            *(u32x4 *)p = v;
                    } else if (r < vm) {
#pragma unroll
                        for (int i = 0; i < W; ++i)
                            if (c * W + i < vn) {
                                if constexpr (C::BF16)
                                    ((uint16_t *)p)[i] = (uint16_t)(v[i / 2] >> (16 * (i & 1)));
                                else
                                    ((uint32_t *)p)[i] = v[i];
                            }
                    }
                }
            };
            if (!C::BF16 || args.d_vec == 2)
                rows(IntC<1>{});
            else
                rows(IntC<0>{});
        } else if (lane < vn) { // rows that start anywhere: one element per lane
            for (int r = 0; r < vm; ++r) {
                const uint8_t *const q = out + place(r, lane / W) + lane % W * ES;
                if constexpr (C::BF16)
                    *(uint16_t *)(d + r * pitch + lane * 2) = *(const uint16_t *)q;
                else
                    *(uint32_t *)(d + r * pitch + lane * 4) = *(const uint32_t *)q;
            }
        }
    }
};

template <class C>
__global__ __launch_bounds__(C::THREADS, 2) void gemm_fp8_tile_kernel(const Fp8Args args)
{
    using Loop = Fp8Loop<C>;
    using Wave = Fp8Wave<C>;
    __shared__ __align__(1024) uint8_t smem[C::STAGES * C::STAGE];
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = uniform(tid >> 6);
    const int wm = wave / C::WN, wn = wave % C::WN;
    Wave w;
    w.init(wm, wn, lane);
    const int total = fp8_total_tiles(args, C::BM);
    const uint32_t lds = lds_address(smem);
    for (int t = blockIdx.x; t < total; t += gridDim.x) {
        Fp8Tile tile;
        if (!fp8_find_tile(args, C::BM, C::BN, static_position(t, total, args.round), tile))
            break;
        Loop loop;
        loop.setup(args, tile, tid);
        w.start_tile();
        barrier_lds(); // every wave has read the last tile's stages
        // A stage that has landed for every wave: its partial end is cleared.
        auto enter = [&](uint8_t *stage, int kb) {
            const int left = args.k - kb * 128;
            if (left < 128) {
                Loop::clear_tail(stage, left, tid);
                barrier_lds();
            }
        };
        // One k block. LAST: none follows. Otherwise the next one's stage is
        // taken over on the way, before the last row of blocks, and the loads of
        // the block STAGES further on go into the stage handed back. STEADY:
        // that one is whole, and its loads are started one by one between the
        // matrix instructions from there into the next block (all at once they
        // hold up every wave: 8% at 8192^3); `pending` says that the block
        // before did so.
        bool pending = false;
        uint32_t here = 0; // the block's stage, byte offset
        auto after = [](uint32_t stage) { return stage + C::STAGE == C::STAGES * C::STAGE ? 0u : stage + C::STAGE; };
        auto k_block = [&](int kb, auto kind) {
            constexpr bool MORE = kind.value != LAST, IN_STEPS = kind.value == STEADY;
            constexpr int HANDOVER = Wave::STEPS - C::NI / Wave::STEP, PER_STEP = C::EXACT ? 2 : Loop::PIECES > Wave::STEPS ? 2 : 1;
            static_assert((Loop::PIECES + PER_STEP - 1) / PER_STEP <= Wave::STEPS, "started before the stage is waited for");
            const uint32_t before = here == 0 ? (C::STAGES - 1) * C::STAGE : here - C::STAGE;
            const uint8_t *const stage = smem + here;
            uint8_t *const next = smem + after(here);
            static_for<Wave::STEPS>([&](auto n) {
                constexpr int N = n.value, I = N * Wave::STEP / C::NI, J = N * Wave::STEP % C::NI;
                if constexpr (J == 0 && I + 1 < C::MI)
                    w.load_a((I + 1) & 1, I + 1, stage);
                if constexpr (J == 0 && I + 1 == C::MI && MORE) {
                    // Everything this wave needs of the stage is in registers: hand it back, take the next one. Of the
                    // loads started, the ones of the STAGES - 2 blocks after that may still be on their way.
                    if (kb + C::STAGES - 1 < args.nk)
                        wait_vmcnt<(C::STAGES - 2) * Loop::PIECES>();
                    else
                        wait_vmcnt<0>();
                    barrier_lds();
                    if constexpr (!IN_STEPS) {
                        if (kb + C::STAGES < args.nk)
                            loop.issue(lds + here, kb + C::STAGES, args.k);
                        enter(next, kb + 1);
                    }
                    w.load_a((I + 1) & 1, 0, next);
                }
                w.template multiply<N>();
                keep_order();
                static_for<PER_STEP>([&](auto u) {
                    if constexpr (N >= HANDOVER && IN_STEPS) {
                        constexpr int P = (N - HANDOVER) * PER_STEP + u.value;
                        if constexpr (P < Loop::PIECES)
                            loop.template issue_piece<P>(lds + here, kb + C::STAGES);
                    } else if constexpr (N < HANDOVER && MORE) {
                        constexpr int P = (N + Wave::STEPS - HANDOVER) * PER_STEP + u.value;
                        if constexpr (P < Loop::PIECES)
                            if (pending)
                                loop.template issue_piece<P>(lds + before, kb - 1 + C::STAGES);
                    }
                });
                w.template add<N - Wave::LAG>();
                if constexpr (C::ROWS && N == Wave::LAG - 1)
                    static_for<C::NI - Wave::EARLY_COL>([&](auto j) { w.load_col(Wave::EARLY_COL + j.value, stage); });
                if constexpr (I + 1 == C::MI && MORE)
                    static_for<Wave::STEP>([&](auto u) { w.load_b(J + u.value, next); });
                keep_order();
            });
            if constexpr (MORE) {
                w.load_scales(next);
                static_for<Wave::EARLY_COL>([&](auto j) { w.load_col(j.value, next); });
            } else {
                static_for<Wave::LAG>([&](auto n) { w.template add<Wave::STEPS + n.value - Wave::LAG>(); });
            }
            here = after(here);
        };
        // A wave whose rows or columns all lie past the tile's edge only loads
        // and meets the others: its partner on the SIMD has the matrix unit to itself.
        auto k_block_idle = [&](int kb) {
            if (kb + C::STAGES - 1 < args.nk)
                wait_vmcnt<(C::STAGES - 2) * Loop::PIECES>();
            else
                wait_vmcnt<0>();
            barrier_lds();
            if (kb + C::STAGES < args.nk)
                loop.issue(lds + here, kb + C::STAGES, args.k);
            here = after(here);
            enter(smem + here, kb + 1);
        };
        const bool idle = wm * C::WTM >= tile.vm || wn * C::WTN >= tile.vn;
        if (args.nk > 0) {
            for (int kb = 0; kb < min(C::STAGES - 1, args.nk); ++kb)
                loop.issue(lds + kb * C::STAGE, kb, args.k);
            if (args.nk >= C::STAGES - 1)
                wait_vmcnt<(C::STAGES - 2) * Loop::PIECES>();
            else
                wait_vmcnt<0>();
            barrier_lds();
            if (args.nk > C::STAGES - 1)
                loop.issue(lds + (C::STAGES - 1) * C::STAGE, C::STAGES - 1, args.k);
            enter(smem, 0);
        }
        if (idle) {
            for (int kb = 0; kb + 1 < args.nk; ++kb)
                k_block_idle(kb);
        } else if (args.nk > 0) {
#pragma unroll
            for (int j = 0; j < C::NI; ++j)
                w.load_b(j, smem);
#pragma unroll
            for (int j = 0; j < Wave::EARLY_COL; ++j)
                w.load_col(j, smem);
            w.load_a(0, 0, smem);
            w.load_scales(smem);
            const int whole = args.k / 128;
            int kb = 0;
            for (; kb + C::STAGES < whole; ++kb) {
                k_block(kb, IntC<STEADY>{});
                pending = true;
            }
            for (; kb + 1 < args.nk; ++kb) {
                k_block(kb, IntC<GENERAL>{});
                pending = false;
            }
            k_block(args.nk - 1, IntC<LAST>{});
        }
        barrier_lds(); // every wave has read the last stage: the ring takes the results
        w.store(args, tile, smem + wave * C::D_BYTES, wm * C::WTM, wn * C::WTN);
    }
}

// ---- few rows ----------------------------------------------------------------

// Up to 16 MB rows against a strip of 16-column tiles per workgroup, straight
// from memory to registers: with so few rows every byte of B is used by one
// workgroup only, so LDS would add a hop and a barrier. The eight waves take the
// k blocks in turn (wave w: w, w + 8, ...), eight independent streams of loads,
// and their partial sums are added in wave order through LDS for each tile; the
// waves go on to the next tile's loads meanwhile.
//
// Memory bound: what counts is how many bytes are on their way. U k blocks per
// wave at once: 4 where a compute unit has one or two workgroups (8 x 4096 x
// 4096: 7 us), 2 where it can have four (59 registers; 128 rows over 55 of 64
// experts, 4096 x 4096 each, 922 MB: 168 us, 5.5 TB/s, against 185 with 4). Two
// tiles per workgroup there spare half the searches for the tile (one: 174 us;
// eight: 179, too few workgroups to even out).
template <int MB, int U, bool ROWS, bool BF16>
__global__ __launch_bounds__(512) void gemm_fp8_rows_kernel(const Fp8Args args)
{
    constexpr int WAVES = 8;
    __shared__ __align__(16) float part[2][WAVES][MB * 16][16];
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = uniform(tid >> 6);
    const int l16 = lane & 15, g = lane >> 4;
    Fp8Tile tile;
    if (!fp8_find_tile(args, MB * 16, 16 * args.strip, blockIdx.x, tile))
        return;
    const uint8_t *ap[MB];
    const float *sap[MB];
#pragma unroll
    for (int i = 0; i < MB; ++i) {
        const int row = fp8_a_row(args, tile.row0 + min(i * 16 + l16, tile.vm - 1));
        ap[i] = args.a + (int64_t)row * args.lda;
        sap[i] = args.sa + (int64_t)row * args.sa_m;
    }
    const uint8_t *const b = args.b + tile.expert * args.b_expert;
    const float *const sbp = args.sb + tile.expert * args.sb_expert;
    const int tiles = (tile.vn + 15) / 16;
    for (int t = 0; t < tiles; ++t) {
        const int col0 = tile.col0 + t * 16;
        const uint8_t *const bp = b + (int64_t)min(col0 + l16, args.n - 1) * args.ldb;
        f32x4 acc[MB];
#pragma unroll
        for (int i = 0; i < MB; ++i)
            acc[i] = f32x4{0.f, 0.f, 0.f, 0.f};
        for (int k0 = wave; k0 < args.nk; k0 += WAVES * U) {
            i32x4 x[U][2], y[U][MB][2];
            float sa[U][MB], sb[U][ROWS ? 4 : 1];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int kb = min(k0 + u * WAVES, args.nk - 1); // past the end: read again, not used
                const int last = min(7, (args.k - kb * 128 - 1) / 16);
                const int64_t lo = (int64_t)kb * 128 + min(g, last) * 16, hi = (int64_t)kb * 128 + min(g + 4, last) * 16;
                x[u][0] = *(const i32x4 *)(bp + lo);
                x[u][1] = *(const i32x4 *)(bp + hi);
#pragma unroll
                for (int i = 0; i < MB; ++i) {
                    y[u][i][0] = *(const i32x4 *)(ap[i] + lo);
                    y[u][i][1] = *(const i32x4 *)(ap[i] + hi);
                    sa[u][i] = sap[i][kb * args.sa_k];
                }
#pragma unroll
                for (int r = 0; r < (ROWS ? 4 : 1); ++r)
                    sb[u][r] = sbp[(ROWS ? min(col0 + g * 4 + r, args.n - 1) : col0 >> 7) * args.sb_n + kb * args.sb_k];
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int kb = k0 + u * WAVES;
                if (kb >= args.nk)
                    break;
                const int left = args.k - kb * 128;
                if (left < 128) { // bytes past the end of the rows are cleared in both operands
#pragma unroll
                    for (int h = 0; h < 2; ++h)
#pragma unroll
                        for (int w = 0; w < 4; ++w) {
                            const int bytes = min(max(left - (g + 4 * h) * 16 - w * 4, 0), 4);
                            const int mask = bytes == 4 ? -1 : (int)((1u << (8 * bytes)) - 1u);
                            x[u][h][w] &= mask;
#pragma unroll
                            for (int i = 0; i < MB; ++i)
                                y[u][i][h][w] &= mask;
                        }
                }
                Fragment<!BF16> fx;
                fx.set(x[u][0], x[u][1]);
#pragma unroll
                for (int i = 0; i < MB; ++i) {
                    Fragment<!BF16> fy;
                    fy.set(y[u][i][0], y[u][i][1]);
                    const f32x4 p = block_sums(fx, fy);
#pragma unroll
                    for (int r = 0; r < 4; ++r)
                        acc[i][r] = fmaf(p[r], sa[u][i] * sb[u][ROWS ? r : 0], acc[i][r]);
                }
            }
        }
        float (*const sums)[MB * 16][16] = part[t & 1];
#pragma unroll
        for (int i = 0; i < MB; ++i)
            *(f32x4 *)&sums[wave][i * 16 + l16][g * 4] = acc[i];
        barrier_lds(); // tile t - 1 was added up before this, so its half may be written next
        if (tid < MB * 64) {
            const int r = tid >> 2, c = (tid & 3) * 4;
            float v[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int w = 0; w < WAVES; ++w) {
                const f32x4 p = *(const f32x4 *)&sums[w][r][c];
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    v[i] += p[i];
            }
            const int valid = tile.vn - t * 16 - c;
            if (r < tile.vm)
                fp8_store4<BF16>(args.d, (int64_t)(tile.row0 + r) * args.ldd + col0 + c, v, valid, args.d_vec);
        }
    }
}

} // namespace pts
