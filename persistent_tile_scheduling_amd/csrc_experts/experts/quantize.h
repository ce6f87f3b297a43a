// Quantisation to e4m3 with one fp32 scale per block of 128.
//
//   scale_b = max(max |x| over block b / 448, 2^-126),  q = e4m3(x / scale_b)
//
// A block is 128 consecutive k of one row, or 128 x 128. Both divisions are
// fp32 divisions rounded to nearest and q is rounded to nearest, ties to even,
// so the codes do not depend on the kernel that writes them. A block holding
// an infinity or a NaN gets a NaN scale and NaN codes.
//
// Memory bound: 2 or 4 bytes read (twice that with the gate) and 1 byte
// written per element; each element is read once and kept in registers between
// the maximum and the conversion. (Loads are ordinary ones: rows need not start
// at a cache line, and a streaming load would fetch the shared lines twice. The
// codes' stores stream: 2% of either form below.)
#pragma once

#include "lanes.h"

namespace pts {

constexpr int QBLOCK = 128;

// |x| as an ordered integer: the maximum then keeps a NaN (its bits are above
// infinity's), which a floating maximum drops.
__device__ __forceinline__ uint32_t abs_bits(float x) { return __float_as_uint(x) & 0x7FFFFFFFu; }

// The scale of a block from the integer maximum of its magnitudes.
__device__ __forceinline__ float block_scale(uint32_t most)
{
    if (most >= 0x7F800000u)
        return __uint_as_float(0x7FC00000u);
    return fmaxf(__uint_as_float(most) / 448.0f, 0x1p-126f);
}

// x / s rounded to nearest, given r = 1 / s rounded to nearest: the product
// x r corrected by its exact residual (Markstein, "Computation of elementary
// functions on the IBM RISC System/6000 processor", 1990). Needs the residual
// to stay normal: the caller divides where s < 2^-60.
__device__ __forceinline__ float divide_by(float x, float s, float r)
{
    const float t = x * r;
    return fmaf(fmaf(-t, s, x), r, t);
}

__device__ __forceinline__ uint32_t pack4(float a, float b, float c, float d)
{
    int v = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false);
    return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(c, d, v, true);
}

// N (4 or 8) values of one block to codes, four to a word.
template <int N> __device__ __forceinline__ void quantize(const float *x, float s, uint32_t (&out)[N / 4])
{
    float t[N];
    if (s >= 0x1p-60f) {
        const float r = 1.0f / s;
#pragma unroll
        for (int i = 0; i < N; ++i)
            t[i] = divide_by(x[i], s, r);
    } else { // tiny or NaN scales
#pragma unroll
        for (int i = 0; i < N; ++i)
            t[i] = x[i] / s;
    }
#pragma unroll
    for (int i = 0; i < N; i += 4)
        out[i / 4] = pack4(t[i], t[i + 1], t[i + 2], t[i + 3]);
}

// A word of codes of which the first `valid` lie inside the row: the others are
// padding, 0 (a block that is not finite makes NaN codes of the zeros there).
__device__ __forceinline__ uint32_t codes_up_to(uint32_t word, int valid)
{
    return valid >= 4 ? word : valid <= 0 ? 0u : word & ((1u << (8 * valid)) - 1u);
}

// silu(g) = g / (1 + exp(-g)) in fp32. Up to |g| = 87, to 6 2^-24 of its value
// (the compiler's expf and division, to 5, made the gated form of 8192 x 7000
// 77 us instead of 62):
//   t = g / ln 2 rounded, and what that misses of exp(-g): l = -g - t ln 2 (ln 2
//   in two parts); exp(-g) = 2^-t (1 + l), |l| < 2^-17; the hardware's 2^x and
//   reciprocal are good to one step, the reciprocal is refined once.
constexpr float SILU_NEAR = 87.0f;
__device__ __forceinline__ float silu_near(float g)
{
    const float t = g * -0x1.715476p+0f;
    const float l = fmaf(0x1.05c61p-29f, t, fmaf(-0x1.62e43p-1f, t, -g));
    const float z = __builtin_amdgcn_exp2f(t);
    const float d = 1.0f + fmaf(z, l, z);
    const float r = __builtin_amdgcn_rcpf(d);
    return g * fmaf(fmaf(-d, r, 1.0f), r, r);
}
// Beyond it the sum would overflow or round to 1: exp(g) itself, down to its
// subnormal values, which the hardware's instructions do not return.
__device__ __forceinline__ float silu_far(float g) { return g < 0.f ? g * expf(g) : g; }

// A thread holds eight elements of a line of x as 16-byte pieces, one of bf16 or
// two of fp32; the pieces of 16 (or 64) lanes side by side are what one load
// instruction reads, so each uses the cache lines it touches whole. Element j
// of the thread at place `at` of `lanes`:
template <bool BF16> __device__ __forceinline__ constexpr int element(int at, int j, int lanes)
{
    return BF16 ? at * 8 + j : j / 4 * lanes * 4 + at * 4 + j % 4;
}

// One piece from p, of which the first `valid` elements exist; the rest read as
// 0. VEC: p is 16-byte aligned.
template <bool BF16, bool VEC>
__device__ __forceinline__ void load_piece(const void *p, int valid, float *x)
{
    constexpr int N = BF16 ? 8 : 4;
    if (VEC && valid >= N) {
        const u32x4 v = *(const u32x4 *)p;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if constexpr (BF16) {
                x[2 * i] = __uint_as_float(v[i] << 16);
                x[2 * i + 1] = __uint_as_float(v[i] & 0xFFFF0000u);
            } else {
                x[i] = __uint_as_float(v[i]);
            }
        }
        return;
    }
#pragma unroll
    for (int i = 0; i < N; ++i) {
        x[i] = 0.f;
        if (i < valid)
            x[i] = BF16 ? __uint_as_float((uint32_t)((const uint16_t *)p)[i] << 16) : ((const float *)p)[i];
    }
}

// The thread's eight elements of a line that starts at p and has `valid`.
template <bool BF16, bool VEC>
__device__ __forceinline__ void load8(const uint8_t *p, int at, int lanes, int valid, float (&x)[8])
{
    constexpr int N = BF16 ? 8 : 4, ES = BF16 ? 2 : 4;
#pragma unroll
    for (int j = 0; j < 8; j += N) {
        const int e = element<BF16>(at, j, lanes);
        load_piece<BF16, VEC>(p + (int64_t)e * ES, valid - e, x + j);
    }
}

struct QuantizeArgs {
    const void *x;
    uint8_t *q;
    float *scale;
    int64_t ldx, ldq;
    int64_t scale_m, scale_k; // element strides of the scale over rows (or row blocks) and k blocks
    int32_t m, k;
    int32_t strips;           // workgroups along k; the grid is flat, strips fastest
    int32_t rows_per_group;   // rows one workgroup walks (row form)
};

__device__ __forceinline__ uint32_t larger(uint32_t a, uint32_t b) { return max(a, b); }

// Row form, x row-major: a wave reads 512 consecutive elements of a row (four
// blocks), so a block's maximum stays inside 16 lanes (bf16) or 32 (fp32). A
// workgroup walks `rows_per_group` rows of one 512-wide strip; the strip's
// scales are collected in LDS and written together, since they are stored with
// the rows next to each other (one k block's scales of consecutive rows are
// what a product's tile reads). 8192 x 8192 bf16: 36 to 40 us (5.0 to 5.6 TB/s; a
// large copy reaches 5.3), fp32 60 us (5.5). 8192 x 7000 with the gate, bf16: 59 to
// 65 us (4.4 to 4.9 TB/s; 55 to 59 with the fast exponential, whose error grows
// with the gate: the gate's instructions count beside the loads) with 8 rows per
// workgroup; 4 take 3 to 6% more, 32 7%, 16 the same. One row of 4096: 2.7 us, the
// latency of one pass.
template <bool BF16, bool GATED, bool VEC>
__global__ __launch_bounds__(256) void quantize_rows_kernel(const QuantizeArgs args)
{
    constexpr int ES = BF16 ? 2 : 4, N = BF16 ? 8 : 4;
    __shared__ float scales[4][64];
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
    const int strip = blockIdx.x % args.strips, group = blockIdx.x / args.strips;
    const int c = strip * 512;
    const int valid = args.k - c, room = (args.k + 15) / 16 * 16 - c;
    const int row0 = group * args.rows_per_group;
    const int rows = min(args.rows_per_group, args.m - row0);
    for (int r = wave; r < rows; r += 4) {
        const int64_t row = row0 + r;
        const uint8_t *p = (const uint8_t *)args.x + (row * args.ldx + c) * ES;
        float x[8];
        load8<BF16, VEC>(p, lane, 64, valid, x);
        if constexpr (GATED) { // silu(gate) up
            float up[8];
            load8<BF16, VEC>(p + (int64_t)args.k * ES, lane, 64, valid, up);
            float most = 0.f;
#pragma unroll
            for (int i = 0; i < 8; ++i)
                most = fmaxf(most, fabsf(x[i]));
            const bool far = __builtin_amdgcn_ballot_w64(most > SILU_NEAR) != 0;
#pragma unroll
            for (int i = 0; i < 8; ++i)
                x[i] = (far && fabsf(x[i]) > SILU_NEAR ? silu_far(x[i]) : silu_near(x[i])) * up[i];
        }
#pragma unroll
        for (int j = 0; j < 8; j += N) {
            uint32_t most = 0;
#pragma unroll
            for (int i = 0; i < N; ++i)
                most = max(most, abs_bits(x[j + i]));
            most = reduce_lanes<16>(most, larger);
            if constexpr (!BF16)
                most = reduce_step<16>(most, larger);
            const float s = block_scale(most);
            uint32_t codes[N / 4];
            quantize<N>(x + j, s, codes);
            const int e = element<BF16>(lane, j, 64);
            if (e < room) { // q's rows are padded to whole 16-byte pieces
                uint8_t *const q = args.q + row * args.ldq + c + e;
#pragma unroll
                for (int w = 0; w < N / 4; ++w)
                    codes[w] = codes_up_to(codes[w], valid - e - 4 * w);
                if constexpr (BF16)
                    __builtin_nontemporal_store((uint64_t)codes[1] << 32 | codes[0], (uint64_t *)q);
                else
                    *(uint32_t *)q = codes[0];
            }
            if (e % QBLOCK == 0)
                scales[e / QBLOCK][r] = s;
        }
    }
    __syncthreads();
    const int kb = strip * 4 + wave; // one wave per k block, lanes along the rows
    if (lane < rows && kb < (args.k + QBLOCK - 1) / QBLOCK)
        args.scale[(row0 + lane) * args.scale_m + kb * args.scale_k] = scales[wave][lane];
}

// Tile form: one 128 x 128 block of the output per workgroup, for x stored
// column by column (COL; the codes are still written row by row) and for
// 128 x 128 scales. x's lines in memory (its rows, or with COL its columns) run
// along the 16 lanes `fast`; a thread holds eight elements of each of eight
// consecutive lines. The codes leave through LDS, so that a row's 128 codes are
// written as whole 16-byte pieces; there, row r's sixteen 8-byte pieces are
// exchanged by a number that follows the thread that writes them, which spreads
// the 16 lanes' rows over the banks. 5000 x 7000 fp32 by columns: 41 us (4.3
// TB/s; its columns start inside cache lines, which adds 16% to what is read).
template <bool BF16, bool COL, bool SQUARE, bool VEC>
__global__ __launch_bounds__(256) void quantize_tile_kernel(const QuantizeArgs args)
{
    constexpr int ES = BF16 ? 2 : 4, N = BF16 ? 8 : 4;
    __shared__ uint32_t most[QBLOCK];
    __shared__ __align__(16) uint8_t codes[QBLOCK * QBLOCK];
    auto place = [](int r, int piece) { // byte of 8-byte piece `piece` of row r
        return r * QBLOCK + ((piece ^ ((COL ? r / N : r / 8) % 8 * 2)) * 8);
    };
    const int tid = threadIdx.x;
    const int fast = tid & 15, slow = tid >> 4;
    const int bk = blockIdx.x % args.strips, bm = blockIdx.x / args.strips;
    const int row0 = bm * QBLOCK, col0 = bk * QBLOCK;
    const int vm = min(QBLOCK, args.m - row0), vk = min(QBLOCK, args.k - col0);
    const int nfast = COL ? vm : vk, nslow = COL ? vk : vm;
    if (tid < QBLOCK)
        most[tid] = 0;
    float x[8][8]; // [slow][fast]
    const int64_t base = COL ? (int64_t)col0 * args.ldx + row0 : (int64_t)row0 * args.ldx + col0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int j = slow * 8 + i;
        load8<BF16, VEC>((const uint8_t *)args.x + (base + (int64_t)j * args.ldx) * ES, fast, 16, j < nslow ? nfast : 0,
                         x[i]);
    }
    __syncthreads();
    if constexpr (SQUARE) {
        uint32_t v = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i)
#pragma unroll
            for (int j = 0; j < 8; ++j)
                v = max(v, abs_bits(x[i][j]));
        v = reduce_lanes<64>(v, larger);
        if ((tid & 63) == 0)
            atomicMax(&most[0], v);
    } else { // COL: a row of the output is a fast index, its maximum runs over the slow ones
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            uint32_t v = 0;
#pragma unroll
            for (int i = 0; i < 8; ++i)
                v = max(v, abs_bits(x[i][j]));
            v = reduce_step<32>(reduce_step<16>(v, larger), larger); // the wave's four lines of lanes
            if ((tid & 48) == 0)
                atomicMax(&most[element<BF16>(fast, j, 16)], v);
        }
    }
    __syncthreads();
#pragma unroll
    for (int r = 0; r < 8; ++r) {
        if constexpr (COL) { // transposed: eight consecutive k of one row
            float row[8];
            uint32_t out[2];
#pragma unroll
            for (int t = 0; t < 8; ++t)
                row[t] = x[t][r];
            const int o = element<BF16>(fast, r, 16);
            quantize<8>(row, block_scale(most[SQUARE ? 0 : o]), out);
            *(uint2 *)(codes + place(o, slow)) = make_uint2(out[0], out[1]);
        } else {
            const int o = slow * 8 + r;
            uint32_t out[2];
            quantize<8>(x[r], block_scale(most[0]), out);
            if constexpr (BF16) {
                *(uint2 *)(codes + place(o, fast)) = make_uint2(out[0], out[1]);
            } else {
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int e = element<BF16>(fast, 4 * h, 16);
                    *(uint32_t *)(codes + place(o, e / 8) + e % 8) = out[h];
                }
            }
        }
    }
    __syncthreads();
    const int room = min(QBLOCK, (args.k + 15) / 16 * 16 - col0);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int r = i * 32 + tid / 8, piece = (tid & 7) * 2;
        if (r < vm && piece * 8 < room) { // q's rows are padded to whole 16-byte pieces
            u32x4 v = *(const u32x4 *)(codes + place(r, piece));
#pragma unroll
            for (int w = 0; w < 4; ++w)
                v[w] = codes_up_to(v[w], vk - piece * 8 - 4 * w);
            __builtin_nontemporal_store(v, (u32x4 *)(args.q + (int64_t)(row0 + r) * args.ldq + col0 + piece * 8));
        }
    }
    if constexpr (SQUARE) {
        if (tid == 0)
            args.scale[bm * args.scale_m + bk * args.scale_k] = block_scale(most[0]);
    } else {
        if (tid < vm)
            args.scale[(row0 + tid) * args.scale_m + bk * args.scale_k] = block_scale(most[tid]);
    }
}

} // namespace pts
