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
// the maximum and the conversion.
#pragma once

#include "device/common.h"

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

// Eight values of one block to eight codes.
__device__ __forceinline__ uint2 quantize8(const float (&x)[8], float s)
{
    float t[8];
    if (s >= 0x1p-60f) {
        const float r = 1.0f / s;
#pragma unroll
        for (int i = 0; i < 8; ++i)
            t[i] = divide_by(x[i], s, r);
    } else { // tiny or NaN scales
#pragma unroll
        for (int i = 0; i < 8; ++i)
            t[i] = x[i] / s;
    }
    return make_uint2(pack4(t[0], t[1], t[2], t[3]), pack4(t[4], t[5], t[6], t[7]));
}

// Eight consecutive elements from p, of which the first `valid` exist; the rest
// read as 0. VEC: p is 16-byte aligned.
template <bool BF16, bool VEC>
__device__ __forceinline__ void load8(const void *p, int valid, float (&x)[8])
{
    if (VEC && valid >= 8) {
        if constexpr (BF16) {
            const u32x4 v = __builtin_nontemporal_load((const u32x4 *)p);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                x[2 * i] = __uint_as_float(v[i] << 16);
                x[2 * i + 1] = __uint_as_float(v[i] & 0xFFFF0000u);
            }
        } else {
            const f32x4 v = __builtin_nontemporal_load((const f32x4 *)p);
            const f32x4 w = __builtin_nontemporal_load((const f32x4 *)p + 1);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                x[i] = v[i];
                x[4 + i] = w[i];
            }
        }
        return;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        x[i] = 0.f;
        if (i < valid) {
            if constexpr (BF16)
                x[i] = __uint_as_float((uint32_t)((const uint16_t *)p)[i] << 16);
            else
                x[i] = ((const float *)p)[i];
        }
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

// Maximum over the 16 lanes of a row of the wave, in every lane.
__device__ __forceinline__ uint32_t max16(uint32_t v)
{
    v = max(v, (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0x128, 0xF, 0xF, false)); // rotate by 8
    v = max(v, (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0x124, 0xF, 0xF, false));
    v = max(v, (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0x122, 0xF, 0xF, false));
    v = max(v, (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0x121, 0xF, 0xF, false));
    return v;
}

// Row form, x row-major: a wave reads 512 consecutive elements of a row (four
// blocks, 16 lanes and 8 elements each), so a block's maximum stays inside a
// DPP row. A workgroup walks `rows_per_group` rows of one 512-wide strip; the
// strip's scales are collected in LDS and written together, since they are
// stored with the rows next to each other (one k block's scales of
// consecutive rows are what a product's tile reads).
template <bool BF16, bool GATED, bool VEC>
__global__ __launch_bounds__(256) void quantize_rows_kernel(const QuantizeArgs args)
{
    __shared__ float scales[4][64];
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
    const int strip = blockIdx.x % args.strips, group = blockIdx.x / args.strips;
    const int c = strip * 512 + lane * 8; // this lane's first column
    const int valid = args.k - c, room = (args.k + 15) / 16 * 16 - c;
    constexpr int ES = BF16 ? 2 : 4;
    const int row0 = group * args.rows_per_group;
    const int rows = min(args.rows_per_group, args.m - row0);
    for (int r = wave; r < rows; r += 4) {
        const int64_t row = row0 + r;
        const uint8_t *p = (const uint8_t *)args.x + (row * args.ldx + c) * ES;
        float x[8];
        load8<BF16, VEC>(p, valid, x);
        if constexpr (GATED) { // silu(gate) up; the reciprocal is good to 1 ulp, a division would take ten instructions
            float up[8];
            load8<BF16, VEC>(p + (int64_t)args.k * ES, valid, up);
#pragma unroll
            for (int i = 0; i < 8; ++i)
                x[i] = x[i] * __builtin_amdgcn_rcpf(1.0f + __expf(-x[i])) * up[i];
        }
        uint32_t most = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i)
            most = max(most, abs_bits(x[i]));
        const float s = block_scale(max16(most));
        if (room > 0) // q's rows are padded to whole 16-byte pieces
            *(uint2 *)(args.q + row * args.ldq + c) = quantize8(x, s);
        if ((lane & 15) == 0)
            scales[lane >> 4][r] = s;
    }
    __syncthreads();
    const int kb = strip * 4 + wave; // one wave per k block, lanes along the rows
    if (lane < rows && kb < (args.k + QBLOCK - 1) / QBLOCK)
        args.scale[(row0 + lane) * args.scale_m + kb * args.scale_k] = scales[wave][lane];
}

// Tile form: one 128 x 128 block of the output per workgroup, for x stored
// column by column (COL; k-major input, codes still written row by row) and
// for 128 x 128 scales. A thread holds an 8 x 8 piece in registers.
//   row-major x: rows 8 a + i, columns 8 b .. 8 b + 7, a = tid / 16, b = tid % 16
//   COL:         the same with the roles exchanged: 8 loads along the rows, each
//                of 8 consecutive rows, then transposed on the way out through
//                the order in which the piece is read.
// Either way the codes leave through LDS, so that a row's 128 codes are
// written as whole 16-byte pieces.
template <bool BF16, bool COL, bool SQUARE, bool VEC>
__global__ __launch_bounds__(256) void quantize_tile_kernel(const QuantizeArgs args)
{
    constexpr int ES = BF16 ? 2 : 4;
    constexpr int PITCH = 144; // bytes per row of codes in LDS, a multiple of 16
    __shared__ uint32_t most[QBLOCK];
    __shared__ __align__(16) uint8_t codes[QBLOCK * PITCH];
    const int tid = threadIdx.x;
    const int fast = tid & 15, slow = tid >> 4;       // along the storage order of x, across it
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
        const uint8_t *p = (const uint8_t *)args.x + (base + (int64_t)j * args.ldx + fast * 8) * ES;
        load8<BF16, VEC>(p, j < nslow ? nfast - fast * 8 : 0, x[i]);
    }
    __syncthreads();
    if constexpr (SQUARE) {
        uint32_t v = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i)
#pragma unroll
            for (int j = 0; j < 8; ++j)
                v = max(v, abs_bits(x[i][j]));
        v = max16(v);
        if (fast == 0)
            atomicMax(&most[0], v);
    } else { // COL: a row of the output is a fast index, its maximum runs over the slow ones
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            uint32_t v = 0;
#pragma unroll
            for (int i = 0; i < 8; ++i)
                v = max(v, abs_bits(x[i][j]));
            atomicMax(&most[fast * 8 + j], v);
        }
    }
    __syncthreads();
#pragma unroll
    for (int r = 0; r < 8; ++r) { // the piece's output rows
        float row[8];
#pragma unroll
        for (int t = 0; t < 8; ++t)
            row[t] = COL ? x[t][r] : x[r][t];
        const int orow = (COL ? fast : slow) * 8 + r, ocol = (COL ? slow : fast) * 8;
        *(uint2 *)(codes + orow * PITCH + ocol) = quantize8(row, block_scale(most[SQUARE ? 0 : orow]));
    }
    __syncthreads();
    const int room = min(QBLOCK, (args.k + 15) / 16 * 16 - col0);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int r = i * 32 + tid / 8, cc = (tid & 7) * 16;
        if (r < vm && cc < room) // q's rows are padded to whole 16-byte pieces
            *(u32x4 *)(args.q + (int64_t)(row0 + r) * args.ldq + col0 + cc) = *(const u32x4 *)(codes + r * PITCH + cc);
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
