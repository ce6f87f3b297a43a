// Newton-Schulz steps of matrices whose short side is at most 64 (ortho.h has the
// formulas): all steps in three launches after the norm's, in fp32.
//
// The Gram matrix follows the steps without the matrix: with Q = a + b A + c A A,
// X' = Q X gives A' = Q A Q, and all of them commute. So one workgroup per matrix
// runs the chain of 64 x 64 products in LDS and leaves each step's b A + c A A;
// then every workgroup takes 64 of the long side's vectors through all the steps.
// Where a step at a time costs three products' launches of 6 us (and the joins of
// split ones), the chain costs 13 products of 64^3 on one compute unit, 1 us each,
// whatever the long side: 64 x 2000 100 -> 40 us. Beyond 64 a chain in LDS would
// grow with the cube of the side and lose.
//
// The matrix unit multiplies fp32 here (16 x 16 x 4), so nothing is rounded to
// fewer bits on the way: A's small eigenvalues grow up to 12-fold a step.
#pragma once

#include "linear/ortho.h"

namespace pts {

constexpr int SMALL = 64;          // the longest short side
constexpr int SMALL_PITCH = 68;    // floats of an LDS row: sixteen rows' 16-byte pieces lie in different banks
constexpr int SMALL_MATRIX = SMALL * SMALL;

struct SmallArgs {
    NormArgs norm;      // x and its norm
    float *parts;       // [matrix][chunk][64][64]: Gram matrices of chunks of the long side
    float *polys;       // [matrix][step][64][64]: b A + c A A
    uint16_t *out;
    int64_t ldo, o_batch;
    float a, b, c;
    int32_t tall, side, lng, chunks, chunk, steps, o_whole; // chunk: vectors each, a multiple of 64
};

__device__ __forceinline__ double small_scale(const SmallArgs &args, int batch)
{
    const int lane = threadIdx.x & 63; // at most 64 blocks
    double sum = lane < args.norm.blocks ? args.norm.sums[(int64_t)batch * args.norm.blocks + lane] : 0.0;
#pragma unroll
    for (int d = 32; d > 0; d /= 2)
        sum += __shfl_xor(sum, d);
    return 1.0 / (sqrt(sum) + args.norm.eps);
}

// Element i of long vector j of x, scaled; 0 outside.
__device__ __forceinline__ float small_x(const SmallArgs &args, int batch, int i, int64_t j, double scale)
{
    if (i >= args.side || j >= args.lng)
        return 0.f;
    const int64_t at = batch * args.norm.x_batch + (args.tall ? j * args.norm.ldx + i : i * args.norm.ldx + j);
    const float v = args.norm.f32 ? ((const float *)args.norm.x)[at] : __uint_as_float((uint32_t)((const uint16_t *)args.norm.x)[at] << 16);
    return (float)((double)v * scale);
}

// acc += (rows of p) . (rows of q) over `blocks` times 16 k: lane l has of row l % 16 the k 4 (l / 16) .. + 3, and gets of the
// result row 4 (l / 16) .. + 3 of p against row l % 16 of q.
__device__ __forceinline__ f32x4 small_product(const float *p, const float *q, int blocks, int lane, f32x4 acc)
{
    const int at = (lane & 15) * SMALL_PITCH + (lane >> 4) * 4;
#pragma unroll
    for (int k = 0; k < SMALL; k += 16) {
        if (k >= blocks * 16)
            break;
        const f32x4 x = *(const f32x4 *)(p + at + k), y = *(const f32x4 *)(q + at + k);
#pragma unroll
        for (int e = 0; e < 4; ++e)
            acc = __builtin_amdgcn_mfma_f32_16x16x4f32(x[e], y[e], acc, 0, 0, 0);
    }
    return acc;
}

// The Gram matrix of one chunk of the long side: sixteen waves, a 16 x 16 block each.
__global__ __launch_bounds__(1024) void small_gram_kernel(const SmallArgs args)
{
    __shared__ __align__(16) float x[SMALL * SMALL_PITCH]; // [element][vector]
    const int tid = threadIdx.x, lane = tid & 63, wave = uniform(tid >> 6);
    const int batch = blockIdx.y, r = wave >> 2, c = wave & 3;
    const double scale = small_scale(args, batch);
    f32x4 acc = {0.f, 0.f, 0.f, 0.f};
    const int64_t first = (int64_t)blockIdx.x * args.chunk;
    for (int64_t j0 = first; j0 < min(first + args.chunk, (int64_t)args.lng); j0 += 64) {
        float v[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const int at = u * 1024 + tid, i = args.tall ? at & 63 : at >> 6, j = args.tall ? at >> 6 : at & 63;
            v[u] = small_x(args, batch, i, j0 + j, scale);
        }
        barrier_lds(); // the vectors before have been read
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const int at = u * 1024 + tid, i = args.tall ? at & 63 : at >> 6, j = args.tall ? at >> 6 : at & 63;
            x[i * SMALL_PITCH + j] = v[u];
        }
        barrier_lds();
        acc = small_product(x + r * 16 * SMALL_PITCH, x + c * 16 * SMALL_PITCH, 4, lane, acc);
    }
    float *const part = args.parts + ((int64_t)batch * args.chunks + blockIdx.x) * SMALL_MATRIX;
#pragma unroll
    for (int e = 0; e < 4; ++e)
        part[(r * 16 + (lane >> 4) * 4 + e) * SMALL + c * 16 + (lane & 15)] = acc[e];
}

// The chain of one matrix: A from the chunks' parts, then for each step b A + c A A, and A' = Q (Q A).
__global__ __launch_bounds__(1024) void small_chain_kernel(const SmallArgs args)
{
    __shared__ __align__(16) float A[SMALL * SMALL_PITCH], Q[SMALL * SMALL_PITCH], T[SMALL * SMALL_PITCH];
    const int tid = threadIdx.x, lane = tid & 63, wave = uniform(tid >> 6);
    const int batch = blockIdx.x, r = wave >> 2, c = wave & 3, blocks = (args.side + 15) / 16;
    const int col = c * 16 + (lane & 15), row = r * 16 + (lane >> 4) * 4;
    const float *const part = args.parts + (int64_t)batch * args.chunks * SMALL_MATRIX;
    float v[4] = {0.f, 0.f, 0.f, 0.f};
    const bool used = r * 16 < args.side && c * 16 < args.side; // blocks past the side are 0 and stay so
#pragma unroll 4
    for (int p = 0; p < args.chunks; ++p)
#pragma unroll
        for (int e = 0; e < 4; ++e)
            v[e] += part[p * SMALL_MATRIX + (row + e) * SMALL + col];
    // a lane's four results are of one column: they go to its row of the (symmetric) matrix
    const int at = col * SMALL_PITCH + row;
    *(f32x4 *)(A + at) = *(f32x4 *)v;
    const f32x4 zero = {0.f, 0.f, 0.f, 0.f};
    if (!used) {
        *(f32x4 *)(Q + at) = zero;
        *(f32x4 *)(T + at) = zero;
    }
    float *poly = args.polys + (int64_t)batch * args.steps * SMALL_MATRIX + row * SMALL + col;
    auto product = [&](const float *p, const float *q) { return small_product(p + r * 16 * SMALL_PITCH, q + c * 16 * SMALL_PITCH, blocks, lane, zero); };
    barrier_lds();
    for (int s = 0; s < args.steps; ++s, poly += SMALL_MATRIX) {
        if (used) {
            const f32x4 square = product(A, A), mine = *(const f32x4 *)(A + at);
            f32x4 q;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                q[e] = fmaf(args.c, square[e], args.b * mine[e]);
                poly[e * SMALL] = q[e];
                if (row + e == col)
                    q[e] += args.a;
            }
            *(f32x4 *)(Q + at) = q;
        }
        if (s + 1 == args.steps)
            return;
        barrier_lds();
        if (used)
            *(f32x4 *)(T + at) = product(Q, A);
        barrier_lds();
        if (used)
            *(f32x4 *)(A + at) = product(Q, T);
        barrier_lds();
    }
}

// 64 vectors of the long side through all the steps: four waves, 16 vectors each, X' = a X + (b A + c A A) X.
__global__ __launch_bounds__(256) void small_update_kernel(const SmallArgs args)
{
    __shared__ __align__(16) float x[SMALL * SMALL_PITCH]; // [vector][element]
    __shared__ __align__(16) float poly[SMALL * SMALL_PITCH];
    const int tid = threadIdx.x, lane = tid & 63, wave = uniform(tid >> 6);
    const int batch = blockIdx.y, blocks = (args.side + 15) / 16;
    const int64_t j0 = (int64_t)blockIdx.x * 64;
    const double scale = small_scale(args, batch);
    constexpr int EACH = SMALL * 64 / 256;
    float v[EACH];
#pragma unroll
    for (int u = 0; u < EACH; ++u) {
        const int at = u * 256 + tid, i = args.tall ? at & 63 : at >> 6, j = args.tall ? at >> 6 : at & 63;
        v[u] = small_x(args, batch, i, j0 + j, scale);
    }
#pragma unroll
    for (int u = 0; u < EACH; ++u) {
        const int at = u * 256 + tid, i = args.tall ? at & 63 : at >> 6, j = args.tall ? at >> 6 : at & 63;
        x[j * SMALL_PITCH + i] = v[u];
    }
    float *const mine = x + wave * 16 * SMALL_PITCH;
    // a step's polynomial is on its way while the step before it runs
    f32x4 p[4];
    const float *from = args.polys + (int64_t)batch * args.steps * SMALL_MATRIX + tid * 4;
    auto fetch = [&] {
#pragma unroll
        for (int u = 0; u < 4; ++u)
            if (u * 16 < args.side) // rows past the side are not written
                p[u] = *(const f32x4 *)(from + u * 1024);
        from += SMALL_MATRIX;
    };
    fetch();
    for (int s = 0; s < args.steps; ++s) {
        barrier_lds(); // the step before has been read
#pragma unroll
        for (int u = 0; u < 4; ++u)
            if (u * 16 < args.side) {
                const int i = u * 16 + tid / 16, k = tid % 16 * 4;
                *(f32x4 *)(poly + i * SMALL_PITCH + k) = k / 16 < blocks ? p[u] : f32x4{0.f, 0.f, 0.f, 0.f};
            }
        if (s + 1 < args.steps)
            fetch();
        barrier_lds();
        f32x4 acc[4];
        const int at = (lane & 15) * SMALL_PITCH + (lane >> 4) * 4; // of vector lane % 16, four elements of each block
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (i < blocks) {
                const f32x4 v = *(const f32x4 *)(mine + at + i * 16);
                acc[i] = small_product(poly + i * 16 * SMALL_PITCH, mine, blocks, lane, f32x4{args.a * v[0], args.a * v[1], args.a * v[2], args.a * v[3]});
            }
        wave_lds_exchange();
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (i < blocks)
                *(f32x4 *)(mine + at + i * 16) = acc[i];
        wave_lds_exchange();
    }
    barrier_lds();
    uint16_t *const out = args.out + batch * args.o_batch;
    for (int at = tid; at < SMALL * 64; at += 256) {
        const int i = args.tall ? at & 63 : at >> 6, j = args.tall ? at >> 6 : at & 63;
        if (i < args.side && j0 + j < args.lng) {
            const __bf16 v = (__bf16)x[j * SMALL_PITCH + i];
            out[args.tall ? (j0 + j) * args.ldo + i : i * args.ldo + j0 + j] = __builtin_bit_cast(uint16_t, v);
        }
    }
}

} // namespace pts
