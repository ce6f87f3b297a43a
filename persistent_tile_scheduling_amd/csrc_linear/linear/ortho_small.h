// Newton-Schulz steps of matrices whose short side is at most 64 (ortho.h has the
// formulas): several steps in three launches.
//
// The Gram matrix follows the steps without the matrix: with Q = a + b A + c A A,
// X' = Q X gives A' = Q A Q, and all of them commute. So one workgroup per matrix
// runs the chain of 64 x 64 products in LDS and leaves each step's b A + c A A;
// then every workgroup takes 64 of the long side's vectors through these steps,
// in fp32. Beyond 64 a chain in LDS would grow with the cube of the side and lose.
//
// What the chain cannot do is see X again. An error of A in a direction of small
// singular values grows by up to a^2 a step (12-fold by the default), where the
// error of a Gram matrix made from X stays what it is, and an eigenvalue that has
// become negative runs away: in fp32 ten steps of a matrix of rank 5 come to 1e23.
// What makes A unsymmetric grows faster still (28-fold), so every product is made
// on and above the diagonal and its values written to both sides. And the Gram
// matrix and the chain are of 64 bits, which leaves the growth 29 bits more, and a
// chain ends, with X written in fp32 and its Gram matrix made anew, before that is
// used up (chain_steps): after eight steps by the default. Against 64-bit steps
// this form is as near as fp32 steps that make A from X each time, for any number
// of steps and whatever the matrix's condition.
//
// Five steps of 16 x 16 take 19 us, of 64 x 2000 57, of 32 matrices of 64 x 500 60
// (a product's launches for each, and the joins of split ones: 75, 104 and 134; a
// chain in fp32, which did not hold: 17, 48 and 50). Of 64 x 2000 the chain, whose
// products are one compute unit's at the matrix unit's rate for 64 bits, takes 31 us
// of the kernels' 58, the update 18.
#pragma once

#include "linear/ortho.h"

namespace pts {

constexpr int SMALL = 64;          // the longest short side
constexpr int SMALL_PITCH = 68;    // floats of an LDS row: sixteen rows' 16-byte pieces lie in different banks
constexpr int SMALL_MATRIX = SMALL * SMALL;

typedef double f64x2 __attribute__((ext_vector_type(2)));
typedef double f64x4 __attribute__((ext_vector_type(4)));

struct SmallArgs {
    NormArgs norm;      // x and its norm, or X as the chain before left it
    double *parts;      // [matrix][chunk][block][lane][4]: Gram matrices of chunks of the long side, 16 x 16 blocks on and
                        //   above the diagonal as the matrix unit leaves them
    float *polys;       // [matrix][step][64][64]: b A + c A A
    float *mid;         // X for the next chain, rows x cols each (it may be norm.x), or null: the last steps
    uint16_t *out;
    int64_t ldo, o_batch;
    float a, b, c;
    int32_t scaled;     // norm.x is X already
    int32_t tall, side, lng, chunks, chunk, steps; // chunk: vectors each, a multiple of 64; steps: of this chain
};

__device__ __forceinline__ double small_scale(const SmallArgs &args, int batch)
{
    if (args.scaled)
        return 1.0;
    const int lane = threadIdx.x & 63; // at most 64 blocks
    double sum = lane < args.norm.blocks ? args.norm.sums[(int64_t)batch * args.norm.blocks + lane] : 0.0;
#pragma unroll
    for (int d = 32; d > 0; d /= 2)
        sum += __shfl_xor(sum, d);
    return norm_scale(sum, args.norm.eps);
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

// The same in 64 bits, of fp32 or fp64 rows. Its instruction's results of lane l are rows l / 16 + 4 v, so the lane with
// row i of p is given row 4 (i % 4) + i / 4, which makes them rows 4 (l / 16) + v.
__device__ __forceinline__ f64x4 four(const float *p)
{
    const f32x4 v = *(const f32x4 *)p;
    return f64x4{(double)v[0], (double)v[1], (double)v[2], (double)v[3]};
}
__device__ __forceinline__ f64x4 four(const double *p)
{
    const f64x2 lo = *(const f64x2 *)p, hi = *(const f64x2 *)(p + 2);
    return f64x4{lo[0], lo[1], hi[0], hi[1]};
}
template <int PITCH, class T>
__device__ __forceinline__ f64x4 small_product64(const T *p, const T *q, int blocks, int lane)
{
    const int l16 = lane & 15, at = (lane >> 4) * 4;
    p += ((l16 & 3) * 4 + (l16 >> 2)) * PITCH + at;
    q += l16 * PITCH + at;
    f64x4 acc = {0.0, 0.0, 0.0, 0.0};
#pragma unroll
    for (int k = 0; k < SMALL; k += 16) {
        if (k >= blocks * 16)
            break;
        const f64x4 x = four(p + k), y = four(q + k);
#pragma unroll
        for (int e = 0; e < 4; ++e)
            acc = __builtin_amdgcn_mfma_f64_16x16x4f64(x[e], y[e], acc, 0, 0, 0);
    }
    return acc;
}

// Block `t` on or above the diagonal: (0, 0); (0, 1), (1, 1); (0, 2), ..; how many there are up to a side.
__device__ __forceinline__ void small_block(int t, int &r, int &c)
{
    c = t < 1 ? 0 : t < 3 ? 1 : t < 6 ? 2 : 3;
    r = t - c * (c + 1) / 2;
}
__host__ __device__ inline int small_blocks(int side)
{
    const int n = (side + 15) / 16;
    return n * (n + 1) / 2;
}

// The Gram matrix of one chunk of the long side: a wave for each of up to ten blocks.
__global__ __launch_bounds__(1024) void small_gram_kernel(const SmallArgs args)
{
    __shared__ __align__(16) float x[SMALL * SMALL_PITCH]; // [element][vector]
    const int tid = threadIdx.x, lane = tid & 63, wave = uniform(tid >> 6);
    const int batch = blockIdx.y, blocks = small_blocks(args.side);
    int r, c;
    small_block(wave, r, c);
    const double scale = small_scale(args, batch);
    f64x4 acc = {0.0, 0.0, 0.0, 0.0};
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
        if (wave < blocks)
            acc += small_product64<SMALL_PITCH>(x + r * 16 * SMALL_PITCH, x + c * 16 * SMALL_PITCH, 4, lane);
    }
    if (wave >= blocks)
        return;
    double *const part = args.parts + ((((int64_t)batch * args.chunks + blockIdx.x) * blocks + wave) * 64 + lane) * 4;
    *(f64x2 *)part = f64x2{acc[0], acc[1]};
    *(f64x2 *)(part + 2) = f64x2{acc[2], acc[3]};
}

// The chain of one matrix: A from the chunks' parts, then for each step b A + c A A, and A' = Q (Q A). A wave has a block
// on or above the diagonal; a lane's four results are of one column.
__global__ __launch_bounds__(640) void small_chain_kernel(const SmallArgs args)
{
    constexpr int PITCH = SMALL + 2; // sixteen rows' 16-byte pieces lie in different banks
    __shared__ __align__(16) double A[SMALL * PITCH], Q[SMALL * PITCH], T[SMALL * PITCH];
    const int tid = threadIdx.x, lane = tid & 63, wave = uniform(tid >> 6);
    const int batch = blockIdx.x, high = (args.side + 15) / 16, blocks = small_blocks(args.side);
    int r, c;
    small_block(wave, r, c);
    const int col = c * 16 + (lane & 15), row = r * 16 + (lane >> 4) * 4;
    const bool used = wave < blocks;
    // v to its place and to the reflected one
    auto put = [&](auto *m, int pitch, const auto &v) {
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if (r < c || row + e <= col)
                m[(row + e) * pitch + col] = m[col * pitch + row + e] = v[e];
    };
    auto product = [&](const double *p, const double *q) {
        return small_product64<PITCH>(p + r * 16 * PITCH, q + c * 16 * PITCH, high, lane);
    };
    if (used) {
        const double *part = args.parts + (((int64_t)batch * args.chunks * blocks + wave) * 64 + lane) * 4;
        f64x4 v = {0.0, 0.0, 0.0, 0.0};
#pragma unroll 8
        for (int p = 0; p < args.chunks; ++p)
            v += four(part + p * blocks * 256);
        put(A, PITCH, v);
    }
    float *poly = args.polys + (int64_t)batch * args.steps * SMALL_MATRIX;
    barrier_lds();
    for (int s = 0; s < args.steps; ++s, poly += SMALL_MATRIX) {
        if (used) {
            const f64x4 square = product(A, A), mine = four(A + col * PITCH + row);
            f64x4 q;
            f32x4 p;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                q[e] = fma((double)args.c, square[e], (double)args.b * mine[e]);
                p[e] = (float)q[e]; // X's products are of 32 bits
                if (row + e == col)
                    q[e] += (double)args.a;
            }
            put(poly, SMALL, p);
            put(Q, PITCH, q);
        }
        if (s + 1 == args.steps)
            return;
        barrier_lds();
        if (used)
            put(T, PITCH, product(Q, A));
        barrier_lds();
        if (used)
            put(A, PITCH, product(Q, T));
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
    const int64_t mid = batch * ((int64_t)args.norm.rows * args.norm.cols);
    uint16_t *const out = args.out + batch * args.o_batch;
    for (int at = tid; at < SMALL * 64; at += 256) {
        const int i = args.tall ? at & 63 : at >> 6, j = args.tall ? at >> 6 : at & 63;
        if (i < args.side && j0 + j < args.lng) {
            const float v = x[j * SMALL_PITCH + i];
            if (args.mid != nullptr)
                args.mid[mid + (args.tall ? (j0 + j) * args.side + i : (int64_t)i * args.lng + j0 + j)] = v;
            else
                out[args.tall ? (j0 + j) * args.ldo + i : i * args.ldo + j0 + j] = __builtin_bit_cast(uint16_t, (__bf16)v);
        }
    }
}

} // namespace pts
