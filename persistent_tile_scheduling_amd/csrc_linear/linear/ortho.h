// Orthogonalising a matrix by Newton-Schulz steps:
//
//   X0 = x / (|x|_F + eps)
//   A = X X^T,  B = b A + c A A,  X' = a X + B X      (rows <= columns)
//   A = X^T X,  B = b A + c A A,  X' = a X + X B      (otherwise)
//
// each of which applies p(s) = a s + b s^3 + c s^5 to the singular values.
//
// Precision. The products' operands are fp16 (11 bits, at bf16's rate), scaled by
// powers of two into its range; sums are fp32. For the term a X, X has 8 bits more
// beside its fp16 form, what that is short of it in e4m3: small singular values
// grow 3.4-fold a step, and a rounding of X would grow with them where X has none.
// In the last step it no longer would. Against 64 bits, five steps, 512 x 512, on
// normal data and on rank 32: bf16 throughout 1.0e-2 and 0.22 of the result, fp16
// throughout 1.3e-3 and 2.8e-2, with the rest of X in fp32 1.5e-3 and 5.8e-4, this
// form 1.4e-3 and 1.0e-3. The rest costs a byte read and written per element and
// step, where fp32 beside fp16 took four: the update of 12 matrices of 1024 x 4096
// is bound by memory.
#pragma once

#include "linear/epilogue.h"

namespace pts {

constexpr float ORTHO_SX = 1024.f; // X entries in fp16, times this (at most 8 before it)
constexpr float ORTHO_SA = 256.f;  // A and B entries
// The rest of an X entry is at most half a step of fp16: 1/2 for entries below 2 (2048 with ORTHO_SX), times this 256, within
// e4m3's 448. Of larger entries, which only coefficients that take singular values past 2 make, it is cut off there: up to 1/8
// (entries up to 4) or 9/16 (up to 8) of the half step stay missing. Scales that keep it whole (512, 256 for ORTHO_SX) gave
// the same errors to two digits in a simulation of such coefficients: the operands' own roundings are larger.
constexpr float ORTHO_SR = 512.f;

typedef float f32x2 __attribute__((ext_vector_type(2)));

struct OrthoArgs {
    const void *r;          // added times beta: null, a matrix of the library's (fp16), or x itself
    const uint8_t *r_rest;  // with fp16: what it is short of its value, or null
    const double *r_scale;  // x: 1 / (|x|_F + eps), one per matrix
    uint16_t *half;         // results, those that are not null: in fp16 times half_scale,
    uint8_t *rest;          //   what that is short of its value (e4m3, times ORTHO_SR more; laid out as half),
    uint16_t *out;          //   in bf16
    int64_t ldr, ldh, ldo;
    int64_t r_batch, h_batch, o_batch;
    float alpha, beta, half_scale;
    int32_t r_type, r_whole, o_whole;
};
enum : int { R_NONE = 0, R_F16 = 1, R_F32 = 2, R_BF16 = 3 };

__device__ __forceinline__ u32x4 to_f16(const float (&v)[8], float scale)
{
    u32x4 w;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
        w[i] = __builtin_bit_cast(uint32_t, f16x2{(_Float16)(v[2 * i] * scale), (_Float16)(v[2 * i + 1] * scale)});
    }
    return w;
}

// v = alpha sum + beta R, to the results asked for. The library's own matrices have rows of whole 16 bytes, written
// whole.
struct OrthoStore {
    static constexpr bool MIRROR = true;
    using Raw = Raw8;
    struct Start {};
    static __device__ __forceinline__ Start start(const OrthoArgs &, int, int, int) { return {}; }
    static __device__ __forceinline__ void fetch(const OrthoArgs &args, int batch, int row, int col, int valid, Raw8 &r)
    {
        const int64_t at = batch * args.r_batch + row * args.ldr + col;
        if (args.r_type == R_F16) {
            fetch8<false>(r, args.r, at);
            if (args.r_rest != nullptr) {
                const u32x2 w = *(const u32x2 *)(args.r_rest + at);
                r.hi[0] = w[0];
                r.hi[1] = w[1];
            }
        } else if (args.r_type == R_F32 && args.r_whole && valid >= 8)
            fetch8<true>(r, args.r, at);
        else if (args.r_type == R_BF16 && args.r_whole && valid >= 8)
            fetch8<false>(r, args.r, at);
    }
    static __device__ __forceinline__ void finish(const OrthoArgs &args, const Start &, const Raw8 &fetched, int batch, int row,
                                                  int col, int valid, float (&v)[8])
    {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            v[i] *= args.alpha;
        if (args.r_type != R_NONE) {
            float r[8];
            const int64_t at = batch * args.r_batch + row * args.ldr + col;
            const bool ahead = args.r_whole && valid >= 8;
            if (args.r_type == R_F16) {
                const f16x8 h = __builtin_bit_cast(f16x8, fetched.lo);
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    r[i] = (float)h[i];
                if (args.r_rest != nullptr) {
#pragma unroll
                    for (int i = 0; i < 8; i += 2) {
                        const f32x2 d = i & 2 ? __builtin_amdgcn_cvt_pk_f32_fp8((int)fetched.hi[i / 4], true)
                                              : __builtin_amdgcn_cvt_pk_f32_fp8((int)fetched.hi[i / 4], false);
                        r[i] = fmaf(d[0], 1.f / ORTHO_SR, r[i]);
                        r[i + 1] = fmaf(d[1], 1.f / ORTHO_SR, r[i + 1]);
                    }
                }
            } else if (args.r_type == R_F32) {
                if (ahead)
                    from_f32(fetched, r);
                else
                    get8((const float *)args.r + at, r, valid, false);
            } else {
                if (ahead)
                    from_bf16(fetched.lo, r);
                else
                    get8((const uint16_t *)args.r + at, r, valid, false);
            }
            if (args.r_scale != nullptr) {
                const double s = args.r_scale[batch];
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    r[i] = (float)((double)r[i] * s);
            }
#pragma unroll
            for (int i = 0; i < 8; ++i)
                v[i] = fmaf(args.beta, r[i], v[i]);
        }
        if (args.half != nullptr) {
            const int64_t at = batch * args.h_batch + row * args.ldh + col;
            const u32x4 w = to_f16(v, args.half_scale);
            *(u32x4 *)(args.half + at) = w;
            if (args.rest != nullptr) {
                const f16x8 h = __builtin_bit_cast(f16x8, w);
                int word[2] = {0, 0};
#pragma unroll
                for (int i = 0; i < 8; i += 2) {
                    float d[2];
#pragma unroll
                    for (int j = 0; j < 2; ++j)
                        d[j] = fminf(fmaxf(fmaf(v[i + j], args.half_scale, -(float)h[i + j]) * ORTHO_SR, -448.f), 448.f);
                    word[i / 4] = i & 2 ? __builtin_amdgcn_cvt_pk_fp8_f32(d[0], d[1], word[i / 4], true)
                                        : __builtin_amdgcn_cvt_pk_fp8_f32(d[0], d[1], word[i / 4], false);
                }
                *(u32x2 *)(args.rest + at) = u32x2{(uint32_t)word[0], (uint32_t)word[1]};
            }
        }
        if (args.out != nullptr)
            put8(args.out + batch * args.o_batch + row * args.ldo + col, to_bf16(v), valid, args.o_whole);
    }
    // The reflected result: rows row .. row + 7 of column col, as columns of row col.
    static __device__ __forceinline__ void mirror(const OrthoArgs &args, int batch, int row, int col, const float (&v)[8])
    {
        *(u32x4 *)(args.half + batch * args.h_batch + col * args.ldh + row) = to_f16(v, args.half_scale);
    }
};
struct OrthoEpilogue {
    using Args = OrthoArgs;
    template <class F> static __device__ __forceinline__ void run(const Args &, F &&f) { f(OrthoStore{}); }
};

struct NormArgs {
    const void *x;
    double *sums;    // [batch][blocks]: squares, summed
    double *scale;   // [batch]
    uint16_t *half;  // X0 in fp16
    int64_t ldx, x_batch, ldh, h_batch;
    double eps;
    int32_t rows, cols, f32, whole, blocks;
};

template <class F> __device__ __forceinline__ void each_piece(const NormArgs &args, F &&f)
{
    const int pieces = (args.cols + 7) / 8, batch = blockIdx.y;
    const int64_t all = (int64_t)args.rows * pieces;
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < all; i += (int64_t)gridDim.x * 256) {
        const int64_t row = i / pieces;
        const int col = (int)(i - row * pieces) * 8;
        const int64_t at = batch * args.x_batch + row * args.ldx + col;
        float v[8];
        if (args.f32)
            get8((const float *)args.x + at, v, args.cols - col, args.whole);
        else
            get8((const uint16_t *)args.x + at, v, args.cols - col, args.whole);
        f(row, col, v);
    }
}

// 1 / (|x|_F + eps); 0 for a matrix of zeros, since 1 / eps may be infinite (and then 0 / eps is NaN).
__device__ __forceinline__ double norm_scale(double squares, double eps) { return squares == 0.0 ? 0.0 : 1.0 / (sqrt(squares) + eps); }

// The sum of v over the workgroup's 256 threads, in every thread.
__device__ __forceinline__ double sum256(double v, double *part)
{
#pragma unroll
    for (int d = 32; d > 0; d /= 2)
        v += __shfl_xor(v, d);
    if ((threadIdx.x & 63) == 0)
        part[threadIdx.x >> 6] = v;
    barrier_lds();
    return (part[0] + part[1]) + (part[2] + part[3]);
}

// Squares in 64 bits: no input's square overflows or vanishes.
__global__ __launch_bounds__(256) void norm_kernel(const NormArgs args)
{
    __shared__ double part[4];
    double sum = 0.0;
    each_piece(args, [&](int64_t, int, const float(&v)[8]) {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            sum = fma((double)v[i], (double)v[i], sum);
    });
    sum = sum256(sum, part);
    if (threadIdx.x == 0)
        args.sums[(int64_t)blockIdx.y * args.blocks + blockIdx.x] = sum;
}

__global__ __launch_bounds__(256) void start_kernel(const NormArgs args)
{
    __shared__ double part[4];
    const double *const sums = args.sums + (int64_t)blockIdx.y * args.blocks;
    const double sum = sum256((int)threadIdx.x < args.blocks ? sums[threadIdx.x] : 0.0, part);
    const double scale = norm_scale(sum, args.eps);
    if (blockIdx.x == 0 && threadIdx.x == 0)
        args.scale[blockIdx.y] = scale;
    each_piece(args, [&](int64_t row, int col, const float(&v)[8]) {
        float x[8];
#pragma unroll
        for (int i = 0; i < 8; ++i)
            x[i] = (float)((double)v[i] * scale);
        *(u32x4 *)(args.half + blockIdx.y * args.h_batch + row * args.ldh + col) = to_f16(x, ORTHO_SX);
    });
}

} // namespace pts
