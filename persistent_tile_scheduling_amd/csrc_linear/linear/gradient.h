// The gradient of a linear layer's sums, and their column sums (the bias's).
#pragma once

#include "linear/epilogue.h"

namespace pts {

struct SlopeArgs {
    const uint16_t *dy, *z; // z null: no activation, dz is dy
    uint16_t *dz;           // null: not written
    float *sums;            // [row blocks][sums_ld], or null
    int64_t ld_dy, ldz, ld_dz, sums_ld;
    int32_t m, n, act, rows; // rows per workgroup
};

// dz = dy act'(z), rounded to bf16 (the matrix unit's type), and the sums of its
// columns over the workgroup's rows from the unrounded values. Sixteen threads
// side by side have 8 columns each, HIGH groups of them every HIGH-th row: memory
// bound, one pass.
template <int ACT, int HIGH> __device__ __forceinline__ void slope_rows(const SlopeArgs &args, int col, int row0, int end, float (&sum)[8])
{
    for (int row = row0; row < end; row += HIGH) { // rows start at whole 16 bytes and are read in whole pieces
        float d[8];
        get8(args.dy + row * args.ld_dy + col, d, 8, true);
        if constexpr (ACT != ACT_NONE) {
            float z[8];
            get8(args.z + row * args.ldz + col, z, 8, true);
#pragma unroll
            for (int i = 0; i < 8; ++i)
                d[i] *= activation_slope<ACT>(z[i]);
        }
        if (args.dz != nullptr)
            *(u32x4 *)(args.dz + row * args.ld_dz + col) = to_bf16(d);
#pragma unroll
        for (int i = 0; i < 8; ++i)
            sum[i] += d[i];
    }
}

template <int HIGH>
__global__ __launch_bounds__(16 * HIGH) void slope_kernel(const SlopeArgs args)
{
    __shared__ __align__(16) float part[HIGH][128 + 4];
    const int tid = threadIdx.x, x = tid & 15, y = tid >> 4;
    const int col = blockIdx.x * 128 + x * 8;
    const int row0 = blockIdx.y * args.rows, end = row0 + min(args.rows, args.m - row0); // row0 + rows can pass 2^31
    float sum[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    if (col < args.n)
        with_activation(args.act, [&](auto act) { slope_rows<decltype(act)::value, HIGH>(args, col, row0 + y, end, sum); });
    if (args.sums == nullptr)
        return;
    *(f32x4 *)&part[y][x * 8] = *(f32x4 *)sum;
    *(f32x4 *)&part[y][x * 8 + 4] = *(f32x4 *)(sum + 4);
    barrier_lds();
    const int c = blockIdx.x * 128 + tid;
    if (tid < 128 && c < args.n) {
        float s = 0.f;
#pragma unroll 16
        for (int i = 0; i < HIGH; ++i)
            s += part[i][tid];
        args.sums[blockIdx.y * args.sums_ld + c] = s;
    }
}

struct SumArgs {
    const float *sums;
    float *out;
    int64_t sums_ld;
    int32_t n, blocks;
};

// out[c] = the sum of the row blocks' sums: 64 columns per workgroup, sixteen
// threads for each, then their sums in order.
__global__ __launch_bounds__(1024) void sum_kernel(const SumArgs args)
{
    __shared__ float part[16][64];
    const int x = threadIdx.x & 63, y = threadIdx.x >> 6;
    const int c = blockIdx.x * 64 + x;
    float s = 0.f;
    if (c < args.n) {
#pragma unroll 4
        for (int b = y; b < args.blocks; b += 16)
            s += args.sums[b * args.sums_ld + c];
    }
    part[y][x] = s;
    barrier_lds();
    if (y == 0 && c < args.n) {
        s = 0.f;
#pragma unroll
        for (int i = 0; i < 16; ++i)
            s += part[i][x];
        args.out[c] = s;
    }
}

} // namespace pts
