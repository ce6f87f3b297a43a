// The weighted sum of each token's expert outputs, and its gradients.
//
//   out[t] = sum_j w[t][j] y[pos[t][j]]
//   dy[pos[t][j]] = w[t][j] dout[t],  dw[t][j] = <dout[t], y[pos[t][j]]>
//
// Sums run over ascending j in 32 bits. A position outside [0, rows) has no
// row: it adds nothing and its dw is 0; a position -2 - p with p a row (a slot
// the order put behind the last expert) makes row p of dy zero.
//
// Memory bound: y is read once in each direction, dy written once. 8192 tokens x
// 8 rows x 4096, bf16: the sum 119 us (5.1 TB/s; a large copy reaches 5.3), the
// gradients 238 us (4.8 TB/s); 16 tokens: 4.3 us, the latency of one pass.
#pragma once

#include "device/common.h"

namespace pts {

struct CombineArgs {
    const void *y;
    const float *weights;
    const int32_t *positions;
    const void *dout;   // backward only
    void *out;          // out, or dy
    float *dweights;    // backward only
    int64_t ldy, ld_out, ld_dout;
    int32_t m, n, top, rows;
    int32_t vec;        // all rows are 16-byte aligned
};

template <bool BF16> struct Piece { // 16 bytes of a row
    static constexpr int N = BF16 ? 8 : 4;
    float v[N];
    // ONCE: past the caches, for what is read once.
    template <bool ONCE = true> __device__ __forceinline__ void load(const void *p, int64_t at, int valid, bool vec)
    {
        if (vec && valid >= N) {
            const u32x4 *const from = (const u32x4 *)((const uint8_t *)p + at * (BF16 ? 2 : 4));
            if constexpr (ONCE)
                set(__builtin_nontemporal_load(from));
            else
                set(*from);
            return;
        }
#pragma unroll
        for (int i = 0; i < N; ++i) {
            v[i] = 0.f;
            if (i < valid)
                v[i] = BF16 ? __uint_as_float((uint32_t)((const uint16_t *)p)[at + i] << 16) : ((const float *)p)[at + i];
        }
    }
    __device__ __forceinline__ void set(u32x4 w)
    {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if constexpr (BF16) {
                v[2 * i] = __uint_as_float(w[i] << 16);
                v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
            } else {
                v[i] = __uint_as_float(w[i]);
            }
        }
    }
    __device__ __forceinline__ void store(void *p, int64_t at, int valid, bool vec) const
    {
        if (vec && valid >= N) {
            u32x4 w;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if constexpr (BF16) {
                    const bf16x2 h = {(__bf16)v[2 * i], (__bf16)v[2 * i + 1]};
                    w[i] = __builtin_bit_cast(uint32_t, h);
                } else {
                    w[i] = __float_as_uint(v[i]);
                }
            }
            __builtin_nontemporal_store(w, (u32x4 *)((uint8_t *)p + at * (BF16 ? 2 : 4)));
            return;
        }
#pragma unroll
        for (int i = 0; i < N; ++i)
            if (i < valid) {
                if constexpr (BF16)
                    ((__bf16 *)p)[at + i] = (__bf16)v[i];
                else
                    ((float *)p)[at + i] = v[i];
            }
    }
};

// Rows in flight per thread: with 8 both directions take 6% longer at that size,
// with 2 the sum 1% and the gradients 6%.
constexpr int COMBINE_UNROLL = 4;

// One token's strip of 256 pieces per workgroup.
template <bool BF16>
__global__ __launch_bounds__(256) void combine_kernel(const CombineArgs args)
{
    using P = Piece<BF16>;
    const int64_t token = blockIdx.x;
    const int col = (blockIdx.y * 256 + threadIdx.x) * P::N, valid = args.n - col;
    if (valid <= 0)
        return;
    float sum[P::N];
#pragma unroll
    for (int i = 0; i < P::N; ++i)
        sum[i] = 0.f;
    for (int j0 = 0; j0 < args.top; j0 += COMBINE_UNROLL) {
        P y[COMBINE_UNROLL];
        float w[COMBINE_UNROLL];
        bool have[COMBINE_UNROLL];
#pragma unroll
        for (int u = 0; u < COMBINE_UNROLL; ++u) {
            const int j = min(j0 + u, args.top - 1);
            const int pos = args.positions[token * args.top + j];
            have[u] = j0 + u < args.top && pos >= 0 && pos < args.rows;
            w[u] = args.weights[token * args.top + j];
            if (have[u])
                y[u].load(args.y, pos * args.ldy + col, valid, args.vec);
        }
#pragma unroll
        for (int u = 0; u < COMBINE_UNROLL; ++u)
            if (have[u]) {
#pragma unroll
                for (int i = 0; i < P::N; ++i)
                    sum[i] = fmaf(w[u], y[u].v[i], sum[i]);
            }
    }
    P out;
#pragma unroll
    for (int i = 0; i < P::N; ++i)
        out.v[i] = sum[i];
    out.store(args.out, token * args.ld_out + col, valid, args.vec);
}

// Both gradients, one token per workgroup: a strip of dout stays in registers
// while the token's rows of y pass by and its rows of dy are written.
template <bool BF16>
__global__ __launch_bounds__(256) void combine_backward_kernel(const CombineArgs args)
{
    using P = Piece<BF16>;
    __shared__ float part[4][COMBINE_UNROLL];
    const int64_t token = blockIdx.x;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    for (int j0 = 0; j0 < args.top; j0 += COMBINE_UNROLL) {
        float dot[COMBINE_UNROLL], w[COMBINE_UNROLL];
        int pos[COMBINE_UNROLL];
#pragma unroll
        for (int u = 0; u < COMBINE_UNROLL; ++u) {
            const int j = min(j0 + u, args.top - 1);
            pos[u] = j0 + u < args.top ? args.positions[token * args.top + j] : -1;
            w[u] = args.weights[token * args.top + j];
            if (pos[u] < -1) { // a row behind the last expert: no weight
                pos[u] = -2 - pos[u];
                w[u] = 0.f;
                dot[u] = 1.f; // marks it until the sums start
            } else {
                dot[u] = 0.f;
            }
            if (pos[u] >= args.rows)
                pos[u] = -1;
        }
        bool dropped[COMBINE_UNROLL];
#pragma unroll
        for (int u = 0; u < COMBINE_UNROLL; ++u) {
            dropped[u] = dot[u] != 0.f;
            dot[u] = 0.f;
        }
        for (int col = threadIdx.x * P::N; col < args.n; col += 256 * P::N) {
            const int valid = args.n - col;
            P d, y[COMBINE_UNROLL];
            d.template load<false>(args.dout, token * args.ld_dout + col, valid, args.vec);
#pragma unroll
            for (int u = 0; u < COMBINE_UNROLL; ++u)
                if (pos[u] >= 0 && !dropped[u])
                    y[u].load(args.y, pos[u] * args.ldy + col, valid, args.vec);
#pragma unroll
            for (int u = 0; u < COMBINE_UNROLL; ++u) {
                if (pos[u] < 0)
                    continue;
                P g;
#pragma unroll
                for (int i = 0; i < P::N; ++i) {
                    if (!dropped[u])
                        dot[u] = fmaf(d.v[i], y[u].v[i], dot[u]);
                    g.v[i] = dropped[u] ? 0.f : w[u] * d.v[i];
                }
                g.store(args.out, pos[u] * args.ld_out + col, valid, args.vec);
            }
        }
#pragma unroll
        for (int u = 0; u < COMBINE_UNROLL; ++u)
#pragma unroll
            for (int s = 32; s > 0; s /= 2)
                dot[u] += __shfl_xor(dot[u], s);
        __syncthreads();
        if (lane == 0)
#pragma unroll
            for (int u = 0; u < COMBINE_UNROLL; ++u)
                part[wave][u] = dot[u];
        __syncthreads();
        if (threadIdx.x < COMBINE_UNROLL && j0 + threadIdx.x < args.top)
            args.dweights[token * args.top + j0 + threadIdx.x] =
                (part[0][threadIdx.x] + part[1][threadIdx.x]) + (part[2][threadIdx.x] + part[3][threadIdx.x]);
    }
}

} // namespace pts
