// A linear layer over few rows: each byte of the weight is used by one workgroup
// only, so it goes straight from memory to the registers of the matrix unit.
//
// A workgroup has 16 NB columns (rows of the weight) and up to 16 MB rows of x. Its
// waves take the blocks of 64 k in turn, U blocks at a time, independent streams
// of loads; their sums are added in wave order through LDS. Which NB, U and waves,
// and when several workgroups share a strip's k, stands with the choice.
#pragma once

#include "linear/epilogue.h"

namespace pts {

// Partial sums of split rows: [split][m][rows_pitch(n)].
__host__ __device__ inline int64_t rows_pitch(int64_t n) { return (n + 7) / 8 * 8; }

template <int MB, int NB, int U, int WAVES, class Epilogue>
__global__ __launch_bounds__(64 * WAVES) void rows_kernel(const TileArgs args, const typename Epilogue::Args epi)
{
    constexpr int WIDE = 16 * NB;
    __shared__ __align__(16) float part[WAVES][MB * 16][WIDE];
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = uniform(tid >> 6);
    const int l16 = lane & 15, g = lane >> 4;
    const int col0 = blockIdx.x * WIDE, split = blockIdx.y;
    const int all = (args.k + 63) / 64;
    const int first = split * args.split_k, end = min(first + args.split_k, all);
    const uint16_t *b[NB], *a[MB];
#pragma unroll
    for (int j = 0; j < NB; ++j)
        b[j] = args.b + (int64_t)min(col0 + j * 16 + l16, args.n - 1) * args.ldb;
#pragma unroll
    for (int i = 0; i < MB; ++i)
        a[i] = args.a + (int64_t)min(i * 16 + l16, args.m - 1) * args.lda;
    f32x4 acc[MB][NB];
#pragma unroll
    for (int i = 0; i < MB; ++i)
#pragma unroll
        for (int j = 0; j < NB; ++j)
            acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
    for (int k0 = first + wave; k0 < end; k0 += WAVES * U) {
        u32x4 x[U][NB][2], y[U][MB][2];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int kb = min(k0 + u * WAVES, end - 1); // past the end: read again, not used
            const int last = min(7, (args.k - kb * 64 - 1) / 8);
            const int64_t lo = (int64_t)kb * 64 + min(g, last) * 8, hi = (int64_t)kb * 64 + min(g + 4, last) * 8;
#pragma unroll
            for (int j = 0; j < NB; ++j) {
                x[u][j][0] = __builtin_nontemporal_load((const u32x4 *)(b[j] + lo));
                x[u][j][1] = __builtin_nontemporal_load((const u32x4 *)(b[j] + hi));
            }
#pragma unroll
            for (int i = 0; i < MB; ++i) {
                y[u][i][0] = *(const u32x4 *)(a[i] + lo);
                y[u][i][1] = *(const u32x4 *)(a[i] + hi);
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int kb = k0 + u * WAVES;
            if (kb >= end)
                break;
            const int left = args.k - kb * 64;
            if (left < 64) { // what lies past the end of the rows is cleared in both operands
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const int have = left - (g + 4 * h) * 8 - 2 * e;
                        const uint32_t mask = have >= 2 ? 0xFFFFFFFFu : have == 1 ? 0xFFFFu : 0u;
#pragma unroll
                        for (int j = 0; j < NB; ++j)
                            x[u][j][h][e] &= mask;
#pragma unroll
                        for (int i = 0; i < MB; ++i)
                            y[u][i][h][e] &= mask;
                    }
            }
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int i = 0; i < MB; ++i)
#pragma unroll
                    for (int j = 0; j < NB; ++j)
                        acc[i][j] = Bf16::mfma(x[u][j][h], y[u][i][h], acc[i][j]);
        }
    }
#pragma unroll
    for (int i = 0; i < MB; ++i)
#pragma unroll
        for (int j = 0; j < NB; ++j)
            *(f32x4 *)&part[wave][i * 16 + l16][j * 16 + g * 4] = acc[i][j];
    barrier_lds();
    for (int at = tid; at < MB * 16 * 2 * NB; at += 64 * WAVES) {
        const int row = at / (2 * NB), c = at % (2 * NB) * 8, valid = args.n - col0 - c;
        if (row >= args.m || valid <= 0)
            continue;
        float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int w = 0; w < WAVES; ++w) {
            const f32x4 lo = *(const f32x4 *)&part[w][row][c], hi = *(const f32x4 *)&part[w][row][c + 4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                v[i] += lo[i];
                v[4 + i] += hi[i];
            }
        }
        if (args.splits > 1) {
            float *const p = args.part + ((int64_t)split * args.m + row) * rows_pitch(args.n) + col0 + c;
            *(f32x4 *)p = *(f32x4 *)v;
            *(f32x4 *)(p + 4) = *(f32x4 *)(v + 4);
            continue;
        }
        Epilogue::run(epi, [&](auto e) {
            Raw8 r;
            e.fetch(epi, 0, row, col0 + c, valid, r);
            e.finish(epi, e.start(epi, 0, col0 + c, valid), r, 0, row, col0 + c, valid, v);
        });
    }
}

// The sum of the splits' sums, in their order, and the epilogue: eight columns per thread.
template <class Epilogue>
__global__ __launch_bounds__(256) void rows_join_kernel(const TileArgs args, const typename Epilogue::Args epi)
{
    const int pieces = (args.n + 7) / 8;
    const int64_t at = (int64_t)blockIdx.x * 256 + threadIdx.x;
    const int row = (int)(at / pieces), col = (int)(at - (int64_t)row * pieces) * 8;
    if (row >= args.m)
        return;
    const float *p = args.part + row * rows_pitch(args.n) + col;
    float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    for (int s = 0; s < args.splits; ++s, p += args.m * rows_pitch(args.n)) {
        const f32x4 lo = *(const f32x4 *)p, hi = *(const f32x4 *)(p + 4);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[i] += lo[i];
            v[4 + i] += hi[i];
        }
    }
    const int valid = args.n - col;
    Epilogue::run(epi, [&](auto e) {
        Raw8 r;
        e.fetch(epi, 0, row, col, valid, r);
        e.finish(epi, e.start(epi, 0, col, valid), r, 0, row, col, valid, v);
    });
}

} // namespace pts
