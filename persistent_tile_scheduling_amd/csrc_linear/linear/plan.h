// Which tiles a 16-bit product takes, and over how many workgroups its
// contraction is split. Host side.
#pragma once

#include <algorithm>
#include <climits>

#include "host_launch.h"
#include "linear/tile.h"

namespace pts {

constexpr int64_t UNITS = 256; // compute units of the card: the choice, and with it every bit of a result, depends on sizes alone
constexpr int64_t MAX_EXTENT = INT32_MAX - 1024; // extents are rounded up to whole tiles in 32 bits

struct Split {
    int edge;   // tiles are edge x edge
    int splits; // workgroups that share a tile's contraction
    int per;    // k tiles (of 64) for each
};

inline Split choose_split(int64_t m, int64_t n, int64_t k, int64_t batch)
{
    const int64_t nk = ceil_div(k, 64);
    auto tiles = [&](int64_t edge) { return ceil_div(m, edge) * ceil_div(n, edge) * batch; };
    Split s{64, 1, (int)std::max<int64_t>(nk, 1)};
    if (20 * tiles(256) >= 11 * UNITS)
        s.edge = 256;
    else if (tiles(128) >= UNITS)
        s.edge = 128;
    else if (tiles(128) * nk >= 16 * UNITS)
        s.edge = 128;
    const int64_t t = tiles(s.edge), room = (s.edge == 256 ? 1 : 2) * UNITS;
    if (t < UNITS && nk >= 16) {
        const int64_t splits = std::max<int64_t>(1, std::min(room / t, nk / 8));
        s.per = (int)ceil_div(nk, splits);
        s.splits = (int)ceil_div(nk, s.per);
    }
    return s;
}

// Partial sums of a split product, in fp32, rows of whole 8 columns.
inline int64_t part_ld(int64_t n) { return (n + 7) / 8 * 8; }
inline int64_t part_bytes(const Split &s, int64_t m, int64_t n, int64_t batch)
{
    return s.splits == 1 ? 0 : batch * s.splits * m * part_ld(n) * (int64_t)sizeof(float);
}

template <class C, class Epilogue>
gemm_status launch_tiles(TileArgs &args, typename Epilogue::Args &epi, void *stream)
{
    args.tiles_m = (int32_t)ceil_div(args.m, C::BM);
    args.tiles_n = (int32_t)ceil_div(args.n, C::BN);
    const int64_t tiles = args.symmetric ? (int64_t)args.tiles_m * (args.tiles_m + 1) / 2 : (int64_t)args.tiles_m * args.tiles_n;
    const int64_t grid = tiles * args.splits * args.batch;
    if (grid > INT32_MAX)
        return fail(GEMM_ERR_UNSUPPORTED, "more than 2^31 output tiles");
    args.tiles = (int32_t)tiles;
    args.round = (int32_t)std::min<int64_t>(grid, UNITS * (160 * 1024 / C::LDS));
    return launch_grid(&tile_kernel<C, Epilogue>, grid, 1, C::THREADS, stream, args, epi);
}

// One product (of a stack of them): the tiles, then the sum of a split's parts.
template <class T, int AF, int BF, class Epilogue>
gemm_status run_product(TileArgs &args, typename Epilogue::Args &epi, const Split &s, void *stream)
{
    if (args.m == 0 || args.n == 0 || args.batch == 0)
        return GEMM_OK;
    args.splits = s.splits;
    args.split_k = s.per;
    args.part_ld = part_ld(args.n);
    gemm_status st;
    if (s.edge == 256)
        st = launch_tiles<TileConfig<256, 256, 2, 4, 2, AF, BF, T>, Epilogue>(args, epi, stream);
    else if (s.edge == 128)
        st = launch_tiles<TileConfig<128, 128, 2, 2, 2, AF, BF, T>, Epilogue>(args, epi, stream);
    else
        st = launch_tiles<TileConfig<64, 64, 2, 2, 3, AF, BF, T>, Epilogue>(args, epi, stream);
    if (st != GEMM_OK || s.splits == 1)
        return st;
    return launch_grid(&join_kernel<Epilogue>, ceil_div((int64_t)args.batch * args.m * ((args.n + 7) / 8), 256), 1, 256, stream, args, epi);
}

} // namespace pts
