// Which tiles a 16-bit product takes, and over how many workgroups its
// contraction is split. Host side.
#pragma once

#include <algorithm>
#include <climits>

#include "host_launch.h"
#include "linear/tile.h"

namespace pts {

constexpr int64_t UNITS = 256; // compute units of the card: the choice, and with it every bit of a result, depends on sizes alone
constexpr int64_t MAX_EXTENT = INT64_C(0x7FFFFC00); // 2^31 - 1024: extents below it are rounded up to whole tiles in 32 bits

struct Split {
    int edge;            // tiles are edge x edge,
    bool wide;           //   128 x 128 ones by eight waves with a ring of four stages, one to a compute unit
    int splits, per;     // workgroups that share a tile's contraction, and k tiles (of 64) for each:
    int64_t whole, rest; //   so many tiles are not shared, so many are
};

// What a tile takes on MI355X, in us: per k tile, and for its first loads and its
// results, alone on its compute unit and with another one of its kind (measured
// with 256 and 512 tiles of 512, 4096 and 8192 k; the three ways the operands can
// lie differ by 10%). So 256 x 256 tiles run at 1470 to 1590 TFLOP/s, 128 x 128 at
// 1190 to 1260 (840 to 1060 alone), 64 x 64 at 650 to 790 (470 to 530 alone).
// Where a unit has one 128 x 128 tile only, eight waves and a ring of four stages
// hide more of the loads' latency than four waves and two (2048^3 21.0 us against
// 25.8, 4096 x 1024 x 4096 36.3 against 44.5; with two tiles to a unit, 4096 x 2048
// x 8192, 132 against 118).
struct TileCost {
    int edge, resident;
    double alone, paired, fixed;
};
constexpr TileCost TILE_COSTS[] = {{256, 1, 1.40, 1.40, 7.0}, {128, 2, 0.54, 0.87, 5.0}, {128, 1, 0.46, 0.46, 5.0}, {64, 2, 0.27, 0.38, 3.0}};
constexpr double JOIN_US = 4.0, JOIN_BYTES_PER_US = 2.5e6; // a launch; a part written and read again

// The tiles, and how the last round of them, which seldom fills the card, is
// shared: whichever takes the least time by the costs above.
inline Split choose_split(int64_t m, int64_t n, int64_t k, int64_t batch, bool symmetric)
{
    const int64_t nk = std::max<int64_t>(ceil_div(k, 64), 1);
    Split best{};
    double least = 1e300;
    for (const TileCost &c : TILE_COSTS) {
        const int64_t tm = ceil_div(m, c.edge), tn = ceil_div(n, c.edge);
        const int64_t tiles = (symmetric ? tm * (tm + 1) / 2 : tm * tn) * batch, round = UNITS * c.resident;
        const int64_t rest = tiles % round, whole = tiles - rest;
        auto tile_us = [&](int64_t workgroups, int64_t per) { // of a last round
            return workgroups == 0 ? 0.0 : c.fixed + (double)per * (workgroups <= UNITS ? c.alone : c.paired);
        };
        const double rounds = (double)(whole / round) * (c.fixed + (double)nk * c.paired);
        for (int64_t splits = 1; splits <= 64 && (splits == 1 || (rest > 0 && nk >= 4 * splits && rest * splits <= round)); ++splits) {
            const int64_t per = ceil_div(nk, splits), used = ceil_div(nk, per);
            double us = rounds + tile_us(rest * used, per);
            if (used > 1)
                us += JOIN_US + (double)(rest * used * c.edge * c.edge * 4) / JOIN_BYTES_PER_US;
            if (us < least) {
                least = us;
                const bool wide = c.edge == 128 && c.resident == 1;
                best = used > 1 ? Split{c.edge, wide, (int)used, (int)per, whole, rest} : Split{c.edge, wide, 1, (int)nk, tiles, 0};
            }
        }
    }
    return best;
}

// Bytes of the shared tiles' sums.
inline int64_t part_bytes(const Split &s) { return s.rest * s.splits * s.edge * s.edge * (int64_t)sizeof(float); }

// Whether its launches keep within HIP's 2^32 - 1 threads.
inline bool launchable(const Split &s) { return s.whole + s.rest * s.splits <= (int64_t)UINT32_MAX / (s.edge == 256 || s.wide ? 512 : 256); }
inline gemm_status check_launches(const Split &s)
{
    const int64_t grid = s.whole + s.rest * s.splits;
    if (!launchable(s))
        return fail(GEMM_ERR_UNSUPPORTED, "%lld workgroups: too large a problem for one launch", (long long)grid);
    return GEMM_OK;
}

template <class C> gemm_status plan_tiles(TileArgs &args, const Split &s, int64_t *grid)
{
    args.tiles_m = (int32_t)ceil_div(args.m, C::BM);
    args.tiles_n = (int32_t)ceil_div(args.n, C::BN);
    const int64_t tiles = args.symmetric ? (int64_t)args.tiles_m * (args.tiles_m + 1) / 2 : (int64_t)args.tiles_m * args.tiles_n;
    *grid = s.whole + s.rest * s.splits;
    const gemm_status st = check_launches(s);
    if (st != GEMM_OK)
        return st;
    args.tiles = (int32_t)tiles;
    args.whole = (int32_t)s.whole;
    args.rest = (int32_t)s.rest;
    args.splits = s.splits;
    args.split_k = s.per;
    args.round = (int32_t)std::min<int64_t>(*grid, UNITS * (160 * 1024 / C::LDS));
    return GEMM_OK;
}

template <class C, class Epilogue>
gemm_status launch_join(TileArgs &args, typename Epilogue::Args &epi, const Split &s, void *stream)
{
    if (s.rest == 0)
        return GEMM_OK;
    return launch_grid(&join_kernel<C, Epilogue>, s.rest * (C::BN / 64) * (C::BM / 8) / 4, 1, 256, stream, args, epi);
}

template <class C, class Epilogue>
gemm_status launch_tiles(TileArgs &args, typename Epilogue::Args &epi, const Split &s, void *stream)
{
    int64_t grid;
    gemm_status st = plan_tiles<C>(args, s, &grid);
    if (st == GEMM_OK)
        st = launch_grid(&tile_kernel<C, Epilogue>, grid, 1, C::THREADS, stream, args, epi);
    return st != GEMM_OK ? st : launch_join<C, Epilogue>(args, epi, s, stream);
}

template <class T, int AF, int BF> using Tiles256 = TileConfig<256, 256, 2, 4, 2, AF, BF, T>;
template <class T, int AF, int BF> using Tiles128 = TileConfig<128, 128, 2, 2, 2, AF, BF, T>;
template <class T, int AF, int BF> using TilesWide128 = TileConfig<128, 128, 2, 4, 4, AF, BF, T>;
template <class T, int AF, int BF> using Tiles64 = TileConfig<64, 64, 2, 2, 3, AF, BF, T>;

// One product (of a stack of them): the tiles, then the sums of those that were shared.
template <class T, int AF, int BF, class Epilogue>
gemm_status run_product(TileArgs &args, typename Epilogue::Args &epi, const Split &s, void *stream)
{
    if (args.m == 0 || args.n == 0 || args.batch == 0)
        return GEMM_OK;
    if (s.edge == 256)
        return launch_tiles<Tiles256<T, AF, BF>, Epilogue>(args, epi, s, stream);
    if (s.wide)
        return launch_tiles<TilesWide128<T, AF, BF>, Epilogue>(args, epi, s, stream);
    if (s.edge == 128)
        return launch_tiles<Tiles128<T, AF, BF>, Epilogue>(args, epi, s, stream);
    return launch_tiles<Tiles64<T, AF, BF>, Epilogue>(args, epi, s, stream);
}

} // namespace pts
