// 16-bit products D = A . B whose operands may lie either way in memory, with an
// epilogue of their own:
//
//   acc[i][j] = sum_k A[i][k] B[k][j]        (fp32, in the matrix unit)
//   D = epilogue(i, j, acc[i][j])
//
// A linear layer needs the three ways its products contract: y = x w^T with the
// contraction contiguous in both operands, dx = dz w with it strided in w, dw =
// dz^T x with it strided in both; an orthogonalised update needs the same three.
// An operand whose contraction is strided is loaded as it lies, 64 k rows of BM
// (BN) elements, and transposed on the way from LDS to the registers
// (ds_read_b64_tr_b16), so no operand is ever transposed in memory.
#pragma once

#include "device/common.h"
#include "device/scheduler.h"

namespace pts {

typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

// The 16-bit type of the operands.
struct Bf16 {
    static __device__ __forceinline__ f32x4 mfma(u32x4 x, u32x4 y, f32x4 c)
    {
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, x), __builtin_bit_cast(bf16x8, y), c, 0, 0, 0);
    }
};
struct F16 {
    static __device__ __forceinline__ f32x4 mfma(u32x4 x, u32x4 y, f32x4 c)
    {
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, x), __builtin_bit_cast(f16x8, y), c, 0, 0, 0);
    }
};

// ROWS: the contraction is contiguous, element (i, k) at i * ld + k.
// COLS: it is strided, element (i, k) at k * ld + i.
enum : int { ROWS = 0, COLS = 1 };

struct TileArgs {
    const uint16_t *a, *b;
    int64_t lda, ldb;           // elements, multiples of 8
    int64_t a_batch, b_batch;   // elements from one problem of a stack to the next
    float *part;                // sums of the tiles that are split: [tile][split][BM][BN]
    int32_t m, n, k;
    int32_t tiles_m, tiles_n;
    int32_t tiles;              // per problem: tiles_m * tiles_n, or the upper triangle's
    int32_t batch;
    int32_t whole, rest;        // tiles of the stack that one workgroup each sums; those shared by `splits`,
    int32_t splits, split_k;    //   of which number s sums k tiles [s * split_k, (s + 1) * split_k)
    int32_t symmetric;          // A B is symmetric: tiles on and above the diagonal, the others by reflection
    int32_t round;              // workgroups dealt to the dies at a time (static_position)
};

template <int BM_, int BN_, int WM_, int WN_, int STAGES_, int AF_, int BF_, class T_>
struct TileConfig {
    static constexpr int BM = BM_, BN = BN_, WM = WM_, WN = WN_, WAVES = WM * WN, THREADS = 64 * WAVES, STAGES = STAGES_;
    static constexpr int AF = AF_, BF = BF_, BK = 64;
    using T = T_;
    static constexpr int WTM = BM / WM, WTN = BN / WN, MI = WTM / 16, NI = WTN / 16;
    static constexpr int A_BYTES = BM * 128, B_BYTES = BN * 128, STAGE = A_BYTES + B_BYTES;
    // Four waves load (with two waves per SIMD the first of each: its partner then always has the matrix unit).
    static constexpr int LOADERS = 4, A_LOADS = BM / 32, B_LOADS = BN / 32, LOADS = A_LOADS + B_LOADS;
    // The epilogue's part of LDS: 512 fp32 per wave, OUT_ROWS rows of the wave's columns, eight per lane.
    static constexpr int OUT_LANES = WTN / 8, OUT_ROWS = 64 / OUT_LANES, OUT_BYTES = 2048;
    static constexpr int LDS = STAGES * STAGE + WAVES * OUT_BYTES;
    static_assert(WAVES == 4 || WAVES == 8, "waves");
    static_assert((BM == 64 || BM == 128 || BM == 256) && (BN == 64 || BN == 128 || BN == 256), "tile");
    static_assert(NI <= MI && 16 % OUT_ROWS == 0 && (WTN == 32 || WTN == 64), "wave tile");
    // the first wait leaves STAGES - 1 stages' loads of a wave under way: what the counter (6 bits) can be told
    static_assert(STAGES >= 2 && LDS <= 160 * 1024 && (STAGES - 1) * LOADS <= 63, "ring");
};

// One operand of a tile: N rows of A (columns of B) by 64 k in a ring stage.
//
// ROWS: row r's 64 k are 128 bytes in eight 16-byte chunks, chunk c at position
// c ^ (r / 2 & 7). A fragment (16 rows x 32 k) is one ds_read_b128 per lane.
//
// COLS: k row r's N elements are 2 N bytes; its 32-byte pieces (16 columns) are
// exchanged by a number f(r) that differs over the eight k rows r, r + 1, .., r + 3
// and r + 8, .. r + 11 that half a wave reads at once, which then lie in
// different banks. A fragment is two ds_read_b64_tr_b16: in each group of 16
// lanes, lane l gives the address of 4 columns of k row l / 4 and gets column l's
// four k.
template <int FORM, int N>
struct Operand {
    static constexpr int LOADS = N / 32;                     // per loading wave and stage
    static constexpr int OFFS = FORM == ROWS || N == 256 ? 2 : 1; // distinct per-lane offsets
    static constexpr int PITCH = FORM == ROWS ? 128 : 2 * N; // bytes of an LDS row
    uint64_t base;      // first byte of the tile's first row (ROWS) or first column (COLS)
    uint64_t step;      // bytes from one k tile to the next
    uint32_t row_bytes; // bytes from one row in memory to the next
    uint32_t off[OFFS], lim[OFFS];

    static __device__ __forceinline__ int swizzle(int r)
    {
        if constexpr (FORM == ROWS)
            return (r >> 1) & 7;
        else if constexpr (N == 64) // two k rows to 256 bytes of banks
            return ((r >> 1) & 1) | ((r >> 2) & 2);
        else
            return (r & 3) | ((r >> 1) & 4);
    }
    // Load i of wave w fills 1 KiB of the stage: the rows from first_row on, whose lanes' offsets are those of
    // off[which] plus `ahead` rows.
    static constexpr int which(int i) { return FORM == ROWS ? i & 1 : N == 256 ? i >> 2 : 0; }
    static constexpr int ahead(int i)
    {
        return FORM == ROWS ? (i >> 1) * 16 : N == 256 ? (i & 3) * 16 : N == 128 ? i * 16 : i * 32;
    }
    static __device__ __forceinline__ int first_row(int w, int p)
    {
        if constexpr (FORM == ROWS)
            return (w * LOADS + p) * 8;
        else
            return N == 256 ? 2 * w + 8 * p : N == 128 ? 4 * w : 8 * w;
    }
    static constexpr int lds_at(int i) { return (FORM == ROWS ? i * 8 : ahead(i) + 8 * which(i)) * PITCH; }
    static __device__ __forceinline__ uint32_t lds_wave(int w) { return (uint32_t)(first_row(w, 0) * PITCH); }

    // This lane's row and 16-byte piece of the row in memory of a load with offsets off[p].
    static __device__ __forceinline__ void lane_at(int w, int p, int lane, int &row, int &piece)
    {
        constexpr int PIECES = PITCH / 16;
        row = first_row(w, p) + lane / PIECES;
        const int at = lane % PIECES;
        if constexpr (FORM == ROWS)
            piece = at ^ swizzle(row);
        else
            piece = (((at >> 1) ^ swizzle(row)) << 1) | (at & 1);
    }

    // valid: rows (ROWS) or columns (COLS) of the tile that exist. Lanes of others read the last one again.
    __device__ __forceinline__ void setup(const uint16_t *p, int64_t ld, int64_t first, int valid, int w, int lane)
    {
        base = (uint64_t)(p + (FORM == ROWS ? first * ld : first));
        step = FORM == ROWS ? 128 : (uint64_t)ld * 128;
        row_bytes = (uint32_t)ld * 2;
#pragma unroll
        for (int q = 0; q < OFFS; ++q) {
            int row, piece;
            lane_at(w, q, lane, row, piece);
            if constexpr (FORM == COLS)
                piece = min(piece, (valid - 1) / 8);
            off[q] = (uint32_t)row * row_bytes + piece * 16;
            lim[q] = (uint32_t)(valid - 1) * row_bytes + piece * 16; // ROWS: the last row's
        }
    }

    // Start this wave's loads of k tile kt into the operand's part `lds` of a stage. WHOLE: every row exists.
    template <bool WHOLE>
    __device__ __forceinline__ void issue(uint32_t lds, int w, int kt) const
    {
        const u32x4 rsrc = buffer_rsrc((const void *)(base + (FORM == COLS ? (uint64_t)kt * step : 0)));
        const uint32_t at = FORM == ROWS ? (uint32_t)kt * 128u : 0u;
        const uint32_t to = lds + lds_wave(w);
        static_for<LOADS>([&](auto i) {
            constexpr int I = decltype(i)::value;
            if constexpr (WHOLE || FORM == COLS)
                dma_load16_at<lds_at(I)>(to, off[which(I)], rsrc, (uint32_t)uniform((int)(at + ahead(I) * row_bytes)));
            else
                dma_load16_at<lds_at(I)>(to, min(off[which(I)] + ahead(I) * row_bytes, lim[which(I)]), rsrc, at);
        });
    }

    // The same for the last, partial k tile, of `left` k: what lies past its end is read from the last place inside.
    __device__ __forceinline__ void issue_tail(uint32_t lds, int w, int kt, int left, int lane) const
    {
        const u32x4 rsrc = buffer_rsrc((const void *)(base + (FORM == COLS ? (uint64_t)kt * step : 0)));
        const uint32_t at = FORM == ROWS ? (uint32_t)kt * 128u : 0u;
        const uint32_t to = lds + lds_wave(w);
        static_for<LOADS>([&](auto i) {
            constexpr int I = decltype(i)::value, P = which(I);
            int row, piece;
            lane_at(w, P, lane, row, piece);
            uint32_t o;
            if constexpr (FORM == ROWS)
                o = min(off[P] + ahead(I) * row_bytes, lim[P]) - max(piece - (left - 1) / 8, 0) * 16;
            else
                o = off[P] + (uint32_t)(min(row + ahead(I), left - 1) - row) * row_bytes;
            dma_load16_at<lds_at(I)>(to, o, rsrc, at);
        });
    }

    // Clear what lies past the end of a partial k tile.
    static __device__ __forceinline__ void clear_tail(uint8_t *part, int left, int tid, int threads)
    {
        if constexpr (FORM == COLS) {
            constexpr int PIECES = PITCH / 16;
            for (int i = left * PIECES + tid; i < 64 * PIECES; i += threads)
                *(u32x4 *)(part + i * 16) = u32x4{0u, 0u, 0u, 0u};
        } else {
            const int c0 = left / 8;
            for (int i = tid; i < N * 8; i += threads) {
                const int r = i / 8, c = i % 8;
                if (c < c0)
                    continue;
                u32x4 *const p = (u32x4 *)(part + r * 128 + ((c ^ swizzle(r)) << 4));
                u32x4 v = {0u, 0u, 0u, 0u};
                if (c == c0 && left % 8 != 0) {
                    v = *p;
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const int have = left % 8 - 2 * e;
                        v[e] = have >= 2 ? v[e] : have == 1 ? v[e] & 0xFFFFu : 0u;
                    }
                }
                *p = v;
            }
        }
    }

    // This lane's place in the part for fragments of the 16-row blocks from `block` (a multiple of the wave's number of
    // blocks) on, k step 0.
    static __device__ __forceinline__ uint32_t fragment_at(int block, int lane)
    {
        const int l16 = lane & 15, g = lane >> 4;
        if constexpr (FORM == ROWS)
            return (uint32_t)((block * 16 + l16) * 128 + ((g ^ swizzle(l16)) << 4));
        const int r = 8 * g + (l16 >> 2);
        return (uint32_t)(r * PITCH + ((swizzle(r) ^ block) << 5) + (l16 & 3) * 8);
    }
    // Fragment of block `block` + I, k step ks (32 k each).
    static __device__ __forceinline__ u32x4 fragment(const uint8_t *part, uint32_t at, int i, int ks)
    {
        if constexpr (FORM == ROWS) {
            return *(const u32x4 *)(part + (at ^ (uint32_t)(ks << 6)) + i * 2048);
        } else {
            const uint8_t *const p = part + (at ^ (uint32_t)(i << 5)) + ks * 32 * PITCH;
            using Ptr = __attribute__((address_space(3))) bf16x4 *;
            const u32x2 lo = __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4bf16((Ptr)(p)));
            const u32x2 hi = __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4bf16((Ptr)(p + 4 * PITCH)));
            return u32x4{lo[0], lo[1], hi[0], hi[1]};
        }
    }
};

struct Tile {
    int batch, split, row0, col0, vm, vn, k0, nk; // split: the sums' place in `part`, or -1; k0: first k tile
    bool diagonal;
};

// Position inside one problem: groups of 8 tile rows walked column by column (one die's share of a round is then a
// compact block whose operands its L2 holds).
__device__ __forceinline__ void tile_raster(int local, int rows, int cols, int &r, int &c)
{
    const int first = local / (8 * cols) * 8;
    const int in = local - first * cols;
    const int high = min(8, rows - first);
    r = first + in % high;
    c = in / high;
}

// Tile t of the stack.
template <class C>
__device__ __forceinline__ Tile find_tile(const TileArgs &args, int t)
{
    Tile tile;
    tile.batch = t / args.tiles;
    t -= tile.batch * args.tiles;
    int tm, tn;
    if (args.symmetric) {
        // The triangle folded into a rectangle: with an odd number e of tile rows (e + 1) / 2 x e, row p holding its own
        // tiles from the diagonal on and, before them, row e - p's; with an even number e / 2 x (e + 1).
        const int e = args.tiles_m, odd = e & 1;
        int p, q;
        tile_raster(t, (e + 1) / 2, e + 1 - odd, p, q);
        const bool own = odd ? q >= p : q > p;
        tm = own ? p : odd ? e - p : e - 1 - p;
        tn = own ? (odd ? q : q - 1) : e - 1 - q;
    } else {
        tile_raster(t, args.tiles_m, args.tiles_n, tm, tn);
    }
    tile.diagonal = tm == tn;
    tile.row0 = tm * C::BM;
    tile.vm = min(C::BM, args.m - tile.row0);
    tile.col0 = tn * C::BN;
    tile.vn = min(C::BN, args.n - tile.col0);
    tile.split = -1;
    tile.k0 = 0;
    tile.nk = (args.k + C::BK - 1) / C::BK;
    return tile;
}

// A workgroup's work: a whole tile, or a split's share of one.
template <class C>
__device__ __forceinline__ Tile find_work(const TileArgs &args, int t)
{
    if (t < args.whole)
        return find_tile<C>(args, t);
    t -= args.whole;
    const int split = t / args.rest, of = t - split * args.rest;
    Tile tile = find_tile<C>(args, args.whole + of);
    tile.split = of * args.splits + split;
    tile.k0 = split * args.split_k;
    tile.nk = max(0, min(args.split_k, tile.nk - tile.k0));
    return tile;
}

// 512 results of a wave at a time, turned around through 2 KiB of LDS so that a
// lane has eight consecutive columns of one row of W. A row's 16-byte chunks are
// exchanged by the row's number, which spreads them over the banks.
template <int W>
struct Piece {
    static constexpr int LANES = W / 8, HIGH = 64 / LANES, CHUNKS = W / 4;
    float *out;
    int lane, row, col; // this lane's row and first column
    static __device__ __forceinline__ int place(int r, int c) { return r * W + ((c ^ (r & (CHUNKS - 1))) << 2); }
    __device__ __forceinline__ void setup(uint8_t *lds, int lane_)
    {
        out = (float *)lds;
        lane = lane_;
        row = lane / LANES;
        col = lane % LANES * 8;
    }
    // Rows H * HIGH to H * HIGH + HIGH - 1 of a row of 16 x 16 blocks: a lane has, of row lane % 16, four columns of each.
    template <int H, int N>
    __device__ __forceinline__ void turn(const f32x4 (&acc)[N], float (&v)[8]) const
    {
        const int l16 = lane & 15, g = lane >> 4;
        if (l16 / HIGH == H) {
#pragma unroll
            for (int j = 0; j < N; ++j)
                *(f32x4 *)(out + place(l16 % HIGH, 4 * j + g)) = acc[j];
        }
        wave_lds_exchange();
        *(f32x4 *)v = *(const f32x4 *)(out + place(row, col / 4));
        *(f32x4 *)(v + 4) = *(const f32x4 *)(out + place(row, col / 4 + 1));
        wave_lds_exchange();
    }
    // v to row row0 + row of D, columns col0 + col on, of which vm x vn from (row0, col0) exist; reflected too: to column
    // row0 + row as well, eight rows of one column per lane.
    template <class E, class Args>
    __device__ __forceinline__ void fetch(E e, const Args &epi, int batch, int row0, int col0, int vm, int vn, typename E::Raw &raw) const
    {
        if (row < vm && col < vn)
            e.fetch(epi, batch, row0 + row, col0 + col, vn - col, raw);
    }
    template <class E, class Args, class Start>
    __device__ __forceinline__ void store(E e, const Args &epi, const Start &start, const typename E::Raw &raw, int batch, int row0,
                                          int col0, int vm, int vn, float (&v)[8], bool reflected) const
    {
        if (row < vm && col < vn)
            e.finish(epi, start, raw, batch, row0 + row, col0 + col, vn - col, v);
        if constexpr (E::MIRROR) {
            if (!reflected)
                return;
            *(f32x4 *)(out + place(row, col / 4)) = *(f32x4 *)v;
            *(f32x4 *)(out + place(row, col / 4 + 1)) = *(f32x4 *)(v + 4);
            wave_lds_exchange();
            const int c = lane % W, r8 = lane / W * 8;
            float x[8];
#pragma unroll
            for (int i = 0; i < 8; ++i)
                x[i] = out[place(r8 + i, c / 4) + c % 4];
            wave_lds_exchange();
            if (c < vn && r8 < vm)
                e.mirror(epi, batch, row0 + r8, col0 + c, x);
        }
    }
};

// Workgroup `block` of `blocks`; smem: C::LDS bytes.
//
// A workgroup has one tile, or a share of one. Workgroups that go on to their next
// tile, whose first loads they start before they write this one's results, were
// level or slower (8192^3 822 us both, 5000 x 7000 x 3000 to fp32 287 against 292,
// 12 matrices of 1024 x 4096 orthogonalised 1385 against 1410): the dispatcher's
// next workgroup goes to whichever unit is free first.
template <class C, class Epilogue>
__device__ __forceinline__ void tile_body(const TileArgs &args, const typename Epilogue::Args &epi, int block, int blocks, uint8_t *smem)
{
    using OpA = Operand<C::AF, C::BM>;
    using OpB = Operand<C::BF, C::BN>;
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = uniform(tid >> 6);
    const int wm = wave / C::WN, wn = wave % C::WN;
    const bool loads = wave < C::LOADERS;
    const uint32_t lds = lds_address(smem);
    const uint32_t at_a = OpA::fragment_at(wm * C::MI, lane), at_b = OpB::fragment_at(wn * C::NI, lane);

    const Tile tile = find_work<C>(args, static_position(block, blocks, args.round));
    OpA a;
    OpB b;
    a.setup(args.a + tile.batch * args.a_batch, args.lda, tile.row0, tile.vm, wave & 3, lane);
    b.setup(args.b + tile.batch * args.b_batch, args.ldb, tile.col0, tile.vn, wave & 3, lane);
    const bool full = tile.vm == C::BM && tile.vn == C::BN; // all rows and columns exist
    // The eight dies start a long k loop an eighth of it apart, so that they do not all ask for the same part of memory at
    // once (the partial last k tile stays last): 8192^3 802 us, 813 with starts 8 k tiles apart, 833 with none; a short
    // one they start together (5000 x 7000 x 3000 to fp32 271 us, apart 280). On another card plain products of k from 2048
    // to 8192 were level both ways (within 1%) and of k = 1024 up to 3% slower apart, so the border is not a sharp one.
    // The order depends on the work's number alone.
    const bool tail = args.k % C::BK != 0 && (tile.k0 + tile.nk) * C::BK > args.k;
    const int left = args.k - (tile.k0 + tile.nk - 1) * C::BK; // k of the last k tile
    const int whole = tile.nk - (tail ? 1 : 0);
    const int turn = whole >= 64 ? block % NUM_XCD * (whole / 8) : 0;
    auto phys = [&](int kt) {
        if (kt >= whole)
            return tile.k0 + kt;
        const int p = kt + turn;
        return tile.k0 + (p >= whole ? p - whole : p);
    };
    auto issue = [&](int kt) {
        if (!loads)
            return;
        const uint32_t stage = lds + (uint32_t)(kt % C::STAGES) * C::STAGE;
        const int p = phys(kt);
        const int ln = (int)lane_id(); // computed afresh: kept through the k loop, what is built on it would cost registers
        if (kt >= whole) {
            a.issue_tail(stage, wave, p, left, ln);
            b.issue_tail(stage + C::A_BYTES, wave, p, left, ln);
        } else if (full) {
            a.template issue<true>(stage, wave, p);
            b.template issue<true>(stage + C::A_BYTES, wave, p);
        } else {
            a.template issue<false>(stage, wave, p);
            b.template issue<false>(stage + C::A_BYTES, wave, p);
        }
    };
    // Stage of k tile kt: landed for every wave, its partial end cleared; the stage before it handed back.
    auto enter = [&](int kt) {
        if (kt + C::STAGES - 2 < tile.nk)
            wait_vmcnt<(C::STAGES - 2) * C::LOADS>();
        else
            wait_vmcnt<0>();
        barrier_lds();
        if (kt >= whole) {
            uint8_t *const stage = smem + kt % C::STAGES * C::STAGE;
            OpA::clear_tail(stage, left, tid, C::THREADS);
            OpB::clear_tail(stage + C::A_BYTES, left, tid, C::THREADS);
            barrier_lds();
        }
    };

    f32x4 acc[C::MI][C::NI];
    u32x4 fa[C::MI], fb[2][C::NI];

    // One k step (32 k) from (fa, fb[S]), while the fragments of the next one, k step KS of `stage`, take their places:
    // a row of A's after its last use, B's in the other set.
    auto k_step = [&](auto set, auto ks, const uint8_t *stage) {
        constexpr int S = decltype(set)::value, KS = decltype(ks)::value;
#pragma unroll
        for (int i = 0; i < C::MI; ++i) {
#pragma unroll
            for (int jj = 0; jj < C::NI; ++jj) {
                const int j = i & 1 ? C::NI - 1 - jj : jj; // neighbours share an operand
                acc[i][j] = C::T::mfma(fb[S][j], fa[i], acc[i][j]);
            }
            fa[i] = OpA::fragment(stage, at_a, i, KS);
            if (i < C::NI)
                fb[S ^ 1][i] = OpB::fragment(stage + C::A_BYTES, at_b, i, KS);
        }
        static_for<C::MI>([](auto row) {
            constexpr int R = (C::AF == COLS ? 2 : 1) + (decltype(row)::value < C::NI ? (C::BF == COLS ? 2 : 1) : 0);
            __builtin_amdgcn_sched_group_barrier(0x008, C::NI, 0); // the row's matrix instructions
            __builtin_amdgcn_sched_group_barrier(0x100, R, 0);     // its reads
        });
    };

#pragma unroll
    for (int i = 0; i < C::MI; ++i)
#pragma unroll
        for (int j = 0; j < C::NI; ++j)
            acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
    if (tile.nk > 0) {
        for (int kt = 0; kt < min(C::STAGES, tile.nk); ++kt)
            issue(kt);
        if (tile.nk >= C::STAGES)
            wait_vmcnt<(C::STAGES - 1) * C::LOADS>();
        else
            wait_vmcnt<0>();
        barrier_lds();
        if (whole == 0) {
            OpA::clear_tail(smem, left, tid, C::THREADS);
            OpB::clear_tail(smem + C::A_BYTES, left, tid, C::THREADS);
            barrier_lds();
        }
        // A wave whose rows or columns all lie past the tile's edge only loads and meets the others.
        const bool idle = wm * C::WTM >= tile.vm || wn * C::WTN >= tile.vn;
        if (idle) {
            for (int kt = 0; kt + 1 < tile.nk; ++kt) {
                enter(kt + 1);
                if (kt + C::STAGES < tile.nk)
                    issue(kt + C::STAGES);
            }
        } else {
#pragma unroll
            for (int i = 0; i < C::MI; ++i)
                fa[i] = OpA::fragment(smem, at_a, i, 0);
#pragma unroll
            for (int j = 0; j < C::NI; ++j)
                fb[0][j] = OpB::fragment(smem + C::A_BYTES, at_b, j, 0);
            int kt = 0, here = 0;
            auto next = [](int s) { return s + 1 == C::STAGES ? 0 : s + 1; };
            // k tiles with nothing special about them or the ones loaded meanwhile
            for (; kt + C::STAGES < whole; ++kt) {
                k_step(IntC<0>{}, IntC<1>{}, smem + here * C::STAGE);
                wait_vmcnt<(C::STAGES - 2) * C::LOADS>();
                barrier_lds();
                issue(kt + C::STAGES);
                here = next(here);
                k_step(IntC<1>{}, IntC<0>{}, smem + here * C::STAGE);
            }
            for (; kt < tile.nk; ++kt) {
                k_step(IntC<0>{}, IntC<1>{}, smem + here * C::STAGE);
                if (kt + 1 < tile.nk) {
                    enter(kt + 1);
                    if (kt + C::STAGES < tile.nk)
                        issue(kt + C::STAGES);
                }
                here = next(here);
                k_step(IntC<1>{}, IntC<0>{}, smem + here * C::STAGE); // past the last: reads a stage nobody uses
            }
        }
    }

    // The wave's piece of the tile's results.
    const int row0 = wm * C::WTM, col0 = wn * C::WTN;
    if (row0 >= tile.vm || col0 >= tile.vn)
        return;
    Piece<C::WTN> piece;
    piece.setup(smem + C::STAGES * C::STAGE + wave * C::OUT_BYTES, lane);
    constexpr int HALVES = 16 / C::OUT_ROWS, PIECES = C::MI * HALVES;
    auto turned = [&](auto i, float(&v)[8]) {
        constexpr int I = decltype(i)::value;
        piece.template turn<I % HALVES>(acc[I / HALVES], v);
    };
    if (tile.split >= 0) {
        float *const part = args.part + (int64_t)tile.split * (C::BM * C::BN) + (row0 + piece.row) * C::BN + col0 + piece.col;
        static_for<PIECES>([&](auto i) {
            float v[8];
            turned(i, v);
            float *const p = part + decltype(i)::value * C::OUT_ROWS * C::BN;
            *(f32x4 *)p = *(f32x4 *)v;
            *(f32x4 *)(p + 4) = *(f32x4 *)(v + 4);
        });
        return;
    }
    const int vm = tile.vm - row0, vn = tile.vn - col0; // rows and columns of the piece
    Epilogue::run(epi, [&](auto e) {
        // what the pieces need from memory is on its way AHEAD pieces before
        constexpr int AHEAD = PIECES < 4 ? PIECES : 4;
        typename decltype(e)::Raw raw[AHEAD];
        auto fetch = [&](auto i) {
            constexpr int I = decltype(i)::value;
            if constexpr (I < PIECES)
                piece.fetch(e, epi, tile.batch, tile.row0 + row0 + I * C::OUT_ROWS, tile.col0 + col0, vm - I * C::OUT_ROWS, vn, raw[I % AHEAD]);
        };
        static_for<AHEAD>(fetch);
        const auto start = e.start(epi, tile.batch, tile.col0 + col0 + piece.col, vn - piece.col);
        static_for<PIECES>([&](auto i) {
            constexpr int I = decltype(i)::value;
            float v[8];
            turned(i, v);
            const auto mine = raw[I % AHEAD];
            fetch(IntC<I + AHEAD>{});
            piece.store(e, epi, start, mine, tile.batch, tile.row0 + row0 + I * C::OUT_ROWS, tile.col0 + col0, vm - I * C::OUT_ROWS,
                        vn, v, args.symmetric && !tile.diagonal);
        });
    });
}

template <class C, class Epilogue>
__global__ __launch_bounds__(C::THREADS, 2) void tile_kernel(const TileArgs args, const typename Epilogue::Args epi)
{
    __shared__ __align__(1024) uint8_t smem[C::LDS];
    tile_body<C, Epilogue>(args, epi, blockIdx.x, gridDim.x, smem);
}

// Two products that do not wait for each other, one launch: the first `blocks` workgroups are the first's.
template <class C, class D, class Epilogue>
__global__ __launch_bounds__(C::THREADS, 2) void tile_pair_kernel(const TileArgs one, const typename Epilogue::Args epi_one, const TileArgs two,
                                                                  const typename Epilogue::Args epi_two, const int blocks)
{
    static_assert(C::THREADS == D::THREADS && C::LDS == D::LDS, "tiles of one shape");
    __shared__ __align__(1024) uint8_t smem[C::LDS];
    if ((int)blockIdx.x < blocks)
        tile_body<C, Epilogue>(one, epi_one, blockIdx.x, blocks, smem);
    else
        tile_body<D, Epilogue>(two, epi_two, blockIdx.x - blocks, gridDim.x - blocks, smem);
}

// The tiles that were split: the sum of their parts, in their order, and the
// epilogue. A wave has eight rows by 64 columns of a tile.
template <class C, class Epilogue>
__global__ __launch_bounds__(256) void join_kernel(const TileArgs args, const typename Epilogue::Args epi)
{
    constexpr int ACROSS = C::BN / 64, WAVES = ACROSS * (C::BM / 8); // waves' pieces of a tile
    __shared__ __align__(16) float out[4][512];
    const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
    const int at = blockIdx.x * 4 + wave, of = at / WAVES, in = at - of * WAVES; // WAVES is a multiple of 4
    const Tile tile = find_tile<C>(args, args.whole + of);
    const int row0 = in / ACROSS * 8, col0 = in % ACROSS * 64;
    if (row0 >= tile.vm || col0 >= tile.vn)
        return;
    Piece<64> piece;
    piece.setup((uint8_t *)out[wave], lane);
    const int vm = tile.vm - row0, vn = tile.vn - col0;
    const float *p = args.part + (int64_t)of * args.splits * (C::BM * C::BN) + (row0 + piece.row) * C::BN + col0 + piece.col;
    Epilogue::run(epi, [&](auto e) {
        typename decltype(e)::Raw raw;
        piece.fetch(e, epi, tile.batch, tile.row0 + row0, tile.col0 + col0, vm, vn, raw);
        const auto start = e.start(epi, tile.batch, tile.col0 + col0 + piece.col, vn - piece.col);
        float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
        for (int s = 0; s < args.splits; ++s, p += C::BM * C::BN) {
            const f32x4 lo = *(const f32x4 *)p, hi = *(const f32x4 *)(p + 4);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                v[i] += lo[i];
                v[4 + i] += hi[i];
            }
        }
        piece.store(e, epi, start, raw, tile.batch, tile.row0 + row0, tile.col0 + col0, vm, vn, v, args.symmetric && !tile.diagonal);
    });
}

} // namespace pts
