// Routing of tokens to experts: scores, choice, weights, the order of the rows
// by expert, and the gradient of the logits.
//
//   p = softmax(x) or 1 / (1 + exp(-x));  c = p + bias
//   groups: a group's score is its largest c, or the sum of its two largest;
//           only the experts of the best `keep` groups stay
//   ids = the k largest c, ties to the lowest index
//   w_j = scale p_j / (sum of the chosen p + 1e-20), or scale p_j
//
// The choice must not depend on rounding, so c is compared in 64 bits; without
// a bias c is in the order of the logits, which are then compared themselves
// (32 bits, exactly). An expert is open to a token if its logit and its c are
// above -inf (and not NaN); a slot for which no open expert is left gets id -1
// and weight 0. A row whose softmax is not a number goes by its logits.
//
// Latency and instruction bound: 16384 tokens x 128 experts, 8 each, fp32 (10 MB
// in all, 2 us of memory time): choice 8.6 us, counts 3.3, order 7.4, gradient 9.5
// (8.2 with its differences taken of whole sums, which loses the gradient of a
// score near one).
// One token of 256 experts with groups: 7.3 us in one launch.
#pragma once

#include "lanes.h"

namespace pts {

constexpr int ROUTE_MAX_EXPERTS = 1024;
constexpr int ROUTE_MAX_TOP = 32;
constexpr int ROUTE_MAX_GROUPS = 64;
constexpr float ROUTE_EPS = 1e-20f;

struct RouteArgs {
    const void *logits;
    const float *bias;     // or null
    int32_t *ids;
    float *weights;
    int32_t *offsets, *rows, *positions; // the order; offsets null: not wanted
    int32_t *counts;       // workspace of the order: per chunk, experts + 1 words
    int64_t ld;
    int32_t m, experts, top, groups, keep;
    int32_t bf16, sigmoid, pair, renorm;
    int32_t fused;         // the one workgroup also puts the slots in order
    int32_t chunk, chunks; // slots per workgroup of the order, their number
    float scale;
};

struct RouteGradArgs {
    const void *logits;
    const float *dweights;
    const int32_t *ids;
    void *dlogits;
    int64_t ld, ld_d;
    int32_t m, experts, top;
    int32_t bf16, sigmoid, renorm;
    float scale;
};

// Order-preserving integers: x < y as numbers iff key(x) < key(y), equal for
// the two zeros; 0 is below every number's.
__device__ __forceinline__ uint32_t sort_key(float x)
{
    const uint32_t b = __float_as_uint(x + 0.0f);
    return b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ uint64_t sort_key(double x)
{
    const uint64_t b = (uint64_t)__double_as_longlong(x + 0.0);
    return b >> 63 ? ~b : b | 0x8000000000000000ull;
}

template <int LPT> __device__ __forceinline__ uint32_t max_lanes(uint32_t v)
{
    return reduce_lanes<LPT>(v, [](uint32_t a, uint32_t b) { return max(a, b); });
}
template <int LPT> __device__ __forceinline__ uint32_t min_lanes(uint32_t v)
{
    return reduce_lanes<LPT>(v, [](uint32_t a, uint32_t b) { return min(a, b); });
}
template <int LPT> __device__ __forceinline__ float max_lanes(float v)
{
    return __uint_as_float(reduce_lanes<LPT>(__float_as_uint(v), [](uint32_t a, uint32_t b) {
        return __float_as_uint(fmaxf(__uint_as_float(a), __uint_as_float(b)));
    }));
}
template <int LPT> __device__ __forceinline__ float sum_lanes(float v)
{
    return __uint_as_float(reduce_lanes<LPT>(__float_as_uint(v), [](uint32_t a, uint32_t b) {
        return __float_as_uint(__uint_as_float(a) + __uint_as_float(b));
    }));
}
template <int LPT> __device__ __forceinline__ double sum_lanes(double v)
{
#pragma unroll
    for (int d = 1; d < LPT; d *= 2)
        v += __shfl_xor(v, d);
    return v;
}

__device__ __forceinline__ float load_logit(const void *x, bool bf16, int64_t at)
{
    return bf16 ? __uint_as_float((uint32_t)((const uint16_t *)x)[at] << 16) : ((const float *)x)[at];
}

// ---- order --------------------------------------------------------------------

// Stable counting sort of the slots (token, j) by expert, in chunks of
// consecutive slots; slots without an expert come last ("expert" E).
constexpr int ORDER_WAVES = 8, ORDER_THREADS = 64 * ORDER_WAVES;

__device__ __forceinline__ int slot_expert(const RouteArgs &args, int64_t slot)
{
    const int e = args.ids[slot];
    return e < 0 ? args.experts : e;
}

__device__ __forceinline__ void place_slot(const RouteArgs &args, int slot, int expert, int p)
{
    args.rows[p] = slot / args.top;
    args.positions[slot] = expert == args.experts ? -2 - p : p;
}

// before[e] = total[0] + .. + total[e - 1] in LDS, by the first wave: each lane
// adds up a run of experts, and the runs are scanned across the lanes.
__device__ __forceinline__ void scan_totals(const RouteArgs &args, const int32_t *total, int32_t *before)
{
    if (threadIdx.x < 64) {
        const int lane = threadIdx.x, n = args.experts + 1, run = (n + 63) / 64;
        const int lo = min(n, lane * run), hi = min(n, lo + run);
        int sum = 0;
        for (int e = lo; e < hi; ++e)
            sum += total[e];
        int at = sum;
#pragma unroll
        for (int d = 1; d < 64; d *= 2) {
            const int v = __shfl_up(at, d);
            if (lane >= d)
                at += v;
        }
        at -= sum;
        for (int e = lo; e < hi; ++e) {
            before[e] = at;
            at += total[e];
        }
    }
    __syncthreads();
}

constexpr int ORDER_KEPT = 4; // slots per lane whose experts stay in registers (a chunk of 2048)

// The experts of slots lo, lo + 64, .. of this lane, below hi (E + 1: no slot).
__device__ __forceinline__ void keep_experts(const RouteArgs &args, int64_t first, int lo, int hi, int (&kept)[ORDER_KEPT])
{
    const int lane = threadIdx.x & 63;
#pragma unroll
    for (int i = 0; i < ORDER_KEPT; ++i)
        kept[i] = lo + i * 64 + lane < hi ? slot_expert(args, first + lo + i * 64 + lane) : args.experts + 1;
}

// Place the slots [first + lo, first + hi) of this wave, 64 at a time: a slot's
// rank among those is the number of lower lanes with the same expert, found by
// one ballot per bit of the expert's index. cursor[e]: the next position.
__device__ __forceinline__ void place_slots(const RouteArgs &args, int64_t first, int lo, int hi, const int (&kept)[ORDER_KEPT],
                                            int32_t *cursor)
{
    const int lane = threadIdx.x & 63, bits = 32 - __builtin_clz(args.experts + 1);
    auto place64 = [&](int i0, int e) {
        const bool on = e <= args.experts;
        uint64_t same = ~0ull;
        for (int b = 0; b < bits; ++b) {
            const bool bit = e >> b & 1;
            const uint64_t set = __ballot(bit);
            same &= bit ? set : ~set;
        }
        const int rank = __builtin_popcountll(same & ((1ull << lane) - 1));
        int p = 0;
        if (on)
            p = cursor[e] + rank;
        wave_lds_exchange();
        if (on) {
            place_slot(args, (int)(first + i0 + lane), e, p);
            if (rank == 0)
                cursor[e] = p + __builtin_popcountll(same);
        }
        wave_lds_exchange();
    };
#pragma unroll
    for (int i = 0; i < ORDER_KEPT; ++i)
        if (lo + i * 64 < hi)
            place64(lo + i * 64, kept[i]);
    for (int i0 = lo + ORDER_KEPT * 64; i0 < hi; i0 += 64)
        place64(i0, i0 + lane < hi ? slot_expert(args, first + i0 + lane) : args.experts + 1);
}

__global__ __launch_bounds__(ORDER_THREADS) void order_count_kernel(const RouteArgs args)
{
    __shared__ int32_t counts[ROUTE_MAX_EXPERTS + 1];
    const int64_t first = (int64_t)blockIdx.x * args.chunk, slots = (int64_t)args.m * args.top;
    const int count = (int)min((int64_t)args.chunk, slots - first);
    for (int e = threadIdx.x; e <= args.experts; e += ORDER_THREADS)
        counts[e] = 0;
    __syncthreads();
    for (int i = threadIdx.x; i < count; i += ORDER_THREADS)
        atomicAdd(&counts[slot_expert(args, first + i)], 1);
    __syncthreads();
    for (int e = threadIdx.x; e <= args.experts; e += ORDER_THREADS)
        args.counts[(int64_t)blockIdx.x * (args.experts + 1) + e] = counts[e];
}

// Up to so many chunks every workgroup of the order counts all slots itself.
constexpr int ORDER_SELF_COUNTED = 4;

// One chunk per workgroup; its waves take consecutive parts. Each workgroup adds
// up all chunks' counts (at most 256 x 1025 words, from L2), or with few chunks
// counts all slots, which saves a launch.
__global__ __launch_bounds__(ORDER_THREADS) void order_place_kernel(const RouteArgs args)
{
    __shared__ int32_t total[ROUTE_MAX_EXPERTS + 1], before[ROUTE_MAX_EXPERTS + 1], earlier[ROUTE_MAX_EXPERTS + 1];
    __shared__ int32_t cursor[ORDER_WAVES * (ROUTE_MAX_EXPERTS + 1)];
    const int n = args.experts + 1, chunk = blockIdx.x, lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int64_t first = (int64_t)chunk * args.chunk, slots = (int64_t)args.m * args.top;
    const int count = (int)min((int64_t)args.chunk, slots - first);
    const int part = (count + ORDER_THREADS - 1) / ORDER_THREADS * 64;
    const int lo = min(count, wave * part), hi = min(count, lo + part);
    int kept[ORDER_KEPT];
    keep_experts(args, first, lo, hi, kept);
    for (int i = threadIdx.x; i < ORDER_WAVES * n; i += ORDER_THREADS)
        cursor[i] = 0;
    const bool self = args.chunks <= ORDER_SELF_COUNTED;
    for (int e = threadIdx.x; e < n; e += ORDER_THREADS) {
        int sum = 0, mine = 0;
        if (!self) {
#pragma unroll 16
            for (int c = 0; c < args.chunks; ++c) {
                const int v = args.counts[(int64_t)c * n + e];
                mine += c < chunk ? v : 0;
                sum += v;
            }
        }
        total[e] = sum;
        earlier[e] = mine;
    }
    __syncthreads();
    int32_t *const mine = cursor + wave * n;
#pragma unroll
    for (int i = 0; i < ORDER_KEPT; ++i)
        if (kept[i] < n)
            atomicAdd(&mine[kept[i]], 1);
    for (int i = lo + ORDER_KEPT * 64 + lane; i < hi; i += 64)
        atomicAdd(&mine[slot_expert(args, first + i)], 1);
    if (self)
        for (int i = threadIdx.x; i < slots; i += ORDER_THREADS) {
            const int e = slot_expert(args, i);
            atomicAdd(&total[e], 1);
            if (i < first)
                atomicAdd(&earlier[e], 1);
        }
    __syncthreads();
    scan_totals(args, total, before);
    for (int e = threadIdx.x; e < n; e += ORDER_THREADS) {
        if (chunk == 0)
            args.offsets[e] = before[e];
        int p = before[e] + earlier[e];
#pragma unroll
        for (int w = 0; w < ORDER_WAVES; ++w) {
            const int c = cursor[w * n + e];
            cursor[w * n + e] = p;
            p += c;
        }
    }
    __syncthreads();
    place_slots(args, first, lo, hi, kept, mine);
}

// Few slots, their experts in LDS (E for none), by the 256 threads of the one
// workgroup that has routed them: each slot's position and each offset is a
// count over all slots, with no atomics and nothing to wait for in between.
constexpr int ROUTE_FUSED_SLOTS = 128;
__device__ __forceinline__ void order_few(const RouteArgs &args, const int32_t *experts, int count)
{
    for (int i = threadIdx.x; i < max(count, args.experts + 1); i += 256) {
        const int mine = i < count ? experts[i] : 0;
        int position = 0, offset = 0;
#pragma unroll 8
        for (int j = 0; j < count; ++j) {
            const int e = experts[j];
            position += e < mine || (e == mine && j < i);
            offset += e < i;
        }
        if (i < count)
            place_slot(args, i, mine, position);
        if (i <= args.experts)
            args.offsets[i] = offset;
    }
}

// ---- choice -------------------------------------------------------------------

// The groups that stay, bit g for group g. `c` holds the token's scores in LDS
// (-inf where closed). Each group is scored by as many lanes as there are to
// spare (a power of two), or each lane scores several groups.
template <int LPT>
__device__ __forceinline__ uint64_t keep_groups(const RouteArgs &args, double *c, int lane)
{
    constexpr int GPL = ROUTE_MAX_GROUPS / LPT;
    const int size = args.experts / args.groups;
    int spare = 1;
    while (2 * spare * args.groups <= LPT)
        spare *= 2;
    double mine[GPL];
#pragma unroll
    for (int q = 0; q < GPL; ++q) {
        const int g = q * LPT + lane / spare;
        double first = -INFINITY, second = -INFINITY;
        if (g < args.groups)
            for (int i = lane % spare; i < size; i += spare) {
                const double s = c[g * size + i];
                second = fmax(second, fmin(first, s));
                first = fmax(first, s);
            }
        for (int d = 1; d < spare; d *= 2) {
            const double f = __shfl_xor(first, d), s = __shfl_xor(second, d);
            second = fmax(fmin(first, f), fmax(second, s));
            first = fmax(first, f);
        }
        mine[q] = args.pair && second > -INFINITY ? first + second : first;
    }
    wave_lds_exchange();
#pragma unroll
    for (int q = 0; q < GPL; ++q)
        if (lane % spare == 0 && q * LPT + lane / spare < args.groups)
            c[q * LPT + lane / spare] = mine[q];
    wave_lds_exchange();
    uint64_t kept = 0;
    const int shift = (threadIdx.x & 63) & ~(LPT - 1); // this token's lanes in a ballot
#pragma unroll
    for (int q = 0; q < GPL; ++q) { // lane g for group g
        const int g = q * LPT + lane;
        const double s = g < args.groups ? c[g] : 0.;
        int ahead = 0; // groups that come before g
#pragma unroll 8
        for (int h = 0; h < args.groups; ++h)
            ahead += c[h] > s || (c[h] == s && h < g);
        const uint64_t stays = __ballot(g < args.groups && ahead < args.keep) >> shift;
        kept |= (LPT == 64 ? stays : stays & ((1ull << (LPT & 63)) - 1)) << (q * LPT & 63);
    }
    wave_lds_exchange();
    return kept;
}

// A token is held by LPT lanes, VPL logits each (expert v LPT + lane). WIDE:
// the choice goes by 64-bit scores (a bias), otherwise by the logits. GROUPED:
// it is limited to the best groups (a kernel of its own: the group arithmetic
// held 90 registers through the choice of the others, 11 us against 8.6 to 10). 16 lanes
// per token keep every reduction inside a row of lanes (four rotations, no
// exchange between rows) and four tokens in a wave; 64 lanes leave the least
// work per lane where there are few tokens or many experts.
template <int LPT, int VPL, bool WIDE, bool GROUPED>
__global__ __launch_bounds__(256) void route_kernel(const RouteArgs args)
{
    constexpr int TOKENS = 256 / LPT; // per workgroup and pass
    __shared__ double group_scores[GROUPED ? TOKENS * LPT * VPL : 1];
    __shared__ int32_t fused_experts[ROUTE_FUSED_SLOTS];
    const int lane = threadIdx.x & (LPT - 1), slot = threadIdx.x / LPT;
    const int experts = args.experts;
    for (int64_t t0 = (int64_t)blockIdx.x * TOKENS; t0 < args.m; t0 += (int64_t)gridDim.x * TOKENS) {
        const int64_t token = t0 + slot;
        const bool live = token < args.m;
        float x[VPL], top = -INFINITY;
#pragma unroll
        for (int v = 0; v < VPL; ++v) {
            const int e = v * LPT + lane;
            x[v] = live && e < experts ? load_logit(args.logits, args.bf16, token * args.ld + e) : -INFINITY;
            top = fmaxf(top, x[v]);
        }
        top = max_lanes<LPT>(top);
        top = top == -INFINITY ? 0.f : top;
        float total = 1.f; // the softmax's denominator
        if (!args.sigmoid) {
            total = 0.f;
#pragma unroll
            for (int v = 0; v < VPL; ++v)
                total += expf(x[v] - top);
            total = sum_lanes<LPT>(total);
            total = total == 0.f ? 1.f : total;
        }
        double c[VPL];
        if (WIDE || (GROUPED && args.pair)) {
            double all = 1.;
            if (!args.sigmoid) {
                all = 0.;
#pragma unroll
                for (int v = 0; v < VPL; ++v) {
                    c[v] = exp((double)x[v] - (double)top);
                    all += c[v];
                }
                all = sum_lanes<LPT>(all);
                all = all == 0. ? 1. : all;
            }
#pragma unroll
            for (int v = 0; v < VPL; ++v) {
                const int e = v * LPT + lane;
                c[v] = args.sigmoid ? 1. / (1. + exp(-(double)x[v])) : c[v] / all;
                if (args.bias != nullptr && e < experts)
                    c[v] += (double)args.bias[e];
                if (all != all)
                    c[v] = (double)x[v];
            }
        } else {
#pragma unroll
            for (int v = 0; v < VPL; ++v)
                c[v] = (double)x[v];
        }
        uint32_t key[VPL], low[VPL]; // of c, or of the logits alone; key 0: closed
#pragma unroll
        for (int v = 0; v < VPL; ++v) {
            const bool open = x[v] > -INFINITY && c[v] > -INFINITY;
            const uint64_t k = WIDE ? sort_key(c[v]) : (uint64_t)sort_key(x[v]) << 32;
            key[v] = open ? (uint32_t)(k >> 32) : 0u;
            low[v] = (uint32_t)k;
        }
        if constexpr (GROUPED) {
            double *const scores = group_scores + slot * LPT * VPL;
            const int size = experts / args.groups;
#pragma unroll
            for (int v = 0; v < VPL; ++v)
                scores[v * LPT + lane] = key[v] == 0 ? -INFINITY : c[v];
            wave_lds_exchange();
            const uint64_t kept = keep_groups<LPT>(args, scores, lane);
#pragma unroll
            for (int v = 0; v < VPL; ++v)
                if (!(kept >> (min(v * LPT + lane, experts - 1) / size) & 1))
                    key[v] = 0;
        }
        // The best ones in turn: the largest key, of those the largest low half, of those the lowest
        // index. Slot j belongs to lane j % 16 (of every row of lanes).
        int id[ROUTE_MAX_TOP / 16];
#pragma unroll
        for (int q = 0; q < ROUTE_MAX_TOP / 16; ++q)
            id[q] = -1;
        for (int j = 0; j < args.top; ++j) {
            uint32_t best = key[0];
#pragma unroll
            for (int v = 1; v < VPL; ++v)
                best = max(best, key[v]);
            best = max_lanes<LPT>(best);
            uint32_t best_low = 0;
            if constexpr (WIDE) {
#pragma unroll
                for (int v = 0; v < VPL; ++v)
                    best_low = max(best_low, key[v] == best ? low[v] : 0u);
                best_low = max_lanes<LPT>(best_low);
            }
            uint32_t at = 0xFFFFFFFFu;
#pragma unroll
            for (int v = VPL - 1; v >= 0; --v)
                at = key[v] == best && (!WIDE || low[v] == best_low) ? (uint32_t)(v * LPT + lane) : at;
            at = min_lanes<LPT>(at);
            const int e = best == 0 ? -1 : (int)at;
#pragma unroll
            for (int v = 0; v < VPL; ++v)
                key[v] = v * LPT + lane == e ? 0u : key[v];
#pragma unroll
            for (int q = 0; q < ROUTE_MAX_TOP / 16; ++q)
                id[q] = j == q * 16 + (lane & 15) ? e : id[q];
        }
        float p[ROUTE_MAX_TOP / 16], sum = 0.f;
#pragma unroll
        for (int q = 0; q < ROUTE_MAX_TOP / 16; ++q) {
            p[q] = 0.f;
            if (id[q] >= 0) { // never where !live: nothing was open
                const float v = load_logit(args.logits, args.bf16, token * args.ld + id[q]);
                p[q] = args.sigmoid ? 1.f / (1.f + expf(-v)) : expf(v - top) / total;
            }
            sum += p[q];
        }
        sum = sum_lanes<16>(sum);
        const float factor = args.renorm ? args.scale / (sum + ROUTE_EPS) : args.scale;
        if (live && lane < 16) {
#pragma unroll
            for (int q = 0; q < ROUTE_MAX_TOP / 16; ++q)
                if (q * 16 + lane < args.top) {
                    const int64_t at = token * args.top + q * 16 + lane;
                    args.ids[at] = id[q];
                    args.weights[at] = id[q] < 0 ? 0.f : p[q] * factor;
                    if (args.fused)
                        fused_experts[at] = id[q] < 0 ? experts : id[q];
                }
        }
    }
    if (args.fused) { // this workgroup has had every token
        __syncthreads();
        order_few(args, fused_experts, args.m * args.top);
    }
}

// ---- gradient -----------------------------------------------------------------

// dL/dx from dL/dw, for the chosen experts of `ids` (the choice itself has no
// gradient; the bias only takes part in the choice). With S = sum p + 1e-20:
//   renormalised:  dL/dp_j = scale / S (dw_j - sum_i dw_i p_i / S)
//   otherwise:     dL/dp_j = scale dw_j
//   softmax:       dL/dx_e = p_e (dL/dp_e - sum_j dL/dp_j p_j)
//   sigmoid:       dL/dx_e = dL/dp_e p_e (1 - p_e)
// As they stand, these lose the gradient of a score near one, which is as small
// as what is left to the others: each difference is of nearly equal values. So
// they are taken term by term:
//   renormalised:  dw_j S - sum_i dw_i p_i = sum_i p_i (dw_j - dw_i) + 1e-20 dw_j,
//                  and softmax's sum_j dL/dp_j p_j keeps only the part of 1e-20
//   softmax:       dL/dx_e = p_e (dL/dp_e rest + sum_{i != e} p_i (dL/dp_e - dL/dp_i)),
//                  rest: the sum of the scores that are not chosen
//   sigmoid:       p (1 - p) = z / (1 + z)^2, z = exp(-|x|)
// The scores are computed again. An id outside [0, experts) has no score. A
// sigmoid's expert that no id names has no part in the weights: 0, also where
// its logit is a NaN, which closes it. An expert that several slots name gets
// the sum; its score counts once among the others'.
template <int SLOT> __device__ __forceinline__ int from_slot(const int (&x)[ROUTE_MAX_TOP / 16])
{ // slot SLOT's value to every lane of its row
    return __builtin_amdgcn_mov_dpp(x[SLOT / 16], 0x150 + SLOT % 16, 0xF, 0xF, true);
}
template <int SLOT> __device__ __forceinline__ float from_slot(const float (&x)[ROUTE_MAX_TOP / 16])
{
    return __uint_as_float(
        (uint32_t)__builtin_amdgcn_mov_dpp((int)__float_as_uint(x[SLOT / 16]), 0x150 + SLOT % 16, 0xF, 0xF, true));
}

template <int LPT, int VPL>
__global__ __launch_bounds__(256) void route_backward_kernel(const RouteGradArgs args)
{
    constexpr int TOKENS = 256 / LPT;
    const int lane = threadIdx.x & (LPT - 1), slot = threadIdx.x / LPT;
    const int experts = args.experts;
    const int64_t token = (int64_t)blockIdx.x * TOKENS + slot;
    const bool live = token < args.m;
    // this lane's slots, j = q 16 + lane % 16, and their logits: asked for first, they are used last
    int id[ROUTE_MAX_TOP / 16];
    float dw[ROUTE_MAX_TOP / 16], chosen[ROUTE_MAX_TOP / 16];
#pragma unroll
    for (int q = 0; q < ROUTE_MAX_TOP / 16; ++q) {
        const int j = q * 16 + (lane & 15);
        id[q] = -1;
        dw[q] = 0.f;
        if (live && j < args.top) {
            id[q] = args.ids[token * args.top + j];
            dw[q] = args.dweights[token * args.top + j];
        }
    }
    float x[VPL], top = -INFINITY;
#pragma unroll
    for (int v = 0; v < VPL; ++v) {
        const int e = v * LPT + lane;
        x[v] = live && e < experts ? load_logit(args.logits, args.bf16, token * args.ld + e) : -INFINITY;
        top = fmaxf(top, x[v]);
    }
#pragma unroll
    for (int q = 0; q < ROUTE_MAX_TOP / 16; ++q) {
        if (id[q] < 0 || id[q] >= experts) {
            id[q] = -1;
            dw[q] = 0.f;
        }
        chosen[q] = id[q] >= 0 ? load_logit(args.logits, args.bf16, token * args.ld + id[q]) : 0.f;
    }
    top = max_lanes<LPT>(top);
    top = top == -INFINITY ? 0.f : top;
    float p[VPL], total = 0.f; // the score, or for the sigmoid its slope
    if (args.sigmoid) {
#pragma unroll
        for (int v = 0; v < VPL; ++v) { // p (1 - p) = z / (1 + z)^2: 1 - p would be lost in the rounding of a p near 1
            const float z = expf(-fabsf(x[v])), r = 1.f / (1.f + z);
            p[v] = z * r * r;
        }
    } else {
#pragma unroll
        for (int v = 0; v < VPL; ++v) {
            p[v] = expf(x[v] - top);
            total += p[v];
        }
        total = sum_lanes<LPT>(total);
        total = total == 0.f ? 1.f : total;
#pragma unroll
        for (int v = 0; v < VPL; ++v)
            p[v] /= total;
    }
    float score[ROUTE_MAX_TOP / 16], sum = 0.f, dot = 0.f;
#pragma unroll
    for (int q = 0; q < ROUTE_MAX_TOP / 16; ++q) {
        score[q] = 0.f;
        if (id[q] >= 0)
            score[q] = args.sigmoid ? 1.f / (1.f + expf(-chosen[q])) : expf(chosen[q] - top) / total;
        sum += score[q];
        dot += dw[q] * score[q];
    }
    sum = sum_lanes<16>(sum) + ROUTE_EPS;
    dot = sum_lanes<16>(dot);
    auto each_slot = [&](auto f) {
        static_for<ROUTE_MAX_TOP>([&](auto slot) {
            if (decltype(slot)::value < args.top)
                f(slot);
        });
    };
    float grad[ROUTE_MAX_TOP / 16], back; // by the slot's score; what softmax takes from every expert
    if (args.renorm) {
#pragma unroll
        for (int q = 0; q < ROUTE_MAX_TOP / 16; ++q)
            grad[q] = ROUTE_EPS * dw[q];
        each_slot([&](auto slot) {
            const float p_i = from_slot<decltype(slot)::value>(score), d_i = from_slot<decltype(slot)::value>(dw);
#pragma unroll
            for (int q = 0; q < ROUTE_MAX_TOP / 16; ++q)
                grad[q] = fmaf(p_i, dw[q] - d_i, grad[q]);
        });
#pragma unroll
        for (int q = 0; q < ROUTE_MAX_TOP / 16; ++q)
            grad[q] = grad[q] / sum * (args.scale / sum);
        back = dot * (ROUTE_EPS / sum) * (args.scale / sum);
    } else {
#pragma unroll
        for (int q = 0; q < ROUTE_MAX_TOP / 16; ++q)
            grad[q] = dw[q];
        back = dot * args.scale;
        if (!args.sigmoid) {
            uint32_t chosen_here = 0; // bit v: expert v LPT + lane
            float first[ROUTE_MAX_TOP / 16]; // 0: an earlier slot names the expert
#pragma unroll
            for (int q = 0; q < ROUTE_MAX_TOP / 16; ++q)
                first[q] = 1.f;
            each_slot([&](auto slot) {
                const int e = from_slot<decltype(slot)::value>(id);
#pragma unroll
                for (int v = 0; v < VPL; ++v)
                    chosen_here |= v * LPT + lane == e ? 1u << v : 0u;
#pragma unroll
                for (int q = 0; q < ROUTE_MAX_TOP / 16; ++q)
                    first[q] = e == id[q] && decltype(slot)::value < q * 16 + (lane & 15) ? 0.f : first[q];
            });
            float rest = 0.f;
#pragma unroll
            for (int v = 0; v < VPL; ++v)
                rest += chosen_here >> v & 1 ? 0.f : p[v];
            rest = sum_lanes<LPT>(rest);
#pragma unroll
            for (int q = 0; q < ROUTE_MAX_TOP / 16; ++q)
                grad[q] *= rest;
            each_slot([&](auto slot) {
                const int e = from_slot<decltype(slot)::value>(id);
                const float p_i = from_slot<decltype(slot)::value>(score), d_i = from_slot<decltype(slot)::value>(dw),
                            f_i = from_slot<decltype(slot)::value>(first);
#pragma unroll
                for (int q = 0; q < ROUTE_MAX_TOP / 16; ++q)
                    grad[q] = e == id[q] ? grad[q] : fmaf(p_i, f_i * dw[q] - first[q] * d_i, grad[q]);
            });
        }
#pragma unroll
        for (int q = 0; q < ROUTE_MAX_TOP / 16; ++q)
            grad[q] *= args.scale;
    }
    float dp[VPL];
    uint32_t named = 0; // bit v: expert v LPT + lane
#pragma unroll
    for (int v = 0; v < VPL; ++v)
        dp[v] = 0.f;
    each_slot([&](auto slot) {
        const int e = from_slot<decltype(slot)::value>(id);
        const float d = from_slot<decltype(slot)::value>(grad);
#pragma unroll
        for (int v = 0; v < VPL; ++v) {
            const bool mine = v * LPT + lane == e;
            dp[v] += mine ? d : 0.f;
            named |= mine ? 1u << v : 0u;
        }
    });
    if (live) {
#pragma unroll
        for (int v = 0; v < VPL; ++v) {
            const int e = v * LPT + lane;
            float d = dp[v];
            if (args.sigmoid)
                d = named >> v & 1 ? d * p[v] : 0.f;
            else
                d = p[v] * (named >> v & 1 && !args.renorm ? d : d - back);
            if (e < experts) {
                if (args.bf16)
                    ((__bf16 *)args.dlogits)[token * args.ld_d + e] = (__bf16)d;
                else
                    ((float *)args.dlogits)[token * args.ld_d + e] = d;
            }
        }
    }
}

} // namespace pts
