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
#pragma once

#include "device/common.h"

namespace pts {

constexpr int ROUTE_MAX_EXPERTS = 1024;
constexpr int ROUTE_MAX_TOP = 32;
constexpr int ROUTE_MAX_GROUPS = 64;
constexpr float ROUTE_EPS = 1e-20f;
constexpr int ORDER_LDS_WORDS = 6 * (ROUTE_MAX_EXPERTS + 1);

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

// The value of the lane D further on, for reductions over the lanes of a token:
// within a row of 16 lanes by a DPP rotation, across rows by a shuffle.
template <int D> __device__ __forceinline__ uint32_t partner(uint32_t v)
{
    if constexpr (D < 16)
        return (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0x120 + D, 0xF, 0xF, false);
    else
        return (uint32_t)__shfl_xor((int)v, D);
}
template <int D> __device__ __forceinline__ int partner(int v) { return (int)partner<D>((uint32_t)v); }
template <int D> __device__ __forceinline__ float partner(float v)
{
    return __uint_as_float(partner<D>(__float_as_uint(v)));
}
template <int D> __device__ __forceinline__ uint64_t partner(uint64_t v)
{
    return (uint64_t)partner<D>((uint32_t)(v >> 32)) << 32 | partner<D>((uint32_t)v);
}
template <int D> __device__ __forceinline__ double partner(double v)
{
    return __longlong_as_double((long long)partner<D>((uint64_t)__double_as_longlong(v)));
}

// Candidates of the choice, larger first: by the logits, the 32-bit key above
// the complement of the expert's index (a tie goes to the lowest index), or by
// 64-bit scores with the index beside them. 0 in the key: none.
template <bool WIDE> struct Candidate;
template <> struct Candidate<false> {
    uint64_t key;
    __device__ __forceinline__ bool none() const { return key == 0; }
    __device__ __forceinline__ int expert() const { return (int)~(uint32_t)key; }
    __device__ __forceinline__ void take(const Candidate o) { key = o.key > key ? o.key : key; } // the better one
    static __device__ __forceinline__ Candidate make(float x, double, int e)
    {
        return Candidate{(uint64_t)sort_key(x) << 32 | (uint32_t)~e};
    }
    static __device__ __forceinline__ Candidate nothing() { return Candidate{0}; }
    template <int D> __device__ __forceinline__ Candidate from_partner() const { return Candidate{partner<D>(key)}; }
};
template <> struct Candidate<true> {
    uint64_t key;
    int index;
    __device__ __forceinline__ bool none() const { return key == 0; }
    __device__ __forceinline__ int expert() const { return index; }
    __device__ __forceinline__ void take(const Candidate o)
    {
        const bool other = o.key > key || (o.key == key && o.index < index);
        key = other ? o.key : key;
        index = other ? o.index : index;
    }
    static __device__ __forceinline__ Candidate make(float, double c, int e) { return Candidate{sort_key(c), e}; }
    static __device__ __forceinline__ Candidate nothing() { return Candidate{0, 0x7FFFFFFF}; }
    template <int D> __device__ __forceinline__ Candidate from_partner() const
    {
        return Candidate{partner<D>(key), partner<D>(index)};
    }
};

template <int LPT, class T, class F> __device__ __forceinline__ T reduce_lanes(T v, F f)
{
    v = f(v, partner<8>(v));
    v = f(v, partner<4>(v));
    v = f(v, partner<2>(v));
    v = f(v, partner<1>(v));
    if constexpr (LPT == 64) {
        v = f(v, partner<16>(v));
        v = f(v, partner<32>(v));
    }
    return v;
}
template <int LPT> __device__ __forceinline__ float sum_lanes(float v)
{
    return reduce_lanes<LPT>(v, [](float a, float b) { return a + b; });
}
template <int LPT, int D, bool WIDE> __device__ __forceinline__ void take_better(Candidate<WIDE> &c)
{
    c.take(c.template from_partner<D>());
}
template <int LPT, bool WIDE> __device__ __forceinline__ Candidate<WIDE> best_of_lanes(Candidate<WIDE> c)
{
    take_better<LPT, 8>(c);
    take_better<LPT, 4>(c);
    take_better<LPT, 2>(c);
    take_better<LPT, 1>(c);
    if constexpr (LPT == 64) {
        take_better<LPT, 16>(c);
        take_better<LPT, 32>(c);
    }
    return c;
}

__device__ __forceinline__ float load_logit(const void *x, bool bf16, int64_t at)
{
    return bf16 ? __uint_as_float((uint32_t)((const uint16_t *)x)[at] << 16) : ((const float *)x)[at];
}

// ---- order --------------------------------------------------------------------

// Stable counting sort of the slots (token, j) by expert, in chunks of
// consecutive slots; slots without an expert come last ("expert" E).

// counts[e] = slots of expert e in [first, first + count), for the 256 threads.
__device__ __forceinline__ void count_slots(const RouteArgs &args, int first, int count, int32_t *counts)
{
    for (int e = threadIdx.x; e <= args.experts; e += 256)
        counts[e] = 0;
    __syncthreads();
    for (int i = threadIdx.x; i < count; i += 256) {
        const int e = args.ids[first + i];
        atomicAdd(&counts[e < 0 ? args.experts : e], 1);
    }
    __syncthreads();
}

// before[e] = total[0] + .. + total[e - 1] in LDS, by the first wave.
__device__ __forceinline__ void scan_totals(const RouteArgs &args, const int32_t *total, int32_t *before)
{
    if (threadIdx.x < 64) {
        const int lane = threadIdx.x;
        int base = 0;
        for (int e0 = 0; e0 <= args.experts; e0 += 64) {
            const int c = e0 + lane <= args.experts ? total[e0 + lane] : 0;
            int sum = c;
#pragma unroll
            for (int d = 1; d < 64; d *= 2) {
                const int v = __shfl_up(sum, d);
                if (lane >= d)
                    sum += v;
            }
            if (e0 + lane <= args.experts)
                before[e0 + lane] = base + sum - c;
            base += __shfl(sum, 63);
        }
    }
    __syncthreads();
}

// Place the slots [first, first + count): `at[e]` is the position of the first
// of them with expert e. Wave w of the four takes the w-th quarter, 64 slots at
// a time: a slot's rank among those is the number of lower lanes with the same
// expert, found by one ballot per bit of the expert's index.
__device__ __forceinline__ void place_slots(const RouteArgs &args, int first, int count, const int32_t *at,
                                            int32_t *cursor)
{
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, n = args.experts + 1;
    for (int i = threadIdx.x; i < 4 * n; i += 256)
        cursor[i] = 0;
    __syncthreads();
    const int quarter = (count + 255) / 256 * 64;
    const int lo = min(count, wave * quarter), hi = min(count, lo + quarter);
    int32_t *const mine = cursor + wave * n;
    for (int i = lo + lane; i < hi; i += 64) {
        const int e = args.ids[first + i];
        atomicAdd(&mine[e < 0 ? args.experts : e], 1);
    }
    __syncthreads();
    for (int e = threadIdx.x; e < n; e += 256) {
        int p = at[e];
        for (int w = 0; w < 4; ++w) {
            const int c = cursor[w * n + e];
            cursor[w * n + e] = p;
            p += c;
        }
    }
    __syncthreads();
    const int bits = 32 - __builtin_clz(args.experts);
    for (int i0 = lo; i0 < hi; i0 += 64) {
        const bool on = i0 + lane < hi;
        const int slot = first + i0 + lane;
        int e = on ? args.ids[slot] : 0;
        e = e < 0 ? args.experts : e;
        uint64_t same = __ballot(on);
        for (int b = 0; b < bits; ++b) {
            const bool bit = e >> b & 1;
            const uint64_t set = __ballot(bit);
            same &= bit ? set : ~set;
        }
        const int rank = __builtin_popcountll(same & ((1ull << lane) - 1));
        int p = 0;
        if (on)
            p = mine[e] + rank;
        wave_lds_exchange();
        if (on) {
            args.rows[p] = slot / args.top;
            args.positions[slot] = e == args.experts ? -2 - p : p;
            if (rank == 0)
                mine[e] = p + __builtin_popcountll(same);
        }
        wave_lds_exchange();
    }
}

__device__ __forceinline__ void store_offsets(const RouteArgs &args, const int32_t *before)
{
    for (int e = threadIdx.x; e <= args.experts; e += 256)
        args.offsets[e] = before[e];
}

// All slots in one workgroup.
__device__ __forceinline__ void order_all(const RouteArgs &args, int32_t *lds)
{
    const int n = args.experts + 1, count = args.m * args.top;
    count_slots(args, 0, count, lds);
    scan_totals(args, lds, lds + n);
    store_offsets(args, lds + n);
    place_slots(args, 0, count, lds + n, lds + 2 * n);
}

__global__ __launch_bounds__(256) void order_all_kernel(const RouteArgs args)
{
    __shared__ int32_t lds[ORDER_LDS_WORDS];
    order_all(args, lds);
}

__global__ __launch_bounds__(256) void order_count_kernel(const RouteArgs args)
{
    __shared__ int32_t lds[ROUTE_MAX_EXPERTS + 1];
    const int64_t first = (int64_t)blockIdx.x * args.chunk, slots = (int64_t)args.m * args.top;
    count_slots(args, (int)first, (int)min((int64_t)args.chunk, slots - first), lds);
    for (int e = threadIdx.x; e <= args.experts; e += 256)
        args.counts[(int64_t)blockIdx.x * (args.experts + 1) + e] = lds[e];
}

__global__ __launch_bounds__(256) void order_place_kernel(const RouteArgs args)
{
    __shared__ int32_t lds[ORDER_LDS_WORDS];
    const int n = args.experts + 1;
    int32_t *const before = lds + n;
    const int chunk = blockIdx.x;
    int32_t mine[ROUTE_MAX_EXPERTS / 256 + 1]; // slots of this thread's experts in earlier chunks
#pragma unroll
    for (int i = 0; i < ROUTE_MAX_EXPERTS / 256 + 1; ++i) {
        const int e = i * 256 + threadIdx.x;
        mine[i] = 0;
        if (e < n) {
            int total = 0;
            for (int c = 0; c < args.chunks; ++c) {
                const int v = args.counts[(int64_t)c * n + e];
                mine[i] += c < chunk ? v : 0;
                total += v;
            }
            lds[e] = total;
        }
    }
    __syncthreads();
    scan_totals(args, lds, before);
    if (chunk == 0)
        store_offsets(args, before);
    __syncthreads();
#pragma unroll
    for (int i = 0; i < ROUTE_MAX_EXPERTS / 256 + 1; ++i)
        if (i * 256 + threadIdx.x < n)
            before[i * 256 + threadIdx.x] += mine[i];
    __syncthreads();
    const int64_t first = (int64_t)chunk * args.chunk, slots = (int64_t)args.m * args.top;
    place_slots(args, (int)first, (int)min((int64_t)args.chunk, slots - first), before, lds + 2 * n);
}

// ---- choice -------------------------------------------------------------------

// The groups that stay, bit g for group g. `c` holds the token's scores in LDS
// (-inf where closed); a lane scores the groups lane, lane + LPT, ...
template <int LPT>
__device__ __forceinline__ uint64_t keep_groups(const RouteArgs &args, double *c, int lane)
{
    constexpr int GPL = ROUTE_MAX_GROUPS / LPT;
    const int size = args.experts / args.groups;
    double mine[GPL];
#pragma unroll
    for (int q = 0; q < GPL; ++q) {
        const int g = q * LPT + lane;
        double first = -INFINITY, second = -INFINITY;
        if (g < args.groups)
            for (int i = 0; i < size; ++i) {
                const double s = c[g * size + i];
                second = fmax(second, fmin(first, s));
                first = fmax(first, s);
            }
        mine[q] = args.pair && second > -INFINITY ? first + second : first;
    }
    wave_lds_exchange();
#pragma unroll
    for (int q = 0; q < GPL; ++q)
        if (q * LPT + lane < args.groups)
            c[q * LPT + lane] = mine[q];
    wave_lds_exchange();
    uint64_t kept = 0;
    for (int g = 0; g < args.groups; ++g) {
        const double s = c[g];
        int ahead = 0; // groups that come before g
#pragma unroll
        for (int q = 0; q < GPL; ++q) {
            const int h = q * LPT + lane;
            ahead += h < args.groups && (mine[q] > s || (mine[q] == s && h < g));
        }
        ahead = reduce_lanes<LPT>(ahead, [](int a, int b) { return a + b; });
        kept |= (uint64_t)(ahead < args.keep) << g;
    }
    wave_lds_exchange();
    return kept;
}

// A token is held by LPT lanes, VPL logits each (expert v LPT + lane). WIDE:
// the choice goes by 64-bit scores (a bias), otherwise by the logits.
template <int LPT, int VPL, bool WIDE>
__global__ __launch_bounds__(256) void route_kernel(const RouteArgs args)
{
    constexpr int TOKENS = 256 / LPT; // per workgroup and pass
    constexpr int CHOICE_BYTES = TOKENS * LPT * VPL * 8;
    __shared__ __align__(8) uint8_t lds[CHOICE_BYTES > ORDER_LDS_WORDS * 4 ? CHOICE_BYTES : ORDER_LDS_WORDS * 4];
    const int lane = threadIdx.x & (LPT - 1), slot = threadIdx.x / LPT;
    double *const scores = (double *)lds + slot * LPT * VPL;
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
        top = reduce_lanes<LPT>(top, [](float a, float b) { return fmaxf(a, b); });
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
        const bool wide = WIDE || (args.groups > 1 && args.pair);
        if (wide) {
            double all = 1.;
            if (!args.sigmoid) {
                all = 0.;
#pragma unroll
                for (int v = 0; v < VPL; ++v) {
                    c[v] = exp((double)x[v] - (double)top);
                    all += c[v];
                }
                all = reduce_lanes<LPT>(all, [](double a, double b) { return a + b; });
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
        Candidate<WIDE> cand[VPL];
#pragma unroll
        for (int v = 0; v < VPL; ++v)
            cand[v] = x[v] > -INFINITY && c[v] > -INFINITY ? Candidate<WIDE>::make(x[v], c[v], v * LPT + lane)
                                                           : Candidate<WIDE>::nothing();
        if (args.groups > 1) {
            const int size = experts / args.groups;
#pragma unroll
            for (int v = 0; v < VPL; ++v)
                scores[v * LPT + lane] = cand[v].none() ? -INFINITY : c[v];
            wave_lds_exchange();
            const uint64_t kept = keep_groups<LPT>(args, scores, lane);
#pragma unroll
            for (int v = 0; v < VPL; ++v)
                if (!(kept >> (min(v * LPT + lane, experts - 1) / size) & 1))
                    cand[v].key = 0;
        }
        // the best ones in turn; slot j belongs to lane j % 16 (of every row of lanes)
        int id[ROUTE_MAX_TOP / 16];
#pragma unroll
        for (int q = 0; q < ROUTE_MAX_TOP / 16; ++q)
            id[q] = -1;
        for (int j = 0; j < args.top; ++j) {
            Candidate<WIDE> best = cand[0];
#pragma unroll
            for (int v = 1; v < VPL; ++v)
                best.take(cand[v]);
            best = best_of_lanes<LPT>(best);
            const int e = best.none() ? -1 : best.expert();
#pragma unroll
            for (int v = 0; v < VPL; ++v)
                cand[v].key = v * LPT + lane == e ? 0 : cand[v].key;
#pragma unroll
            for (int q = 0; q < ROUTE_MAX_TOP / 16; ++q)
                if (j == q * 16 + (lane & 15))
                    id[q] = e;
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
                    args.ids[token * args.top + q * 16 + lane] = id[q];
                    args.weights[token * args.top + q * 16 + lane] = id[q] < 0 ? 0.f : p[q] * factor;
                }
        }
    }
    if (args.fused) { // this workgroup has had every token
        __threadfence_block();
        __syncthreads();
        order_all(args, (int32_t *)lds);
    }
}

// ---- gradient -----------------------------------------------------------------

// dL/dx from dL/dw, for the chosen experts of `ids` (the choice itself has no
// gradient; the bias only takes part in the choice):
//   renormalised:  dL/dp_j = scale / S (dw_j - sum_i dw_i p_i / S), S = sum p + 1e-20
//   otherwise:     dL/dp_j = scale dw_j
//   softmax:       dL/dx_e = p_e (dL/dp_e - sum_j dL/dp_j p_j)
//   sigmoid:       dL/dx_e = dL/dp_e p_e (1 - p_e)
// The scores are computed again. An id outside [0, experts) has no score.
template <int LPT, int VPL>
__global__ __launch_bounds__(256) void route_backward_kernel(const RouteGradArgs args)
{
    constexpr int TOKENS = 256 / LPT;
    const int lane = threadIdx.x & (LPT - 1), slot = threadIdx.x / LPT;
    const int experts = args.experts;
    const int64_t token = (int64_t)blockIdx.x * TOKENS + slot;
    const bool live = token < args.m;
    float x[VPL], top = -INFINITY;
#pragma unroll
    for (int v = 0; v < VPL; ++v) {
        const int e = v * LPT + lane;
        x[v] = live && e < experts ? load_logit(args.logits, args.bf16, token * args.ld + e) : -INFINITY;
        top = fmaxf(top, x[v]);
    }
    top = reduce_lanes<LPT>(top, [](float a, float b) { return fmaxf(a, b); });
    top = top == -INFINITY ? 0.f : top;
    float p[VPL], total = 0.f;
#pragma unroll
    for (int v = 0; v < VPL; ++v) {
        p[v] = args.sigmoid ? 1.f / (1.f + expf(-x[v])) : expf(x[v] - top);
        total += p[v];
    }
    if (!args.sigmoid) {
        total = sum_lanes<LPT>(total);
        total = total == 0.f ? 1.f : total;
#pragma unroll
        for (int v = 0; v < VPL; ++v)
            p[v] /= total;
    }
    // this lane's slots: j = q 16 + lane % 16
    int id[ROUTE_MAX_TOP / 16];
    float dw[ROUTE_MAX_TOP / 16], score[ROUTE_MAX_TOP / 16], sum = 0.f, dot = 0.f;
#pragma unroll
    for (int q = 0; q < ROUTE_MAX_TOP / 16; ++q) {
        const int j = q * 16 + (lane & 15);
        id[q] = live && j < args.top ? args.ids[token * args.top + j] : -1;
        if (id[q] >= experts)
            id[q] = -1;
        dw[q] = score[q] = 0.f;
        if (id[q] >= 0) {
            dw[q] = args.dweights[token * args.top + j];
            const float v = load_logit(args.logits, args.bf16, token * args.ld + id[q]);
            score[q] = args.sigmoid ? 1.f / (1.f + expf(-v)) : expf(v - top) / total;
        }
        sum += score[q];
        dot += dw[q] * score[q];
    }
    sum = sum_lanes<16>(sum) + ROUTE_EPS;
    dot = sum_lanes<16>(dot) / sum;
    float back = 0.f;
#pragma unroll
    for (int q = 0; q < ROUTE_MAX_TOP / 16; ++q) {
        dw[q] = args.renorm ? (dw[q] - dot) * (args.scale / sum) : dw[q] * args.scale;
        back += id[q] >= 0 ? dw[q] * score[q] : 0.f;
    }
    back = sum_lanes<16>(back);
    float dp[VPL];
#pragma unroll
    for (int v = 0; v < VPL; ++v)
        dp[v] = 0.f;
    for (int j = 0; j < args.top; ++j) {
        int e = -1;
        float d = 0.f;
#pragma unroll
        for (int q = 0; q < ROUTE_MAX_TOP / 16; ++q)
            if (j / 16 == q) {
                e = __shfl(id[q], (threadIdx.x & 48) + j % 16);
                d = __shfl(dw[q], (threadIdx.x & 48) + j % 16);
            }
#pragma unroll
        for (int v = 0; v < VPL; ++v)
            if (v * LPT + lane == e)
                dp[v] += d;
    }
    if (live) {
#pragma unroll
        for (int v = 0; v < VPL; ++v) {
            const int e = v * LPT + lane;
            const float d = args.sigmoid ? dp[v] * p[v] * (1.f - p[v]) : p[v] * (dp[v] - back);
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
