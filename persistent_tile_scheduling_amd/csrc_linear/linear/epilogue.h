// What a linear layer's products do with a sum before they write it: eight
// consecutive columns of one row at a time, all in fp32 and rounded once.
#pragma once

#include "linear/activation.h"
#include "linear/tile.h"

namespace pts {

// Eight (or the first `valid`) values of a row to and from memory; whole: `p` is 16-byte aligned.
__device__ __forceinline__ void put8(uint16_t *p, const u32x4 &v, int valid, bool whole)
{
    if (whole && valid >= 8) {
        __builtin_nontemporal_store(v, (u32x4 *)p);
        return;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i)
        if (i < valid)
            p[i] = (uint16_t)(v[i / 2] >> (16 * (i & 1)));
}
__device__ __forceinline__ u32x4 to_bf16(const float (&v)[8])
{
    u32x4 w;
#pragma unroll
    for (int i = 0; i < 4; ++i)
        w[i] = __builtin_bit_cast(uint32_t, bf16x2{(__bf16)v[2 * i], (__bf16)v[2 * i + 1]});
    return w;
}
__device__ __forceinline__ void put8(float *p, const float (&v)[8], int valid, bool whole)
{
    if (whole && valid >= 8) {
        __builtin_nontemporal_store(*(const f32x4 *)v, (f32x4 *)p);
        __builtin_nontemporal_store(*(const f32x4 *)(v + 4), (f32x4 *)(p + 4));
        return;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i)
        if (i < valid)
            p[i] = v[i];
}
__device__ __forceinline__ void from_bf16(const u32x4 &w, float (&v)[8])
{
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[2 * i] = __uint_as_float(w[i] << 16);
        v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
}
__device__ __forceinline__ void get8(const uint16_t *p, float (&v)[8], int valid, bool whole)
{
    if (whole && valid >= 8) {
        from_bf16(*(const u32x4 *)p, v);
        return;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i)
        v[i] = i < valid ? __uint_as_float((uint32_t)p[i] << 16) : 0.f;
}
__device__ __forceinline__ void get8(const float *p, float (&v)[8], int valid, bool whole)
{
    if (whole && valid >= 8) {
        *(f32x4 *)v = *(const f32x4 *)p;
        *(f32x4 *)(v + 4) = *(const f32x4 *)(p + 4);
        return;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i)
        v[i] = i < valid ? p[i] : 0.f;
}

// Eight values as they lie in memory, loaded ahead of their use.
struct Raw8 {
    u32x4 lo, hi;
};
template <bool F32> __device__ __forceinline__ void fetch8(Raw8 &r, const void *p, int64_t at)
{
    if constexpr (F32) {
        r.lo = *(const u32x4 *)((const float *)p + at);
        r.hi = *(const u32x4 *)((const float *)p + at + 4);
    } else {
        r.lo = *(const u32x4 *)((const uint16_t *)p + at);
    }
}
__device__ __forceinline__ void from_f32(const Raw8 &r, float (&v)[8])
{
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[i] = __uint_as_float(r.lo[i]);
        v[4 + i] = __uint_as_float(r.hi[i]);
    }
}
// An epilogue's store has three parts: start, once for a lane's columns; fetch, what a row's results need from memory,
// ahead of them; finish, the results.
struct LinearArgs {
    void *d;
    const void *bias;     // of n, or null
    const void *residual; // of D's type, or null
    uint16_t *z;          // the sums before the activation, or null
    int64_t ldd, ldr, ldz;
    int32_t d_f32, bias_f32, act;
    int32_t d_whole, r_whole, z_whole; // rows start at whole 16 bytes
};

// z = sum + bias; D = act(z) + residual.
template <int ACT> struct LinearStore {
    static constexpr bool MIRROR = false;
    using Raw = Raw8;
    struct Start {
        float bias[8];
    };
    static __device__ __forceinline__ Start start(const LinearArgs &args, int, int col, int valid)
    {
        Start s;
#pragma unroll
        for (int i = 0; i < 8; ++i)
            s.bias[i] = 0.f;
        if (args.bias != nullptr) {
            if (args.bias_f32)
                get8((const float *)args.bias + col, s.bias, valid, false);
            else
                get8((const uint16_t *)args.bias + col, s.bias, valid, false);
        }
        return s;
    }
    static __device__ __forceinline__ void fetch(const LinearArgs &args, int, int row, int col, int valid, Raw8 &r)
    {
        if (args.residual != nullptr && args.r_whole && valid >= 8) {
            if (args.d_f32)
                fetch8<true>(r, args.residual, row * args.ldr + col);
            else
                fetch8<false>(r, args.residual, row * args.ldr + col);
        }
    }
    static __device__ __forceinline__ void finish(const LinearArgs &args, const Start &s, const Raw8 &fetched, int, int row,
                                                  int col, int valid, float (&v)[8])
    {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            v[i] += s.bias[i];
        if (args.z != nullptr)
            put8(args.z + row * args.ldz + col, to_bf16(v), valid, args.z_whole);
#pragma unroll
        for (int i = 0; i < 8; ++i)
            v[i] = activate<ACT>(v[i]);
        if (args.residual != nullptr) {
            float r[8];
            if (args.d_f32) {
                if (args.r_whole && valid >= 8)
                    from_f32(fetched, r);
                else
                    get8((const float *)args.residual + row * args.ldr + col, r, valid, false);
            } else {
                if (args.r_whole && valid >= 8)
                    from_bf16(fetched.lo, r);
                else
                    get8((const uint16_t *)args.residual + row * args.ldr + col, r, valid, false);
            }
#pragma unroll
            for (int i = 0; i < 8; ++i)
                v[i] += r[i];
        }
        if (args.d_f32)
            put8((float *)args.d + row * args.ldd + col, v, valid, args.d_whole);
        else
            put8((uint16_t *)args.d + row * args.ldd + col, to_bf16(v), valid, args.d_whole);
    }
};

struct LinearEpilogue {
    using Args = LinearArgs;
    template <class F> static __device__ __forceinline__ void run(const Args &args, F &&f)
    {
        with_activation(args.act, [&](auto act) { f(LinearStore<decltype(act)::value>{}); });
    }
};

// D = sum (the gradients' products).
struct PlainStore {
    static constexpr bool MIRROR = false;
    using Raw = Raw8;
    struct Start {};
    static __device__ __forceinline__ Start start(const LinearArgs &, int, int, int) { return {}; }
    static __device__ __forceinline__ void fetch(const LinearArgs &, int, int, int, int, Raw8 &) {}
    static __device__ __forceinline__ void finish(const LinearArgs &args, const Start &, const Raw8 &, int, int row, int col,
                                                  int valid, float (&v)[8])
    {
        if (args.d_f32)
            put8((float *)args.d + row * args.ldd + col, v, valid, args.d_whole);
        else
            put8((uint16_t *)args.d + row * args.ldd + col, to_bf16(v), valid, args.d_whole);
    }
};
struct PlainEpilogue {
    using Args = LinearArgs;
    template <class F> static __device__ __forceinline__ void run(const Args &, F &&f) { f(PlainStore{}); }
};

} // namespace pts
