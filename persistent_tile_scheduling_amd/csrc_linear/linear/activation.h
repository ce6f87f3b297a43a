// The activations of a linear layer and their slopes, in fp32.
//
// An activation stands in a product's epilogue, where eight waves put 65536 values
// through it with nothing else to do, its slope in a pass that gelu's would bound
// by its instructions (5000 x 7000: 53 us with corrected exponentials and
// reciprocals, 48 without). So both take the hardware's as they are. An
// activation is good to 16 steps of 2^-24 of its value and, from the rounding of
// its exponential's argument, 3 |argument| more: 2^-20 of the value for |z| < 5. A
// slope is good to as many steps of its two terms, Phi(z) and z Phi'(z) (p and z p'),
// in the tails too; its value is as good but near its own zero, where they cancel.
// Measured over every bf16: 5 steps for arguments below 4, 36 at 40. What lies below
// 2^-119, and silu and gelu_tanh left of an argument of -88, is 0.
//
// gelu is z Phi(z). With a = |z|, Phi(-a) = exp(-a^2 / 2) G(a), where G(a) =
// erfcx(a / sqrt 2) / 2 falls smoothly from 1/2 like 1 / (a sqrt(2 pi)); it is a
// polynomial of degree 9 in t = 1 / (1 + 0.35 a), without a constant term, fitted
// here to the least relative error on Chebyshev points of t (3.2e-8; 3.3e-7 with
// its evaluation in fp32). 1 + erf would lose the left tail to cancellation.
#pragma once

#include "device/common.h"

namespace pts {

// -2 sqrt(2 / pi) / ln 2 and 0.044715 of it
constexpr float GELU_C = -0x1.26aec2p+1f, GELU_D = -0x1.a5a7d0p-4f;

enum : int { ACT_NONE = 0, ACT_RELU = 1, ACT_GELU = 2, ACT_GELU_TANH = 3, ACT_SILU = 4 };

// v within [-most, most]; NaN stays.
__device__ __forceinline__ float within(float v, float most) { return v > most ? most : v < -most ? -most : v; }

// G(a) / t of a polynomial of degree 9 in t, above.
__device__ __forceinline__ float normal_poly(float t)
{
    float g = -0x1.ddb7c2p-6f;
    g = fmaf(g, t, 0x1.26f8e2p-3f);
    g = fmaf(g, t, -0x1.05f9cep-2f);
    g = fmaf(g, t, 0x1.464764p-3f);
    g = fmaf(g, t, -0x1.7c4432p-6f);
    g = fmaf(g, t, 0x1.b05690p-4f);
    g = fmaf(g, t, 0x1.eaca10p-4f);
    g = fmaf(g, t, 0x1.1e70bep-3f);
    return fmaf(g, t, 0x1.1df1c6p-3f);
}

// exp(-a^2 / 2) and Phi(-a), a >= 0.
struct Normal {
    float bell, below;
};
__device__ __forceinline__ Normal normal(float a)
{
    Normal n;
    n.bell = __builtin_amdgcn_exp2f(a * a * -0x1.715476p-1f); // -1 / (2 ln 2)
    const float t = __builtin_amdgcn_rcpf(fmaf(0.35f, a, 1.0f));
    n.below = n.bell * (normal_poly(t) * t);
    return n;
}

// The logistic function p of an argument whose negative over ln 2 is u, and p (1 - p), from 2^-|u|, since 1 - p is lost in
// the rounding of a p near 1.
struct Logistic {
    float p, slope;
};
__device__ __forceinline__ Logistic logistic(float u)
{
    const float e = __builtin_amdgcn_exp2f(-fabsf(u));
    const float r = __builtin_amdgcn_rcpf(1.0f + e);
    return Logistic{u > 0.f ? e * r : r, e * r * r};
}

template <int ACT> __device__ __forceinline__ float activate(float z)
{
    if constexpr (ACT == ACT_RELU)
        return z < 0.f ? 0.f : z;
    if constexpr (ACT == ACT_GELU) {
        const float a = fminf(fabsf(z), 16.0f); // beyond, Phi(-a) is 0
        return (z < 0.f ? 0.f : z) - a * normal(a).below;
    }
    if constexpr (ACT == ACT_GELU_TANH) { // z / (1 + 2^(z (c + d z^2))), c = -2 sqrt(2 / pi) / ln 2, d = 0.044715 c
        const float e = __builtin_amdgcn_exp2f(z * fmaf(z * z, GELU_D, GELU_C));
        return z * __builtin_amdgcn_rcpf(1.0f + e);
    }
    if constexpr (ACT == ACT_SILU)
        return z * __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(z * -0x1.715476p+0f));
    return z;
}

template <int ACT> __device__ __forceinline__ float activation_slope(float z)
{
    if constexpr (ACT == ACT_RELU)
        return z > 0.f ? 1.f : 0.f;
    if constexpr (ACT == ACT_GELU) { // Phi(z) + z exp(-z^2 / 2) / sqrt(2 pi)
        const float c = within(z, 16.0f);
        const Normal n = normal(fabsf(c));
        return fmaf(c * 0x1.988454p-2f, n.bell, z > 0.f ? 1.0f - n.below : n.below);
    }
    if constexpr (ACT == ACT_GELU_TANH) { // p + z p (1 - p) u', u = 2 sqrt(2 / pi) (z + 0.044715 z^3)
        const float c = within(z, 16.0f), s = c * c;
        const Logistic l = logistic(c * fmaf(s, GELU_D, GELU_C));
        return fmaf(c * fmaf(s, 3.0f * 0x1.2444f2p-4f, 0x1.988454p+0f), l.slope, l.p);
    }
    if constexpr (ACT == ACT_SILU) {
        const float c = within(z, 128.0f);
        const Logistic l = logistic(c * -0x1.715476p+0f);
        return fmaf(c, l.slope, l.p);
    }
    return 1.f;
}

// f(IntC<activation>{}) for an activation known at run time.
template <class F> __device__ __forceinline__ void with_activation(int act, F &&f)
{
    switch (act) {
    case ACT_RELU:
        return f(IntC<ACT_RELU>{});
    case ACT_GELU:
        return f(IntC<ACT_GELU>{});
    case ACT_GELU_TANH:
        return f(IntC<ACT_GELU_TANH>{});
    case ACT_SILU:
        return f(IntC<ACT_SILU>{});
    default:
        return f(IntC<ACT_NONE>{});
    }
}

} // namespace pts
