// Reductions across the lanes of a wave without LDS.
#pragma once

#include "device/common.h"

namespace pts {

// v combined with the value of another lane, so that after D = 8, 4, 2, 1 (and
// 16, 32) every lane of a token has the combination of all: within a row of 16
// lanes by a DPP rotation, across rows by the lane-swap instructions, which
// leave both sides' values in two registers.
template <int D, class F> __device__ __forceinline__ uint32_t reduce_step(uint32_t v, F f)
{
    if constexpr (D < 16) {
        return f(v, (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0x120 + D, 0xF, 0xF, true));
    } else {
        const auto r = D == 16 ? __builtin_amdgcn_permlane16_swap(v, v, false, false)
                               : __builtin_amdgcn_permlane32_swap(v, v, false, false);
        return f(r[0], r[1]);
    }
}
template <int LPT, class F> __device__ __forceinline__ uint32_t reduce_lanes(float v, F f) = delete; // by its bits
template <int LPT, class F> __device__ __forceinline__ uint32_t reduce_lanes(uint32_t v, F f)
{
    v = reduce_step<8>(v, f);
    v = reduce_step<4>(v, f);
    v = reduce_step<2>(v, f);
    v = reduce_step<1>(v, f);
    if constexpr (LPT == 64) {
        v = reduce_step<16>(v, f);
        v = reduce_step<32>(v, f);
    }
    return v;
}

} // namespace pts
