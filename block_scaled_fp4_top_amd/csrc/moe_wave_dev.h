// Sums and maxima over the lanes of a wave by DPP rotations and lane reads (no LDS),
// and over the waves of a block. Every lane gets the same bits; the order is fixed.
#pragma once

#include "moe_internal.h"

namespace moe {

template <int CTRL>
__device__ __forceinline__ uint32_t dpp_move(uint32_t v) {
    return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, 0xF, 0xF, false);
}
constexpr int kRor8 = 0x128, kRor4 = 0x124, kRor2 = 0x122, kRor1 = 0x121;  // rotations in a row of 16 lanes

__device__ __forceinline__ float lane_f32(float v, int lane) {
    return u2f((uint32_t)__builtin_amdgcn_readlane((int)f2u(v), lane));
}

// over the 16 lanes of a row
__device__ __forceinline__ float row_sum(float v) {
    v += u2f(dpp_move<kRor8>(f2u(v)));
    v += u2f(dpp_move<kRor4>(f2u(v)));
    v += u2f(dpp_move<kRor2>(f2u(v)));
    v += u2f(dpp_move<kRor1>(f2u(v)));
    return v;
}
__device__ __forceinline__ uint32_t row_max(uint32_t v) {
    v = max(v, dpp_move<kRor8>(v));
    v = max(v, dpp_move<kRor4>(v));
    v = max(v, dpp_move<kRor2>(v));
    v = max(v, dpp_move<kRor1>(v));
    return v;
}

// over the wave
__device__ __forceinline__ float lanes_sum(float v) {
    v = row_sum(v);
    return (lane_f32(v, 0) + lane_f32(v, 16)) + (lane_f32(v, 32) + lane_f32(v, 48));
}
__device__ __forceinline__ uint32_t lanes_max(uint32_t v) {
    v = row_max(v);
    auto at = [&](int lane) { return (uint32_t)__builtin_amdgcn_readlane((int)v, lane); };
    return max(max(at(0), at(16)), max(at(32), at(48)));
}

}  // namespace moe
