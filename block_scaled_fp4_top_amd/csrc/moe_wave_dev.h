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

template <int CTRL>
__device__ __forceinline__ float dpp_move(float v) { return u2f(dpp_move<CTRL>(f2u(v))); }
template <int CTRL>
__device__ __forceinline__ double dpp_move(double v) {
    const uint64_t b = __builtin_bit_cast(uint64_t, v);
    const uint32_t lo = dpp_move<CTRL>((uint32_t)b), hi = dpp_move<CTRL>((uint32_t)(b >> 32));
    return __builtin_bit_cast(double, ((uint64_t)hi << 32) | lo);
}
__device__ __forceinline__ double lane_f64(double v, int lane) {
    const uint64_t b = __builtin_bit_cast(uint64_t, v);
    const uint32_t lo = __builtin_amdgcn_readlane((int)(uint32_t)b, lane), hi = __builtin_amdgcn_readlane((int)(b >> 32), lane);
    return __builtin_bit_cast(double, ((uint64_t)hi << 32) | lo);
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
__device__ __forceinline__ double lanes_max(double v) {
    auto more = [](double a, double b) { return a > b ? a : b; };
    v = more(v, dpp_move<kRor8>(v));
    v = more(v, dpp_move<kRor4>(v));
    v = more(v, dpp_move<kRor2>(v));
    v = more(v, dpp_move<kRor1>(v));
    return more(more(lane_f64(v, 0), lane_f64(v, 16)), more(lane_f64(v, 32), lane_f64(v, 48)));
}

}  // namespace moe
