// Element types of activations and their 16-byte vectors at any element
// alignment.
#pragma once

#include "moe_internal.h"

namespace moe {

struct Bf16 { uint16_t v; };
struct Fp16 { _Float16 v; };
__device__ __forceinline__ float to_f32(Bf16 x) { return u2f((uint32_t)x.v << 16); }
__device__ __forceinline__ float to_f32(Fp16 x) { return (float)x.v; }
__device__ __forceinline__ float to_f32(float x) { return x; }
// round to nearest even by the hardware converters (a NaN stays one)
template <typename T> __device__ __forceinline__ T from_f32(float f);
template <> __device__ __forceinline__ Bf16 from_f32<Bf16>(float f) {
    return Bf16{__builtin_bit_cast(uint16_t, (__bf16)f)};
}
template <> __device__ __forceinline__ Fp16 from_f32<Fp16>(float f) { return Fp16{(_Float16)f}; }
template <> __device__ __forceinline__ float from_f32<float>(float f) { return f; }

// 16 bytes of a row at any alignment of its elements (gfx950 loads and stores
// global memory at any byte address).
template <typename T>
struct __attribute__((packed, aligned(sizeof(T)))) Vec {
    T e[16 / sizeof(T)];
};

}  // namespace moe
