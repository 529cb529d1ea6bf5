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

// 16 bytes of a row, read and written in one access at any alignment of its
// elements (gfx950 takes global memory at any byte address).
template <typename T>
struct Vec {
    T e[16 / sizeof(T)];
};
typedef uint32_t words4_at2 __attribute__((ext_vector_type(4), aligned(2)));
template <typename T>
__device__ __forceinline__ Vec<T> load_vec(const T* p) {
    const words4_at2 v = *reinterpret_cast<const words4_at2*>(p);
    return __builtin_bit_cast(Vec<T>, v);
}
// PAST: a store that leaves the caches to others.
template <bool PAST, typename T>
__device__ __forceinline__ void store_vec(T* p, const Vec<T>& v) {
    const words4_at2 w = __builtin_bit_cast(words4_at2, v);
    if constexpr (PAST) __builtin_nontemporal_store(w, reinterpret_cast<words4_at2*>(p));
    else *reinterpret_cast<words4_at2*>(p) = w;
}

// N consecutive elements (16 or 32 bytes of them) at any alignment of one, as floats.
template <int N, typename T>
__device__ __forceinline__ void load_floats(const T* p, float* f) {
    constexpr int V = 16 / sizeof(T);
    if constexpr (N < V) {  // 8 bytes of 16-bit elements
        static_assert(N * sizeof(T) == 8, "half a vector");
        typedef uint32_t words2_at2 __attribute__((ext_vector_type(2), aligned(2)));
        struct Half { T e[N]; };
        const Half h = __builtin_bit_cast(Half, *reinterpret_cast<const words2_at2*>(p));
#pragma unroll
        for (int i = 0; i < N; ++i) f[i] = to_f32(h.e[i]);
    } else {
#pragma unroll
        for (int g = 0; g < N / V; ++g) {
            const Vec<T> v = load_vec(p + g * V);
#pragma unroll
            for (int i = 0; i < V; ++i) f[g * V + i] = to_f32(v.e[i]);
        }
    }
}

}  // namespace moe
