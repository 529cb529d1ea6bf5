// Codes of the symmetric 8-bit quantizer: the correctly rounded quotients of a row's
// values by the row's fp32 scale.
#pragma once

#include "moe_internal.h"

namespace moe {

// Codes are the correctly rounded quotients x / s of the row's fp32 scale s (ties
// to even). q = x * fl(1/s) is within 127 * 2^-23 of the quotient, so rint(q) is
// the code unless q lies within kNear of a half; there the sign of the exact
// remainder x - n s (one fma: at most 24 bits remain) against s / 2 decides.
constexpr float kNear = 2e-5f;            // > 127 * 2^-23
constexpr float kRoundInt = 12582912.0f;  // 1.5 * 2^23: adding it rounds to an integer, held in the low bits
constexpr float kTinyScale = 1e-37f;      // 1/s overflows below 2^-128: such rows divide in fp64

__device__ __forceinline__ int int8_code_exact(float x, float s, float inv) {
    if (s < kTinyScale) return (int)fmin(fmax(rint((double)x / (double)s), -127.0), 127.0);
    float n = __builtin_rintf(x * inv);
    const float r2 = 2.0f * __fmaf_rn(-n, s, x);  // twice the remainder, exact
    const bool odd = ((int)n) & 1;
    if (r2 > s || (r2 == s && odd)) n += 1.0f;
    else if (r2 < -s || (r2 == -s && odd)) n -= 1.0f;
    return (int)n;
}

// What a row's codes need: its scale and the quotient's factor. Zero, infinity and
// NaN: codes 0, by a factor of 0 (and no careful rounding).
struct Int8Row {
    float s, inv;
    bool plain, tiny;
};
// top: the bits of the row's largest |x|, which order like the values, NaN above infinity
__device__ __forceinline__ Int8Row int8_row(uint32_t top) {
    Int8Row r;
    r.s = __fdiv_rn(u2f(top), 127.0f);
    r.plain = r.s > 0.0f && top < 0x7F800000u;
    r.tiny = r.plain && r.s < kTinyScale;
    r.inv = r.plain && !r.tiny ? __fdiv_rn(1.0f, r.s) : 0.0f;
    return r;
}

template <int N>
struct Codes {
    uint32_t w[N / 4];
};

// Four codes in one word, from values rounded by adding kRoundInt.
__device__ __forceinline__ uint32_t int8_word(const uint32_t* b) {
    const uint32_t lo = __builtin_amdgcn_perm(b[1], b[0], 0x0C0C0400u), hi = __builtin_amdgcn_perm(b[3], b[2], 0x0C0C0400u);
    return lo | (hi << 16);
}

// The codes of N values, packed.
template <int N>
__device__ __forceinline__ Codes<N> int8_codes(const float* f, const Int8Row& r) {
    Codes<N> c;
    float far = 0.0f;
#pragma unroll
    for (int g = 0; g < N / 4; ++g) {
        uint32_t b[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float x = f[4 * g + i];
            const float n = __fmaf_rn(x, r.inv, kRoundInt);
            b[i] = f2u(n);
            far = fmaxf(far, fabsf(__fmaf_rn(x, r.inv, -(n - kRoundInt))));
        }
        c.w[g] = int8_word(b);
    }
    if (!r.plain) {
#pragma unroll
        for (int g = 0; g < N / 4; ++g) c.w[g] = 0;
    } else if (r.tiny || far > 0.5f - kNear) {
#pragma unroll
        for (int g = 0; g < N / 4; ++g) {
            c.w[g] = 0;
#pragma unroll
            for (int i = 0; i < 4; ++i)
                c.w[g] |= (uint32_t)(int8_code_exact(f[4 * g + i], r.s, r.inv) & 0xFF) << (8 * i);
        }
    }
    return c;
}

template <int N>
__device__ __forceinline__ void store_codes(int8_t* dst, const Codes<N>& c) {
    typedef uint32_t words __attribute__((ext_vector_type(N / 4), aligned(1)));
    *reinterpret_cast<words*>(dst) = __builtin_bit_cast(words, c);
}

}  // namespace moe
