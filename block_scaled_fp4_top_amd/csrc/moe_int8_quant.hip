// Symmetric 8-bit integer quantization of each row:
//   s[m] = fl32(max_j |x[m,j]| / 127),  c[m,j] = round(x[m,j] / s[m])
#include "moe_args.h"
#include "moe_rows_dev.h"

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

// One row per TPT threads (a wave, or a block of 256), read once: each thread keeps
// up to NV vectors of 16 bytes in registers between the maximum and the rounding
// (LONG: rows of any length, read twice). Bound by memory: 16384 x 7168 bf16
// (352 MB) takes 66 us, 5.3 TB/s.
template <typename T, int TPT, int NV, bool LONG>
__global__ __launch_bounds__(256) void int8_quantize_kernel(const T* __restrict__ x, int64_t ld, int rows, int H,
                                                            int8_t* __restrict__ codes, int64_t ld_codes,
                                                            float* __restrict__ scales) {
    constexpr int V = 16 / sizeof(T);
    __shared__ uint32_t s_top[256 / 64];
    const int lane = threadIdx.x & 63, at = threadIdx.x % TPT;
    const int m = __builtin_amdgcn_readfirstlane(blockIdx.x * (256 / TPT) + (TPT == 64 ? threadIdx.x >> 6 : 0));
    if (m >= rows) return;  // (a whole block for TPT = 256, which alone has barriers)
    const T* row = x + (int64_t)m * ld;
    int8_t* dst = codes + (int64_t)m * ld_codes;
    const int whole = H / V;  // vectors; the H % V elements behind them belong to the first threads
    const int tail = H - whole * V;
    // the bits of |x| order like the values, NaN above infinity
    uint32_t top = 0;
    Vec<T> v[NV];
    T last{};
#pragma unroll
    for (int j = 0; j < NV; ++j)
        if (at + j * TPT < whole) v[j] = load_vec(row + (at + j * TPT) * V);
    if (at < tail) last = row[whole * V + at];
#pragma unroll
    for (int j = 0; j < NV; ++j)
        if (at + j * TPT < whole) {
#pragma unroll
            for (int i = 0; i < V; ++i) top = max(top, f2u(to_f32(v[j].e[i])) & 0x7FFFFFFFu);
        }
    if (at < tail) top = max(top, f2u(to_f32(last)) & 0x7FFFFFFFu);
    if (LONG) {
        for (int c = at + NV * TPT; c < whole; c += TPT) {
            const Vec<T> u = load_vec(row + (int64_t)c * V);
#pragma unroll
            for (int i = 0; i < V; ++i) top = max(top, f2u(to_f32(u.e[i])) & 0x7FFFFFFFu);
        }
    }
#pragma unroll
    for (int off = 32; off >= 1; off >>= 1) top = max(top, (uint32_t)__shfl_xor((int)top, off));
    if (TPT == 256) {
        if (lane == 0) s_top[threadIdx.x >> 6] = top;
        __syncthreads();
        top = max(max(s_top[0], s_top[1]), max(s_top[2], s_top[3]));
    }
    top = __builtin_amdgcn_readfirstlane(top);
    const float s = __fdiv_rn(u2f(top), 127.0f);
    if (at == 0) scales[m] = s;
    // zero, infinity and NaN: codes 0, by a factor of 0 (and no careful rounding)
    const bool plain = s > 0.0f && top < 0x7F800000u;
    const bool tiny = plain && s < kTinyScale;
    const float inv = plain && !tiny ? __fdiv_rn(1.0f, s) : 0.0f;
    auto put = [&](const Vec<T>& u, int c) {
        uint32_t w[V / 4];
        float far = 0.0f;
#pragma unroll
        for (int g = 0; g < V / 4; ++g) {
            uint32_t b[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float f = to_f32(u.e[4 * g + i]);
                const float n = __fmaf_rn(f, inv, kRoundInt);
                b[i] = f2u(n);
                far = fmaxf(far, fabsf(__fmaf_rn(f, inv, -(n - kRoundInt))));
            }
            const uint32_t lo = __builtin_amdgcn_perm(b[1], b[0], 0x0C0C0400u), hi = __builtin_amdgcn_perm(b[3], b[2], 0x0C0C0400u);
            w[g] = lo | (hi << 16);
        }
        if (!plain) {
#pragma unroll
            for (int g = 0; g < V / 4; ++g) w[g] = 0;
        } else if (tiny || far > 0.5f - kNear) {
#pragma unroll
            for (int g = 0; g < V / 4; ++g) {
                w[g] = 0;
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    w[g] |= (uint32_t)(int8_code_exact(to_f32(u.e[4 * g + i]), s, inv) & 0xFF) << (8 * i);
            }
        }
        typedef uint32_t words __attribute__((ext_vector_type(V / 4), aligned(1)));
        *reinterpret_cast<words*>(dst + (int64_t)c * V) = __builtin_bit_cast(words, w);
    };
#pragma unroll
    for (int j = 0; j < NV; ++j)
        if (at + j * TPT < whole) put(v[j], at + j * TPT);
    if (at < tail) dst[whole * V + at] = plain ? (int8_t)int8_code_exact(to_f32(last), s, inv) : (int8_t)0;
    if (LONG)
        for (int c = at + NV * TPT; c < whole; c += TPT) put(load_vec(row + (int64_t)c * V), c);
}

template <typename T>
static hipError_t launch_int8_quantize(const T* x, int64_t ld, int rows, int H, int8_t* codes, int64_t ld_codes,
                                       float* scales, hipStream_t s) {
    constexpr int V = 16 / (int)sizeof(T);
    const int vecs = (H + V - 1) / V;
#define Q(TPT, NV, LONG)                                                                                       \
    hipLaunchKernelGGL((int8_quantize_kernel<T, TPT, NV, LONG>), dim3((rows + 256 / TPT - 1) / (256 / TPT)),   \
                       dim3(256), 0, s, x, ld, rows, H, codes, ld_codes, scales)
    // a wave per row for many rows of up to 256 vectors, a block for few and for longer
    // ones. bf16 in a graph, us, with a wave (with a block): 16384 x 1024 12.3 (17.6), x 1536
    // 17.2 (19.9), x 2048 25.5 (25.0), 65536 x 2048 77 (87); 4096 x 1024 5.2 (6.2), x 1536 7.7
    // (7.4), x 2048 9.8 (8.4); 256 x 2048 6.4 (3.3); 16384 x 4096 46 (34), x 7168 97 (66)
    const bool wave = vecs <= 64 || (vecs <= 256 && rows >= 4096);
    if (wave && vecs <= 64) Q(64, 1, false);
    else if (wave && vecs <= 128) Q(64, 2, false);
    else if (wave) Q(64, 4, false);
    else if (vecs <= 256) Q(256, 1, false);
    else if (vecs <= 512) Q(256, 2, false);
    else if (vecs <= 1024) Q(256, 4, false);
    else if (vecs <= 2048) Q(256, 8, false);
    else Q(256, 8, true);
#undef Q
    return hipGetLastError();
}

}  // namespace moe

using namespace moe;

extern "C" int moe_int_quantize(const void* x, int64_t x_stride, int32_t dtype, int32_t rows, int32_t cols,
                                int8_t* codes, int64_t codes_stride, float* scales, hipStream_t stream) {
    if (!dtype_ok(dtype)) return reject(MOE_ERR_INVALID, "dtype=%d is not a moe_dtype", dtype);
    if (rows < 0) return reject(MOE_ERR_INVALID, "rows=%d is negative", rows);
    if (rows > kMaxRows) return reject(MOE_ERR_UNSUPPORTED, "rows=%d above %lld", rows, (long long)kMaxRows);
    if (cols < 1 || cols > (1 << 20)) return reject(MOE_ERR_UNSUPPORTED, "cols=%d outside [1, %d]", cols, 1 << 20);
    if (rows == 0) return MOE_OK;
    if (!x || !codes || !scales) return reject(MOE_ERR_INVALID, "NULL pointer argument");
    const int64_t far = (int64_t)1 << 32;
    if (x_stride < 0 || x_stride > far || codes_stride > far || (rows > 1 && codes_stride < cols))
        return reject(MOE_ERR_INVALID, "row strides %lld and %lld", (long long)x_stride, (long long)codes_stride);
    const size_t es = dtype_bytes(dtype);
    if (!is_aligned(x, es) || !is_aligned(scales, 4)) return reject(MOE_ERR_INVALID, "misaligned pointer");
    const Bytes bx = matrix(x, rows, x_stride, cols, (int)es), bc = matrix(codes, rows, codes_stride, cols, 1),
                bs = flat(scales, (int64_t)rows * 4);
    if (overlap(bx, bc) || overlap(bx, bs) || overlap(bc, bs)) return reject(MOE_ERR_INVALID, "buffers overlap");
    hipError_t e;
    if (dtype == MOE_DT_BF16) e = launch_int8_quantize((const Bf16*)x, x_stride, rows, cols, codes, codes_stride, scales, stream);
    else if (dtype == MOE_DT_FP16) e = launch_int8_quantize((const Fp16*)x, x_stride, rows, cols, codes, codes_stride, scales, stream);
    else e = launch_int8_quantize((const float*)x, x_stride, rows, cols, codes, codes_stride, scales, stream);
    return launched(e, "8-bit integer quantizer");
}
