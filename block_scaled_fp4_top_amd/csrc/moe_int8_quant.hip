// Symmetric 8-bit integer quantization of each row:
//   s[m] = fl32(max_j |x[m,j]| / 127),  c[m,j] = round(x[m,j] / s[m])
#include "moe_args.h"
#include "moe_int8_dev.h"
#include "moe_rows_dev.h"

namespace moe {

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
    const Int8Row r = int8_row(top);
    if (at == 0) scales[m] = r.s;
    auto put = [&](const Vec<T>& u, int c) {
        float f[V];
#pragma unroll
        for (int i = 0; i < V; ++i) f[i] = to_f32(u.e[i]);
        store_codes<V>(dst + (int64_t)c * V, int8_codes<V>(f, r));
    };
#pragma unroll
    for (int j = 0; j < NV; ++j)
        if (at + j * TPT < whole) put(v[j], at + j * TPT);
    if (at < tail) dst[whole * V + at] = r.plain ? (int8_t)int8_code_exact(to_f32(last), r.s, r.inv) : (int8_t)0;
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
