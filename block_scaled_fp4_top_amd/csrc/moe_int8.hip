// Products of 8-bit integer matrices with a scale for each token (row of A)
// and each output channel (row of B), dense or expert by expert, and the
// quantizer of their activations.
//   quantize: s[m] = max_j |x[m,j]| / 127, c[m,j] = round(x[m,j] / s[m])
//   product:  y[m,n] = sa[m] sb[n] sum_k a[m,k] b[n,k] (+ bias[n])
// The sums are exact 32-bit integers (|sum| <= 2^14 * 131056 < 2^31), the scales
// are applied in fp32 and the result is rounded once to the output's type.
#include "moe_args.h"
#include "moe_rows_dev.h"

namespace moe {

typedef int i32x4 __attribute__((ext_vector_type(4)));

// ---------------------------------------------------------------------------
// quantizer
// ---------------------------------------------------------------------------
// One block per row, two passes. Codes are the correctly rounded quotients
// x / s of the row's fp32 scale s (ties to even): n = rint(x * (1/s)) is at
// most one off, and the sign of the exact remainder x - n s (one fma: at most
// 24 bits remain) against s / 2 decides. A scale that is not finite (a row with
// an infinity or a NaN) or zero leaves codes 0.
__device__ __forceinline__ int int8_code(float x, float s, float inv) {
    float n = __builtin_rintf(x * inv);
    const float r2 = 2.0f * __fmaf_rn(-n, s, x);  // twice the remainder, exact
    const bool odd = ((int)n) & 1;
    if (r2 > s || (r2 == s && odd)) n += 1.0f;
    else if (r2 < -s || (r2 == -s && odd)) n -= 1.0f;
    return (int)fminf(fmaxf(n, -127.0f), 127.0f);
}

template <typename T>
__global__ __launch_bounds__(256) void int8_quantize_kernel(const T* __restrict__ x, int64_t ld, int H,
                                                            int8_t* __restrict__ codes, int64_t ld_codes,
                                                            float* __restrict__ scales) {
    __shared__ uint32_t smax[4];
    const size_t m = blockIdx.x;
    const T* row = x + (int64_t)m * ld;
    // the bits of |x| order like the values, NaN above infinity
    uint32_t top = 0;
    for (int i = threadIdx.x; i < H; i += 256) top = max(top, f2u(to_f32(row[i])) & 0x7FFFFFFFu);
#pragma unroll
    for (int off = 32; off >= 1; off >>= 1) top = max(top, (uint32_t)__shfl_xor((int)top, off));
    if ((threadIdx.x & 63) == 0) smax[threadIdx.x >> 6] = top;
    __syncthreads();
    top = max(max(smax[0], smax[1]), max(smax[2], smax[3]));
    const float s = __fdiv_rn(u2f(top), 127.0f);
    const bool zero = !(s > 0.0f) || top >= 0x7F800000u;
    for (int i = threadIdx.x; i < H; i += 256) {
        int c = 0;
        if (!zero) {
            const float v = to_f32(row[i]);
            // 1/s overflows below 2^-126: such rows divide in fp64
            if (s < 1e-37f) c = (int)fmin(fmax(rint((double)v / (double)s), -127.0), 127.0);
            else c = int8_code(v, s, __fdiv_rn(1.0f, s));
        }
        codes[(int64_t)m * ld_codes + i] = (int8_t)c;
    }
    if (threadIdx.x == 0) scales[m] = s;
}

// ---------------------------------------------------------------------------
// products
// ---------------------------------------------------------------------------
struct Int8Args {
    const int8_t* a;
    int64_t lda;
    const float* sa;
    const int8_t* b;
    int64_t ldb, b_expert;  // row stride, and bytes from one expert's matrix to the next
    const float* sb;
    const float* bias;      // [N] or [E][N], or null
    int M, N, Kd;           // rows of the output, columns, depth
    int a_rows;             // rows of A
    // grouped: rows offsets[e] .. offsets[e+1] use expert e; null: dense
    const int32_t* offsets;
    int E;
    const int32_t* row_to_route;  // gather: row r reads A's row row_to_route[r] / topk; else null
    int topk;
    void* y;
    int64_t ldy;
};

// The tile's expert and rows. Tiles are counted expert by expert, ceil(rows / BM)
// each; every wave finds the tile by itself from the offsets, 64 experts at a
// time. Offsets are clamped to [0, M], so a damaged list stays in range.
// Returns false when there is no such tile.
template <int BM>
__device__ __forceinline__ bool find_tile(const Int8Args& p, int tile, int lane, int* e_out, int* row0, int* rows) {
    if (!p.offsets) {
        *e_out = 0;
        *row0 = tile * BM;
        *rows = min(BM, p.M - *row0);
        return *rows > 0;
    }
    int before = 0;
    for (int base = 0; base < p.E; base += 64) {
        const int e = base + lane;
        int lo = 0, hi = 0;
        if (e < p.E) {
            lo = min(max(p.offsets[e], 0), p.M);
            hi = min(max(p.offsets[e + 1], lo), p.M);
        }
        const int n = (hi - lo + BM - 1) / BM;
        int incl = n;
#pragma unroll
        for (int off = 1; off < 64; off <<= 1) {
            const int v = __shfl_up(incl, off);
            if (lane >= off) incl += v;
        }
        const int excl = before + incl - n;
        const uint64_t hit = __ballot(tile >= excl && tile < excl + n);
        if (hit) {
            const int src = __ffsll((unsigned long long)hit) - 1;
            const int first = __shfl(lo, src) + (tile - __shfl(excl, src)) * BM;
            *e_out = base + src;
            *row0 = first;
            *rows = min(BM, __shfl(hi, src) - first);
            return true;
        }
        before += __shfl(incl, 63);
    }
    return false;
}

// 64 x 64 tiles of four waves, 64 bytes of depth a step, both operands through
// the LDS.
template <typename T>
__global__ __launch_bounds__(256) void int8_matmul_kernel(Int8Args p) {
    constexpr int BM = 64, BN = 64, LD = 64 + 16;
    __shared__ __attribute__((aligned(16))) int8_t sA[BM * LD], sB[BN * LD];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    int e, row0, rows;
    if (!find_tile<BM>(p, blockIdx.x, lane, &e, &row0, &rows)) return;
    const int n0 = blockIdx.y * BN;
    const int r = tid >> 2, kc = (tid & 3) * 16;
    int arow = -1;
    if (r < rows) {
        arow = row0 + r;
        if (p.row_to_route) arow = p.row_to_route[row0 + r] / p.topk;
        if ((uint32_t)arow >= (uint32_t)p.a_rows) arow = -1;
    }
    const int brow = n0 + r < p.N ? n0 + r : -1;
    i32x4 acc[4] = {};
    for (int k = 0; k < p.Kd; k += 64) {
        uint4 av = make_uint4(0, 0, 0, 0), bv = av;
        if (k + kc < p.Kd) {
            if (arow >= 0) av = *reinterpret_cast<const uint4*>(p.a + (int64_t)arow * p.lda + k + kc);
            if (brow >= 0) bv = *reinterpret_cast<const uint4*>(p.b + (int64_t)e * p.b_expert + (int64_t)brow * p.ldb + k + kc);
        }
        __syncthreads();
        *reinterpret_cast<uint4*>(&sA[r * LD + kc]) = av;
        *reinterpret_cast<uint4*>(&sB[r * LD + kc]) = bv;
        __syncthreads();
        const i32x4 bf = *reinterpret_cast<const i32x4*>(&sB[(wave * 16 + (lane & 15)) * LD + 16 * (lane >> 4)]);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const i32x4 af = *reinterpret_cast<const i32x4*>(&sA[(i * 16 + (lane & 15)) * LD + 16 * (lane >> 4)]);
            acc[i] = __builtin_amdgcn_mfma_i32_16x16x64_i8(af, bf, acc[i], 0, 0, 0);
        }
    }
    const int n = n0 + wave * 16 + (lane & 15);
    if (n >= p.N) return;
    const float sb = p.sb[(size_t)e * p.N + n], bias = p.bias ? p.bias[(size_t)e * p.N + n] : 0.0f;
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int m = i * 16 + 4 * (lane >> 4) + j;
            if (m >= rows) continue;
            int ar = row0 + m;
            if (p.row_to_route) ar = p.row_to_route[row0 + m] / p.topk;
            if ((uint32_t)ar >= (uint32_t)p.a_rows) continue;
            const float v = __fmaf_rn((float)acc[i][j] * p.sa[ar], sb, bias);
            static_cast<T*>(p.y)[(int64_t)(row0 + m) * p.ldy + n] = from_f32<T>(v);
        }
}

template <typename T>
static hipError_t launch_int8_matmul(const Int8Args& p, hipStream_t s) {
    const int tiles = (p.M + 63) / 64 + (p.offsets ? p.E : 0);
    hipLaunchKernelGGL(int8_matmul_kernel<T>, dim3(tiles, (p.N + 63) / 64), dim3(256), 0, s, p);
    return hipGetLastError();
}

// Checks shared by both products (grouped: offsets not null), then the launch.
static int run_int8_matmul(Int8Args p, int out_dtype, bool grouped, hipStream_t stream) {
    if (!dtype_ok(out_dtype)) return reject(MOE_ERR_INVALID, "out_dtype=%d is not a moe_dtype", out_dtype);
    if (p.M < 0) return reject(MOE_ERR_INVALID, "M=%d is negative", p.M);
    if (p.N < 1 || p.Kd < 1) return reject(MOE_ERR_INVALID, "N=%d, K=%d must be positive", p.N, p.Kd);
    if (p.Kd % 16) return reject(MOE_ERR_UNSUPPORTED, "the depth K=%d must be a multiple of 16", p.Kd);
    if (p.Kd >= 131072) return reject(MOE_ERR_UNSUPPORTED, "depth K=%d: 32-bit sums hold up to 131071 products", p.Kd);
    if (p.N > (1 << 20)) return reject(MOE_ERR_UNSUPPORTED, "N=%d above %d", p.N, 1 << 20);
    if (p.M > (1 << 26)) return reject(MOE_ERR_UNSUPPORTED, "M=%d rows above %d", p.M, 1 << 26);
    if (grouped && (p.E < 1 || p.E > kMaxE)) return reject(MOE_ERR_INVALID, "E=%d outside [1, %d]", p.E, kMaxE);
    if (p.row_to_route && (p.topk < 1 || p.topk > kMaxK))
        return reject(MOE_ERR_INVALID, "topk=%d outside [1, %d]", p.topk, kMaxK);
    if (p.row_to_route && (long long)p.a_rows * p.topk != p.M)
        return reject(MOE_ERR_INVALID, "%d tokens of %d routes are not %d rows", p.a_rows, p.topk, p.M);
    if (p.M == 0) return MOE_OK;
    if (!p.a || !p.sa || !p.b || !p.sb || !p.y || (grouped && !p.offsets))
        return reject(MOE_ERR_INVALID, "NULL pointer argument");
    if ((p.a_rows > 1 && p.lda < p.Kd) || (p.N > 1 && p.ldb < p.Kd) || (p.M > 1 && p.ldy < p.N) ||
        (grouped && p.E > 1 && p.b_expert < 0))
        return reject(MOE_ERR_INVALID, "a row stride is below the row");
    const int64_t far = (int64_t)1 << 31;
    if (p.lda > far || p.ldb > far || p.ldy > far) return reject(MOE_ERR_UNSUPPORTED, "a row stride above 2^31");
    if ((p.a_rows > 1 && p.lda % 16) || (p.N > 1 && p.ldb % 16) || (grouped && p.E > 1 && p.b_expert % 16))
        return reject(MOE_ERR_UNSUPPORTED, "the strides of a and b must be multiples of 16");
    const size_t es = dtype_bytes(out_dtype);
    if (!is_aligned(p.a, 16) || !is_aligned(p.b, 16)) return reject(MOE_ERR_INVALID, "a and b must be 16-byte aligned");
    if (!is_aligned(p.y, es) || !is_aligned(p.sa, 4) || !is_aligned(p.sb, 4) || !is_aligned(p.bias, 4) ||
        !is_aligned(p.offsets, 4) || !is_aligned(p.row_to_route, 4))
        return reject(MOE_ERR_INVALID, "misaligned pointer");
    const size_t n_y = extent(p.M, p.ldy, p.N, (int)es);
    const size_t E = grouped ? p.E : 1;
    const struct { const void* p; size_t n; } in[] = {
        {p.a, extent(p.a_rows, p.lda, p.Kd, 1)}, {p.sa, (size_t)p.a_rows * 4},
        {p.b, (E - 1) * (size_t)p.b_expert + extent(p.N, p.ldb, p.Kd, 1)}, {p.sb, E * p.N * 4},
        {p.bias, p.bias ? E * p.N * 4 : 0}, {p.offsets, grouped ? (E + 1) * 4 : 0},
        {p.row_to_route, p.row_to_route ? (size_t)p.M * 4 : 0}};
    for (const auto& b : in)
        if (overlap(b.p, b.n, p.y, n_y)) return reject(MOE_ERR_INVALID, "the output overlaps an input");
    hipError_t e;
    if (out_dtype == MOE_DT_BF16) e = launch_int8_matmul<Bf16>(p, stream);
    else if (out_dtype == MOE_DT_FP16) e = launch_int8_matmul<Fp16>(p, stream);
    else e = launch_int8_matmul<float>(p, stream);
    return launched(e, "8-bit integer product");
}

}  // namespace moe

using namespace moe;

extern "C" int moe_int_quantize(const void* x, int64_t x_stride, int32_t dtype, int32_t rows, int32_t cols,
                                int8_t* codes, int64_t codes_stride, float* scales, hipStream_t stream) {
    if (!dtype_ok(dtype)) return reject(MOE_ERR_INVALID, "dtype=%d is not a moe_dtype", dtype);
    if (rows < 0) return reject(MOE_ERR_INVALID, "rows=%d is negative", rows);
    if (cols < 1 || cols > (1 << 20)) return reject(MOE_ERR_UNSUPPORTED, "cols=%d outside [1, %d]", cols, 1 << 20);
    if (rows == 0) return MOE_OK;
    if (!x || !codes || !scales) return reject(MOE_ERR_INVALID, "NULL pointer argument");
    const int64_t far = (int64_t)1 << 32;
    if (x_stride < 0 || x_stride > far || codes_stride > far || (rows > 1 && codes_stride < cols))
        return reject(MOE_ERR_INVALID, "row strides %lld and %lld", (long long)x_stride, (long long)codes_stride);
    const size_t es = dtype_bytes(dtype);
    if (!is_aligned(x, es) || !is_aligned(scales, 4)) return reject(MOE_ERR_INVALID, "misaligned pointer");
    const size_t nx = extent(rows, x_stride, cols, (int)es), nc = extent(rows, codes_stride, cols, 1), ns = (size_t)rows * 4;
    if (overlap(x, nx, codes, nc) || overlap(x, nx, scales, ns) || overlap(codes, nc, scales, ns))
        return reject(MOE_ERR_INVALID, "buffers overlap");
    const dim3 grid(rows), block(256);
    if (dtype == MOE_DT_BF16) hipLaunchKernelGGL(int8_quantize_kernel<Bf16>, grid, block, 0, stream, (const Bf16*)x, x_stride, cols, codes, codes_stride, scales);
    else if (dtype == MOE_DT_FP16) hipLaunchKernelGGL(int8_quantize_kernel<Fp16>, grid, block, 0, stream, (const Fp16*)x, x_stride, cols, codes, codes_stride, scales);
    else hipLaunchKernelGGL(int8_quantize_kernel<float>, grid, block, 0, stream, (const float*)x, x_stride, cols, codes, codes_stride, scales);
    return launched(hipGetLastError(), "8-bit integer quantizer");
}

extern "C" int moe_int_matmul(const int8_t* a, int64_t a_stride, const float* a_scales, const int8_t* b,
                              int64_t b_stride, const float* b_scales, const float* bias, int32_t M, int32_t N,
                              int32_t K, int32_t out_dtype, void* y, int64_t y_stride, hipStream_t stream) {
    return run_int8_matmul(Int8Args{a, a_stride, a_scales, b, b_stride, 0, b_scales, bias, M, N, K, M, nullptr, 0,
                                    nullptr, 1, y, y_stride},
                           out_dtype, false, stream);
}

extern "C" int moe_int_grouped_matmul(const int8_t* a, int64_t a_stride, const float* a_scales, int32_t a_rows,
                                      const int8_t* b, int64_t b_stride, int64_t b_expert_stride,
                                      const float* b_scales, const float* bias, const int32_t* offsets,
                                      const int32_t* row_to_route, int32_t topk, int32_t M, int32_t N,
                                      int32_t K, int32_t E, int32_t out_dtype, void* y, int64_t y_stride,
                                      hipStream_t stream) {
    if (a_rows < 0 || (!row_to_route && a_rows != M))
        return reject(MOE_ERR_INVALID, "a has %d rows, the output %d", a_rows, M);
    return run_int8_matmul(Int8Args{a, a_stride, a_scales, b, b_stride, b_expert_stride, b_scales, bias, M, N, K,
                                    a_rows, offsets, E, row_to_route, topk, y, y_stride},
                           out_dtype, true, stream);
}
