// Root-mean-square norm of each row with the residual's addition before it, an output
// in the rows' type, one in 8-bit codes, and the gradient.
//
//   h = round(x + residual)              stored: the residual stream
//   r = 1 / sqrt(mean_j h_j^2 + eps)
//   y_j = h_j r w_j
//
// The norm reads h as it is stored, so that a gradient and a recomputation from h see
// the numbers that the forward saw. 8 bits: r is one positive factor of the row, which
// leaves the codes alone, so they are those of p_j = fl32(h_j w_j) (exact for 16-bit
// h and w) by the quantizer's rule, s = fl32(max |p| / 127), code = round(p / s), and
// only the scale, s r, depends on r. So the codes are the same in any correct
// implementation, and no rounding of y to 16 bits lies under them.
#include <algorithm>

#include "moe_args.h"
#include "moe_int8_dev.h"
#include "moe_rows_dev.h"
#include "moe_wave_dev.h"

#define INLINE __attribute__((always_inline))

namespace moe {

constexpr int kMaxNormCols = 32768;

// Squares outside fp32's range: such rows are summed again with h times a power of two.
// Below 2^-90 a sum may have lost squares to underflow, which shows unless eps is far
// above them.
constexpr float kBigSum = 0x1p120f, kSmallSum = 0x1p-90f;
__device__ __forceinline__ bool out_of_range(float ss, float eps) {
    return !(ss < kBigSum) || (ss < kSmallSum && eps < kSmallSum);
}
__device__ __forceinline__ float rescale(float ss) { return ss < 1.0f ? 0x1p100f : 0x1p-80f; }
// r / f for the sum of (h f)^2
__device__ __forceinline__ float inverse_rms(float ss, float f, int H, float eps) {
    return __fdiv_rn(1.0f, __fsqrt_rn(__fdiv_rn(ss, (float)H) + (eps * f) * f));
}

template <typename T, typename W>
struct NormArgs {
    const T* x;
    int64_t ld_x;
    const T* residual;  // or null
    int64_t ld_residual;
    const W* weight;    // or null: ones
    T* total;           // with residual; may be residual itself
    int64_t ld_total;
    T* y;               // or null
    int64_t ld_y;
    int8_t* codes;      // or null
    int64_t ld_codes;
    float* scales;
    int rows, H;
    float eps;
};

// The sum and the maximum of a row's threads (a wave, or the block). s: one word each
// per wave; two sets that alternate, so that one barrier per row is enough.
template <int TPT>
__device__ __forceinline__ void row_reduce(float* ss, uint32_t* top, float (*s_sum)[TPT / 64], uint32_t (*s_top)[TPT / 64], int set) {
    *ss = lanes_sum(*ss);
    *top = lanes_max(*top);
    if constexpr (TPT > 64) {
        constexpr int NW = TPT / 64;
        const int wave = threadIdx.x >> 6;
        if ((threadIdx.x & 63) == 0) {
            s_sum[set][wave] = *ss;
            s_top[set][wave] = *top;
        }
        __syncthreads();
        float a = 0.0f;
        uint32_t m = 0;
#pragma unroll
        for (int w = 0; w < NW; ++w) {
            a += s_sum[set][w];
            m = max(m, s_top[set][w]);
        }
        *ss = a;
        *top = m;
    }
}

// A row per TPT threads (a wave, or a block); each thread keeps its NV vectors of 16
// bytes between the sum and the output, so a row is read once. Blocks walk over rows.
// Bound by memory: 16384 x 7168 bf16 with residual, y and codes (1.06 GB) 206 us, 5.1 TB/s;
// y alone 91 us. 64 x 7168: 5.6 us, latency.
template <typename T, typename W, int TPT, int NV>
__global__ __launch_bounds__(TPT < 256 ? 256 : TPT) void rms_norm_kernel(NormArgs<T, W> p) {
    constexpr int V = 16 / sizeof(T), PER = TPT < 256 ? 256 / TPT : 1;
    __shared__ float s_sum[2][TPT / 64];
    __shared__ uint32_t s_top[2][TPT / 64];
    const int at = threadIdx.x % TPT;
    const int whole = p.H / V, tail = p.H - whole * V;  // the H % V elements belong to the first threads
    float w[NV][V];
#pragma unroll
    for (int j = 0; j < NV; ++j) {
#pragma unroll
        for (int i = 0; i < V; ++i) w[j][i] = 1.0f;
        if (p.weight && at + j * TPT < whole) load_floats<V>(p.weight + (at + j * TPT) * V, w[j]);
    }
    const float w_last = p.weight && at < tail ? to_f32(p.weight[whole * V + at]) : 1.0f;
    int set = 0;
    const int first = __builtin_amdgcn_readfirstlane(blockIdx.x * PER + (PER > 1 ? threadIdx.x / TPT : 0));
    for (int m = first; m < p.rows; m += gridDim.x * PER, set ^= 1) {
        const T* x = p.x + m * p.ld_x;
        Vec<T> h[NV];
        T last{};
#pragma unroll
        for (int j = 0; j < NV; ++j)
            if (at + j * TPT < whole) h[j] = load_vec(x + (at + j * TPT) * V);
        if (at < tail) last = x[whole * V + at];
        if (p.residual) {
            const T* res = p.residual + m * p.ld_residual;
            T* total = p.total + m * p.ld_total;
            Vec<T> u[NV];
#pragma unroll
            for (int j = 0; j < NV; ++j)
                if (at + j * TPT < whole) u[j] = load_vec(res + (at + j * TPT) * V);
#pragma unroll
            for (int j = 0; j < NV; ++j)
                if (at + j * TPT < whole) {
#pragma unroll
                    for (int i = 0; i < V; ++i) h[j].e[i] = from_f32<T>(to_f32(h[j].e[i]) + to_f32(u[j].e[i]));
                    store_vec<false>(total + (at + j * TPT) * V, h[j]);
                }
            if (at < tail) {
                last = from_f32<T>(to_f32(last) + to_f32(res[whole * V + at]));
                total[whole * V + at] = last;
            }
        }
        float ss = 0.0f;
        uint32_t top = 0;
        auto each = [&](float v, float wt) INLINE {
            ss = __fmaf_rn(v, v, ss);
            top = max(top, f2u(v * wt) & 0x7FFFFFFFu);
        };
#pragma unroll
        for (int j = 0; j < NV; ++j)
            if (at + j * TPT < whole) {
#pragma unroll
                for (int i = 0; i < V; ++i) each(to_f32(h[j].e[i]), w[j][i]);
            }
        if (at < tail) each(to_f32(last), w_last);
        row_reduce<TPT>(&ss, &top, s_sum, s_top, set);
        float f = 1.0f;
        if (out_of_range(ss, p.eps)) {  // (the same for all threads of the row)
            f = rescale(ss);
            ss = 0.0f;
            auto again = [&](float v) INLINE { ss = __fmaf_rn(v * f, v * f, ss); };
#pragma unroll
            for (int j = 0; j < NV; ++j)
                if (at + j * TPT < whole) {
#pragma unroll
                    for (int i = 0; i < V; ++i) again(to_f32(h[j].e[i]));
                }
            if (at < tail) again(to_f32(last));
            set ^= 1;
            row_reduce<TPT>(&ss, &top, s_sum, s_top, set);
        }
        float r = inverse_rms(ss, f, p.H, p.eps);
        if (f < 1.0f) r *= f, f = 1.0f;  // (a row of large values: h f would take the bits of its small ones)
        if (p.y) {
            T* y = p.y + m * p.ld_y;
#pragma unroll
            for (int j = 0; j < NV; ++j)
                if (at + j * TPT < whole) {
                    Vec<T> o;
#pragma unroll
                    for (int i = 0; i < V; ++i) o.e[i] = from_f32<T>(to_f32(h[j].e[i]) * f * r * w[j][i]);
                    store_vec<false>(y + (at + j * TPT) * V, o);
                }
            if (at < tail) y[whole * V + at] = from_f32<T>(to_f32(last) * f * r * w_last);
        }
        if (p.codes) {
            const Int8Row q = int8_row(top);
            int8_t* dst = p.codes + m * p.ld_codes;
            if (at == 0) p.scales[m] = q.s * f * r;
#pragma unroll
            for (int j = 0; j < NV; ++j)
                if (at + j * TPT < whole) {
                    float v[V];
#pragma unroll
                    for (int i = 0; i < V; ++i) v[i] = to_f32(h[j].e[i]) * w[j][i];
                    store_codes<V>(dst + (at + j * TPT) * V, int8_codes<V>(v, q));
                }
            if (at < tail) dst[whole * V + at] = q.plain ? (int8_t)int8_code_exact(to_f32(last) * w_last, q.s, q.inv) : (int8_t)0;
        }
    }
}

// ---------------------------------------------------------------------------
// gradient
// ---------------------------------------------------------------------------
// With n = h r and g = dy w:  dx = r (g - n mean(g n)) (+ dtotal),  dw = sum over rows of dy n.
// dw: every block sums its rows in registers, in order, and leaves one row of partial
// sums in the workspace, which a second kernel adds in the order of the blocks.
// Bound by memory: 4096 x 4096 bf16 with dtotal (134 MB and 17 MB of partial sums) 25 - 27 and
// 4.2 us from memory, 16384 x 7168 without (705 MB) 140 us. In a graph 25 and 141 us with 512 blocks, 29 and 161 with
// 256 (too little on its way), 25 and 156 with 1024 (partial sums).
template <typename T, typename W>
struct NormGradArgs {
    const T* dy;
    int64_t ld_dy;
    const T* h;
    int64_t ld_h;
    const W* weight;  // or null: ones
    const T* dtotal;  // or null
    int64_t ld_dtotal;
    T* dx;
    int64_t ld_dx;
    float* part;      // [blocks][H], or null
    int rows, H;
    float eps;
};

template <int NW>
__device__ __forceinline__ void block_sum2(float* a, float* b, float (*s)[2][NW], int set) {
    *a = lanes_sum(*a);
    *b = lanes_sum(*b);
    if constexpr (NW > 1) {
        const int wave = threadIdx.x >> 6;
        if ((threadIdx.x & 63) == 0) {
            s[set][0][wave] = *a;
            s[set][1][wave] = *b;
        }
        __syncthreads();
        float c = 0.0f, d = 0.0f;
#pragma unroll
        for (int w = 0; w < NW; ++w) {
            c += s[set][0][w];
            d += s[set][1][w];
        }
        *a = c;
        *b = d;
    }
}

template <typename T, typename W, int TPT, int NV>
__global__ __launch_bounds__(TPT) void rms_norm_grad_kernel(NormGradArgs<T, W> p) {
    constexpr int V = 16 / sizeof(T), NW = TPT / 64;
    __shared__ float s[2][2][NW];
    const int at = threadIdx.x;
    const int whole = p.H / V, tail = p.H - whole * V;
    float w[NV][V], dw[NV][V];
#pragma unroll
    for (int j = 0; j < NV; ++j) {
#pragma unroll
        for (int i = 0; i < V; ++i) w[j][i] = 1.0f, dw[j][i] = 0.0f;
        if (p.weight && at + j * TPT < whole) load_floats<V>(p.weight + (at + j * TPT) * V, w[j]);
    }
    const float w_last = p.weight && at < tail ? to_f32(p.weight[whole * V + at]) : 1.0f;
    float dw_last = 0.0f;
    int set = 0;
    for (int m = blockIdx.x; m < p.rows; m += gridDim.x, set ^= 1) {
        const T *dy = p.dy + m * p.ld_dy, *h = p.h + m * p.ld_h;
        Vec<T> a[NV], b[NV], c[NV];
        T a_last{}, b_last{}, c_last{};
#pragma unroll
        for (int j = 0; j < NV; ++j)
            if (at + j * TPT < whole) {
                a[j] = load_vec(dy + (at + j * TPT) * V);
                b[j] = load_vec(h + (at + j * TPT) * V);
                if (p.dtotal) c[j] = load_vec(p.dtotal + m * p.ld_dtotal + (at + j * TPT) * V);
            }
        if (at < tail) {
            a_last = dy[whole * V + at];
            b_last = h[whole * V + at];
            if (p.dtotal) c_last = p.dtotal[m * p.ld_dtotal + whole * V + at];
        }
        float f = 1.0f, ss = 0.0f, sg = 0.0f;
        auto sums = [&]() INLINE {
            ss = sg = 0.0f;
            auto each = [&](float d, float v, float wt) INLINE {
                v *= f;
                ss = __fmaf_rn(v, v, ss);
                sg = __fmaf_rn(d * wt, v, sg);
            };
#pragma unroll
            for (int j = 0; j < NV; ++j)
                if (at + j * TPT < whole) {
#pragma unroll
                    for (int i = 0; i < V; ++i) each(to_f32(a[j].e[i]), to_f32(b[j].e[i]), w[j][i]);
                }
            if (at < tail) each(to_f32(a_last), to_f32(b_last), w_last);
            block_sum2<NW>(&ss, &sg, s, set);
        };
        sums();
        if (out_of_range(ss, p.eps)) {
            f = rescale(ss);
            set ^= 1;
            sums();
        }
        float r = inverse_rms(ss, f, p.H, p.eps);
        const float mean = __fdiv_rn(sg * r, (float)p.H);  // of g n
        if (f < 1.0f) r *= f, f = 1.0f;  // (as in rms_norm_kernel)
        T* dx = p.dx + m * p.ld_dx;
        auto one = [&](float d, float v, float wt, float more, float* sum) INLINE {
            const float n = v * f * r;
            *sum = __fmaf_rn(d, n, *sum);
            return __fmaf_rn(-n, mean, d * wt) * r * f + more;
        };
#pragma unroll
        for (int j = 0; j < NV; ++j)
            if (at + j * TPT < whole) {
                Vec<T> o;
#pragma unroll
                for (int i = 0; i < V; ++i)
                    o.e[i] = from_f32<T>(one(to_f32(a[j].e[i]), to_f32(b[j].e[i]), w[j][i], p.dtotal ? to_f32(c[j].e[i]) : 0.0f, &dw[j][i]));
                store_vec<false>(dx + (at + j * TPT) * V, o);
            }
        if (at < tail)
            dx[whole * V + at] = from_f32<T>(one(to_f32(a_last), to_f32(b_last), w_last, p.dtotal ? to_f32(c_last) : 0.0f, &dw_last));
    }
    if (p.part) {
        float* part = p.part + (size_t)blockIdx.x * p.H;
#pragma unroll
        for (int j = 0; j < NV; ++j)
            if (at + j * TPT < whole) {
#pragma unroll
                for (int g = 0; g < V / 4; ++g) {
                    Vec<float> o;
#pragma unroll
                    for (int i = 0; i < 4; ++i) o.e[i] = dw[j][4 * g + i];
                    store_vec<false>(part + (at + j * TPT) * V + 4 * g, o);
                }
            }
        if (at < tail) part[whole * V + at] = dw_last;
    }
}

// Column sums of the blocks' partial sums, in the order of the blocks within each of sixteen
// parts; 64 columns per block.
__global__ __launch_bounds__(1024) void norm_weight_grad_kernel(const float* __restrict__ part, int blocks, int H,
                                                                float* __restrict__ dweight) {
    __shared__ float s[16][64];
    const int lane = threadIdx.x & 63, q = threadIdx.x >> 6, c = blockIdx.x * 64 + lane;
    const int each = (blocks + 15) / 16, hi = min(blocks, (q + 1) * each);
    float a = 0.0f;
    if (c < H)
#pragma unroll 8
        for (int b = q * each; b < hi; ++b) a += part[(size_t)b * H + c];
    s[q][lane] = a;
    __syncthreads();
    if (q == 0 && c < H) {
#pragma unroll
        for (int i = 1; i < 16; ++i) a += s[i][lane];
        dweight[c] = a;
    }
}

// ---------------------------------------------------------------------------
// launches
// ---------------------------------------------------------------------------
constexpr int kGradBlocks = 512;  // rows of partial sums, at most
static int grad_blocks(int rows) { return std::min(rows, kGradBlocks); }

template <typename T, typename W>
static hipError_t launch_norm(const NormArgs<T, W>& p, hipStream_t s) {
    constexpr int V = 16 / (int)sizeof(T);
    const int vecs = std::max((p.H + V - 1) / V, 1);
#define N(TPT, NV)                                                                                     \
    hipLaunchKernelGGL((rms_norm_kernel<T, W, TPT, NV>),                                              \
                       dim3(std::min((p.rows + (TPT < 256 ? 256 / TPT : 1) - 1) / (TPT < 256 ? 256 / TPT : 1), 2048)), \
                       dim3(TPT < 256 ? 256 : TPT), 0, s, p)
    // Few rows: many threads each, latency is all there is. Many: as few as hold the row, down to a
    // wave. Codes, y and residual, bf16, in a graph, us, with 256 threads (512, 1024):
    // 64 x 7168 9.5 (6.5, 5.8), 256 x 7168 10.1 (7.8, 7.1), 1024 x 7168 17.0 (15.9, 17.9),
    // 16384 x 7168 208 (210, 223); 64 x 4096 6.2 (4.7, 4.8), 4096 x 4096 27.7 (27.2, 39.6);
    // 16384 x 2048 64 (75, 140), with a wave 60; 4096 x 2048 17.1 (19.0, 34), with a wave 19.2
    const bool few = p.rows <= 512, many = p.rows >= 8192;
    if (vecs <= 64) N(64, 1);
    else if (many && vecs <= 128) N(64, 2);
    else if (many && vecs <= 256) N(64, 4);
    else if (vecs <= 256) N(256, 1);
    else if (few && vecs <= 512) N(512, 1);
    else if (vecs <= 512) N(256, 2);
    else if (few && vecs <= 1024) N(1024, 1);
    else if (vecs <= 1024) N(512, 2);
    else if (vecs <= 2048) N(1024, 2);
    else if (V == 8 || vecs <= 4096) N(1024, 4);
    else if constexpr (V == 4) N(1024, 8);
#undef N
    return hipGetLastError();
}

template <typename T, typename W>
static hipError_t launch_norm_grad(const NormGradArgs<T, W>& p, float* dweight, hipStream_t s) {
    constexpr int V = 16 / (int)sizeof(T);
    const int vecs = std::max((p.H + V - 1) / V, 1), blocks = grad_blocks(p.rows);
#define N(TPT, NV) hipLaunchKernelGGL((rms_norm_grad_kernel<T, W, TPT, NV>), dim3(blocks), dim3(TPT), 0, s, p)
    if (!blocks) {}
    else if (vecs <= 64) N(64, 1);
    else if (vecs <= 256) N(256, 1);
    else if (vecs <= 512) N(256, 2);
    else if (vecs <= 1024) N(512, 2);
    else if (vecs <= 2048) N(1024, 2);
    else if (V == 8 || vecs <= 4096) N(1024, 4);
    else if constexpr (V == 4) N(1024, 8);
#undef N
    if (dweight)
        hipLaunchKernelGGL(norm_weight_grad_kernel, dim3((p.H + 63) / 64), dim3(1024), 0, s, p.part, blocks, p.H, dweight);
    return hipGetLastError();
}

static int check_norm_sizes(int32_t dtype, int32_t weight_dtype, int32_t rows, int32_t cols, float eps) {
    if (!dtype_ok(dtype)) return reject(MOE_ERR_INVALID, "dtype=%d is not a moe_dtype", dtype);
    if (weight_dtype != dtype && weight_dtype != MOE_DT_FP32)
        return reject(MOE_ERR_INVALID, "weight_dtype=%d must be the rows' type or fp32", weight_dtype);
    if (rows < 0) return reject(MOE_ERR_INVALID, "rows=%d is negative", rows);
    if (rows > kMaxRows) return reject(MOE_ERR_UNSUPPORTED, "rows=%d above %lld", rows, (long long)kMaxRows);
    if (cols < 1 || cols > kMaxNormCols) return reject(MOE_ERR_UNSUPPORTED, "cols=%d outside [1, %d]", cols, kMaxNormCols);
    if (!(eps >= 0.0f) || eps > 3.4e38f) return reject(MOE_ERR_INVALID, "eps must be finite and not negative");
    return MOE_OK;
}

// stride: of an input (0 and more) or of an output (rows apart)
static bool stride_ok(int64_t stride, int rows, int cols, bool output) {
    return stride >= (output && rows > 1 ? cols : 0) && stride <= ((int64_t)1 << 32);
}

// Calls f(T(), W()) for the element types.
template <typename F>
static hipError_t with_types(int dtype, int weight_dtype, F f) {
    const bool wide = weight_dtype == MOE_DT_FP32;
    if (dtype == MOE_DT_BF16) return wide ? f(Bf16(), float()) : f(Bf16(), Bf16());
    if (dtype == MOE_DT_FP16) return wide ? f(Fp16(), float()) : f(Fp16(), Fp16());
    return f(float(), float());
}

}  // namespace moe

using namespace moe;

extern "C" int moe_rms_norm(const void* x, int64_t x_stride, const void* residual, int64_t residual_stride, int32_t dtype,
                            const void* weight, int32_t weight_dtype, int32_t rows, int32_t cols, float eps, void* total,
                            int64_t total_stride, void* y, int64_t y_stride, int8_t* codes, int64_t codes_stride,
                            float* scales, hipStream_t stream) {
    const int rc = check_norm_sizes(dtype, weight_dtype, rows, cols, eps);
    if (rc) return rc;
    if ((residual == nullptr) != (total == nullptr)) return reject(MOE_ERR_INVALID, "residual and total come together");
    if ((codes == nullptr) != (scales == nullptr)) return reject(MOE_ERR_INVALID, "codes and scales come together");
    if (rows == 0) return MOE_OK;
    if (!x || (!y && !codes)) return reject(MOE_ERR_INVALID, "NULL pointer argument");
    if (!stride_ok(x_stride, rows, cols, false) || (residual && !stride_ok(residual_stride, rows, cols, false)) ||
        (total && !stride_ok(total_stride, rows, cols, true)) || (y && !stride_ok(y_stride, rows, cols, true)) ||
        (codes && !stride_ok(codes_stride, rows, cols, true)))
        return reject(MOE_ERR_INVALID, "a row stride is out of range");
    const int es = dtype_bytes(dtype), ws = dtype_bytes(weight_dtype);
    if (!is_aligned(x, es) || !is_aligned(residual, es) || !is_aligned(total, es) || !is_aligned(y, es) ||
        !is_aligned(weight, ws) || !is_aligned(scales, 4))
        return reject(MOE_ERR_INVALID, "misaligned pointer");
    const bool in_place = total && total == residual && (rows == 1 || total_stride == residual_stride);
    const Bytes in[] = {matrix(x, rows, x_stride, cols, es), matrix(in_place ? nullptr : residual, rows, residual_stride, cols, es),
                        flat(weight, (int64_t)cols * ws)};
    const Bytes out[] = {matrix(total, rows, total_stride, cols, es), matrix(y, rows, y_stride, cols, es),
                         matrix(codes, rows, codes_stride, cols, 1), flat(scales, (int64_t)rows * 4)};
    for (const Bytes& o : out)
        for (const Bytes& i : in)
            if (overlap(i, o)) return reject(MOE_ERR_INVALID, "an output overlaps an input");
    for (int i = 0; i < 4; ++i)
        for (int j = i + 1; j < 4; ++j)
            if (overlap(out[i], out[j])) return reject(MOE_ERR_INVALID, "the outputs overlap");
    return launched(with_types(dtype, weight_dtype, [&](auto t, auto w) {
        typedef decltype(t) T;
        typedef decltype(w) W;
        return launch_norm(NormArgs<T, W>{(const T*)x, x_stride, (const T*)residual, residual_stride, (const W*)weight, (T*)total,
                                          total_stride, (T*)y, y_stride, codes, codes_stride, scales, rows, cols, eps}, stream);
    }), "RMS norm");
}

extern "C" size_t moe_rms_norm_grad_workspace_bytes(int32_t rows, int32_t cols) {
    if (check_norm_sizes(MOE_DT_FP32, MOE_DT_FP32, rows, cols, 0.0f) != MOE_OK) return 0;
    return align256((size_t)std::max(grad_blocks(rows), 1) * cols * 4);
}

extern "C" int moe_rms_norm_grad(const void* dy, int64_t dy_stride, const void* h, int64_t h_stride, int32_t dtype,
                                 const void* weight, int32_t weight_dtype, const void* dtotal, int64_t dtotal_stride,
                                 int32_t rows, int32_t cols, float eps, void* workspace, size_t workspace_bytes, void* dx,
                                 int64_t dx_stride, float* dweight, hipStream_t stream) {
    const int rc = check_norm_sizes(dtype, weight_dtype, rows, cols, eps);
    if (rc) return rc;
    if ((rows && (!dy || !h || !dx)) || (dweight && !workspace)) return reject(MOE_ERR_INVALID, "NULL pointer argument");
    const int es = dtype_bytes(dtype), ws = dtype_bytes(weight_dtype);
    if (!is_aligned(dy, es) || !is_aligned(h, es) || !is_aligned(dtotal, es) || !is_aligned(dx, es) ||
        !is_aligned(weight, ws) || !is_aligned(dweight, 4) || !is_aligned(workspace, 16))
        return reject(MOE_ERR_INVALID, "misaligned pointer");
    if (!stride_ok(dy_stride, rows, cols, false) || !stride_ok(h_stride, rows, cols, false) ||
        (dtotal && !stride_ok(dtotal_stride, rows, cols, false)) || !stride_ok(dx_stride, rows, cols, true))
        return reject(MOE_ERR_INVALID, "a row stride is out of range");
    const size_t need = dweight ? moe_rms_norm_grad_workspace_bytes(rows, cols) : 0;
    if (workspace_bytes < need) return reject(MOE_ERR_WORKSPACE, "workspace %zu bytes < %zu needed", workspace_bytes, need);
    const Bytes in[] = {matrix(dy, rows, dy_stride, cols, es), matrix(h, rows, h_stride, cols, es),
                        matrix(dtotal, rows, dtotal_stride, cols, es), flat(weight, (int64_t)cols * ws)};
    const Bytes out[] = {matrix(dx, rows, dx_stride, cols, es), flat(dweight, (int64_t)cols * 4), flat(workspace, (int64_t)need)};
    for (const Bytes& o : out)
        for (const Bytes& i : in)
            if (overlap(i, o)) return reject(MOE_ERR_INVALID, "an output overlaps an input");
    for (int i = 0; i < 3; ++i)
        for (int j = i + 1; j < 3; ++j)
            if (overlap(out[i], out[j])) return reject(MOE_ERR_INVALID, "the outputs overlap");
    if (!rows && !dweight) return MOE_OK;
    return launched(with_types(dtype, weight_dtype, [&](auto t, auto w) {
        typedef decltype(t) T;
        typedef decltype(w) W;
        return launch_norm_grad(NormGradArgs<T, W>{(const T*)dy, dy_stride, (const T*)h, h_stride, (const W*)weight, (const T*)dtotal,
                                                   dtotal_stride, (T*)dx, dx_stride, dweight ? (float*)workspace : nullptr, rows,
                                                   cols, eps}, dweight, stream);
    }), "RMS norm gradient");
}
