// Token rows to the experts' rows and back, and the gradients of both.
//
// With row(t, k) the sorted row of route t*K + k (none for a dropped route):
//   spread:  out[row(t,k)] = w[t,k] * token[t]          dispatch, and combine's gradient
//   collect: out[t] = sum_k w[t,k] * rows[row(t,k)]     combine, and dispatch's gradient
//   dots:    dw[t,k] = <token[t], rows[row(t,k)]>       both gradients, of the weights
// w missing means 1. Sums run in fp32, k ascending, with one rounding to the
// type of the rows at the end; a dropped route contributes nothing and its dw
// is 0. Everything is bound by memory: a token's row is read once and its K
// expert rows are written or read once each.
#include "moe_args.h"
#include "moe_rows_dev.h"

namespace moe {

constexpr int kRowThreads = 256;

// The row of route r, or -1 where it is dropped or names no row (so that a
// damaged map reads and writes nothing out of range).
__device__ __forceinline__ int row_of(const int32_t* __restrict__ route_to_row, size_t r, uint32_t R) {
    const int row = route_to_row[r];
    return (uint32_t)row < R ? row : -1;
}

__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
    for (int off = 32; off >= 1; off >>= 1) v += __shfl_xor(v, off);
    return v;
}

// out[row(t,k)] = w * token[t]: one block per token and chunk of columns; the
// chunk is read once and stored K times.
template <typename T>
__global__ __launch_bounds__(kRowThreads) void spread_kernel(const T* __restrict__ token, int64_t ld_token,
                                                             const int32_t* __restrict__ route_to_row,
                                                             const float* __restrict__ w, int K, int H,
                                                             uint32_t R, T* __restrict__ out, int64_t ld_out) {
    constexpr int V = 16 / sizeof(T);
    const size_t t = blockIdx.x;
    const int c = (blockIdx.y * kRowThreads + threadIdx.x) * V;
    if (c >= H) return;
    const T* src = token + (int64_t)t * ld_token + c;
    const int n = min(V, H - c);
    Vec<T> v;
    if (n == V) v = *reinterpret_cast<const Vec<T>*>(src);
    else for (int i = 0; i < n; ++i) v.e[i] = src[i];
    for (int k = 0; k < K; ++k) {
        const int row = row_of(route_to_row, t * K + k, R);
        if (row < 0) continue;
        T* dst = out + (int64_t)row * ld_out + c;
        Vec<T> o = v;
        if (w) {
            const float f = w[t * K + k];
#pragma unroll
            for (int i = 0; i < V; ++i) o.e[i] = from_f32<T>(f * to_f32(v.e[i]));
        }
        if (n == V) *reinterpret_cast<Vec<T>*>(dst) = o;
        else for (int i = 0; i < n; ++i) dst[i] = o.e[i];
    }
}

// out[t] = sum_k w * rows[row(t,k)]: one block per token and chunk of columns.
template <typename T>
__global__ __launch_bounds__(kRowThreads) void collect_kernel(const T* __restrict__ rows, int64_t ld_rows,
                                                              const int32_t* __restrict__ route_to_row,
                                                              const float* __restrict__ w, int K, int H,
                                                              uint32_t R, T* __restrict__ out, int64_t ld_out) {
    constexpr int V = 16 / sizeof(T);
    const size_t t = blockIdx.x;
    const int c = (blockIdx.y * kRowThreads + threadIdx.x) * V;
    if (c >= H) return;
    const int n = min(V, H - c);
    float acc[V] = {};
    for (int k = 0; k < K; ++k) {
        const int row = row_of(route_to_row, t * K + k, R);
        if (row < 0) continue;
        const T* src = rows + (int64_t)row * ld_rows + c;
        Vec<T> v;
        if (n == V) v = *reinterpret_cast<const Vec<T>*>(src);
        else for (int i = 0; i < V; ++i) v.e[i] = i < n ? src[i] : from_f32<T>(0.0f);
        const float f = w ? w[t * K + k] : 1.0f;
#pragma unroll
        for (int i = 0; i < V; ++i) acc[i] = __fmaf_rn(f, to_f32(v.e[i]), acc[i]);
    }
    T* dst = out + (int64_t)t * ld_out + c;
    Vec<T> o;
#pragma unroll
    for (int i = 0; i < V; ++i) o.e[i] = from_f32<T>(acc[i]);
    if (n == V) *reinterpret_cast<Vec<T>*>(dst) = o;
    else for (int i = 0; i < n; ++i) dst[i] = o.e[i];
}

// dw[t,k] = <token[t], rows[row(t,k)]>: one wave per route.
template <typename T>
__global__ __launch_bounds__(kRowThreads) void dots_kernel(const T* __restrict__ token, int64_t ld_token,
                                                           const T* __restrict__ rows, int64_t ld_rows,
                                                           const int32_t* __restrict__ route_to_row, int K,
                                                           int H, uint32_t R, float* __restrict__ dw) {
    constexpr int V = 16 / sizeof(T);
    const size_t r = (size_t)blockIdx.x * (kRowThreads / 64) + (threadIdx.x >> 6);
    if (r >= R) return;
    const int lane = threadIdx.x & 63;
    const int row = row_of(route_to_row, r, R);
    float s = 0.0f;
    if (row >= 0) {
        const T* a = token + (int64_t)(r / K) * ld_token;
        const T* b = rows + (int64_t)row * ld_rows;
        int c = lane * V;
        for (; c + V <= H; c += 64 * V) {
            const Vec<T> x = *reinterpret_cast<const Vec<T>*>(a + c), y = *reinterpret_cast<const Vec<T>*>(b + c);
#pragma unroll
            for (int i = 0; i < V; ++i) s = __fmaf_rn(to_f32(x.e[i]), to_f32(y.e[i]), s);
        }
        for (int i = c; i < H && i < c + V; ++i) s = __fmaf_rn(to_f32(a[i]), to_f32(b[i]), s);
    }
    s = wave_sum(s);
    if (lane == 0) dw[r] = s;
}

struct RowArgs {
    const void* token_in;   // spread's source, and the tokens of the dots
    int64_t ld_token_in;
    const void* rows_in;    // collect's source, and the rows of the dots
    int64_t ld_rows_in;
    const int32_t* route_to_row;
    const float* w;
    int T, K, H;
    void* out;
    int64_t ld_out;
    float* dw;              // null: no dots
};

template <typename T>
static hipError_t launch_rows_t(bool spread, const RowArgs& a, hipStream_t s) {
    const uint32_t R = (uint32_t)a.T * a.K;
    constexpr int cols = kRowThreads * 16 / (int)sizeof(T);
    const dim3 grid(a.T, (a.H + cols - 1) / cols);
    if (spread)
        hipLaunchKernelGGL(spread_kernel<T>, grid, dim3(kRowThreads), 0, s, (const T*)a.token_in, a.ld_token_in,
                           a.route_to_row, a.w, a.K, a.H, R, (T*)a.out, a.ld_out);
    else
        hipLaunchKernelGGL(collect_kernel<T>, grid, dim3(kRowThreads), 0, s, (const T*)a.rows_in, a.ld_rows_in,
                           a.route_to_row, a.w, a.K, a.H, R, (T*)a.out, a.ld_out);
    if (a.dw)
        hipLaunchKernelGGL(dots_kernel<T>, dim3((R + 3) / 4), dim3(kRowThreads), 0, s, (const T*)a.token_in,
                           a.ld_token_in, (const T*)a.rows_in, a.ld_rows_in, a.route_to_row, a.K, a.H, R, a.dw);
    return hipGetLastError();
}

static hipError_t launch_rows(bool spread, int dtype, const RowArgs& a, hipStream_t s) {
    if (dtype == MOE_DT_BF16) return launch_rows_t<Bf16>(spread, a, s);
    if (dtype == MOE_DT_FP16) return launch_rows_t<Fp16>(spread, a, s);
    return launch_rows_t<float>(spread, a, s);
}

// Every check of the four entry points, then the launch. spread: the output has
// R rows; else T.
static int run_rows(bool spread, const char* what, int dtype, const RowArgs& a, hipStream_t stream) {
    const int64_t R = (int64_t)a.T * a.K;
    if (!dtype_ok(dtype)) return reject(MOE_ERR_INVALID, "dtype=%d is not a moe_dtype", dtype);
    if (a.T < 0) return reject(MOE_ERR_INVALID, "T=%d is negative", a.T);
    if (a.K < 1 || a.K > kMaxK) return reject(MOE_ERR_INVALID, "K=%d outside [1, %d]", a.K, kMaxK);
    if (a.H < 1 || a.H > (1 << 20)) return reject(MOE_ERR_UNSUPPORTED, "H=%d outside [1, %d]", a.H, 1 << 20);
    if (R > (1 << 26)) return reject(MOE_ERR_UNSUPPORTED, "T*K=%lld routes above %d", (long long)R, 1 << 26);
    if (a.dw && !a.w) return reject(MOE_ERR_INVALID, "a gradient of weights that are not there");
    if (a.T == 0) return MOE_OK;
    const bool tok = spread || a.dw, rows = !spread || a.dw;
    if (!a.route_to_row || !a.out || (tok && !a.token_in) || (rows && !a.rows_in))
        return reject(MOE_ERR_INVALID, "NULL pointer argument");
    const int64_t out_rows = spread ? R : a.T;
    if ((tok && a.ld_token_in < 0) || (rows && a.ld_rows_in < 0))
        return reject(MOE_ERR_INVALID, "a row stride is negative");
    if (out_rows > 1 && a.ld_out < a.H)
        return reject(MOE_ERR_INVALID, "the output's row stride %lld is below H=%d", (long long)a.ld_out, a.H);
    const int64_t far = (int64_t)1 << 32;
    if (a.ld_out > far || (tok && a.ld_token_in > far) || (rows && a.ld_rows_in > far))
        return reject(MOE_ERR_UNSUPPORTED, "a row stride above 2^32 elements");
    const size_t es = dtype_bytes(dtype);
    if (!is_aligned(a.out, es) || (tok && !is_aligned(a.token_in, es)) || (rows && !is_aligned(a.rows_in, es)) ||
        !is_aligned(a.route_to_row, 4) || !is_aligned(a.w, 4) || !is_aligned(a.dw, 4))
        return reject(MOE_ERR_INVALID, "misaligned pointer");
    const size_t n_out = extent(out_rows, a.ld_out, a.H, (int)es), n_dw = a.dw ? (size_t)R * 4 : 0;
    const struct { const void* p; size_t n; } in[] = {
        {tok ? a.token_in : nullptr, tok ? extent(a.T, a.ld_token_in, a.H, (int)es) : 0},
        {rows ? a.rows_in : nullptr, rows ? extent(R, a.ld_rows_in, a.H, (int)es) : 0},
        {a.route_to_row, (size_t)R * 4}, {a.w, a.w ? (size_t)R * 4 : 0}};
    for (const auto& b : in)
        if (overlap(b.p, b.n, a.out, n_out) || overlap(b.p, b.n, a.dw, n_dw))
            return reject(MOE_ERR_INVALID, "an output overlaps an input");
    if (overlap(a.out, n_out, a.dw, n_dw)) return reject(MOE_ERR_INVALID, "the outputs overlap");
    return launched(launch_rows(spread, dtype, a, stream), what);
}

}  // namespace moe

using namespace moe;

extern "C" int moe_dispatch(const void* x, int64_t x_stride, int32_t dtype, const int32_t* route_to_row,
                            const float* weights, int32_t T, int32_t K, int32_t H, void* rows,
                            int64_t rows_stride, hipStream_t stream) {
    return run_rows(true, "dispatch", dtype,
                    RowArgs{x, x_stride, nullptr, 0, route_to_row, weights, T, K, H, rows, rows_stride, nullptr}, stream);
}

extern "C" int moe_dispatch_grad(const void* drows, int64_t drows_stride, int32_t dtype,
                                 const int32_t* route_to_row, const float* weights, const void* x,
                                 int64_t x_stride, int32_t T, int32_t K, int32_t H, void* dx,
                                 int64_t dx_stride, float* dweights, hipStream_t stream) {
    return run_rows(false, "dispatch gradient", dtype,
                    RowArgs{x, x_stride, drows, drows_stride, route_to_row, weights, T, K, H, dx, dx_stride, dweights},
                    stream);
}

extern "C" int moe_combine(const void* rows, int64_t rows_stride, int32_t dtype, const int32_t* route_to_row,
                           const float* weights, int32_t T, int32_t K, int32_t H, void* y, int64_t y_stride,
                           hipStream_t stream) {
    return run_rows(false, "combine", dtype,
                    RowArgs{nullptr, 0, rows, rows_stride, route_to_row, weights, T, K, H, y, y_stride, nullptr}, stream);
}

extern "C" int moe_combine_grad(const void* dy, int64_t dy_stride, int32_t dtype, const int32_t* route_to_row,
                                const float* weights, const void* rows, int64_t rows_stride, int32_t T,
                                int32_t K, int32_t H, void* drows, int64_t drows_stride, float* dweights,
                                hipStream_t stream) {
    return run_rows(true, "combine gradient", dtype,
                    RowArgs{dy, dy_stride, rows, rows_stride, route_to_row, weights, T, K, H, drows, drows_stride, dweights},
                    stream);
}
