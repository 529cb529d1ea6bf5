// Token rows to the experts' rows and back, and the gradients of both.
//
// With row(t, k) the sorted row of route t*K + k (none for a dropped route):
//   spread:  out[row(t,k)] = w[t,k] * token[t]          dispatch, and combine's gradient
//   collect: out[t] = sum_k w[t,k] * rows[row(t,k)]     combine, and dispatch's gradient
//   dots:    dw[t,k] = <token[t], rows[row(t,k)]>       both gradients, of the weights
// w missing means 1. Sums run in fp32, k ascending, with one rounding to the
// type of the rows at the end; a dropped route contributes nothing and its dw
// is 0. Everything is bound by memory: a token's row is read once and its K
// expert rows are written or read once each. 16384 tokens x 7168 bf16 with 8 experts:
// dispatch 434 us, combine 398 us (4.9 and 5.3 TB/s, a large copy runs at 4.9).
#include "moe_args.h"
#include "moe_rows_dev.h"

namespace moe {

// Columns of one token are dealt to TPT threads, 16 bytes each at a time: a wave
// for short rows (several tokens per block), a block of 256 for long ones.
constexpr int kBlock = 256;
constexpr int kBatch = 8;  // routes whose loads are on their way together

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

// This block's token (one of several for TPT = 64), the same in every lane of a wave.
template <int TPT>
__device__ __forceinline__ int my_token() {
    return __builtin_amdgcn_readfirstlane(blockIdx.x * (kBlock / TPT) + (TPT == 64 ? threadIdx.x >> 6 : 0));
}

// out[row(t,k)] = w * token[t]. A block of TPT = 256 owns 256 vectors of the
// token's columns (blockIdx.y), a wave of TPT = 64 all of them; each is read once
// and stored K times.
template <typename T, int TPT, bool PAST, bool WEIGHTED>
__global__ __launch_bounds__(kBlock) void spread_kernel(const T* __restrict__ token, int64_t ld_token,
                                                        const int32_t* __restrict__ route_to_row,
                                                        const float* __restrict__ w, int n_tokens, int K, int H,
                                                        uint32_t R, T* __restrict__ out, int64_t ld_out) {
    constexpr int V = 16 / sizeof(T);
    const int t = my_token<TPT>();
    if (t >= n_tokens) return;
    const size_t r0 = (size_t)t * K;
    const T* src = token + (int64_t)t * ld_token;
    for (int k0 = 0; k0 < K; k0 += kBatch) {
        int row[kBatch];
        float f[kBatch];
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
            row[u] = k0 + u < K ? row_of(route_to_row, r0 + k0 + u, R) : -1;
            f[u] = WEIGHTED && row[u] >= 0 ? w[r0 + k0 + u] : 0.0f;
        }
        for (int c = (blockIdx.y * TPT + threadIdx.x % TPT) * V; c < H; c += gridDim.y * TPT * V) {
            if (c + V <= H) {
                const Vec<T> v = load_vec(src + c);
#pragma unroll
                for (int u = 0; u < kBatch; ++u) {
                    if (row[u] < 0) continue;
                    Vec<T> o = v;
                    if (WEIGHTED) {
#pragma unroll
                        for (int i = 0; i < V; ++i) o.e[i] = from_f32<T>(f[u] * to_f32(v.e[i]));
                    }
                    store_vec<PAST>(out + (int64_t)row[u] * ld_out + c, o);
                }
            } else {
                for (int i = c; i < H; ++i)
#pragma unroll
                    for (int u = 0; u < kBatch; ++u)
                        if (row[u] >= 0)
                            out[(int64_t)row[u] * ld_out + i] = WEIGHTED ? from_f32<T>(f[u] * to_f32(src[i])) : src[i];
            }
        }
    }
}

// out[t] = sum_k w * rows[row(t,k)], k ascending; the loads of kBatch routes go
// out together.
template <typename T, int TPT, bool PAST>
__global__ __launch_bounds__(kBlock) void collect_kernel(const T* __restrict__ rows, int64_t ld_rows,
                                                         const int32_t* __restrict__ route_to_row,
                                                         const float* __restrict__ w, int n_tokens, int K, int H,
                                                         uint32_t R, T* __restrict__ out, int64_t ld_out) {
    constexpr int V = 16 / sizeof(T);
    const int t = my_token<TPT>();
    if (t >= n_tokens) return;
    const size_t r0 = (size_t)t * K;
    T* dst = out + (int64_t)t * ld_out;
    for (int c = (blockIdx.y * TPT + threadIdx.x % TPT) * V; c < H; c += gridDim.y * TPT * V) {
        if (c + V <= H) {
            float acc[V] = {};
            for (int k0 = 0; k0 < K; k0 += kBatch) {
                Vec<T> v[kBatch];
                float f[kBatch];
#pragma unroll
                for (int u = 0; u < kBatch; ++u) {
                    const int row = k0 + u < K ? row_of(route_to_row, r0 + k0 + u, R) : -1;
                    f[u] = 0.0f;
                    v[u] = Vec<T>{};
                    if (row >= 0) {  // a dropped route adds 0 * 0
                        v[u] = load_vec(rows + (int64_t)row * ld_rows + c);
                        f[u] = w ? w[r0 + k0 + u] : 1.0f;
                    }
                }
#pragma unroll
                for (int u = 0; u < kBatch; ++u)
#pragma unroll
                    for (int i = 0; i < V; ++i) acc[i] = __fmaf_rn(f[u], to_f32(v[u].e[i]), acc[i]);
            }
            Vec<T> o;
#pragma unroll
            for (int i = 0; i < V; ++i) o.e[i] = from_f32<T>(acc[i]);
            store_vec<PAST>(dst + c, o);
        } else {
            for (int i = c; i < H; ++i) {
                float a = 0.0f;
                for (int k = 0; k < K; ++k) {
                    const int row = row_of(route_to_row, r0 + k, R);
                    if (row >= 0) a = __fmaf_rn(w ? w[r0 + k] : 1.0f, to_f32(rows[(int64_t)row * ld_rows + i]), a);
                }
                dst[i] = from_f32<T>(a);
            }
        }
    }
}

// Both gradients with the weights' one, a token per TPT threads: the rows are
// read once for the dots and the other output together.
//   SPREAD:  out[row(t,k)] = w * token[t]              dw[t,k] = <token[t], rows[row(t,k)]>
//   else:    out[t] = sum_k w * rows[row(t,k)] (K <= kBatch), dw as above
// A dot is summed by each thread over its columns, then over the lanes of a wave
// and the waves, always in the same order.
template <typename T, int TPT, bool PAST, bool SPREAD>
__global__ __launch_bounds__(kBlock) void grad_kernel(const T* __restrict__ token, int64_t ld_token,
                                                      const T* __restrict__ rows, int64_t ld_rows,
                                                      const int32_t* __restrict__ route_to_row,
                                                      const float* __restrict__ w, int n_tokens, int K, int H,
                                                      uint32_t R, T* __restrict__ out, int64_t ld_out,
                                                      float* __restrict__ dw) {
    constexpr int V = 16 / sizeof(T);
    __shared__ float s_dot[kBlock / 64][kBatch];
    const int t = my_token<TPT>(), lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    if (t >= n_tokens) return;  // (TPT = 64 has no barrier below; else every block has a token)
    const size_t r0 = (size_t)t * K;
    const T* tok = token + (int64_t)t * ld_token;
    for (int k0 = 0; k0 < K; k0 += kBatch) {
        float dot[kBatch] = {};
        int row[kBatch];
        float f[kBatch];
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
            row[u] = k0 + u < K ? row_of(route_to_row, r0 + k0 + u, R) : -1;
            f[u] = row[u] >= 0 ? w[r0 + k0 + u] : 0.0f;
        }
        for (int c = (threadIdx.x % TPT) * V; c < H; c += TPT * V) {
            if (c + V <= H) {
                const Vec<T> x = load_vec(tok + c);
                Vec<T> v[kBatch];
#pragma unroll
                for (int u = 0; u < kBatch; ++u) {
                    v[u] = Vec<T>{};
                    if (row[u] >= 0) v[u] = load_vec(rows + (int64_t)row[u] * ld_rows + c);
                }
                float acc[V] = {};
#pragma unroll
                for (int u = 0; u < kBatch; ++u) {
                    if (row[u] < 0) continue;
                    Vec<T> o;
#pragma unroll
                    for (int i = 0; i < V; ++i) {
                        dot[u] = __fmaf_rn(to_f32(x.e[i]), to_f32(v[u].e[i]), dot[u]);
                        if (SPREAD) o.e[i] = from_f32<T>(f[u] * to_f32(x.e[i]));
                        else acc[i] = __fmaf_rn(f[u], to_f32(v[u].e[i]), acc[i]);
                    }
                    if (SPREAD) store_vec<PAST>(out + (int64_t)row[u] * ld_out + c, o);
                }
                if (!SPREAD) {
                    Vec<T> o;
#pragma unroll
                    for (int i = 0; i < V; ++i) o.e[i] = from_f32<T>(acc[i]);
                    store_vec<PAST>(out + (int64_t)t * ld_out + c, o);
                }
            } else {
                for (int i = c; i < H; ++i) {
                    const float x = to_f32(tok[i]);
                    float acc = 0.0f;
#pragma unroll
                    for (int u = 0; u < kBatch; ++u) {
                        if (row[u] < 0) continue;
                        const float v = to_f32(rows[(int64_t)row[u] * ld_rows + i]);
                        dot[u] = __fmaf_rn(x, v, dot[u]);
                        if (SPREAD) out[(int64_t)row[u] * ld_out + i] = from_f32<T>(f[u] * x);
                        else acc = __fmaf_rn(f[u], v, acc);
                    }
                    if (!SPREAD) out[(int64_t)t * ld_out + i] = from_f32<T>(acc);
                }
            }
        }
#pragma unroll
        for (int u = 0; u < kBatch; ++u) dot[u] = wave_sum(dot[u]);
        if (TPT == 64) {
#pragma unroll
            for (int u = 0; u < kBatch; ++u)
                if (lane == u && k0 + u < K) dw[r0 + k0 + u] = dot[u];
        } else {
            if (lane == 0) {
#pragma unroll
                for (int u = 0; u < kBatch; ++u) s_dot[wave][u] = dot[u];
            }
            __syncthreads();
            if (threadIdx.x < kBatch && k0 + threadIdx.x < K) {
                float s = 0.0f;
                for (int q = 0; q < kBlock / 64; ++q) s += s_dot[q][threadIdx.x];
                dw[r0 + k0 + threadIdx.x] = s;
            }
            __syncthreads();
        }
    }
}

// dw[t,k] = <token[t], rows[row(t,k)]> alone: one wave per route.
template <typename T>
__global__ __launch_bounds__(kBlock) void dots_kernel(const T* __restrict__ token, int64_t ld_token,
                                                      const T* __restrict__ rows, int64_t ld_rows,
                                                      const int32_t* __restrict__ route_to_row, int K,
                                                      int H, uint32_t R, float* __restrict__ dw) {
    constexpr int V = 16 / sizeof(T);
    const uint32_t r = __builtin_amdgcn_readfirstlane(blockIdx.x * (kBlock / 64) + (threadIdx.x >> 6));
    if (r >= R) return;
    const int lane = threadIdx.x & 63;
    const int row = row_of(route_to_row, r, R);
    float s = 0.0f;
    if (row >= 0) {
        const T* a = token + (int64_t)(r / K) * ld_token;
        const T* b = rows + (int64_t)row * ld_rows;
        int c = lane * V;
        for (; c + V <= H; c += 64 * V) {
            const Vec<T> x = load_vec(a + c), y = load_vec(b + c);
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

// Whether the output is stored past the caches: large ones whose rows begin on 16
// bytes. Inputs and outputs changing from call to call, bf16, 8 experts a token:
// combine of 16384 x 7168 428 -> 398 us and of 4096 x 4096 61 -> 58, its gradient 119
// -> 115, dispatch of 4096 x 4096 59 -> 52 and of 16384 x 7168 the same (430, 434);
// with rows of 129 fp32 values (16384 tokens, 4 experts), whose stores split lines,
// 13 -> 18.5. Small outputs stay in the caches for whoever reads them next.
static bool store_past_caches(bool spread, const RowArgs& a, size_t es) {
    const size_t rows = spread ? (size_t)a.T * a.K : (size_t)a.T;
    return rows * a.H * es >= ((size_t)32 << 20) && is_aligned(a.out, 16) && (size_t)a.ld_out * es % 16 == 0;
}

template <typename T, int TPT, bool PAST>
static void launch_rows_tpt(bool spread, const RowArgs& a, hipStream_t s) {
    const uint32_t R = (uint32_t)a.T * a.K;
    constexpr int cols = TPT * 16 / (int)sizeof(T);
    const T *tok = (const T*)a.token_in, *rows = (const T*)a.rows_in;
    const dim3 block(kBlock), tokens((a.T + kBlock / TPT - 1) / (kBlock / TPT));
    const dim3 grid(tokens.x, TPT == 64 ? 1 : (a.H + cols - 1) / cols);
    if (a.dw && spread) {
        hipLaunchKernelGGL((grad_kernel<T, TPT, PAST, true>), tokens, block, 0, s, tok, a.ld_token_in, rows, a.ld_rows_in,
                           a.route_to_row, a.w, a.T, a.K, a.H, R, (T*)a.out, a.ld_out, a.dw);
        return;
    }
    if (a.dw && a.K <= kBatch) {
        hipLaunchKernelGGL((grad_kernel<T, TPT, PAST, false>), tokens, block, 0, s, tok, a.ld_token_in, rows, a.ld_rows_in,
                           a.route_to_row, a.w, a.T, a.K, a.H, R, (T*)a.out, a.ld_out, a.dw);
        return;
    }
    if (!spread)
        hipLaunchKernelGGL((collect_kernel<T, TPT, PAST>), grid, block, 0, s, rows, a.ld_rows_in, a.route_to_row, a.w, a.T,
                           a.K, a.H, R, (T*)a.out, a.ld_out);
    else if (a.w)
        hipLaunchKernelGGL((spread_kernel<T, TPT, PAST, true>), grid, block, 0, s, tok, a.ld_token_in, a.route_to_row, a.w,
                           a.T, a.K, a.H, R, (T*)a.out, a.ld_out);
    else
        hipLaunchKernelGGL((spread_kernel<T, TPT, PAST, false>), grid, block, 0, s, tok, a.ld_token_in, a.route_to_row, a.w,
                           a.T, a.K, a.H, R, (T*)a.out, a.ld_out);
    if (a.dw)
        hipLaunchKernelGGL(dots_kernel<T>, dim3((R + 3) / 4), block, 0, s, tok, a.ld_token_in, rows, a.ld_rows_in,
                           a.route_to_row, a.K, a.H, R, a.dw);
}

template <typename T>
static hipError_t launch_rows_t(bool spread, const RowArgs& a, hipStream_t s) {
    // A wave per token for rows of up to 2 KB, or 4 KB with dots (16384 tokens x 1536,
    // 4 experts, bf16: combine's gradient 122 -> 98 us, dispatch's 92 -> 64, the others
    // the same; 64 tokens x 7168: 13 -> 33 us, one wave is too slow there).
    const bool wave = (size_t)a.H * sizeof(T) <= (a.dw ? 4096 : 2048);
    if (store_past_caches(spread, a, sizeof(T))) {
        if (wave) launch_rows_tpt<T, 64, true>(spread, a, s);
        else launch_rows_tpt<T, 256, true>(spread, a, s);
    } else {
        if (wave) launch_rows_tpt<T, 64, false>(spread, a, s);
        else launch_rows_tpt<T, 256, false>(spread, a, s);
    }
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
    if (R > kMaxRows) return reject(MOE_ERR_UNSUPPORTED, "T*K=%lld routes above %lld", (long long)R, (long long)kMaxRows);
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
    const Bytes out = matrix(a.out, out_rows, a.ld_out, a.H, (int)es), dw = flat(a.dw, R * 4);
    const Bytes in[] = {matrix(tok ? a.token_in : nullptr, a.T, a.ld_token_in, a.H, (int)es),
                        matrix(rows ? a.rows_in : nullptr, R, a.ld_rows_in, a.H, (int)es),
                        flat(a.route_to_row, R * 4), flat(a.w, R * 4)};
    for (const Bytes& b : in)
        if (overlap(b, out) || overlap(b, dw)) return reject(MOE_ERR_INVALID, "an output overlaps an input");
    if (overlap(out, dw)) return reject(MOE_ERR_INVALID, "the outputs overlap");
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
