// The activation between an expert's two products, over the sorted rows, with an output
// in the rows' type or in 8-bit codes, and its gradient.
//
//   swiglu: a_j = silu(g_j) u_j, a row of h being [g | u];   relu2: a_j = max(h_j, 0)^2
//   out = w a, with w the router's weight of the row's route (1 without weights)
//
// With sig = 1 / (1 + exp(-g)) and e = exp(-|g|), both sig and 1 - sig are e / (1 + e)
// and 1 / (1 + e), one or the other by the sign of g: neither overflows or cancels.
//
// The rows from offsets[E] on (routes of experts elsewhere) are neither read nor
// written: the number of rows is read on the device, and blocks walk over them.
#include <algorithm>

#include "moe_args.h"
#include "moe_int8_dev.h"
#include "moe_rows_dev.h"
#include "moe_wave_dev.h"

#define INLINE __attribute__((always_inline))

namespace moe {

constexpr int kMaxActCols = 32768;

struct ActArgs {
    const void* h;
    int64_t ld_h;
    const int32_t* row_to_route;  // with weights
    const int32_t* route_to_row;  // with dweights
    const int32_t* kept;          // offsets + E, or null: all rows
    const float* weights;         // [routes], or null
    void* out;                    // activation, or dh
    int64_t ld_out;
    const void* da;               // gradient
    int64_t ld_da;
    float* dweights;              // or null
    int8_t* codes;
    int64_t ld_codes;
    float* scales;
    int rows, I;
};

__device__ __forceinline__ int kept_rows(const ActArgs& p) {
    return p.kept ? min(max(*p.kept, 0), p.rows) : p.rows;
}
// The row's route, -1 where the map names none.
__device__ __forceinline__ int route_of(const ActArgs& p, int m) {
    const int r = p.row_to_route[m];
    return (uint32_t)r < (uint32_t)p.rows ? r : -1;
}

struct Silu {
    float sig, rest;  // 1 / (1 + exp(-g)) and 1 - that
};
__device__ __forceinline__ Silu silu_parts(float g) {
    const float e = expf(-fabsf(g)), r = __builtin_amdgcn_rcpf(1.0f + e);
    return g >= 0.0f ? Silu{r, e * r} : Silu{e * r, r};  // (NaN: e is NaN)
}

template <bool SWIGLU>
__device__ __forceinline__ float act_of(float g, float u) {
    if constexpr (SWIGLU) return g * silu_parts(g).sig * u;
    const float z = fmaxf(g, 0.0f);
    return g != g ? g : z * z;
}

// Threads of a row: a wave, or the block; blocks walk over rows.
template <int TPT>
struct RowThreads {
    static constexpr int kPer = TPT < 256 ? 256 / TPT : 1, kBlock = TPT < 256 ? 256 : TPT, kWaves = TPT / 64;
};
template <int TPT>
__device__ __forceinline__ int first_row() {
    return __builtin_amdgcn_readfirstlane(blockIdx.x * RowThreads<TPT>::kPer + (TPT < 256 ? threadIdx.x / TPT : 0));
}

// Bound by memory: 16384 x 2048 bf16 (201 MB) 32 us partly from the caches, 65536 x 2048 154 us (5.2 TB/s).
template <typename T, bool SWIGLU, int TPT, int NV>
__global__ __launch_bounds__(RowThreads<TPT>::kBlock) void act_kernel(ActArgs p) {
    constexpr int V = 16 / sizeof(T);
    const int at = threadIdx.x % TPT, whole = p.I / V, tail = p.I - whole * V, n = kept_rows(p);
    for (int m = first_row<TPT>(); m < n; m += gridDim.x * RowThreads<TPT>::kPer) {
        const int r = p.weights ? route_of(p, m) : 0;  // (the row's loads do not wait for it)
        const T* h = (const T*)p.h + m * p.ld_h;
        T* out = (T*)p.out + m * p.ld_out;
        Vec<T> g[NV], u[NV];
#pragma unroll
        for (int j = 0; j < NV; ++j)
            if (at + j * TPT < whole) {
                g[j] = load_vec(h + (at + j * TPT) * V);
                if (SWIGLU) u[j] = load_vec(h + p.I + (at + j * TPT) * V);
            }
        if (r < 0) continue;
        const float w = p.weights ? p.weights[r] : 1.0f;
#pragma unroll
        for (int j = 0; j < NV; ++j)
            if (at + j * TPT < whole) {
                Vec<T> o;
#pragma unroll
                for (int i = 0; i < V; ++i)
                    o.e[i] = from_f32<T>(act_of<SWIGLU>(to_f32(g[j].e[i]), SWIGLU ? to_f32(u[j].e[i]) : 0.0f) * w);
                store_vec<false>(out + (at + j * TPT) * V, o);
            }
        if (at < tail) {
            const int c = whole * V + at;
            out[c] = from_f32<T>(act_of<SWIGLU>(to_f32(h[c]), SWIGLU ? to_f32(h[p.I + c]) : 0.0f) * w);
        }
    }
}

// ---------------------------------------------------------------------------
// 8-bit codes
// ---------------------------------------------------------------------------
// s = fl32(max_j |a_j| / 127) and code_j = round(a_j / s), of the values a_j in 64 bits, so
// that the codes are those of any implementation that is careful enough. fp32 values
// decide all but a few: the largest ones, of which the maximum is taken in fp64, and those
// whose quotient lies next to a half, which are computed again in fp64 (a vector of a
// lane at a time, by as many lanes). Rows whose largest value is below kSmallAct (fp32 loses
// bits there) are computed in fp64 altogether; one that fp32 has as 0 has scale 0.
//
// kActError, relative, from kDeep on: exp2's argument is off by 1.25 |g| half steps (2^-24), exp2
// and the reciprocal by 2 each, 1 + e, both products and the quotient by 5.5 in all: 30
// half steps at g = -16. Gates below kDeep go the exact way. The sigmoid meets u first: it lies
// between 1e-7 and 1 here, while g sigmoid(g) of a subnormal g would keep few bits. (What
// sigmoid(g) u loses below 2^-126 shows in the product only where g is beyond 2^36, whose
// sigmoid is 1 and loses nothing.)
constexpr float kActError = 0x1p-19f;
constexpr float kDeep = -16.0f;
constexpr float kSmallAct = 0x1p-90f;

template <bool SWIGLU>
__device__ __forceinline__ float act_fast(float g, float u) {
    if constexpr (SWIGLU) return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(g * -1.44269504f)) * u * g;
    const float z = fmaxf(g, 0.0f);
    return g != g ? g : z * z;
}
template <bool SWIGLU>
__device__ __forceinline__ double act_exact(double g, double u) {
    if constexpr (SWIGLU) {
        const double e = exp(-fabs(g));
        return g * ((g >= 0.0 ? 1.0 : e) / (1.0 + e)) * u;
    }
    const double z = fmax(g, 0.0);
    return z * z;
}

// Four waves per SIMD (128 registers) for rows of a wave each: 65536 x 2048 bf16 161 -> 142 us,
// 16384 x 2048 from memory 49 -> 44 (3.8 TB/s; 141 registers let three run, five spill: 117).
// Bound by memory and by the vector units. Gates below kDeep cost more, as a vector that
// has one is computed again: with gates of deviation 6 (0.4 % of them) 16384 x 2048 35 -> 73 us,
// and the wave of a row that lies there altogether takes 70 us longer than others.
template <typename T, bool SWIGLU, int TPT, int NV>
__global__ __launch_bounds__(RowThreads<TPT>::kBlock, TPT == 64 ? 4 : 1) void act_int8_kernel(ActArgs p) {
    constexpr int V = 16 / sizeof(T), NW = RowThreads<TPT>::kWaves;
    static_assert(NV * V <= 64, "a lane for each of a lane's elements");
    __shared__ uint32_t s_top[2][NW];
    __shared__ double s_max[2][NW];
    const int at = threadIdx.x % TPT, lane = threadIdx.x & 63, at0 = at - lane;  // at0: lane 0's
    const int whole = p.I / V, tail = p.I - whole * V, n = kept_rows(p);
    int set = 0;
    for (int m = first_row<TPT>(); m < n; m += gridDim.x * RowThreads<TPT>::kPer) {
        const int r = p.weights ? route_of(p, m) : 0;
        const T* h = (const T*)p.h + m * p.ld_h;
        int8_t* dst = p.codes + m * p.ld_codes;
        Vec<T> g[NV], u[NV];
        T g_last{}, u_last{};
#pragma unroll
        for (int j = 0; j < NV; ++j)
            if (at + j * TPT < whole) {
                g[j] = load_vec(h + (at + j * TPT) * V);
                if (SWIGLU) u[j] = load_vec(h + p.I + (at + j * TPT) * V);
            }
        if (at < tail) {
            g_last = h[whole * V + at];
            if (SWIGLU) u_last = h[p.I + whole * V + at];
        }
        if (r < 0) continue;  // (for all threads of the row)
        const float w = p.weights ? p.weights[r] : 1.0f;
        float a[NV][V], a_last = 0.0f;
        uint32_t mine = 0, doubt = 0;  // the lane's largest |a|; its vectors to be computed again
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            float low = 0.0f;
#pragma unroll
            for (int i = 0; i < V; ++i) {
                a[j][i] = 0.0f;
                if (at + j * TPT < whole) {
                    const float gv = to_f32(g[j].e[i]);
                    a[j][i] = act_fast<SWIGLU>(gv, SWIGLU ? to_f32(u[j].e[i]) : 0.0f);
                    if (SWIGLU) low = fminf(low, gv);
                }
            }
            if (SWIGLU && low < kDeep) doubt |= 1u << j;
#pragma unroll
            for (int i = 0; i < V; ++i) mine = max(mine, f2u(a[j][i]) & 0x7FFFFFFFu);
        }
        bool odd = doubt != 0;  // has elements that fp32 says too little about
        if (at < tail) {
            a_last = act_fast<SWIGLU>(to_f32(g_last), SWIGLU ? to_f32(u_last) : 0.0f);
            odd |= SWIGLU && to_f32(g_last) < kDeep;
            mine = max(mine, f2u(a_last) & 0x7FFFFFFFu);
        }
        if (odd) mine = max(mine, 1u);  // (fp32 may have had 0 for all of a row that is not)
        uint32_t top = lanes_max(mine);
        if constexpr (NW > 1) {
            if (lane == 0) s_top[set][threadIdx.x >> 6] = top;
            __syncthreads();
#pragma unroll
            for (int v = 0; v < NW; ++v) top = max(top, s_top[set][v]);
        }
        top = __builtin_amdgcn_readfirstlane(top);
        const float big = u2f(top);
        const bool plain = top < 0x7F800000u && top > 0, small = plain && big < kSmallAct;
        auto exact = [&](int c) INLINE {  // column c, again from memory
            return act_exact<SWIGLU>((double)to_f32(h[c]), SWIGLU ? (double)to_f32(h[p.I + c]) : 0.0);
        };
        float s = 0.0f;
        if (plain) {
            const float near = small ? 0.0f : big * (1.0f - 2.0f * kActError);
            double most = 0.0;
            // all elements of each lane that has one that may be the largest, a lane each
            for (uint64_t left = __ballot(u2f(mine) >= near || odd); left; left &= left - 1) {
                const int owner = at0 + __ffsll((unsigned long long)left) - 1, v = owner + (lane / V) * TPT;
                if (lane < NV * V && v < whole) most = fmax(most, fabs(exact(v * V + lane % V)));
                if (owner < tail && lane == 0) most = fmax(most, fabs(exact(whole * V + owner)));
            }
            most = lanes_max(most);
            if constexpr (NW > 1) {
                if (lane == 0) s_max[set][threadIdx.x >> 6] = most;
                __syncthreads();
#pragma unroll
                for (int v = 0; v < NW; ++v) most = fmax(most, s_max[set][v]);
            }
            s = (float)(most / 127.0);
        } else if (top > 0) {
            s = __fdiv_rn(big, 127.0f);  // an infinity or a NaN stays one
        }
        if (at == 0) p.scales[m] = w * s;
        const bool coded = plain && s > 0.0f;
        const float inv = coded && !small ? __fdiv_rn(1.0f, s) : 0.0f;
#pragma unroll
        for (int j = 0; j < NV; ++j)
            if (at + j * TPT < whole) {
                Codes<V> c;
                float far = 0.0f;  // distance from the code, and what the quotient may be off
#pragma unroll
                for (int k = 0; k < V / 4; ++k) {
                    uint32_t b[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float x = a[j][4 * k + i], r = __fmaf_rn(x, inv, kRoundInt), code = r - kRoundInt;
                        b[i] = f2u(r);
                        far = fmaxf(far, __fmaf_rn(fabsf(code), kActError, fabsf(__fmaf_rn(x, inv, -code))));
                    }
                    c.w[k] = coded ? int8_word(b) : 0;
                }
                store_codes<V>(dst + (at + j * TPT) * V, c);
                // (|code| is within a half of the quotient)
                if (far > 0.5f - 1.5f * kActError || small) doubt |= 1u << j;
            }
        auto code_exact = [&](int c) INLINE {
            return (int8_t)(int)fmin(fmax(rint(exact(c) / (double)s), -127.0), 127.0);
        };
        if (at < tail) dst[whole * V + at] = coded ? code_exact(whole * V + at) : (int8_t)0;
        if (!coded) doubt = 0;
        if (uint64_t left = __ballot(doubt != 0)) {
            asm volatile("s_waitcnt vmcnt(0)" ::: "memory");  // behind the stores of the other lanes
            do {
                const int l = __ffsll((unsigned long long)left) - 1, j = __ffs(__builtin_amdgcn_readlane((int)doubt, l)) - 1;
                const int c = (at0 + l + j * TPT) * V + lane;
                if (lane < V) dst[c] = code_exact(c);
                if (lane == l) doubt &= doubt - 1;
                left = __ballot(doubt != 0);
            } while (left);
        }
        set ^= 1;
    }
}

// ---------------------------------------------------------------------------
// gradient
// ---------------------------------------------------------------------------
// d = w da:  dg = d u sig (1 + g (1 - sig)), du = d g sig;  relu2: dh = 2 d max(h, 0);
// dweights[route] = <da, a>, 0 for a route without a row. Bound by memory: 32768 x 2048 bf16
// (671 MB) 127 us, 5.3 TB/s.
template <typename T, bool SWIGLU, int TPT, int NV>
__global__ __launch_bounds__(RowThreads<TPT>::kBlock) void act_grad_kernel(ActArgs p) {
    constexpr int V = 16 / sizeof(T), NW = RowThreads<TPT>::kWaves;
    __shared__ float s_dot[2][NW];
    const int at = threadIdx.x % TPT, whole = p.I / V, tail = p.I - whole * V, n = kept_rows(p);
    if (p.dweights)
        for (int64_t r = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; r < p.rows; r += (int64_t)gridDim.x * blockDim.x)
            if ((uint32_t)p.route_to_row[r] >= (uint32_t)p.rows) p.dweights[r] = 0.0f;
    int set = 0;
    for (int m = first_row<TPT>(); m < n; m += gridDim.x * RowThreads<TPT>::kPer) {
        const int r = p.weights ? route_of(p, m) : 0;
        const T *h = (const T*)p.h + m * p.ld_h, *da = (const T*)p.da + m * p.ld_da;
        T* dh = (T*)p.out + m * p.ld_out;
        Vec<T> g[NV], u[NV], d[NV];
#pragma unroll
        for (int j = 0; j < NV; ++j)
            if (at + j * TPT < whole) {
                g[j] = load_vec(h + (at + j * TPT) * V);
                if (SWIGLU) u[j] = load_vec(h + p.I + (at + j * TPT) * V);
                d[j] = load_vec(da + (at + j * TPT) * V);
            }
        if (r < 0) continue;
        const float w = p.weights ? p.weights[r] : 1.0f;
        float dot = 0.0f;
        auto one = [&](float gv, float uv, float dv, T* dg, T* du) INLINE {
            const float dw = dv * w;
            if constexpr (SWIGLU) {
                const Silu s = silu_parts(gv);
                const float gs = gv * s.sig;
                dot = __fmaf_rn(dv, gs * uv, dot);
                *dg = from_f32<T>(dw * uv * (s.sig * __fmaf_rn(gv, s.rest, 1.0f)));
                *du = from_f32<T>(dw * gs);
            } else {
                const float z = gv != gv ? gv : fmaxf(gv, 0.0f);
                dot = __fmaf_rn(dv, z * z, dot);
                *dg = from_f32<T>(dw * (2.0f * z));
            }
        };
#pragma unroll
        for (int j = 0; j < NV; ++j)
            if (at + j * TPT < whole) {
                Vec<T> dg, du;
#pragma unroll
                for (int i = 0; i < V; ++i)
                    one(to_f32(g[j].e[i]), SWIGLU ? to_f32(u[j].e[i]) : 0.0f, to_f32(d[j].e[i]), &dg.e[i], &du.e[i]);
                store_vec<false>(dh + (at + j * TPT) * V, dg);
                if (SWIGLU) store_vec<false>(dh + p.I + (at + j * TPT) * V, du);
            }
        if (at < tail) {
            const int c = whole * V + at;
            T dg, du;
            one(to_f32(h[c]), SWIGLU ? to_f32(h[p.I + c]) : 0.0f, to_f32(da[c]), &dg, &du);
            dh[c] = dg;
            if (SWIGLU) dh[p.I + c] = du;
        }
        if (p.dweights) {
            dot = lanes_sum(dot);
            if constexpr (NW > 1) {
                if ((threadIdx.x & 63) == 0) s_dot[set][threadIdx.x >> 6] = dot;
                __syncthreads();
                dot = 0.0f;
#pragma unroll
                for (int v = 0; v < NW; ++v) dot += s_dot[set][v];
            }
            if (at == 0) p.dweights[r] = dot;
            set ^= 1;
        }
    }
}

// ---------------------------------------------------------------------------
// launches
// ---------------------------------------------------------------------------
// Threads of a row: as few as keep it in registers, a block from 64 vectors on; the codes of
// many rows a wave up to 256, which needs no barrier. bf16, I = 2048, in a graph, us, with a
// block (with a wave): 4096 rows 10.1 (12.0), gradient 14.5 (17.4), codes 13.3 (12.9); 16384
// rows 33.5 (37.6), 63 (68), codes 42 (39); codes of 16384 x 1024 32 (21).
template <typename T, bool SWIGLU>
static hipError_t launch_act(const ActArgs& p, hipStream_t s) {
    constexpr int V = 16 / (int)sizeof(T);
    const int vecs = std::max((p.I + V - 1) / V, 1);
#define A(KERNEL, TPT, NV)                                                                                             \
    hipLaunchKernelGGL((KERNEL<T, SWIGLU, TPT, NV>),                                                                   \
                       dim3(std::min((p.rows + RowThreads<TPT>::kPer - 1) / RowThreads<TPT>::kPer, blocks)),           \
                       dim3(RowThreads<TPT>::kBlock), 0, s, p)
#define SHAPES(KERNEL, BLOCKS, WAVE)                                                                                   \
    do {                                                                                                               \
        const int blocks = BLOCKS;                                                                                     \
        if (vecs <= 64) A(KERNEL, 64, 1);                                                                              \
        else if (WAVE && vecs <= 128) A(KERNEL, 64, 2);                                                                \
        else if (WAVE && vecs <= 256) A(KERNEL, 64, 4);                                                                \
        else if (vecs <= 256) A(KERNEL, 256, 1);                                                                       \
        else if (vecs <= 512) A(KERNEL, 256, 2);                                                                       \
        else if (vecs <= 1024) A(KERNEL, 256, 4);                                                                      \
        else if (V == 8 || vecs <= 4096) A(KERNEL, 1024, 4);                                                           \
        else if constexpr (V == 4) A(KERNEL, 1024, 8);                                                                 \
    } while (0)
    const bool many = p.rows >= 4096;
    if (p.da) SHAPES(act_grad_kernel, 8192, false);
    else if (p.codes) SHAPES(act_int8_kernel, 4096, many);
    else SHAPES(act_kernel, 8192, false);
#undef SHAPES
#undef A
    return hipGetLastError();
}

template <typename T>
static hipError_t launch_act(const ActArgs& p, int act, hipStream_t s) {
    return act == MOE_ACT_SWIGLU ? launch_act<T, true>(p, s) : launch_act<T, false>(p, s);
}

static bool act_stride_ok(int64_t stride, int rows, int64_t cols, bool output) {
    return stride >= (output && rows > 1 ? cols : 0) && stride <= ((int64_t)1 << 32);
}

// The checks of all three calls, then the launch. routes: rows of the order (0: none).
static int run_act(ActArgs p, int dtype, int act, const int32_t* offsets, int E, hipStream_t stream) {
    if (!dtype_ok(dtype)) return reject(MOE_ERR_INVALID, "dtype=%d is not a moe_dtype", dtype);
    if (act != MOE_ACT_SWIGLU && act != MOE_ACT_RELU2) return reject(MOE_ERR_INVALID, "act=%d is not a moe_act", act);
    if (p.rows < 0) return reject(MOE_ERR_INVALID, "rows=%d is negative", p.rows);
    if (p.rows > kMaxRows) return reject(MOE_ERR_UNSUPPORTED, "rows=%d above %lld", p.rows, (long long)kMaxRows);
    if (p.I < 1 || p.I > kMaxActCols) return reject(MOE_ERR_UNSUPPORTED, "I=%d outside [1, %d]", p.I, kMaxActCols);
    if (offsets && (E < 1 || E > kMaxE)) return reject(MOE_ERR_INVALID, "E=%d outside [1, %d]", E, kMaxE);
    if (p.weights && (!p.row_to_route || !offsets)) return reject(MOE_ERR_INVALID, "weights need row_to_route and offsets");
    if (p.dweights && (!p.weights || !p.route_to_row)) return reject(MOE_ERR_INVALID, "dweights needs weights and route_to_row");
    if (p.rows == 0) return MOE_OK;
    const int es = dtype_bytes(dtype);
    const int64_t wide = act == MOE_ACT_SWIGLU ? 2 * (int64_t)p.I : p.I;
    if (!act_stride_ok(p.ld_h, p.rows, wide, false) || (p.da && !act_stride_ok(p.ld_da, p.rows, p.I, false)) ||
        (p.out && !act_stride_ok(p.ld_out, p.rows, p.da ? wide : p.I, true)) ||
        (p.codes && !act_stride_ok(p.ld_codes, p.rows, p.I, true)))
        return reject(MOE_ERR_INVALID, "a row stride is out of range");
    if (!is_aligned(p.h, es) || !is_aligned(p.da, es) || !is_aligned(p.out, es) || !is_aligned(p.scales, 4) ||
        !is_aligned(p.weights, 4) || !is_aligned(p.dweights, 4) || !is_aligned(offsets, 4) || !is_aligned(p.row_to_route, 4) ||
        !is_aligned(p.route_to_row, 4))
        return reject(MOE_ERR_INVALID, "misaligned pointer");
    const int64_t r4 = (int64_t)p.rows * 4;
    const Bytes in[] = {matrix(p.h, p.rows, p.ld_h, wide, es), matrix(p.da, p.rows, p.ld_da, p.I, es), flat(p.weights, r4),
                        flat(p.row_to_route, r4), flat(p.route_to_row, r4), flat(offsets, ((int64_t)E + 1) * 4)};
    const Bytes out[] = {matrix(p.out, p.rows, p.ld_out, p.da ? wide : p.I, es), matrix(p.codes, p.rows, p.ld_codes, p.I, 1),
                         flat(p.scales, r4), flat(p.dweights, r4)};
    for (const Bytes& o : out)
        for (const Bytes& i : in)
            if (overlap(i, o)) return reject(MOE_ERR_INVALID, "an output overlaps an input");
    for (int i = 0; i < 4; ++i)
        for (int j = i + 1; j < 4; ++j)
            if (overlap(out[i], out[j])) return reject(MOE_ERR_INVALID, "the outputs overlap");
    p.kept = offsets ? offsets + E : nullptr;
    hipError_t e;
    if (dtype == MOE_DT_BF16) e = launch_act<Bf16>(p, act, stream);
    else if (dtype == MOE_DT_FP16) e = launch_act<Fp16>(p, act, stream);
    else e = launch_act<float>(p, act, stream);
    return launched(e, "activation");
}

}  // namespace moe

using namespace moe;

extern "C" int moe_activate(const void* h, int64_t h_stride, int32_t dtype, int32_t act, int32_t rows, int32_t I,
                            const int32_t* offsets, int32_t E, const int32_t* row_to_route, const float* weights, void* out,
                            int64_t out_stride, hipStream_t stream) {
    if (rows > 0 && (!h || !out)) return reject(MOE_ERR_INVALID, "NULL pointer argument");
    ActArgs p{};
    p.h = h, p.ld_h = h_stride, p.rows = rows, p.I = I, p.row_to_route = weights ? row_to_route : nullptr, p.weights = weights;
    p.out = out, p.ld_out = out_stride;
    return run_act(p, dtype, act, offsets, E, stream);
}

extern "C" int moe_activate_int(const void* h, int64_t h_stride, int32_t dtype, int32_t act, int32_t rows, int32_t I,
                                const int32_t* offsets, int32_t E, const int32_t* row_to_route, const float* weights,
                                int8_t* codes, int64_t codes_stride, float* scales, hipStream_t stream) {
    if (rows > 0 && (!h || !codes || !scales)) return reject(MOE_ERR_INVALID, "NULL pointer argument");
    ActArgs p{};
    p.h = h, p.ld_h = h_stride, p.rows = rows, p.I = I, p.row_to_route = weights ? row_to_route : nullptr, p.weights = weights;
    p.codes = codes, p.ld_codes = codes_stride, p.scales = scales;
    return run_act(p, dtype, act, offsets, E, stream);
}

extern "C" int moe_activate_grad(const void* da, int64_t da_stride, const void* h, int64_t h_stride, int32_t dtype, int32_t act,
                                 int32_t rows, int32_t I, const int32_t* offsets, int32_t E, const int32_t* row_to_route,
                                 const int32_t* route_to_row, const float* weights, void* dh, int64_t dh_stride, float* dweights,
                                 hipStream_t stream) {
    if (rows > 0 && (!da || !h || !dh)) return reject(MOE_ERR_INVALID, "NULL pointer argument");
    ActArgs p{};
    p.h = h, p.ld_h = h_stride, p.rows = rows, p.I = I, p.row_to_route = weights ? row_to_route : nullptr, p.weights = weights;
    p.route_to_row = dweights ? route_to_row : nullptr, p.da = da, p.ld_da = da_stride, p.out = dh, p.ld_out = dh_stride;
    p.dweights = dweights;
    return run_act(p, dtype, act, offsets, E, stream);
}
