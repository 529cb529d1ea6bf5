// Low-rank adapters of many requests beside a shared projection:
//   out[t] = base[t] + scales[e] b[e] (a[e] x[t]),   e the adapter of token t,
// and out[t] = base[t] for a token without one. The tokens are sorted by adapter.
//
// Two launches. The first multiplies the tokens of one adapter with its a[e] ([r][H]); the
// depth is split over blocks where there are few tokens, each leaving one fp32 partial
// sum of v = a x in the workspace. The second adds them in a fixed order and multiplies
// with b[e] ([N][r]). v stays as exact as fp32 there: it is split in two parts of the
// operands' type, hi + lo (16 bits or more of it), which costs a second matrix
// instruction where the matrix cores have nothing else to do. fp16 parts are scaled by a
// power of two per token, as v may lie outside fp16's range.
//
// Matrix operands come straight from memory: a lane holds 8 consecutive elements of one
// row (16x16x32, rows lane % 16); any order of the depth serves as long as both operands
// have the same, so a lane takes 16 consecutive ones for two instructions, and the four
// lanes of a row read one line.
#include <algorithm>

#include "moe_args.h"
#include "moe_rows_dev.h"
#include "moe_tiles_dev.h"

#define INLINE __attribute__((always_inline))

namespace moe {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

__device__ __forceinline__ f32x4 mma(const Vec<Bf16>& a, const Vec<Bf16>& b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
}
__device__ __forceinline__ f32x4 mma(const Vec<Fp16>& a, const Vec<Fp16>& b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
}

struct AdaptArgs {
    const void* base;
    int64_t ld_base;
    const void* x;
    int64_t ld_x;
    const int32_t* row_to_token;
    const int32_t* token_to_row;
    const int32_t* offsets;
    const void* a;
    int64_t a_adapter, ld_a;
    const void* b;
    int64_t b_adapter, ld_b;
    const float* scales;  // or null: ones
    int T, n, H, r, N;
    float* part;          // [splits][T][r]
    int splits;
    void* out;
    int64_t ld_out;
};

constexpr int kStep = 64;  // depth of two matrix instructions

// v of the tile's rows, NT * 16 ranks, over one part of the depth. WK of the block's four
// waves share it among them, the others have rows of their own.
template <typename T, int MS, int NT, int WK>
__global__ __launch_bounds__(256) void adapt_down_kernel(AdaptArgs p, int most) {
    constexpr int WM = 4 / WK, BM = WM * MS * 16;
    __shared__ f32x4 s_acc[WK > 1 ? WK : 1][WK > 1 ? MS * NT : 1][64];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wm = wave / WK, wk = wave % WK, c = lane & 15, q = lane >> 4;
    const int split = blockIdx.x % p.splits;
    int e, row0, rows;
    if (!find_tile<BM>(p.offsets, p.n, p.T, blockIdx.x / p.splits, lane, &e, &row0, &rows)) return;
    const int r0 = blockIdx.y * NT * 16;
    const T* xr[MS];
    const T* ar[NT];
#pragma unroll
    for (int m = 0; m < MS; ++m) {
        // (rows behind the last one and entries that name no token: any token, not used)
        const int row = row0 + min(wm * MS * 16 + m * 16 + c, rows - 1), t = p.row_to_token[row];
        xr[m] = (const T*)p.x + (int64_t)((uint32_t)t < (uint32_t)p.T ? t : 0) * p.ld_x + 16 * q;
    }
#pragma unroll
    for (int j = 0; j < NT; ++j)
        ar[j] = (const T*)p.a + e * p.a_adapter + (int64_t)min(r0 + j * 16 + c, p.r - 1) * p.ld_a + 16 * q;
    f32x4 acc[MS][NT] = {};
    const int steps = (p.H + kStep - 1) / kStep, each = (steps + p.splits - 1) / p.splits;
    const int hi = min(steps, (split + 1) * each);
    for (int s = split * each + wk; s < hi; s += WK) {
        const int k = s * kStep;
        Vec<T> xv[MS][2] = {}, av[NT][2] = {};
        if (k + 16 * q < p.H) {  // (H is a multiple of 16)
#pragma unroll
            for (int j = 0; j < NT; ++j)
#pragma unroll
                for (int h = 0; h < 2; ++h) av[j][h] = load_vec(ar[j] + k + 8 * h);
#pragma unroll
            for (int m = 0; m < MS; ++m)
#pragma unroll
                for (int h = 0; h < 2; ++h) xv[m][h] = load_vec(xr[m] + k + 8 * h);
        }
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int m = 0; m < MS; ++m)
#pragma unroll
                for (int j = 0; j < NT; ++j) acc[m][j] = mma(av[j][h], xv[m][h], acc[m][j]);
    }
    // acc[m][j]: token m * 16 + c, ranks j * 16 + 4 q + 0..3
    float* part = p.part + (int64_t)split * p.T * p.r;
    auto put = [&](int m, int j, f32x4 v) INLINE {
        const int row = wm * MS * 16 + m * 16 + c, rank = r0 + j * 16 + 4 * q;
        if (row < rows && rank < p.r) *reinterpret_cast<f32x4*>(part + (int64_t)(row0 + row) * p.r + rank) = v;
    };
    if constexpr (WK == 1) {
#pragma unroll
        for (int m = 0; m < MS; ++m)
#pragma unroll
            for (int j = 0; j < NT; ++j) put(m, j, acc[m][j]);
    } else {
        static_assert(WK == 4, "a tile's waves are the block's");
#pragma unroll
        for (int m = 0; m < MS; ++m)
#pragma unroll
            for (int j = 0; j < NT; ++j) s_acc[wk][m * NT + j][lane] = acc[m][j];
        __syncthreads();
#pragma unroll
        for (int f = 0; f < MS * NT; ++f)
            if (f % WK == wk) put(f / NT, f % NT, (s_acc[0][f][lane] + s_acc[1][f][lane]) + (s_acc[2][f][lane] + s_acc[3][f][lane]));
    }
}

// out = base + scale b v: MS * 16 rows by 256 columns per block, 64 columns per wave. A lane ends
// up with 16 consecutive columns of a row: the rows of b that it multiplies are dealt so.
// Blocks behind the tiles copy the rows of tokens without an adapter.
constexpr int kCopyTokens = 16;

template <typename T, int MS>
__global__ __launch_bounds__(256) void adapt_up_kernel(AdaptArgs p, int most, int nblocks) {
    constexpr int BM = MS * 16;
    extern __shared__ __align__(16) char s_room[];
    __shared__ float s_back[BM];  // what undoes the tokens' powers of two, times the adapter's scale
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6), c = lane & 15, q = lane >> 4;
    const int tile = blockIdx.x / nblocks;
    if (tile >= most) {
        const int t0 = (blockIdx.x - most * nblocks) * kCopyTokens, t = t0 + c;
        uint32_t none = (uint32_t)__ballot(lane < kCopyTokens && t < p.T && (uint32_t)p.token_to_row[min(t, p.T - 1)] >= (uint32_t)p.T);
        for (; none; none &= none - 1) {
            const int64_t u = t0 + __ffs(none) - 1;
            const T* src = (const T*)p.base + u * p.ld_base;
            T* dst = (T*)p.out + u * p.ld_out;
            for (int n = tid * 8; n < p.N; n += 256 * 8) {
                if (n + 8 <= p.N) store_vec<false>(dst + n, load_vec(src + n));
                else
                    for (int i = n; i < p.N; ++i) dst[i] = src[i];
            }
        }
        return;
    }
    int e, row0, rows;
    if (!find_tile<BM>(p.offsets, p.n, p.T, tile, lane, &e, &row0, &rows)) return;
    const int n0 = (blockIdx.x % nblocks) * 256 + wave * 64, n = n0 + 16 * q;
    int token[MS];
    Vec<T> base[MS][2];
#pragma unroll
    for (int m = 0; m < MS; ++m) {
        const int row = m * 16 + c, t = row < rows ? p.row_to_token[row0 + row] : -1;
        token[m] = (uint32_t)t < (uint32_t)p.T ? t : -1;
        if (token[m] >= 0 && n + 16 <= p.N) {
            base[m][0] = load_vec((const T*)p.base + token[m] * p.ld_base + n);
            base[m][1] = load_vec((const T*)p.base + token[m] * p.ld_base + n + 8);
        }
    }
    // v: fp32 [BM][wide], then its parts hi and lo [BM][wide] each
    const int deep = (p.r + 31) / 32 * 32, wide = deep + 8;
    float* v = (float*)s_room;
    T *v_hi = (T*)(v + BM * wide), *v_lo = v_hi + BM * wide;
    {
        constexpr int TPR = 256 / BM;  // threads of a row
        const int row = tid / TPR, at = tid % TPR;
        uint32_t top = 0;
        for (int j = at * 4; j < deep; j += TPR * 4) {
            f32x4 sum = {};
            if (row < rows && j < p.r) {
                const float* src = p.part + (int64_t)(row0 + row) * p.r + j;
                for (int s = 0; s < p.splits; ++s) sum += *reinterpret_cast<const f32x4*>(src + (int64_t)s * p.T * p.r);
            }
            *reinterpret_cast<f32x4*>(v + row * wide + j) = sum;
#pragma unroll
            for (int i = 0; i < 4; ++i) top = max(top, f2u(sum[i]) & 0x7FFFFFFFu);
        }
        // fp16: the largest |v| of the row to [2^12, 2^13). (0, infinity, NaN: as they are)
        int up = 0;
        if constexpr (std::is_same<T, Fp16>::value) {
#pragma unroll
            for (int off = TPR / 2; off >= 1; off >>= 1) top = max(top, (uint32_t)__shfl_xor((int)top, off));
            if (top && top < 0x7F800000u) up = 12 - (ilogbf(u2f(top)));
        }
        if (at == 0) s_back[row] = ldexpf(p.scales ? p.scales[e] : 1.0f, -up);
        for (int j = at * 4; j < deep; j += TPR * 4)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float f = ldexpf(v[row * wide + j + i], up);
                const T h = from_f32<T>(f);
                const float rest = f - to_f32(h);
                v_hi[row * wide + j + i] = h;
                v_lo[row * wide + j + i] = from_f32<T>(fabsf(to_f32(h)) < __builtin_huge_valf() ? rest : 0.0f);
            }
    }
    __syncthreads();
    if (n0 >= p.N) return;
    f32x4 acc[MS][4] = {};
    const T* b = (const T*)p.b + e * p.b_adapter;
    for (int k = 8 * q; k < deep; k += 32) {
        Vec<T> bv[4] = {};
        if (k < p.r) {  // (r is a multiple of 8)
#pragma unroll
            for (int u = 0; u < 4; ++u)  // row i = 4 (c / 4) + c % 4 of instruction u is column 16 (c / 4) + 4 u + c % 4
                bv[u] = load_vec(b + (int64_t)min(n0 + 16 * (c >> 2) + 4 * u + (c & 3), p.N - 1) * p.ld_b + k);
        }
#pragma unroll
        for (int m = 0; m < MS; ++m) {
            const Vec<T> hi = *reinterpret_cast<const Vec<T>*>(v_hi + (m * 16 + c) * wide + k);
            const Vec<T> lo = *reinterpret_cast<const Vec<T>*>(v_lo + (m * 16 + c) * wide + k);
#pragma unroll
            for (int u = 0; u < 4; ++u) acc[m][u] = mma(bv[u], hi, mma(bv[u], lo, acc[m][u]));
        }
    }
    // acc[m][u]: token m * 16 + c, columns n + 4 u + 0..3
#pragma unroll
    for (int m = 0; m < MS; ++m) {
        if (token[m] < 0) continue;
        const float back = s_back[m * 16 + c];
        T* dst = (T*)p.out + token[m] * p.ld_out + n;
        if (n + 16 <= p.N) {
#pragma unroll
            for (int g = 0; g < 2; ++g) {
                Vec<T> o;
#pragma unroll
                for (int i = 0; i < 8; ++i) o.e[i] = from_f32<T>(__fmaf_rn(acc[m][2 * g + i / 4][i % 4], back, to_f32(base[m][g].e[i])));
                store_vec<false>(dst + 8 * g, o);
            }
        } else {
            const T* src = (const T*)p.base + token[m] * p.ld_base + n;
#pragma unroll
            for (int i = 0; i < 16; ++i)
                if (n + i < p.N) dst[i] = from_f32<T>(__fmaf_rn(acc[m][i / 4][i % 4], back, to_f32(src[i])));
        }
    }
}

// ---------------------------------------------------------------------------
// launches
// ---------------------------------------------------------------------------
constexpr int kMaxRank = 256, kMaxSplits = 16;

// Tiles of bm rows there can be: whole ones, and a last one for each adapter with rows.
static int64_t most_tiles(int T, int n, int bm) { return T / bm + std::min(n, T); }

struct AdaptPlan {
    bool wide;  // 128-row tiles in the first product, 64-row ones in the second
    int splits;
};
static AdaptPlan plan_adapt(int T, int n, int H) {
    AdaptPlan q;
    q.wide = T >= 64 * (int64_t)std::min(n, T);
    const int64_t tiles = q.wide ? T / 128 + 1 : most_tiles(T, n, 16);
    const int64_t most = std::max((H + kStep * 4 - 1) / (kStep * 4), 1);
    q.splits = (int)std::max<int64_t>(1, std::min<int64_t>({512 / tiles, most, kMaxSplits}));
    return q;
}

template <typename T, int MS, int WK>
static void launch_down(const AdaptArgs& p, hipStream_t s) {
    const int most = (int)most_tiles(p.T, p.n, 4 / WK * MS * 16);
#define D(NT)                                                                                                         \
    hipLaunchKernelGGL((adapt_down_kernel<T, MS, NT, WK>), dim3(most * p.splits, (p.r + NT * 16 - 1) / (NT * 16)),     \
                       dim3(256), 0, s, p, most)
    if (p.r <= 16) D(1);
    else if (p.r <= 32) D(2);
    else D(4);
#undef D
}

template <typename T, int MS>
static void launch_up(const AdaptArgs& p, hipStream_t s) {
    const int most = (int)most_tiles(p.T, p.n, MS * 16), nblocks = (p.N + 255) / 256;
    const int copy = p.out == p.base ? 0 : (p.T + kCopyTokens - 1) / kCopyTokens;
    const int wide = (p.r + 31) / 32 * 32 + 8;
    hipLaunchKernelGGL((adapt_up_kernel<T, MS>), dim3(most * nblocks + copy), dim3(256), MS * 16 * wide * 8, s, p, most, nblocks);
}

template <typename T>
static hipError_t launch_adapt(AdaptArgs p, hipStream_t s) {
    const AdaptPlan q = plan_adapt(p.T, p.n, p.H);
    p.splits = q.splits;
    if (q.wide) launch_down<T, 2, 1>(p, s);
    else launch_down<T, 1, 4>(p, s);
    if (q.wide && p.r <= 96) launch_up<T, 4>(p, s);
    else launch_up<T, 1>(p, s);
    return hipGetLastError();
}

static int check_adapt_sizes(int T, int n, int H, int r, int N) {
    if (T < 0) return reject(MOE_ERR_INVALID, "T=%d is negative", T);
    if (T > (1 << 22)) return reject(MOE_ERR_UNSUPPORTED, "T=%d above %d", T, 1 << 22);
    if (n < 1 || n > kMaxE) return reject(MOE_ERR_INVALID, "adapters=%d outside [1, %d]", n, kMaxE);
    if (H < 1 || N < 1 || r < 1) return reject(MOE_ERR_INVALID, "H=%d, rank=%d, N=%d must be positive", H, r, N);
    if (H % 16) return reject(MOE_ERR_UNSUPPORTED, "H=%d must be a multiple of 16", H);
    if (r % 8 || r > kMaxRank) return reject(MOE_ERR_UNSUPPORTED, "rank=%d must be a multiple of 8 up to %d", r, kMaxRank);
    if (H > (1 << 20) || N > (1 << 20)) return reject(MOE_ERR_UNSUPPORTED, "H=%d, N=%d above %d", H, N, 1 << 20);
    const int64_t blocks = (most_tiles(T, n, 16) + T / kCopyTokens + 1) * ((N + 255) / 256 + 1);
    if (blocks >= ((int64_t)1 << 24)) return reject(MOE_ERR_UNSUPPORTED, "T=%d, N=%d: too many tiles", T, N);
    return MOE_OK;
}

}  // namespace moe

using namespace moe;

extern "C" size_t moe_adapt_workspace_bytes(int32_t T, int32_t adapters, int32_t H, int32_t rank) {
    if (check_adapt_sizes(T, adapters, H, rank, 1) != MOE_OK) return 0;
    return align256((size_t)std::max(T, 1) * rank * 4 * plan_adapt(std::max(T, 1), adapters, H).splits);
}

extern "C" int moe_adapt(const void* base, int64_t base_stride, const void* x, int64_t x_stride, int32_t dtype,
                         const int32_t* row_to_token, const int32_t* token_to_row, const int32_t* offsets, const void* a,
                         int64_t a_adapter_stride, int64_t a_stride, const void* b, int64_t b_adapter_stride, int64_t b_stride,
                         const float* scales, int32_t T, int32_t adapters, int32_t H, int32_t rank, int32_t N, void* workspace,
                         size_t workspace_bytes, void* out, int64_t out_stride, hipStream_t stream) {
    if (dtype != MOE_DT_BF16 && dtype != MOE_DT_FP16) return reject(MOE_ERR_INVALID, "dtype=%d must be bf16 or fp16", dtype);
    const int rc = check_adapt_sizes(T, adapters, H, rank, N);
    if (rc) return rc;
    if (T == 0) return MOE_OK;
    if (!base || !x || !row_to_token || !token_to_row || !offsets || !a || !b || !workspace || !out)
        return reject(MOE_ERR_INVALID, "NULL pointer argument");
    const int64_t far = (int64_t)1 << 32;
    auto in_ok = [&](int64_t ld) { return ld >= 0 && ld <= far; };
    if (!in_ok(base_stride) || !in_ok(x_stride) || !in_ok(a_stride) || !in_ok(b_stride) || out_stride > far ||
        (T > 1 && out_stride < N))
        return reject(MOE_ERR_INVALID, "a row stride is out of range");
    if (adapters > 1 && (a_adapter_stride < 0 || a_adapter_stride > ((int64_t)1 << 48) || b_adapter_stride < 0 ||
                         b_adapter_stride > ((int64_t)1 << 48)))
        return reject(MOE_ERR_INVALID, "an adapter stride is out of range");
    if (!is_aligned(base, 2) || !is_aligned(x, 2) || !is_aligned(a, 2) || !is_aligned(b, 2) || !is_aligned(out, 2) ||
        !is_aligned(row_to_token, 4) || !is_aligned(token_to_row, 4) || !is_aligned(offsets, 4) || !is_aligned(scales, 4) ||
        !is_aligned(workspace, 16))
        return reject(MOE_ERR_INVALID, "misaligned pointer");
    const size_t need = moe_adapt_workspace_bytes(T, adapters, H, rank);
    if (workspace_bytes < need) return reject(MOE_ERR_WORKSPACE, "workspace %zu bytes < %zu needed", workspace_bytes, need);
    if (adapters == 1) a_adapter_stride = b_adapter_stride = 0;
    const bool in_place = out == base && (T == 1 || out_stride == base_stride);
    if (out == base && !in_place) return reject(MOE_ERR_INVALID, "the output overlaps an input");
    const int64_t t4 = (int64_t)T * 4, last = adapters - 1;
    const Bytes in[] = {matrix(in_place ? nullptr : base, T, base_stride, N, 2), matrix(x, T, x_stride, H, 2), flat(row_to_token, t4),
                        flat(token_to_row, t4), flat(offsets, ((int64_t)adapters + 1) * 4), flat(scales, (int64_t)adapters * 4),
                        // (all of the adapters as one piece)
                        flat(a, 2 * (last * a_adapter_stride + (int64_t)(rank - 1) * a_stride + H)),
                        flat(b, 2 * (last * b_adapter_stride + (int64_t)(N - 1) * b_stride + rank))};
    const Bytes o = matrix(out, T, out_stride, N, 2), ws = flat(workspace, (int64_t)need);
    for (const Bytes& i : in)
        if (overlap(i, o) || overlap(i, ws)) return reject(MOE_ERR_INVALID, "the output or the workspace overlaps an input");
    if (overlap(o, ws)) return reject(MOE_ERR_INVALID, "the output and the workspace overlap");
    const AdaptArgs p{base, base_stride, x, x_stride, row_to_token, token_to_row, offsets, a, a_adapter_stride, a_stride, b,
                      b_adapter_stride, b_stride, scales, T, adapters, H, rank, N, (float*)workspace, 1, out, out_stride};
    return launched(dtype == MOE_DT_BF16 ? launch_adapt<Bf16>(p, stream) : launch_adapt<Fp16>(p, stream), "low-rank adapters");
}
