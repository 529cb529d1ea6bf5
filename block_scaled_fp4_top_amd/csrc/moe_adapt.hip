// Low-rank adapters of many requests beside a shared projection:
//   out[t] = base[t] + scales[e] b[e] (a[e] x[t]),   e the adapter of token t,
// and out[t] = base[t] for a token without one. The tokens are sorted by adapter.
//
// Two launches. The first multiplies the tokens of one adapter with its a[e] ([r][H]); the
// depth is split over blocks where there are few tokens, each leaving one fp32 partial
// sum of v = a x in the workspace. The second adds them in a fixed order and multiplies
// with b[e] ([N][r]). v stays what it is in fp32: three parts of the operands' type, each the
// rounded rest of those before it, hold all 24 bits (3 x 8 in bf16, 11 + 11 + 2 in fp16), at
// the price of two more matrix instructions where the matrix cores have nothing else to do.
// (With two parts, 17 bits in bf16, seven of 4096 columns of a token were rounded to the other
// neighbour.) fp16 parts are scaled by a power of two per token, as v may lie outside fp16's
// range; they end 2^-37 below the token's largest |v|.
//
// A lane's part of a matrix operand is 8 consecutive elements of row lane % 16, so 16
// neighbouring lanes read 16 rows: straight from memory that costs the address units about
// 50 cycles a load instead of 16, which is what bounds the narrow kernels, for few tokens an
// adapter, where nothing but latency counts. The wide ones go through the LDS, filled by
// direct loads of whole lines, and end with whole lines of base and out.
//
// 16384 tokens of 16 adapters of rank 64, H = 7168, N = 4096, bf16 (503 MB, 103 us of memory): 69
// us each (3.6 and 4.0 TB/s), straight from memory 108 and 126. 64 tokens of 32 adapters of
// rank 16: 4.3 and 5.3 us; one token 3.5 and 4.7. (One launch for few tokens, whose blocks each
// make all of v, takes 13 us: the address units again.)
#include <algorithm>

#include "moe_args.h"
#include "moe_lds_dev.h"
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

// v of the tile's 16 rows, NT * 16 ranks, over one part of the depth, which the block's four
// waves share among them. P steps are on their way.
template <typename T, int NT, int P>
__global__ __launch_bounds__(256) void adapt_down_kernel(AdaptArgs p) {
    __shared__ f32x4 s_acc[4][NT][64];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), c = lane & 15, q = lane >> 4;
    const int split = blockIdx.x % p.splits;
    int e, row0, rows;
    if (!find_tile<16>(p.offsets, p.n, p.T, blockIdx.x / p.splits, lane, &e, &row0, &rows)) return;
    const int r0 = blockIdx.y * NT * 16;
    // (rows behind the last one and entries that name no token: any token, not used)
    const int t = p.row_to_token[row0 + min(c, rows - 1)];
    const T* xr = (const T*)p.x + (int64_t)((uint32_t)t < (uint32_t)p.T ? t : 0) * p.ld_x + 8 * q;
    const T* ar[NT];
#pragma unroll
    for (int j = 0; j < NT; ++j)
        ar[j] = (const T*)p.a + e * p.a_adapter + (int64_t)min(r0 + j * 16 + c, p.r - 1) * p.ld_a + 8 * q;
    f32x4 acc[NT] = {};
    const int steps = (p.H + kStep - 1) / kStep, each = (steps + p.splits - 1) / p.splits;
    const int lo = split * each + wave, hi = min(steps, (split + 1) * each);
    Vec<T> xv[P][2], av[P][NT][2];
    auto load = [&](int u, int s) INLINE {
        const int k = s * kStep;
        if (s >= hi) return;
        if (k + kStep <= p.H) {
#pragma unroll
            for (int h = 0; h < 2; ++h) xv[u][h] = load_vec(xr + k + 32 * h);
#pragma unroll
            for (int j = 0; j < NT; ++j)
#pragma unroll
                for (int h = 0; h < 2; ++h) av[u][j][h] = load_vec(ar[j] + k + 32 * h);
        } else {
            const bool in[2] = {k + 8 * q < p.H, k + 32 + 8 * q < p.H};  // (H is a multiple of 16)
#pragma unroll
            for (int h = 0; h < 2; ++h) xv[u][h] = in[h] ? load_vec(xr + k + 32 * h) : Vec<T>{};
#pragma unroll
            for (int j = 0; j < NT; ++j)
#pragma unroll
                for (int h = 0; h < 2; ++h) av[u][j][h] = in[h] ? load_vec(ar[j] + k + 32 * h) : Vec<T>{};
        }
    };
#pragma unroll
    for (int u = 0; u < P; ++u) load(u, lo + u * 4);
    for (int s = lo; s < hi; s += P * 4) {
#pragma unroll
        for (int u = 0; u < P; ++u) {
            if (s + u * 4 >= hi) break;
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int j = 0; j < NT; ++j) acc[j] = mma(av[u][j][h], xv[u][h], acc[j]);
            load(u, s + (u + P) * 4);
        }
    }
    // acc[j]: token c, ranks j * 16 + 4 q + 0..3
#pragma unroll
    for (int j = 0; j < NT; ++j) s_acc[wave][j][lane] = acc[j];
    __syncthreads();
    float* part = p.part + (int64_t)split * p.T * p.r;
#pragma unroll
    for (int j = 0; j < NT; ++j) {
        const int rank = r0 + j * 16 + 4 * q;
        if (j % 4 == wave && c < rows && rank < p.r)
            *reinterpret_cast<f32x4*>(part + (int64_t)(row0 + c) * p.r + rank) =
                (s_acc[0][j][lane] + s_acc[1][j][lane]) + (s_acc[2][j][lane] + s_acc[3][j][lane]);
    }
}

constexpr int kCopyTokens = 16;

// The copy of one group of tokens without an adapter.
template <typename T>
__device__ __forceinline__ void copy_tokens(const AdaptArgs& p, int group) {
    const int tid = threadIdx.x, lane = tid & 63, t0 = group * kCopyTokens, t = t0 + (lane & 15);
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
}

// fp16: the power of two that brings a row's largest |v| (its bits) to [2^12, 2^13). (0,
// infinity, NaN: as they are)
__device__ __forceinline__ int power_for(uint32_t top) { return top && top < 0x7F800000u ? 12 - ilogbf(u2f(top)) : 0; }

// f as hi + mid + lo of type T (an infinity or a NaN in hi alone). The rests are exact: what a
// rounding leaves of a float is a float.
template <typename T>
__device__ __forceinline__ void split_value(float f, T* hi, T* mid, T* lo) {
    *hi = from_f32<T>(f);
    const float h = to_f32(*hi), rest = fabsf(h) < __builtin_huge_valf() ? f - h : 0.0f;
    *mid = from_f32<T>(rest);
    *lo = from_f32<T>(rest - to_f32(*mid));
}

// out = base + scale b v: 16 rows per block, 256 columns at a time (64 per wave), `chunks`
// times, with the next columns' b and base on their way. A lane ends up with twice 8
// consecutive columns of a row: the rows of b that it multiplies are dealt so.
// KS: b's rows are at most 32 KS long and wait in registers (0: any length, read as
// needed). Blocks behind the tiles copy the rows of tokens without an adapter.
template <typename T, int KS>
__global__ __launch_bounds__(256) void adapt_up_kernel(AdaptArgs p, int most, int nblocks, int chunks) {
    constexpr int BM = 16, KR = KS ? KS : 1;
    extern __shared__ __align__(16) char s_room[];
    __shared__ float s_back[BM];  // what undoes the tokens' powers of two, times the adapter's scale
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6), c = lane & 15, q = lane >> 4;
    const int tile = blockIdx.x / nblocks;
    if (tile >= most) {
        copy_tokens<T>(p, blockIdx.x - most * nblocks);
        return;
    }
    int e, row0, rows;
    if (!find_tile<BM>(p.offsets, p.n, p.T, tile, lane, &e, &row0, &rows)) return;
    const int t = c < rows ? p.row_to_token[row0 + c] : -1;
    const int64_t token = (uint32_t)t < (uint32_t)p.T ? t : -1;
    const int first = (blockIdx.x % nblocks) * chunks * 256 + wave * 64;
    const T* b = (const T*)p.b + e * p.b_adapter;
    Vec<T> base[2], bv[KR][4];
    auto load_base = [&](int n0) INLINE {
#pragma unroll
        for (int g = 0; g < 2; ++g) {
            const int n = n0 + 32 * g + 8 * q;
            if (token >= 0 && n + 8 <= p.N) base[g] = load_vec((const T*)p.base + token * p.ld_base + n);
        }
    };
    auto load_b = [&](int n0, int k, Vec<T>* v) INLINE {
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            v[u] = Vec<T>{};
            // row 4 i + j of instruction u is column 32 (u / 2) + 8 i + 4 (u % 2) + j (r is a multiple of 8)
            if (k < p.r) v[u] = load_vec(b + (int64_t)min(n0 + 32 * (u >> 1) + 8 * (c >> 2) + 4 * (u & 1) + (c & 3), p.N - 1) * p.ld_b + k);
        }
    };
    if (KS) {
#pragma unroll
        for (int s = 0; s < KR; ++s) load_b(first, 32 * s + 8 * q, bv[s]);
    }
    load_base(first);
    // v: fp32 [BM][wide], then its parts hi, mid and lo [BM][wide] each
    const int deep = KS ? 32 * KS : (p.r + 31) / 32 * 32, wide = deep + 8;
    float* v = (float*)s_room;
    T *v_hi = (T*)(v + BM * wide), *v_mid = v_hi + BM * wide, *v_lo = v_mid + BM * wide;
    {
        constexpr int TPR = 256 / BM;  // threads of a row
        const int row = tid / TPR, at = tid % TPR;
        uint32_t top = 0;
        for (int j = at * 4; j < deep; j += TPR * 4) {
            f32x4 sum = {};
            if (row < rows && j < p.r) {
                const float* src = p.part + (int64_t)(row0 + row) * p.r + j;
                const int64_t far = (int64_t)p.T * p.r;
                for (int s = 0; s < p.splits; s += 8) {  // eight loads on their way, added in order
                    f32x4 w[8];
#pragma unroll
                    for (int i = 0; i < 8; ++i) w[i] = *reinterpret_cast<const f32x4*>(src + min(s + i, p.splits - 1) * far);
#pragma unroll
                    for (int i = 0; i < 8; ++i) sum += s + i < p.splits ? w[i] : f32x4{};
                }
            }
            *reinterpret_cast<f32x4*>(v + row * wide + j) = sum;
#pragma unroll
            for (int i = 0; i < 4; ++i) top = max(top, f2u(sum[i]) & 0x7FFFFFFFu);
        }
        int up = 0;
        if constexpr (std::is_same<T, Fp16>::value) {
#pragma unroll
            for (int off = TPR / 2; off >= 1; off >>= 1) top = max(top, (uint32_t)__shfl_xor((int)top, off));
            up = power_for(top);
        }
        if (at == 0) s_back[row] = ldexpf(p.scales ? p.scales[e] : 1.0f, -up);
        for (int j = at * 4; j < deep; j += TPR * 4)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int o = row * wide + j + i;
                split_value(ldexpf(v[o], up), &v_hi[o], &v_mid[o], &v_lo[o]);
            }
    }
    __syncthreads();
    for (int i = 0; i < chunks; ++i) {
        const int n0 = first + i * 256;
        if (n0 >= p.N) return;
        const bool more = i + 1 < chunks && n0 + 256 < p.N;
        f32x4 acc[4] = {};
        auto multiply = [&](int k, const Vec<T>* w) INLINE {
            const Vec<T> hi = *reinterpret_cast<const Vec<T>*>(v_hi + c * wide + k);
            const Vec<T> mid = *reinterpret_cast<const Vec<T>*>(v_mid + c * wide + k);
            const Vec<T> lo = *reinterpret_cast<const Vec<T>*>(v_lo + c * wide + k);
#pragma unroll
            for (int u = 0; u < 4; ++u) acc[u] = mma(w[u], hi, mma(w[u], mid, mma(w[u], lo, acc[u])));
        };
        if constexpr (KS > 0) {
#pragma unroll
            for (int s = 0; s < KS; ++s) multiply(32 * s + 8 * q, bv[s]);
            if (more) {
#pragma unroll
                for (int s = 0; s < KS; ++s) load_b(n0 + 256, 32 * s + 8 * q, bv[s]);
            }
        } else {
            for (int k = 8 * q; k < deep; k += 32) {
                load_b(n0, k, bv[0]);
                multiply(k, bv[0]);
            }
        }
        // acc[u]: token c, columns n0 + 32 (u / 2) + 8 q + 4 (u % 2) + 0..3
        if (token >= 0) {
            const float back = s_back[c];
#pragma unroll
            for (int g = 0; g < 2; ++g) {
                const int n = n0 + 32 * g + 8 * q;
                T* dst = (T*)p.out + token * p.ld_out + n;
                if (n + 8 <= p.N) {
                    Vec<T> o;
#pragma unroll
                    for (int j = 0; j < 8; ++j) o.e[j] = from_f32<T>(__fmaf_rn(acc[2 * g + j / 4][j % 4], back, to_f32(base[g].e[j])));
                    store_vec<false>(dst, o);
                } else {
                    const T* src = (const T*)p.base + token * p.ld_base + n;
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        if (n + j < p.N) dst[j] = from_f32<T>(__fmaf_rn(acc[2 * g + j / 4][j % 4], back, to_f32(src[j])));
                }
            }
        }
        if (more) load_base(n0 + 256);
    }
}

// ---------------------------------------------------------------------------
// many tokens an adapter
// ---------------------------------------------------------------------------
// v of 64 * MS rows, 16 * MS a wave, NT * 16 ranks, over one part of the depth: steps of 128
// bytes of depth through P LDS buffers. The wave's own rows of x and its share of those of
// a: one load brings 8 rows of 128 bytes, chunk (l % 8) ^ mix(row) of row l / 8 to lane l, so
// that an operand read (one chunk of 16 rows) uses all banks.
template <typename T, int MS, int NT, int P>
__global__ __launch_bounds__(256) void adapt_down_wide_kernel(AdaptArgs p, uint32_t x_bytes) {
    constexpr int LX = 2 * MS, LA = NT > 2 ? NT / 2 : 1, L = LX + LA, kRow = 128, kRows = 64 * MS;
    constexpr int kA = kRows * kRow, BUF = kA + 4 * LA * 8 * kRow;
    __shared__ __attribute__((aligned(1024))) uint8_t lds[P * BUF];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), c = lane & 15, q = lane >> 4;
    const int split = blockIdx.x % p.splits;
    int e, row0, rows;
    if (!find_tile<kRows>(p.offsets, p.n, p.T, blockIdx.x / p.splits, lane, &e, &row0, &rows)) return;
    const int r0 = blockIdx.y * NT * 16;
    auto mix = [](int row) INLINE { return (row >> 1) & 7; };
    // (rows behind the last one and entries that name no token: any token, not used)
    uint32_t xo[LX], ao[LA];  // where a lane's rows begin
    int xk[LX], ak[LA];       // where its chunk begins in a step
#pragma unroll
    for (int i = 0; i < LX; ++i) {
        const int row = (wave * LX + i) * 8 + (lane >> 3), t = p.row_to_token[row0 + min(row, rows - 1)];
        xk[i] = ((lane & 7) ^ mix(row)) * 8;
        xo[i] = ((uint32_t)t < (uint32_t)p.T ? t : 0) * (uint32_t)(p.ld_x * 2) + xk[i] * 2;
    }
    const T* a = (const T*)p.a + e * p.a_adapter + r0 * p.ld_a;
    const int ranks = min(NT * 16, p.r - r0);
    const uint32_t a_bytes = (uint32_t)((ranks - 1) * p.ld_a + p.H) * 2;
#pragma unroll
    for (int i = 0; i < LA; ++i) {
        const int row = (wave + 4 * i) * 8 + (lane >> 3);
        ak[i] = ((lane & 7) ^ mix(row)) * 8;
        ao[i] = (uint32_t)min(row, ranks - 1) * (uint32_t)(p.ld_a * 2) + ak[i] * 2;
    }
    const int steps = (p.H + kStep - 1) / kStep, each = (steps + p.splits - 1) / p.splits;
    const int lo = split * each, hi = min(steps, lo + each);
    // (always L loads: those of steps behind the last bring zeros that nothing reads)
    auto issue = [&](int s, int buf) INLINE {
        const int k = s * kStep, left = s < hi ? p.H - k : 0;
        uint8_t* at = lds + buf * BUF;
        if (left >= kStep) {
#pragma unroll
            for (int i = 0; i < LX; ++i) buffer_load_lds16<false>(p.x, x_bytes, xo[i] + k * 2, at + (wave * LX + i) * 8 * kRow);
#pragma unroll
            for (int i = 0; i < LA; ++i) buffer_load_lds16<false>(a, a_bytes, ao[i] + k * 2, at + kA + (wave + 4 * i) * 8 * kRow);
        } else {
#pragma unroll
            for (int i = 0; i < LX; ++i)
                buffer_load_lds16<false>(p.x, x_bytes, xk[i] < left ? xo[i] + k * 2 : kOutOfRange, at + (wave * LX + i) * 8 * kRow);
#pragma unroll
            for (int i = 0; i < LA; ++i)
                buffer_load_lds16<false>(a, a_bytes, ak[i] < left ? ao[i] + k * 2 : kOutOfRange, at + kA + (wave + 4 * i) * 8 * kRow);
        }
    };
    f32x4 acc[MS][NT] = {};
#pragma unroll
    for (int u = 0; u < P - 1; ++u) issue(lo + u, u);
    const uint32_t base = lds_address(lds) + c * kRow;
    int buf = 0, next = P - 1;
    for (int s = lo; s < hi; ++s) {
        wait_and_barrier<L*(P - 2)>();
        issue(s + P - 1, next);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const uint32_t at = base + buf * BUF + (((4 * h + q) ^ mix(c)) << 4);
            uint32_t from[MS + NT];
            u32x4 v[MS + NT];
#pragma unroll
            for (int m = 0; m < MS; ++m) from[m] = at + (wave * MS + m) * 16 * kRow;
#pragma unroll
            for (int j = 0; j < NT; ++j) from[MS + j] = at + kA + j * 16 * kRow;
            lds_read(v, from);
#pragma unroll
            for (int j = 0; j < NT; ++j)
#pragma unroll
                for (int m = 0; m < MS; ++m)
                    acc[m][j] = mma(__builtin_bit_cast(Vec<T>, v[MS + j]), __builtin_bit_cast(Vec<T>, v[m]), acc[m][j]);
        }
        buf = buf + 1 == P ? 0 : buf + 1;
        next = next + 1 == P ? 0 : next + 1;
    }
    // acc[m][j]: token m * 16 + c, ranks j * 16 + 4 q + 0..3
    float* part = p.part + (int64_t)split * p.T * p.r;
#pragma unroll
    for (int m = 0; m < MS; ++m)
#pragma unroll
        for (int j = 0; j < NT; ++j) {
            const int row = (wave * MS + m) * 16 + c, rank = r0 + j * 16 + 4 * q;
            if (row < rows && rank < p.r) *reinterpret_cast<f32x4*>(part + (int64_t)(row0 + row) * p.r + rank) = acc[m][j];
        }
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");  // no load into the LDS outlives the block
}

// out = base + scale b v for 64 rows, 16 a wave, 128 columns at a time, `chunks` times. The block's
// waves share the columns' rows of b in the LDS (two buffers) and have rows of their own,
// whose v waits in registers. Lane (c, q) holds columns 8 c .. 8 c + 7 of tokens 4 q .. 4 q + 3:
// row 8 c + u of b is column c of instruction u and lies in row 16 u + c of the buffer, its
// chunks mixed (where their number is a power of two) so that 16 rows use all banks.
//
// Ranks of 65 to 128 take 264 registers, of which 256 let two waves of a SIMD run: held to
// them (six are spilled) the call of 16384 tokens, H = 7168, N = 4096, rank 128, takes 228 us
// instead of 268.
template <typename T, int KS>
__global__ __launch_bounds__(256, KS == 4 ? 2 : 1) void adapt_up_wide_kernel(AdaptArgs p, int most, int nblocks, int chunks) {
    constexpr int BM = 64, kColumns = 128;
    extern __shared__ __align__(1024) char s_room[];
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6), c = lane & 15, q = lane >> 4;
    const int tile = blockIdx.x / nblocks;
    if (tile >= most) {
        copy_tokens<T>(p, blockIdx.x - most * nblocks);
        return;
    }
    int e, row0, rows;
    if (!find_tile<BM>(p.offsets, p.n, p.T, tile, lane, &e, &row0, &rows)) return;
    const int first = (blockIdx.x % nblocks) * chunks * kColumns;
    const int rc = p.r / 8, pitch = p.r * 2, size = kColumns * pitch;
    // 2^shift chunks of 16 bytes: a row of 16 (c) lies 128 bytes behind the row 8 / chunks before it
    const int shift = rc & (rc - 1) ? -1 : __builtin_ctz(rc);
    auto mix = [&](int row) INLINE { return shift < 0 ? 0 : shift >= 3 ? (row >> 1) & 7 : (row >> (4 - shift)) & ((1 << shift) - 1); };
    const T* b = (const T*)p.b + e * p.b_adapter;
    auto issue = [&](int n0, int buf) INLINE {
        const int last = min(kColumns, p.N - n0) - 1;  // (rows may share memory: their stride may lie below the rank)
        const uint32_t bytes = (uint32_t)(last * p.ld_b + p.r) * 2;
        for (int i = wave; i < 2 * rc; i += 4) {
            const int slot = i * 64 + lane, at = slot / rc, chunk = (slot - at * rc) ^ mix(at & 15);
            const int n = min(8 * (at & 15) + (at >> 4), last);
            buffer_load_lds16<false>(b + n0 * p.ld_b, bytes, (uint32_t)n * (uint32_t)(p.ld_b * 2) + chunk * 16,
                                     s_room + buf * size + i * 1024);
        }
    };
    const uint32_t room = lds_address(s_room);
    issue(first, 0);
    // v of the wave's rows (those behind the last are the last one's again)
    Vec<T> hi[KS], mid[KS], lo[KS];
    float back[4];
    int token[4];
    {
        const int row = wave * 16 + c, t = p.row_to_token[row0 + min(row, rows - 1)];
        const int named = (uint32_t)t < (uint32_t)p.T && row < rows ? t : -1;
        float f[KS][8];
        uint32_t top = 0;
#pragma unroll
        for (int s = 0; s < KS; ++s) {
            const int k = 32 * s + 8 * q;
#pragma unroll
            for (int i = 0; i < 8; ++i) f[s][i] = 0.0f;
            if (k < p.r) {
                const float* src = p.part + (int64_t)(row0 + min(row, rows - 1)) * p.r + k;
                for (int z = 0; z < p.splits; ++z, src += (int64_t)p.T * p.r) {
                    const f32x4 u = *reinterpret_cast<const f32x4*>(src), w = *reinterpret_cast<const f32x4*>(src + 4);
#pragma unroll
                    for (int i = 0; i < 4; ++i) f[s][i] += u[i], f[s][4 + i] += w[i];
                }
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) top = max(top, f2u(f[s][i]) & 0x7FFFFFFFu);
        }
        int up = 0;
        if constexpr (std::is_same<T, Fp16>::value) {
            top = max(top, (uint32_t)__shfl_xor((int)top, 16));
            top = max(top, (uint32_t)__shfl_xor((int)top, 32));
            up = power_for(top);
        }
        const float undo = ldexpf(p.scales ? p.scales[e] : 1.0f, -up);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            back[i] = __shfl(undo, 4 * q + i);
            token[i] = __shfl(named, 4 * q + i);
        }
#pragma unroll
        for (int s = 0; s < KS; ++s)
#pragma unroll
            for (int i = 0; i < 8; ++i) split_value(ldexpf(f[s][i], up), &hi[s].e[i], &mid[s].e[i], &lo[s].e[i]);
    }
    // Base of a pass, always four loads (none where a row has no 8 columns: then there is one
    // pass), so that the wait below can count them.
    typedef u32x4 Base[4];
    auto load_base = [&](int n0, Base& base) INLINE {
        if (p.N < 8) return;
        const int n = min(n0 + 8 * c, p.N - 8);
#pragma unroll
        for (int i = 0; i < 4; ++i) base[i] = __builtin_bit_cast(u32x4, load_vec((const T*)p.base + max(token[i], 0) * p.ld_base + n));
    };
    // Makes the compiler wait for these loads here, and not where the values are used.
    auto have = [](Base& base) INLINE {
#pragma unroll
        for (int i = 0; i < 4; ++i) asm volatile("" : "+v"(base[i]));
    };
    bool named = true;  // all rows of the wave
#pragma unroll
    for (int i = 0; i < 4; ++i) named &= token[i] >= 0;
    named = __ballot(!named) == 0;
    const int end = min(first + chunks * kColumns, p.N);
    auto pass = [&](int n0, int buf, Base& base, Base& next) INLINE {
        have(base);
        if (n0 + kColumns < end) {
            issue(n0 + kColumns, buf ^ 1);
            asm volatile("" ::: "memory");  // (the count below wants them in this order)
            load_base(n0 + kColumns, next);
        }
        f32x4 acc[8] = {};
        const uint32_t rows_of_b = room + buf * size + c * pitch;
#pragma unroll
        for (int s = 0; s < KS; ++s) {
            const int k = 4 * s + q;  // chunk
            uint32_t from[8];
            u32x4 v[8];
#pragma unroll
            for (int u = 0; u < 8; ++u) from[u] = rows_of_b + 16 * u * pitch + ((min(k, rc - 1) ^ mix(c)) << 4);
            lds_read(v, from);
#pragma unroll
            for (int u = 0; u < 8; ++u) {
                if (p.r % 32 && k >= rc) v[u] = u32x4{};
                const Vec<T> bv = __builtin_bit_cast(Vec<T>, v[u]);
                acc[u] = mma(hi[s], bv, mma(mid[s], bv, mma(lo[s], bv, acc[u])));
            }
        }
        const int n = n0 + 8 * c;
        auto result = [&](int i) INLINE {
            const Vec<T> old = __builtin_bit_cast(Vec<T>, base[i]);
            Vec<T> o;
#pragma unroll
            for (int u = 0; u < 8; ++u) o.e[u] = from_f32<T>(__fmaf_rn(acc[u][i], back[i], to_f32(old.e[u])));
            return o;
        };
        if (named && n0 + kColumns <= p.N) {
#pragma unroll
            for (int i = 0; i < 4; ++i) store_vec<false>((T*)p.out + token[i] * p.ld_out + n, result(i));
            return;
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (token[i] < 0) continue;
            T* dst = (T*)p.out + token[i] * p.ld_out + n;
            if (n + 8 <= p.N) {
                store_vec<false>(dst, result(i));
            } else {
                const T* src = (const T*)p.base + token[i] * p.ld_base + n;
#pragma unroll
                for (int u = 0; u < 8; ++u)
                    if (n + u < p.N) dst[u] = from_f32<T>(__fmaf_rn(acc[u][i], back[i], to_f32(src[u])));
            }
        }
        have(next);
    };
    Base one, two;
    load_base(first, one);
    wait_and_barrier<0>();
    for (int n0 = first; n0 < end; n0 += 2 * kColumns) {
        pass(n0, 0, one, two);
        if (n0 + kColumns >= end) break;
        // the next columns' rows of b have landed once no more than four operations are left: behind
        // them came as many loads of base, and whatever stores
        wait_and_barrier<4>();
        pass(n0 + kColumns, 1, two, one);
        if (n0 + 2 * kColumns < end) wait_and_barrier<4>();
    }
}

// ---------------------------------------------------------------------------
// launches
// ---------------------------------------------------------------------------
constexpr int kMaxRank = 256, kMaxSplits = 16;

// Tiles of bm rows there can be: whole ones, and a last one for each adapter with rows.
static int64_t most_tiles(int T, int n, int bm) { return T / bm + std::min(n, T); }

constexpr int kWideRows = 128;  // of a tile of the first product

struct AdaptPlan {
    bool wide;  // the kernels for many tokens an adapter
    int splits;
};
// The wide kernels from 2048 tokens and 32 an adapter on. H = 7168, N = 4096, in a graph, us, wide
// (narrow): rank 16, 1024 tokens of one adapter 17.8 (14.9), 2048 of 64 28.2 (30.2), 4096 of 64
// 35 (56), of 128 43 (51), of 256 78 (53); rank 64 31 (25), 60 (62), 70 (114), 100 (118), 144 (134).
// All n adapters have tokens there, which is what the rule takes for granted (the host does not
// know how many do): 16384 tokens of 4 adapters take 148 us of rank 64 out of 4 or 166 out of
// 512, but 275 out of 1024, by the narrow kernels.
static AdaptPlan plan_adapt(int T, int n, int H) {
    AdaptPlan q;
    q.wide = T >= 2048 && T >= 32 * (int64_t)std::min(n, T);
    const int64_t tiles = q.wide ? T / kWideRows + 1 : most_tiles(T, n, 16);
    const int64_t most = std::max((H + kStep * 4 - 1) / (kStep * 4), 1);
    q.splits = (int)std::max<int64_t>(1, std::min<int64_t>({512 / tiles, most, kMaxSplits}));
    return q;
}

// Bytes from the first token's row to the last one's end.
static int64_t x_extent(const AdaptArgs& p) { return ((p.T - 1) * p.ld_x + p.H) * 2; }

template <typename T>
static void launch_down(const AdaptArgs& p, bool wide, hipStream_t s) {
    const int most = (int)most_tiles(p.T, p.n, wide ? kWideRows : 16);
#define D(KERNEL, NT)                                                                                                  \
    hipLaunchKernelGGL(KERNEL, dim3(most * p.splits, (p.r + NT * 16 - 1) / (NT * 16)), dim3(256), 0, s, MORE)
    if (wide) {
#define MORE p, (uint32_t)x_extent(p)
        constexpr int MS = kWideRows / 64;
        if (p.r <= 16) D((adapt_down_wide_kernel<T, MS, 1, 3>), 1);
        else if (p.r <= 32) D((adapt_down_wide_kernel<T, MS, 2, 3>), 2);
        else D((adapt_down_wide_kernel<T, MS, 4, 3>), 4);
#undef MORE
    } else {
#define MORE p
        if (p.r <= 16) D((adapt_down_kernel<T, 1, 3>), 1);
        else if (p.r <= 32) D((adapt_down_kernel<T, 2, 3>), 2);
        else D((adapt_down_kernel<T, 4, 3>), 4);
#undef MORE
    }
#undef D
}

template <typename T>
static hipError_t launch_up(const AdaptArgs& p, bool wide, hipStream_t s) {
    const int rows = wide ? 64 : 16, step = wide ? 128 : 256;
    const int64_t most = most_tiles(p.T, p.n, rows), columns = (p.N + step - 1) / step;
    // columns a block walks over: about 1024 blocks, no more than 8 times (wide: what is left)
    const int chunks = (int)std::min<int64_t>(std::max<int64_t>(most * columns / 1024, 1), wide ? 16 : 8);
    const int nblocks = (int)((columns + chunks - 1) / chunks);
    const int copy = p.out == p.base ? 0 : (p.T + kCopyTokens - 1) / kCopyTokens;
    const int lds = wide ? 2 * 128 * p.r * 2 : 16 * ((p.r + 31) / 32 * 32 + 8) * 10;
#define U(KERNEL)                                                                                                      \
    hipLaunchKernelGGL((KERNEL), dim3((int)most * nblocks + copy), dim3(256), lds, s, p, (int)most, nblocks, chunks)
    if (wide) {
        if (p.r <= 32) U((adapt_up_wide_kernel<T, 1>));
        else if (p.r <= 64) U((adapt_up_wide_kernel<T, 2>));
        else if (p.r <= 128) U((adapt_up_wide_kernel<T, 4>));
        else U((adapt_up_wide_kernel<T, 8>));
    } else {
        if (p.r <= 32) U((adapt_up_kernel<T, 1>));
        else if (p.r <= 64) U((adapt_up_kernel<T, 2>));
        else U((adapt_up_kernel<T, 0>));
    }
#undef U
    return hipGetLastError();
}

template <typename T>
static hipError_t launch_adapt(AdaptArgs p, hipStream_t s) {
    const AdaptPlan q = plan_adapt(p.T, p.n, p.H);
    p.splits = q.splits;
    // (the wide kernels address the rows of x, 64 of a and 128 of b by 32-bit offsets; the
    // workspace fits either)
    const bool wide = q.wide && x_extent(p) <= (int64_t)kOutOfRange && p.ld_a <= (1 << 24) && p.ld_b <= (1 << 23);
    launch_down<T>(p, wide, s);
    return launch_up<T>(p, wide, s);
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
