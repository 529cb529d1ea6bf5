// Products of 8-bit integer matrices with a scale for each token (row of A)
// and each output channel (row of B), dense or expert by expert:
//   y[m,n] = sa[m] sb[n] sum_k a[m,k] b[n,k] (+ bias[n])
// The sums are exact 32-bit integers (|sum| <= 2^14 * 131056 < 2^31), the scales
// are applied in fp32 and the result is rounded once to the output's type.
#include <algorithm>
#include <atomic>
#include <type_traits>

#include "moe_args.h"
#include "moe_rows_dev.h"
#include "moe_route_dev.h"

// for the kernels' lambdas: what one captures would go through scratch memory if it
// were called
#define INLINE __attribute__((always_inline))

namespace moe {

typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

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

// Row of A of row r of the result, -1 if there is none.
__device__ __forceinline__ int row_of_route(const Int8Args& p, int route) {
    const int ar = p.row_to_route ? route / p.topk : route;
    return route >= 0 && ar < p.a_rows ? ar : -1;
}
__device__ __forceinline__ int row_of_a(const Int8Args& p, int r) {
    return row_of_route(p, p.row_to_route ? p.row_to_route[r] : r);
}

// The integer sum times both scales, plus the bias, by one product and one fma.
// |sum| < 2^31, so sum * sa is finite for |sa| <= 2^96. A larger one waits for sb:
// where sum * sb overflows too, both scales are above 2^96 and so is the result.
// Small scales lose nothing in either order: an integer times a subnormal is a whole
// number of the smallest subnormals, and an integer times a normal number a normal
// one (or 0). The selects cost nothing that shows (16384 x 4096 x 7168 407 us with
// them and without, x 2048 156 and 154, 4096 x 4096 x 1024 26 and 27); a branch around
// the whole epilogue made the 256 x 256 tile spill registers.
constexpr float kBigScale = 0x1p96f;
__device__ __forceinline__ float scaled(int sum, float sa, float sb, float bias) {
    const bool big = fabsf(sa) > kBigScale;
    return __fmaf_rn((float)sum * (big ? sb : sa), big ? sa : sb, bias);
}

// Rows of expert e. Offsets are clamped to [0, M], so a damaged list stays in range. (One
// that goes back lets experts share rows: there may then be more tiles than most_mtiles
// says, and the kernels leave out those behind.)
__device__ __forceinline__ void expert_rows(const Int8Args& p, int e, int* lo, int* hi) {
    *lo = *hi = 0;
    if (e < p.E) {
        *lo = min(max(p.offsets[e], 0), p.M);
        *hi = min(max(p.offsets[e + 1], *lo), p.M);
    }
}

// Tiles are counted expert by expert, ceil(rows / BM) each. The host knows only
// their largest number, so every wave counts them, 64 experts at a time.
template <int BM>
__device__ __forceinline__ int count_tiles(const Int8Args& p, int lane) {
    if (!p.offsets) return (p.M + BM - 1) / BM;
    int n = 0;
    for (int base = 0; base < p.E; base += 64) {
        int lo, hi;
        expert_rows(p, base + lane, &lo, &hi);
        n += (hi - lo + BM - 1) / BM;
    }
#pragma unroll
    for (int off = 32; off >= 1; off >>= 1) n += __shfl_xor(n, off);
    return __builtin_amdgcn_readfirstlane(n);
}

// The tile's expert and rows; false when there is no such tile.
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
        int lo, hi;
        expert_rows(p, base + lane, &lo, &hi);
        const int n = (hi - lo + BM - 1) / BM;
        const int incl = wave_incl_scan(n);
        const int excl = before + incl - n;
        const uint64_t hit = __ballot(tile >= excl && tile < excl + n);
        if (hit) {
            const int src = __ffsll((unsigned long long)hit) - 1;
            const int first = __builtin_amdgcn_readlane(lo, src) + (tile - __builtin_amdgcn_readlane(excl, src)) * BM;
            *e_out = base + src;
            *row0 = first;
            *rows = min(BM, __builtin_amdgcn_readlane(hi, src) - first);
            return true;
        }
        before += __builtin_amdgcn_readlane(incl, 63);
    }
    return false;
}

// ---------------------------------------------------------------------------
// wide tiles
// ---------------------------------------------------------------------------
template <typename T, int N>
struct __attribute__((packed, aligned(sizeof(T)))) Few {
    T e[N];
};

// Direct buffer -> LDS load of 16 bytes per lane from `base` + `off` (zeros from
// `bytes` on): lane l's bytes land at dst + 16 l (dst is uniform across the wave).
// ONCE: a non-temporal load, for lines that are read once: the rows of B of an
// expert with one M-tile. 64 x 8 routes over 256 experts of 4096 x 7168 801 -> 714 us then;
// mean rows of 16, 48, 64, 128 over 128 experts of 4096 x 4096 359 -> 325, 406 -> 377,
// 422 -> 404, 516 -> 504 (with all of B non-temporal 326, 391, 443, 540: experts with
// several tiles then lose their L2).
template <bool ONCE>
__device__ __forceinline__ void buffer_load_lds16(const void* base, uint32_t bytes, uint32_t off, void* dst) {
    __builtin_amdgcn_raw_ptr_buffer_load_lds(__builtin_amdgcn_make_buffer_rsrc((void*)base, 0, bytes, 0x00020000),
                                             (__attribute__((address_space(3))) void*)dst, 16, off, 0, 0, ONCE ? 2 : 0);
}

// s_waitcnt until no vector-memory and no LDS operation of this wave is
// outstanding, then the workgroup barrier.
template <int N>
__device__ __forceinline__ void wait_and_barrier() {
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(N) : "memory");
}

// The workgroup barrier once this wave's LDS operations are done (loads into the
// LDS may still be on their way).
__device__ __forceinline__ void wait_lds_and_barrier() {
    asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
}

// Stores N consecutive results of one row past the caches (nothing reads them here
// again; with normal stores they push rows of A and B out of the L2: 16384 x 4096 x
// 7168 went from 454 to 437 us, 98304 x 2048 x 2048 in 64 groups from 525 to 482).
template <typename T, int N>
__device__ __forceinline__ void store_past_caches(T* dst, const Few<T, N>& v) {
    typedef uint32_t words4 __attribute__((ext_vector_type(4), aligned(2)));
    typedef uint32_t words2 __attribute__((ext_vector_type(2), aligned(2)));
    constexpr int B = N * (int)sizeof(T);
    static_assert(B % 8 == 0, "whole stores");
    const char* src = reinterpret_cast<const char*>(&v);
    char* to = reinterpret_cast<char*>(dst);
#pragma unroll
    for (int i = 0; i + 16 <= B; i += 16)
        __builtin_nontemporal_store(*reinterpret_cast<const words4*>(src + i), reinterpret_cast<words4*>(to + i));
    if constexpr (B % 16)
        __builtin_nontemporal_store(*reinterpret_cast<const words2*>(src + B - 8), reinterpret_cast<words2*>(to + B - 8));
}

// Until this wave's loads (and stores) are done.
__device__ __forceinline__ void wait_loads() { asm volatile("s_waitcnt vmcnt(0)" ::: "memory"); }

// Byte offset that lies behind every buffer (their extents are checked on the
// host to be at most this): loads there return zeros.
constexpr uint32_t kOutOfRange = 0xFFFF0000u;

// One block per CU walks tiles of BM x BN (BM rows of one expert); NW = WM * WN
// waves of ME * 16 rows x NT * 16 columns each (row group g of the tile belongs to
// wave row g % WM, so that an expert's last, partly filled tile shortens every
// wave's work: the products run over ME = MT, MT / 2 or MT / 4 groups).
//  - A and B go through S LDS buffers of 128 bytes of depth, filled by direct
//    loads of whole 128-byte lines.
//  - The first S steps of the next tile are requested between a tile's last step
//    and its epilogue.
// 16384 x 4096 x 7168 in bf16 with 256 x 256 tiles: 405 to 431 us from card to card,
// 2.2 to 2.4 POP/s (the plain library product of that size: 465 us, 2.07). Built up to
// whole-line stores it took 340 us without its loads and 366 without its products;
// neither the matrix cores (54 % busy) nor the LDS (no bank conflicts) are full, the chip
// is at its power limit (1.7 - 2.0 GHz instead of 2.4), which is why fewer bytes through
// the LDS and the L2 per product, and the cheaper matrix instruction, are what made it
// faster: 32x32x32 products 516 us, 16x16x64 450, whole-line stores past the caches 427,
// every lambda inlined 408. Half lines (64 bytes of depth per step, four or five buffers)
// and requests of lines ahead into the L2 were slower (556, 490).
// 128 groups of 32768 x 4096 x 4096 (mean 256 rows, up to 1300): 750 to 775 us: weights
// of 2.1 GB, read by 1.5 M-tiles each (of the second readings about 60 % miss the L2),
// and the matrix work of partly filled tiles.
template <typename T, int BM, int BN, int WM, int WN, int S>
__global__ __launch_bounds__(WM * WN * 64) void int8_wide_kernel(Int8Args p, int most_mtiles, int ntiles) {
    constexpr int NW = WM * WN, MT = BM / WM / 16, NT = BN / WN / 16;
    constexpr int BK = 128, SL = BK / 64;               // bytes of depth per step, slices per step
    constexpr int LA = BM / 8 / NW, LB = BN / 8 / NW;   // 1 KB loads of A and of B per wave and step
    constexpr int BUF = (BM + BN) * BK;
    static_assert(BM % (8 * NW) == 0 && BN % (8 * NW) == 0 && MT >= 1 && BM <= NW * 64 && BN <= NW * 64, "tile shape");
    __shared__ __attribute__((aligned(1024))) uint8_t lds[S * BUF];
    __shared__ int s_first[kMaxE];   // grouped: tiles of the lower experts
    __shared__ int s_arow[2][BM];    // row of A of each row of the tile, -1 for none
    __shared__ __attribute__((aligned(16))) float s_sa[2][BM], s_sb[2][BN], s_bias[2][BN];
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wm = wave / WN, wn = wave % WN;

    int mtiles = (p.M + BM - 1) / BM;
    if (p.offsets) {  // every wave writes the same list
        mtiles = 0;
        for (int base = 0; base < p.E; base += 64) {
            int lo, hi;
            expert_rows(p, base + lane, &lo, &hi);
            const int n = (hi - lo + BM - 1) / BM;
            const int incl = wave_incl_scan(n);
            if (base + lane < p.E) s_first[base + lane] = min(mtiles + incl - n, most_mtiles);
            mtiles += __builtin_amdgcn_readlane(incl, 63);
        }
        // (the host has checked that most_mtiles * ntiles fits 32 bits)
        mtiles = min(mtiles, most_mtiles);
    }
    // Tile order: one contiguous range per XCD (blocks are dealt to the 8 XCDs in
    // turn), dealt to the XCD's blocks in turn. Inside it expert by expert, and there
    // groups of 8 M-tiles walk the N-blocks together: the tiles an XCD works on at a
    // time share rows of B (and of A) in its L2.
    constexpr int GM = 8;
    const int per = (mtiles * ntiles + 7) >> 3;
    const int last = min((int)(blockIdx.x & 7) * per + per, mtiles * ntiles);
    int id = (blockIdx.x & 7) * per + (blockIdx.x >> 3);
    const int stride = gridDim.x >> 3;

    struct Tile {
        int e, row0, rows, n0, cols;
        bool once;  // the only M-tile of its rows of B
    };
    auto locate = [&](int i) INLINE {
        Tile t;
        int lo = 0, hi = p.M;
        t.e = 0;
        if (p.offsets) {
            int cnt = 0;  // the last expert whose first tile is not behind i (an empty one has the next one's)
            for (int base = 0; base < p.E; base += 64)
                cnt += __popcll(__ballot(base + lane < p.E && s_first[base + lane] * ntiles <= i));
            t.e = cnt - 1;
            i -= s_first[t.e] * ntiles;
            // (the constant address space: scalar loads, which do not wait for this wave's stores)
            const auto* off = (const __attribute__((address_space(4))) int32_t*)p.offsets;
            const int e = __builtin_amdgcn_readfirstlane(t.e);
            lo = min(max(off[e], 0), p.M);
            hi = min(max(off[e + 1], lo), p.M);
        }
        const int tiles = (hi - lo + BM - 1) / BM;
        const int group = i / (GM * ntiles), in = i - group * GM * ntiles;
        const int gm = min(GM, tiles - group * GM);
        const int nb = in / gm, mt = group * GM + in - nb * gm;
        t.once = tiles == 1;
        t.n0 = nb * BN;
        t.cols = min(BN, p.N - t.n0);
        t.e = __builtin_amdgcn_readfirstlane(t.e);
        t.row0 = __builtin_amdgcn_readfirstlane(lo + mt * BM);
        t.rows = __builtin_amdgcn_readfirstlane(min(BM, hi - lo - mt * BM));
        return t;
    };
    // Thread r < BM looks up row r of the tile: first the route, later the row of A
    // and its scale (rows behind the tile's last repeat its first).
    auto route_of_row = [&](const Tile& t) INLINE {
        int r = 0;
        if (tid < BM) {
            r = t.row0 + (tid < t.rows ? tid : 0);
            if (p.row_to_route) r = p.row_to_route[r];
        }
        return r;
    };

    // Staging: one load brings 8 rows of 128 bytes; lane l lands at byte 16 l of its
    // 1 KB, i.e. in slot l % 8 of row l / 8, and fetches chunk (l % 8) ^ mix(row). The
    // LDS serves 16 lanes of an operand read (one chunk of 16 rows) at a time over 256
    // bytes of banks: every second row has the same banks, and mix() gives the eight
    // of them another slot each. An operand of A has rows 0 .. 15 of its group; one of
    // B, number j, rows CQ q + 4 j + c (q, c < 4) of its wave's 4 CQ: a lane then
    // ends up with CQ consecutive columns of the result.
    constexpr int CQ = 4 * NT;
    auto mix_a = [](int row) { return (row >> 1) & 7; };
    auto mix_b = [](int row) { return ((row / CQ) & 3) * 2 + ((row >> 1) & 1); };
    const int lr = lane >> 3;
    auto chunk_a = [&](int i) { return ((lane & 7) ^ mix_a((wave + NW * i) * 8 + lr)) << 4; };  // of the wave's load i
    auto chunk_b = [&](int i) { return ((lane & 7) ^ mix_b((wave + NW * i) * 8 + lr)) << 4; };
    const int KT = (p.Kd + BK - 1) / BK;
    const int8_t *abase, *bbase;
    uint32_t a_bytes, b_bytes, aoff[LA], boff[LB];
    bool b_once;
    auto address = [&](const Tile& t, int par) INLINE {
        abase = p.row_to_route ? p.a : p.a + (int64_t)t.row0 * p.lda;
        bbase = p.b + (int64_t)t.e * p.b_expert + (int64_t)t.n0 * p.ldb;
        b_once = t.once;
        a_bytes = (uint32_t)((int64_t)((p.row_to_route ? p.a_rows : t.rows) - 1) * p.lda + p.Kd);
        b_bytes = (uint32_t)((int64_t)(t.cols - 1) * p.ldb + p.Kd);
#pragma unroll
        for (int i = 0; i < LA; ++i) {
            const int ar = max(s_arow[par][(wave + NW * i) * 8 + lr], 0) - (p.row_to_route ? 0 : t.row0);
            aoff[i] = (uint32_t)ar * (uint32_t)p.lda + chunk_a(i);
        }
#pragma unroll
        for (int i = 0; i < LB; ++i)
            boff[i] = (uint32_t)min((wave + NW * i) * 8 + lr, t.cols - 1) * (uint32_t)p.ldb + chunk_b(i);
    };
    // loads of A that bring rows of the tile (or its first row's repeats up to the
    // groups that are multiplied)
    auto loads_of_a = [](int rows) { return rows > BM / 2 ? LA : rows > BM / 4 ? (LA + 1) / 2 : (LA + 3) / 4; };
    auto issue = [&](int kt, int buf, int la) INLINE {
        const int k = kt * BK;
        // the last step of a depth that is no multiple of 128: chunks behind the row's
        // end take an offset that the buffer's range check answers with zeros
        const int left = p.Kd - k;
#pragma unroll
        for (int i = 0; i < LA; ++i)
            if (i < la) buffer_load_lds16<false>(abase, a_bytes, left < BK && chunk_a(i) >= left ? kOutOfRange : aoff[i] + (uint32_t)k,
                                          lds + buf * BUF + (wave + NW * i) * 1024);
        auto load_b = [&](auto once) INLINE {
#pragma unroll
            for (int i = 0; i < LB; ++i)
                buffer_load_lds16<decltype(once)::value>(
                    bbase, b_bytes, left < BK && chunk_b(i) >= left ? kOutOfRange : boff[i] + (uint32_t)k,
                    lds + buf * BUF + BM * BK + (wave + NW * i) * 1024);
        };
        if (b_once) load_b(std::true_type{});
        else load_b(std::false_type{});
    };
    auto issue_first = [&](const Tile& t) INLINE {
        const int la = loads_of_a(t.rows);
#pragma unroll
        for (int u = 0; u < S; ++u)
            if (u < KT) issue(u, u, la);
    };

    if (id >= last) return;
    __syncthreads();
    Tile t = locate(id), nt = t;
    int par = 0;
    float my_sa = 0.0f, my_sb = 0.0f, my_bias = 0.0f;
    // Row r < BM of a tile and column c < BN belong to thread r, c: row of A, scales, bias.
    auto look_up = [&](const Tile& t, int route, int par) INLINE {
        if (tid < BM) {
            const int ar = row_of_route(p, route);
            s_arow[par][tid] = ar;
            my_sa = p.sa[max(ar, 0)];
        }
        if (tid < t.cols) {
            const size_t ne = (size_t)t.e * p.N + t.n0 + tid;
            my_sb = p.sb[ne];
            if (p.bias) my_bias = p.bias[ne];
        }
    };
    look_up(t, route_of_row(t), 0);
    __syncthreads();
    address(t, 0);
    issue_first(t);
    wait_loads();

    // Operands of 16 rows x 64 bytes: lane l holds row l % 16, chunk 4 s + l / 16 of slice s.
    const int r16 = lane & 15, quad = lane >> 4;
    const int b_row = wn * NT * 16 + CQ * (r16 >> 2) + (r16 & 3);  // of operand 0
    const int a_at = (wm * 16 + r16) * BK, b_at = BM * BK + b_row * BK;
    const int slot_a = (quad ^ mix_a(r16)) << 4, slot_b = (quad ^ mix_b(b_row)) << 4;
    T* const y = static_cast<T*>(p.y);
    bool more;

    auto tile = [&](auto me_tag, int next_route) INLINE {
        constexpr int ME = decltype(me_tag)::value;
        constexpr int LE = ME == MT ? LA : ME == (MT + 1) / 2 ? (LA + 1) / 2 : (LA + 3) / 4;  // loads_of_a
        // A slice's rows of A come in H parts of HM groups, which bounds the operands held
        constexpr int HM = ME > 4 ? 4 : ME, H = ME / HM, UNITS = SL * H;
        i32x4 fa[2][HM], fb[2][NT];
        auto fetch_b = [&](int buf, int sl) INLINE {
            const int o = buf * BUF + (slot_b ^ (sl << 6)) + b_at;
#pragma unroll
            for (int j = 0; j < NT; ++j) fb[sl & 1][j] = *reinterpret_cast<const i32x4*>(&lds[o + j * 4 * BK]);
        };
        auto fetch_a = [&](int buf, int sl, int h) INLINE {
            const int o = buf * BUF + (slot_a ^ (sl << 6)) + a_at;
#pragma unroll
            for (int i = 0; i < HM; ++i)
                fa[(sl * H + h) & 1][i] = *reinterpret_cast<const i32x4*>(&lds[o + (h * HM + i) * WM * 16 * BK]);
        };
        i32x4 acc[NT][ME];
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
            for (int i = 0; i < ME; ++i) acc[j][i] = i32x4{0, 0, 0, 0};

        // One barrier per step: at the end of step kt every wave has read its last
        // operands from the step's buffer and its loads of step kt + 1 have landed, so
        // behind the barrier the loads of step kt + S may overwrite the one while the
        // first operands come from the next; the last products cover both.
        static_assert(UNITS % 2 == 0 && SL % 2 == 0, "operand buffers alternate across steps");
        fetch_b(0, 0);
        fetch_a(0, 0, 0);
        int buf = 0;
        for (int kt = 0; kt < KT; ++kt) {
            const int next = buf + 1 == S ? 0 : buf + 1;
#pragma unroll
            for (int u = 0; u < UNITS; ++u) {
                const int sl = u / H, h = u % H;
                if (u + 1 == UNITS) {
                    if (kt + S <= KT) wait_and_barrier<(S - 2) * (LE + LB)>();
                    else wait_and_barrier<0>();
                    if (kt + 1 < KT) {
                        fetch_b(next, 0);
                        fetch_a(next, 0, 0);
                    }
                    if (kt + S < KT) issue(kt + S, buf, LE);
                } else if (h + 1 < H) {
                    fetch_a(buf, sl, h + 1);
                } else {
                    fetch_b(buf, sl + 1);
                    fetch_a(buf, sl + 1, 0);
                }
                // B in the place of the left operand: a lane then holds four consecutive
                // columns of one row of the result. (16x16x64: register-only loops over
                // normal data reach 4.0 POP/s of it and 3.4 of 32x32x32, at the power limit.)
#pragma unroll
                for (int j = 0; j < NT; ++j)
#pragma unroll
                    for (int i = 0; i < HM; ++i)
                        acc[j][h * HM + i] =
                            __builtin_amdgcn_mfma_i32_16x16x64_i8(fb[sl & 1][j], fa[u & 1][i], acc[j][h * HM + i], 0, 0, 0);
            }
            buf = next;
        }

        // every wave has read its last operands (the last step's barrier): the next
        // tile's loads may start
        if (more) {
            look_up(nt, next_route, par ^ 1);
            wait_lds_and_barrier();
            address(nt, par ^ 1);
            issue_first(nt);
        }

        // acc[j][i][c]: row (i*WM + wm)*16 + lane % 16, column CQ (lane / 16) + 4 j + c
        float sa[ME];
        bool ok[ME];
#pragma unroll
        for (int i = 0; i < ME; ++i) {
            const int m = (i * WM + wm) * 16 + r16;
            ok[i] = m < t.rows && s_arow[par][m] >= 0;
            sa[i] = s_sa[par][m];
        }
        const int col = wn * NT * 16 + CQ * quad, n = t.n0 + col, left = p.N - n;
        Few<T, CQ> o[ME];
#pragma unroll
        for (int j = 0; j < NT; ++j) {
            const f32x4 sb = *reinterpret_cast<const f32x4*>(&s_sb[par][col + 4 * j]);
            f32x4 bias = {0.0f, 0.0f, 0.0f, 0.0f};
            if (p.bias) bias = *reinterpret_cast<const f32x4*>(&s_bias[par][col + 4 * j]);
#pragma unroll
            for (int i = 0; i < ME; ++i)
#pragma unroll
                for (int c = 0; c < 4; ++c)
                    o[i].e[4 * j + c] = from_f32<T>(scaled(acc[j][i][c], sa[i], sb[c], bias[c]));
        }
        // the next tile's first steps have landed before any store is on its way, so
        // that no wait at the tile's start has to wait for stores
        wait_loads();
#pragma unroll
        for (int i = 0; i < ME; ++i) {
            if (!ok[i]) continue;
            T* dst = y + (int64_t)(t.row0 + (i * WM + wm) * 16 + r16) * p.ldy + n;
            if (left >= CQ) {
                store_past_caches<T, CQ>(dst, o[i]);
            } else {
#pragma unroll
                for (int c = 0; c < CQ - 1; ++c)
                    if (c < left) dst[c] = o[i].e[c];
            }
        }
    };

    for (;;) {
        if (tid < BM) s_sa[par][tid] = my_sa;
        if (tid < BN) {
            s_sb[par][tid] = my_sb;
            s_bias[par][tid] = my_bias;
        }
        wait_lds_and_barrier();  // every wave's share of the tile's first steps has landed
        id += stride;
        more = id < last;
        int next_route = 0;
        if (more) {
            nt = locate(id);
            next_route = route_of_row(nt);  // consumed after the main loop
        }
        if (MT < 2 || t.rows > BM / 2) tile(std::integral_constant<int, MT>{}, next_route);
        else if (MT < 4 || t.rows > BM / 4) tile(std::integral_constant<int, (MT + 1) / 2>{}, next_route);
        else tile(std::integral_constant<int, (MT + 3) / 4>{}, next_route);
        if (!more) break;
        t = nt;
        par ^= 1;
    }
}

// CUs of the current device (0 if the runtime cannot say), asked once per device.
static int cu_count() {
    static std::atomic<int> cache[64];
    int dev = 0;
    if (hipGetDevice(&dev) != hipSuccess || dev < 0 || dev >= 64) return 0;
    int c = cache[dev].load(std::memory_order_relaxed);
    if (c == 0) {
        if (hipDeviceGetAttribute(&c, hipDeviceAttributeMultiprocessorCount, dev) != hipSuccess) return 0;
        cache[dev].store(c, std::memory_order_relaxed);
    }
    return c;
}

// M-tiles there can be: whole ones, and a last one for each expert with rows.
static int64_t most_mtiles(const Int8Args& p, int bm) {
    return p.offsets ? p.M / bm + std::min(p.E, p.M) : (p.M + bm - 1) / bm;
}

template <typename T, int BM, int BN, int WM, int WN, int S>
static void launch_wide(const Int8Args& p, hipStream_t s) {
    const int64_t mtiles = most_mtiles(p, BM), ntiles = (p.N + BN - 1) / BN;
    const int64_t blocks = std::min<int64_t>(std::max(cu_count(), 8), mtiles * ntiles);
    hipLaunchKernelGGL((int8_wide_kernel<T, BM, BN, WM, WN, S>), dim3((unsigned)((blocks + 7) / 8 * 8)),
                       dim3(WM * WN * 64), 0, s, p, (int)mtiles, (int)ntiles);
}

// ---------------------------------------------------------------------------
// narrow tiles
// ---------------------------------------------------------------------------
// MS * 16 rows x NS * 16 columns per block, for few rows (where B's bytes are
// what counts) and small products (where latency is). The depth is dealt to the
// block's NW waves, 128 bytes at a time, each wave keeps P such pieces of both
// operands on their way straight into its registers, and the waves' integer sums
// are joined through the LDS, which is exact in any order.
template <typename T, int MS, int NS, int NW, int P>
__global__ __launch_bounds__(NW * 64) void int8_narrow_kernel(Int8Args p, int most_mtiles, int ntiles) {
    constexpr int BM = MS * 16, BN = NS * 16;
    __shared__ __attribute__((aligned(16))) i32x4 part[NW][MS * NS][64];
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int r16 = lane & 15, quad = lane >> 4;
    // one contiguous range of tiles per XCD, M-tiles of a column block side by side
    const int mtiles = min(count_tiles<BM>(p, lane), most_mtiles);
    const int per = (mtiles * ntiles + 7) >> 3, j8 = blockIdx.x >> 3;
    const int id = (blockIdx.x & 7) * per + j8;
    if (j8 >= per || id >= mtiles * ntiles) return;
    int e, row0, rows;
    if (!find_tile<BM>(p, id % mtiles, lane, &e, &row0, &rows)) return;
    const int n0 = id / mtiles * BN;

    const int8_t *ap[MS], *bp[NS];
#pragma unroll
    for (int i = 0; i < MS; ++i) {
        const int ar = max(row_of_a(p, row0 + min(i * 16 + r16, rows - 1)), 0);
        ap[i] = p.a + (int64_t)ar * p.lda + quad * 16;
    }
#pragma unroll
    for (int j = 0; j < NS; ++j)
        bp[j] = p.b + (int64_t)e * p.b_expert + (int64_t)min(n0 + j * 16 + r16, p.N - 1) * p.ldb + quad * 16;

    // the result's fragment that this wave joins in the end: its scales are requested
    // first, so that they are there by then
    static_assert(MS * NS <= NW, "one fragment per wave");
    const int f = wave, m = (f % MS) * 16 + r16, n = n0 + (f / MS) * 16 + 4 * quad, left = p.N - n;
    bool mine = f < MS * NS && m < rows && left > 0;
    float sa = 0.0f;
    Few<float, 4> sb = {}, bias = {};
    if (mine) {
        const int ar = row_of_a(p, row0 + m);
        mine = ar >= 0;
        const size_t ne = (size_t)e * p.N + n;
        if (mine) sa = p.sa[ar];
        if (left >= 4) {
            sb = *reinterpret_cast<const Few<float, 4>*>(p.sb + ne);
            if (p.bias) bias = *reinterpret_cast<const Few<float, 4>*>(p.bias + ne);
        } else {
#pragma unroll
            for (int c = 0; c < 3; ++c)
                if (c < left) {
                    sb.e[c] = p.sb[ne + c];
                    if (p.bias) bias.e[c] = p.bias[ne + c];
                }
        }
    }

    i32x4 fa[P][2][MS], fb[P][2][NS];
    i32x4 acc[NS][MS];
#pragma unroll
    for (int j = 0; j < NS; ++j)
#pragma unroll
        for (int i = 0; i < MS; ++i) acc[j][i] = i32x4{0, 0, 0, 0};
    // B stays cacheable: column blocks with several M-tiles share it, and weights that the
    // last-level cache still holds come from there. Non-temporal loads took 11.2 us instead
    // of 9.6 for 16 x 4096 x 7168, 18.9 instead of 16.3 with 64 rows, and from memory 12.0
    // instead of 11.8 and 19.7 instead of 19.0.
    auto load = [&](int st, int k) INLINE {
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            const bool in = k + s * 64 + quad * 16 < p.Kd;
#pragma unroll
            for (int j = 0; j < NS; ++j)
                fb[st][s][j] = in ? *reinterpret_cast<const i32x4*>(bp[j] + k + s * 64) : i32x4{0, 0, 0, 0};
#pragma unroll
            for (int i = 0; i < MS; ++i)
                fa[st][s][i] = in ? *reinterpret_cast<const i32x4*>(ap[i] + k + s * 64) : i32x4{0, 0, 0, 0};
        }
    };
    auto multiply = [&](int st) INLINE {
#pragma unroll
        for (int s = 0; s < 2; ++s)
#pragma unroll
            for (int j = 0; j < NS; ++j)
#pragma unroll
                for (int i = 0; i < MS; ++i)
                    acc[j][i] = __builtin_amdgcn_mfma_i32_16x16x64_i8(fb[st][s][j], fa[st][s][i], acc[j][i], 0, 0, 0);
    };
    constexpr int STRIDE = NW * 128;
    int k = wave * 128;
#pragma unroll
    for (int u = 0; u < P; ++u) load(u, k + u * STRIDE);
    for (; k < p.Kd; k += P * STRIDE) {
#pragma unroll
        for (int u = 0; u < P; ++u) {
            multiply(u);
            load(u, k + (P + u) * STRIDE);
        }
    }
#pragma unroll
    for (int j = 0; j < NS; ++j)
#pragma unroll
        for (int i = 0; i < MS; ++i) part[wave][j * MS + i][lane] = acc[j][i];
    __syncthreads();
    // part[w][j * MS + i][lane][c]: row i * 16 + lane % 16, column j * 16 + 4 (lane / 16) + c
    if (!mine) return;
    i32x4 sum = part[0][f][lane];
#pragma unroll
    for (int w = 1; w < NW; ++w) sum += part[w][f][lane];
    T* dst = static_cast<T*>(p.y) + (int64_t)(row0 + m) * p.ldy + n;
    Few<T, 4> o;
#pragma unroll
    for (int c = 0; c < 4; ++c) o.e[c] = from_f32<T>(scaled(sum[c], sa, sb.e[c], bias.e[c]));
    if (left >= 4) {
        *reinterpret_cast<Few<T, 4>*>(dst) = o;
    } else {
#pragma unroll
        for (int c = 0; c < 3; ++c)
            if (c < left) dst[c] = o.e[c];
    }
}

template <typename T, int MS, int NS, int NW, int P>
static void launch_narrow(const Int8Args& p, hipStream_t s) {
    const int64_t mtiles = most_mtiles(p, MS * 16), ntiles = (p.N + NS * 16 - 1) / (NS * 16);
    hipLaunchKernelGGL((int8_narrow_kernel<T, MS, NS, NW, P>), dim3((unsigned)((mtiles * ntiles + 7) / 8 * 8)),
                       dim3(NW * 64), 0, s, p, (int)mtiles, (int)ntiles);
}

// The tile shape: the largest that still gives about one block per CU. A larger
// tile moves fewer bytes per product, but a product that does not fill the CUs is
// bound by the time of one block. Columns N = 4096, depth 7168, bf16, in us from
// call to call (a call takes the host 9 to 10 us):
//   rows      256x256  128x256  128x128  64x128  64x32  32x32  16x32  16x16
//   16384         409      459
//    2048          82       58       67
//    1024          81       51       36      48
//     512          81       51       33      27     86
//     256          91       51       32      25     44
//     128          79       58       39      25     24     30
//      64                             29      30     23     17     22
//      32                             25             19     16     13     16
//      16                             23             17     14     13     10
// (weights of 29 MB that are still in the last-level cache; from memory the narrow
// tiles take 2 to 3 us more, in the same order.) For experts the host knows an upper
// bound of the mean rows only: the rows of dropped routes are among M. Without any, 64
// tokens with 8 of 256 experts, depth 7168: 685 us with 128x256, 1044 or more with 16 rows;
// 256-row tiles pay from about 192 mean rows on (128: 576 against 521 us, 1536: 482
// against 528). With 32 of 256 experts here and 4096 x 4096 weights the rule takes 256x256
// for 4096 tokens, 164 us (128x256: 142), and 2048 tokens, 146 (128x128: 115), as for eight
// times the rows. Narrow tiles are no higher than the rows: 16 x 7168 x 7168 takes 13 us
// with 16x32 and 17 with 64x32, 32 rows 17 with 32x32 and 19 with 64x32. A single
// token's rows are broadcast, which favours 16x16 (1 x 14336 x 4096: 13.6 us, 64x128
// 16.8; with 16 rows both 17.9) until the wide tiles fill the CUs (1 x 28672 x 8192: 43.4
// and 41.8).
template <typename T>
static hipError_t launch_int8_matmul(const Int8Args& p, hipStream_t s) {
    const int64_t groups = p.offsets ? std::min(p.E, p.M) : 1;
    const int64_t mean = (p.M + groups - 1) / groups;
    auto blocks = [&](int bm, int bn) { return groups * ((mean + bm - 1) / bm) * ((p.N + bn - 1) / bn); };
    const int64_t cus = std::max(cu_count(), 8), full = cus * 7 / 8;
    const bool one = !p.offsets && p.M <= 4;
    if (mean >= 192 && blocks(256, 256) >= full) launch_wide<T, 256, 256, 2, 4, 2>(p, s);
    else if (blocks(128, 256) >= full) launch_wide<T, 128, 256, 2, 4, 3>(p, s);
    else if (blocks(128, 128) >= full) launch_wide<T, 128, 128, 2, 4, 4>(p, s);
    else if (blocks(64, 128) >= (one ? full : cus * 3 / 8)) launch_wide<T, 64, 128, 1, 8, 5>(p, s);
    else if (mean > 32 && blocks(64, 32) >= full) launch_narrow<T, 4, 2, 8, 2>(p, s);
    else if (mean > 16 && blocks(32, 32) >= full) launch_narrow<T, 2, 2, 8, 3>(p, s);
    else if (!one && blocks(16, 32) >= full) launch_narrow<T, 1, 2, 8, 3>(p, s);
    else launch_narrow<T, 1, 1, 8, 4>(p, s);
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
    if (p.M > kMaxRows) return reject(MOE_ERR_UNSUPPORTED, "M=%d rows above %lld", p.M, (long long)kMaxRows);
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
    const int64_t far = (int64_t)1 << 23;  // 256 rows of a tile are addressed by 32-bit offsets
    if ((p.a_rows > 1 && p.lda > far) || (p.N > 1 && p.ldb > far) || (p.M > 1 && p.ldy > ((int64_t)1 << 31)))
        return reject(MOE_ERR_UNSUPPORTED, "a row stride above 2^23 bytes (a, b) or 2^31 elements (y)");
    if (grouped && p.E > 1 && p.b_expert > ((int64_t)1 << 48))
        return reject(MOE_ERR_UNSUPPORTED, "experts more than 2^48 bytes apart");
    if (p.row_to_route && (int64_t)(p.a_rows - 1) * p.lda + p.Kd > (int64_t)kOutOfRange)
        return reject(MOE_ERR_UNSUPPORTED, "gathered rows of 4 GiB or more");
    const int64_t most = ((int64_t)(p.M + 15) / 16 + (grouped ? p.E : 0)) * ((p.N + 15) / 16);
    if (most >= ((int64_t)1 << 31)) return reject(MOE_ERR_UNSUPPORTED, "M=%d, N=%d: too many tiles", p.M, p.N);
    if ((p.a_rows > 1 && p.lda % 16) || (p.N > 1 && p.ldb % 16) || (grouped && p.E > 1 && p.b_expert % 16))
        return reject(MOE_ERR_UNSUPPORTED, "the strides of a and b must be multiples of 16");
    const size_t es = dtype_bytes(out_dtype);
    if (!is_aligned(p.a, 16) || !is_aligned(p.b, 16)) return reject(MOE_ERR_INVALID, "a and b must be 16-byte aligned");
    if (!is_aligned(p.y, es) || !is_aligned(p.sa, 4) || !is_aligned(p.sb, 4) || !is_aligned(p.bias, 4) ||
        !is_aligned(p.offsets, 4) || !is_aligned(p.row_to_route, 4))
        return reject(MOE_ERR_INVALID, "misaligned pointer");
    const Bytes y = matrix(p.y, p.M, p.ldy, p.N, (int)es);
    const int64_t E = grouped ? p.E : 1;
    const Bytes in[] = {matrix(p.a, p.a_rows, p.lda, p.Kd, 1), flat(p.sa, (int64_t)p.a_rows * 4),
                        // (all of the experts as one piece)
                        flat(p.b, (E - 1) * p.b_expert + (int64_t)(p.N - 1) * p.ldb + p.Kd), flat(p.sb, E * p.N * 4),
                        flat(p.bias, E * p.N * 4), flat(p.offsets, (E + 1) * 4), flat(p.row_to_route, (int64_t)p.M * 4)};
    for (const Bytes& b : in)
        if (overlap(b, y)) return reject(MOE_ERR_INVALID, "the output overlaps an input");
    hipError_t e;
    if (out_dtype == MOE_DT_BF16) e = launch_int8_matmul<Bf16>(p, stream);
    else if (out_dtype == MOE_DT_FP16) e = launch_int8_matmul<Fp16>(p, stream);
    else e = launch_int8_matmul<float>(p, stream);
    return launched(e, "8-bit integer product");
}

}  // namespace moe

using namespace moe;

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
