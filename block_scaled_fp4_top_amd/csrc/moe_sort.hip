// Routes sorted by expert, from the caller's expert ids: the stable order that
// groups routes r = t*K + k by expert, with the routes of experts outside
// [0, E) left out (experts of other GPUs, dropped tokens).
//
// A counting sort. A block of 16 waves owns `chunk` consecutive routes, each
// wave a contiguous 16th of them. Inside a wave the 64 routes of one step find
// their peers (routes of the same expert) by one ballot per bit of the key, so
// the rank among the peers is a population count and no atomic decides a
// position. Positions follow as base of the expert (routes of lower experts,
// and of this expert in earlier blocks) + routes of the expert in earlier waves
// + in earlier steps of the wave + the rank. Left-out routes form a last group
// with key E, which gives every entry of both maps a writer.
#include <algorithm>

#include "moe_args.h"
#include "moe_route_dev.h"

namespace moe {

constexpr int kSortWaves = 16;
constexpr int kSortMinChunk = kSortWaves * 64;
constexpr int kSortMaxChunk = 32768;         // per-wave counters are 16-bit
constexpr int kSortBlocks = 256;              // at most (kMaxRows / kSortMaxChunk)
static_assert(kMaxRows <= (int64_t)kSortBlocks * kSortMaxChunk, "every size has a chunk");
// Routes sorted by a single block, in one launch. 4096 routes to 256 experts: 7.9 us in
// a graph and 8.3 from call to call; two launches take 7.6 and 10.5 (E = 32: 5.9 and
// 8.4 against 6.2 and 10.6), with 6144 routes one block already takes 11. What bounds
// either is latency: the ballots of each step, and the phases between barriers.
constexpr long long kSortOneBlock = 4096;

__host__ __device__ inline int sort_row_words(int E) { return (E + 2) / 2; }  // E + 1 16-bit counts

template <typename ID>
__device__ __forceinline__ int sort_key(const ID* __restrict__ ids, long long r, int R, int E) {
    if (r >= R) return -1;
    const ID v = ids[r];
    return v >= 0 && v < (ID)E ? (int)v : E;
}

// Lanes with the same key as this one (lanes without a route, key -1, aside): for
// each bit of the key, the lanes whose bit is this lane's.
__device__ __forceinline__ uint64_t peers_of(int key, int nbits) {
    const uint64_t valid = __ballot(key >= 0);
    uint32_t lo = (uint32_t)valid, hi = (uint32_t)(valid >> 32);
    for (int b = 0; b < nbits; ++b) {
        const int mine = __builtin_amdgcn_sbfe(key, b, 1);  // 0 or -1
        const uint64_t set = __ballot(mine);
        lo &= ~((uint32_t)set ^ (uint32_t)mine);
        hi &= ~((uint32_t)(set >> 32) ^ (uint32_t)mine);
    }
    return ((uint64_t)hi << 32) | lo;
}

// Routes of each expert in one chunk, as 16-bit counts, two per word.
template <typename ID>
__global__ __launch_bounds__(1024) void sort_count_kernel(const ID* __restrict__ ids, int R, int E,
                                                          int chunk, uint32_t* __restrict__ counts) {
    __shared__ int32_t h[kMaxE + 2];
    const int words = sort_row_words(E);
    for (int e = threadIdx.x; e < 2 * words; e += 1024) h[e] = 0;
    __syncthreads();
    const long long base = (long long)blockIdx.x * chunk;
    for (int i = threadIdx.x; i < chunk; i += 1024) {
        const int key = sort_key(ids, base + i, R, E);
        if (key >= 0) atomicAdd(&h[key], 1);
    }
    __syncthreads();
    for (int w = threadIdx.x; w < words; w += 1024)
        counts[(size_t)blockIdx.x * words + w] = (uint32_t)h[2 * w] | ((uint32_t)h[2 * w + 1] << 16);
}

// The positions of one chunk's routes. counts: the chunks' counts (null when
// one block sorts everything). Every block sums the counts of all chunks and of
// those before its own by itself: that reads nblk * (E + 1) 16-bit values from
// the L2 and saves a launch for a scan.
// KEEP: a wave has at most KEEP steps, whose keys and peers it keeps between the
// two passes; 0: any number, found twice.
constexpr int kKeep = 4;
template <typename ID, int KEEP>
__global__ __launch_bounds__(1024) void sort_place_kernel(const ID* __restrict__ ids, int R, int E,
                                                          int chunk, const uint32_t* __restrict__ counts,
                                                          int32_t* __restrict__ row_to_route,
                                                          int32_t* __restrict__ route_to_row,
                                                          int32_t* __restrict__ offsets) {
    __shared__ uint16_t wcount[kSortWaves][kMaxE + 2];
    __shared__ int32_t total[kMaxE + 2], before[kMaxE + 2];
    __shared__ int32_t base[kMaxE + 1];
    __shared__ int32_t wsum[kSortWaves];
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int words = sort_row_words(E), nblk = gridDim.x, blk = blockIdx.x;
    int nbits = 0;
    while ((1 << nbits) <= E) ++nbits;
    for (int i = tid; i < kSortWaves * 2 * words; i += 1024) wcount[i / (2 * words)][i % (2 * words)] = 0;
    for (int e = tid; e < 2 * words; e += 1024) total[e] = before[e] = 0;
    __syncthreads();

    // routes per expert of this wave
    const int per = chunk / kSortWaves;
    const long long r0 = (long long)blk * chunk + (long long)wave * per;
    const uint64_t below = (1ull << lane) - 1ull;
    auto count = [&](int key, uint64_t peers) {
        if (key >= 0 && (peers & below) == 0) wcount[wave][key] = (uint16_t)(wcount[wave][key] + __popcll(peers));
        asm volatile("" ::: "memory");  // the next step reads what other lanes wrote (LDS keeps a wave's order)
    };
    int keys[KEEP ? KEEP : 1];
    uint64_t peers_at[KEEP ? KEEP : 1];
    if (KEEP) {
#pragma unroll
        for (int u = 0; u < KEEP; ++u) keys[u] = 64 * u < per ? sort_key(ids, r0 + 64 * u + lane, R, E) : -1;
#pragma unroll
        for (int u = 0; u < KEEP; ++u) {
            peers_at[u] = 0;
            if (64 * u >= per) continue;
            peers_at[u] = peers_of(keys[u], nbits);
            count(keys[u], peers_at[u]);
        }
    } else {
        for (int s = 0; s < per; s += 64) {
            const int key = sort_key(ids, r0 + s + lane, R, E);
            count(key, peers_of(key, nbits));
        }
    }
    // routes per expert of all chunks and of the chunks before this one
    if (counts) {
        // the chunks are dealt to groups of `words` threads, one word (two experts) per thread
        const int groups = 1024 / words, w = tid % words, q = tid / words;
        if (q < groups) {
            int a0 = 0, a1 = 0, b0 = 0, b1 = 0;
            for (int b = q; b < nblk; b += groups) {
                const uint32_t v = counts[(size_t)b * words + w];
                const int lo = (int)(v & 0xFFFF), hi = (int)(v >> 16);
                a0 += lo;
                a1 += hi;
                b0 += b < blk ? lo : 0;
                b1 += b < blk ? hi : 0;
            }
            atomicAdd(&total[2 * w], a0);
            atomicAdd(&total[2 * w + 1], a1);
            atomicAdd(&before[2 * w], b0);
            atomicAdd(&before[2 * w + 1], b1);
        }
    }
    __syncthreads();
    // exclusive prefix over the waves; the chunk's counts are the totals when it is the only one
    for (int e = tid; e <= E; e += 1024) {
        int run = 0, v[kSortWaves];
#pragma unroll
        for (int w = 0; w < kSortWaves; ++w) v[w] = wcount[w][e];
#pragma unroll
        for (int w = 0; w < kSortWaves; ++w) {
            wcount[w][e] = (uint16_t)run;
            run += v[w];
        }
        if (!counts) total[e] = run;
    }
    __syncthreads();
    // exclusive prefix over the experts (E <= 1024, one thread each)
    const int mine = tid < E ? total[tid] : 0;
    const int incl = wave_incl_scan(mine);
    if (lane == 63) wsum[wave] = incl;
    __syncthreads();
    int lower = 0, kept = 0;
    for (int w = 0; w < kSortWaves; ++w) {
        if (w < wave) lower += wsum[w];
        kept += wsum[w];
    }
    const int off = lower + incl - mine;
    if (tid < E) {
        base[tid] = off + before[tid];
        if (blk == 0) offsets[tid] = off;
    }
    if (tid == 0) {
        base[E] = kept + before[E];
        if (blk == 0) offsets[E] = kept;
    }
    __syncthreads();
    auto place = [&](int s, int key, uint64_t peers) {
        const long long r = r0 + s + lane;
        const int rank = __popcll(peers & below);
        int prior = 0;
        if (key >= 0) prior = wcount[wave][key];
        asm volatile("" ::: "memory");
        if (key >= 0 && rank == 0) wcount[wave][key] = (uint16_t)(prior + __popcll(peers));
        asm volatile("" ::: "memory");
        if (key >= 0) {
            const int row = base[key] + prior + rank;
            row_to_route[row] = key < E ? (int)r : -1;
            route_to_row[r] = key < E ? row : -1;
        }
    };
    if (KEEP) {
#pragma unroll
        for (int u = 0; u < KEEP; ++u)
            if (64 * u < per) place(64 * u, keys[u], peers_at[u]);
    } else {
        for (int s = 0; s < per; s += 64) {
            const int key = sort_key(ids, r0 + s + lane, R, E);
            place(s, key, peers_of(key, nbits));
        }
    }
}

// Routes per block: the smallest power of two from kSortMinChunk that keeps the
// blocks at kSortBlocks or fewer (each reads every block's counts).
static int sort_chunk(long long R) {
    int c = kSortMinChunk;
    while (c < kSortMaxChunk && (R + c - 1) / c > kSortBlocks) c *= 2;
    return c;
}

template <typename ID>
static hipError_t launch_sort(const ID* ids, int R, int E, uint32_t* counts, int32_t* row_to_route,
                              int32_t* route_to_row, int32_t* offsets, hipStream_t s) {
    const bool one = R <= kSortOneBlock;
    const int chunk = one ? (R + kSortMinChunk - 1) / kSortMinChunk * kSortMinChunk : sort_chunk(R);
    const int nblk = one ? 1 : (R + chunk - 1) / chunk;
    if (!one) hipLaunchKernelGGL(sort_count_kernel<ID>, dim3(nblk), dim3(1024), 0, s, ids, R, E, chunk, counts);
    const uint32_t* c = one ? nullptr : counts;
    if (chunk <= kKeep * kSortMinChunk)
        hipLaunchKernelGGL((sort_place_kernel<ID, kKeep>), dim3(nblk), dim3(1024), 0, s, ids, R, E, chunk, c,
                           row_to_route, route_to_row, offsets);
    else
        hipLaunchKernelGGL((sort_place_kernel<ID, 0>), dim3(nblk), dim3(1024), 0, s, ids, R, E, chunk, c,
                           row_to_route, route_to_row, offsets);
    return hipGetLastError();
}

static int check_sort_sizes(int32_t T, int32_t K, int32_t E) {
    if (E < 1 || E > kMaxE) return reject(MOE_ERR_INVALID, "E=%d outside [1, %d]", E, kMaxE);
    if (T < 0) return reject(MOE_ERR_INVALID, "T=%d is negative", T);
    if (K < 1 || K > kMaxK) return reject(MOE_ERR_INVALID, "K=%d outside [1, %d]", K, kMaxK);
    if ((long long)T * K > (long long)kMaxRows)
        return reject(MOE_ERR_UNSUPPORTED, "T*K=%lld routes above %lld", (long long)T * K, (long long)kMaxRows);
    return MOE_OK;
}

}  // namespace moe

using namespace moe;

extern "C" size_t moe_sort_workspace_bytes(int32_t T, int32_t K, int32_t E) {
    if (check_sort_sizes(T, K, E) != MOE_OK) return 0;
    const long long R = (long long)T * K;
    // never less for fewer tokens: a workspace for T serves every smaller batch
    const long long blocks = std::min((R + kSortMinChunk - 1) / kSortMinChunk, (long long)kSortBlocks);
    return align256((size_t)std::max(blocks, 1LL) * sort_row_words(E) * 4);
}

extern "C" int moe_sort_routes(const void* ids, int32_t ids_are_wide, int32_t T, int32_t K, int32_t E,
                               void* workspace, size_t workspace_bytes, int32_t* row_to_route,
                               int32_t* route_to_row, int32_t* offsets, hipStream_t stream) {
    const int rc = check_sort_sizes(T, K, E);
    if (rc) return rc;
    if (ids_are_wide != 0 && ids_are_wide != 1) return reject(MOE_ERR_INVALID, "ids_are_wide must be 0 or 1");
    const size_t R = (size_t)T * K;
    if (!offsets || !workspace || (R && (!ids || !row_to_route || !route_to_row)))
        return reject(MOE_ERR_INVALID, "NULL pointer argument");
    if (!is_aligned(ids, ids_are_wide ? 8 : 4) || !is_aligned(row_to_route, 4) || !is_aligned(route_to_row, 4) ||
        !is_aligned(offsets, 4) || !is_aligned(workspace, 16))
        return reject(MOE_ERR_INVALID, "misaligned pointer");
    const size_t need = moe_sort_workspace_bytes(T, K, E);
    if (workspace_bytes < need)
        return reject(MOE_ERR_WORKSPACE, "workspace %zu bytes < %zu needed", workspace_bytes, need);
    const int64_t r4 = (int64_t)R * 4;
    const Bytes b[] = {flat(ids, r4 * (ids_are_wide ? 2 : 1)), flat(workspace, (int64_t)need), flat(row_to_route, r4),
                       flat(route_to_row, r4), flat(offsets, ((int64_t)E + 1) * 4)};
    for (int i = 0; i < 5; ++i)
        for (int j = i + 1; j < 5; ++j)
            if (overlap(b[i], b[j])) return reject(MOE_ERR_INVALID, "buffers overlap");
    uint32_t* counts = static_cast<uint32_t*>(workspace);
    return launched(ids_are_wide ? launch_sort(static_cast<const int64_t*>(ids), (int)R, E, counts, row_to_route,
                                               route_to_row, offsets, stream)
                                 : launch_sort(static_cast<const int32_t*>(ids), (int)R, E, counts, row_to_route,
                                               route_to_row, offsets, stream),
                    "sort routes");
}
