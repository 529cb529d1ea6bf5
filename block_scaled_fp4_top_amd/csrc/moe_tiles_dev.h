// The M-tiles of products over sorted rows: ceil(rows / BM) for each expert, counted
// expert by expert on the device, as the host does not know the offsets.
#pragma once

#include "moe_route_dev.h"

namespace moe {

// Rows of expert e of E. Offsets are clamped to [0, M], so a damaged list stays in range.
// (One that goes back lets experts share rows: there may then be more tiles than the host
// has counted on, and the kernels leave out those behind.)
__device__ __forceinline__ void expert_rows(const int32_t* offsets, int E, int M, int e, int* lo, int* hi) {
    *lo = *hi = 0;
    if (e < E) {
        *lo = min(max(offsets[e], 0), M);
        *hi = min(max(offsets[e + 1], *lo), M);
    }
}

// The tile's expert and rows, found by a whole wave, 64 experts at a time; false when there
// is no such tile.
template <int BM>
__device__ __forceinline__ bool find_tile(const int32_t* offsets, int E, int M, int tile, int lane, int* e_out, int* row0,
                                          int* rows) {
    int before = 0;
    for (int base = 0; base < E; base += 64) {
        int lo, hi;
        expert_rows(offsets, E, M, base + lane, &lo, &hi);
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

}  // namespace moe
