// window.cuh -- the active range of a windowed sequence over a paged cache.
//
// schedule.cuh starts a windowed sequence's tiles at the first position any query sees.  In a
// paged cache a tile must not straddle two pages, so there the range starts at the tile
// boundary (a multiple of the tile, hence inside one page) at or below that position; the
// per-column visibility mask hides the positions before the window.
#pragma once
#include "schedule.cuh"

namespace kvattn {

__host__ __device__ __forceinline__ int active_start_on(int align, int len, int q_len, int window) {
    const int s = active_start(len, q_len, window);
    return align > 1 ? s - s % align : s;
}

// build_tile_prefix (schedule.cuh) over those ranges; a sequence with tiles counts `cost` more, what a
// unit's start and end cost in tiles.
__device__ __forceinline__ void build_tile_prefix_on(int align, int cost, const int32_t *seq_lens, int B, int T_max, int tile,
                                                     int *s_prefix, int lane, int q_len, int window) {
    int running = 0;
    if (lane == 0) s_prefix[0] = 0;
    for (int base = 0; base < B; base += 32) {
        const int idx = base + lane;
        int v = 0;
        if (idx < B) {
            const int len = clamp_len(__ldg(seq_lens + idx), T_max);
            v = tiles_of(len - active_start_on(align, len, q_len, window), tile);
            if (v > 0) v += cost;
        }
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const int n = __shfl_up_sync(0xffffffffu, v, off);
            if (lane >= off) v += n;
        }
        if (idx < B) s_prefix[idx + 1] = running + v;
        running += __shfl_sync(0xffffffffu, v, 31);
    }
}

}  // namespace kvattn
