// groups.cuh -- the ragged groups of the linear products: rows of group e are
// [offsets[e], offsets[e+1]), cut into items of at most `item_rows` rows. Every
// CTA builds the item list's prefix in shared memory from the offsets itself
// (E <= 256: one load per thread and a scan), so no list lives in a workspace
// and no kernel has to run before.
#pragma once

#include "common.cuh"
#include "internal.h"
#include "tiles.cuh"

namespace moe {

struct GroupSmem {
    int row0[MOE_MAX_E + 1];    // first row of each group, so [e + 1] is the end of group e
    int first[MOE_MAX_E + 1];   // first item of each group; [E]: number of items
    int warp[17];
    int bad;
};

// Fills G. All threads of a block of >= 256 threads (a multiple of 32) call it;
// the first 256 work. offsets NULL: one group of all rows. Offsets that decrease
// or leave [0, rows] make every group empty and flag MOE_ERR_CHECK.
__device__ __forceinline__ void build_groups(GroupSmem &G, const int32_t *offsets, int E, int rows,
                                             int item_rows, uint32_t *status)
{
    const int t = threadIdx.x;
    if (t == 0)
        G.bad = 0;
    __syncthreads();
    int a = 0, b = 0;
    if (t < E) {
        a = offsets ? offsets[t] : 0;
        b = offsets ? offsets[t + 1] : rows;
        if (a < 0 || b < a || b > rows)
            G.bad = 1;
    }
    __syncthreads();
    const bool bad = G.bad != 0;
    if (bad) {
        a = b = 0;
        if (t == 0 && blockIdx.x == 0 && blockIdx.y == 0 && blockIdx.z == 0)
            flag_status(status, MOE_ERR_CHECK);
    }
    const int n = (b - a + item_rows - 1) / item_rows;
    // exclusive scan over the first 256 threads
    const int lane = t & 31, warp = t >> 5;
    int inc = n;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const int o = __shfl_up_sync(kFullMask, inc, off);
        if (lane >= off)
            inc += o;
    }
    if (warp < 8 && lane == 31)
        G.warp[warp] = inc;
    __syncthreads();
    if (t < E) {
        int base = 0;
        for (int w = 0; w < warp; ++w)
            base += G.warp[w];
        G.first[t] = base + inc - n;
        G.row0[t] = a;
        if (t == E - 1) {
            G.first[E] = base + inc;
            G.row0[E] = b;
        }
    }
    __syncthreads();
}

// Group of an item (item < G.first[E]): the e with first[e] <= item < first[e+1].
__device__ __forceinline__ int item_group(const GroupSmem &G, int E, int item)
{
    int lo = 0, hi = E - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (G.first[mid] <= item)
            lo = mid;
        else
            hi = mid - 1;
    }
    return lo;
}

} // namespace moe
