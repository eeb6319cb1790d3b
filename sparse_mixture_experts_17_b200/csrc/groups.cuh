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
    int group[MOE_MAX_E];       // ORDER: the group at each place of first[]
    int cls[4];                 // ORDER: first item of each class, and the end of the last
    unsigned long long warp[8];
    int bad;
};

// Fills G. All threads of a block of >= 256 threads (a multiple of 32) call it;
// the first 256 work. offsets NULL: one group of all rows. Offsets that decrease
// or leave [0, rows] make every group empty and flag MOE_ERR_CHECK. With ORDER
// (item_rows >= kClass1Rows), first[] runs over the groups by class, and group[i] is the
// group at place i (row0 stays by group): class 0 has more than kClass1Rows rows,
// class 1 more than kClass2Rows, class 2 at least one; empty groups come last.
constexpr int kClass1Rows = 128, kClass2Rows = 64;

template <bool ORDER = false>
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
    // exclusive scan over the first 256 threads: the items (26 bits: at most 2^24 + 256), with
    // ORDER those of class 0 only, and the groups of each class (9 bits each)
    const int c = b - a > kClass1Rows ? 0 : b - a > kClass2Rows ? 1 : 2;
    unsigned long long mine = (unsigned long long)n;
    if (ORDER)
        mine = n == 0 ? 0 : c == 0 ? mine | 1ull << 26 : 1ull << (26 + 9 * c);
    const int lane = t & 31, warp = t >> 5;
    unsigned long long inc = mine;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const unsigned long long o = __shfl_up_sync(kFullMask, inc, off);
        if (lane >= off)
            inc += o;
    }
    if (warp < 8 && lane == 31)
        G.warp[warp] = inc;
    __syncthreads();
    if (t < E) {
        unsigned long long base = 0, sum = 0;
        for (int w = 0; w < 8; ++w) {
            if (w == warp)
                base = sum;
            sum += G.warp[w];
        }
        const unsigned long long ex = base + inc - mine;
        const int mask = (1 << 26) - 1;
        const int items = (int)(ex & mask), all = (int)(sum & mask);
        if (ORDER) {
            const auto part = [](unsigned long long v, int c) { return (int)(v >> (26 + 9 * c)) & 511; };
            const int r0 = part(ex, 0), r1 = part(ex, 1), r2 = part(ex, 2);
            const int n0 = part(sum, 0), n1 = part(sum, 1), n2 = part(sum, 2);
            const int end1 = all + n1, end2 = end1 + n2;
            int place, first;
            if (n == 0) {
                place = n0 + n1 + n2 + t - r0 - r1 - r2;
                first = end2;
            } else if (c == 0) {
                place = r0;
                first = items;
            } else if (c == 1) {
                place = n0 + r1;
                first = all + r1;
            } else {
                place = n0 + n1 + r2;
                first = end1 + r2;
            }
            G.first[place] = first;
            G.group[place] = t;
            if (t == 0) {
                G.cls[0] = 0;
                G.cls[1] = all;
                G.cls[2] = end1;
                G.cls[3] = G.first[E] = end2;
            }
        } else {
            G.first[t] = items;
            if (t == 0)
                G.first[E] = all;
        }
        G.row0[t] = a;
        if (t == E - 1)
            G.row0[E] = b;
    }
    __syncthreads();
}

// Group of an item (item < G.first[E]): the e with first[e] <= item < first[e+1]
// (with ORDER its place). Empty groups never come out: the last one that fits is taken.
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
