// Rows that belong to groups (a mixture's experts), as a kernel finds them.
//
// ends[e] is the row behind group e's last; the groups follow one another from
// row 0.  The counts are on the device, so each CTA works out by itself which
// group a unit of work falls into: one pass over `ends` by all threads (a
// running maximum, then a running sum of the groups' units), two tables in
// shared memory, and a binary search a unit.  It takes a microsecond or two; a
// launch of its own for the tables would cost as much, and a buffer (1024 groups
// at most: two tables of 4 KB).
//
// Whatever `ends` holds, no group reaches past [0, rows) and no two groups
// meet: it is taken as its running maximum, held within [0, rows].
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "rlk_ptx.cuh"

namespace rlk {
namespace {

constexpr int kMaxGroups = 1024;

struct GroupTable {
    int begin[kMaxGroups + 2];  // group e's rows are [begin[e], begin[e + 1]); e = G: the rows behind the groups
    int first[kMaxGroups + 2];  // its units are [first[e], first[e + 1])
    int carry[2][32];
};

// By all THREADS threads (whole warps); the caller's next __syncthreads
// publishes the table.  A group has ceil(rows / unit) * per units, and where
// `rest`, so have the rows behind the last group (else they have none).
template <int THREADS>
__device__ __forceinline__ void groups_build(GroupTable* tab, const int32_t* ends, int G, int rows, int unit, int per,
                                             bool rest) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int each = (G + THREADS - 1) / THREADS, e0 = threadIdx.x * each, e1 = min(e0 + each, G);
    auto units_of = [&](int n) { return (n + unit - 1) / unit * per; };

    int top = 0;
    for (int e = e0; e < e1; ++e) top = max(top, min(ends[e], rows));
    int scan = top;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xFFFFFFFFu, scan, o);
        if (lane >= o) scan = max(scan, v);
    }
    if (lane == 31) tab->carry[0][warp] = scan;
    __syncthreads();
    int before = __shfl_up_sync(0xFFFFFFFFu, scan, 1);
    if (lane == 0) before = 0;
    for (int w = 0; w < warp; ++w) before = max(before, tab->carry[0][w]);

    int units = 0, at = before;
    for (int e = e0; e < e1; ++e) {
        const int v = max(at, min(ends[e], rows));
        tab->begin[e] = at;
        units += units_of(v - at);
        at = v;
    }
    int sum = units;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xFFFFFFFFu, sum, o);
        if (lane >= o) sum += v;
    }
    if (lane == 31) tab->carry[1][warp] = sum;
    __syncthreads();
    int u = sum - units;
    for (int w = 0; w < warp; ++w) u += tab->carry[1][w];
    at = before;
    for (int e = e0; e < e1; ++e) {
        const int v = max(at, min(ends[e], rows));
        tab->first[e] = u;
        u += units_of(v - at);
        at = v;
        if (e == G - 1) {
            tab->begin[G] = at;
            tab->first[G] = u;
            tab->begin[G + 1] = rows;
            tab->first[G + 1] = u + (rest ? units_of(rows - at) : 0);
        }
    }
}

// The group of unit u < first[G + 1] (G: the rows behind the groups).
__device__ __forceinline__ int group_of(const GroupTable* tab, int G, int u) {
    int lo = 0, hi = G;  // first[lo] <= u < first[hi + 1]
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (tab->first[mid] <= u)
            lo = mid;
        else
            hi = mid - 1;
    }
    return lo;
}

}  // namespace
}  // namespace rlk
