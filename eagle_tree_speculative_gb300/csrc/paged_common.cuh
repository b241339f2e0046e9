// What the calls on the paged K/V cache share: page sizes, limits, places of rows, a warp's view of a
// draft tree.
#pragma once

#include "common.cuh"

namespace eagle {
namespace paged {

constexpr int64_t kMaxPool = 0x7fffffffLL;        // N * Hkv * page: rows of all pages and heads, as 32-bit places
// P * page: rows of a sequence.  The attention goes through them in 2^20 tiles of 3 500 cycles at most, during which the
// roles that are done with them wait; waits give up from 2^32 cycles on.
constexpr int64_t kMaxRows = 1LL << 27;

inline bool page_ok(int page) { return page == 16 || page == 32 || page == 64 || page == 128; }
inline int page_shift(int page) { return page == 16 ? 4 : page == 32 ? 5 : page == 64 ? 6 : 7; }

// First element of row r (within its page) of head h.
__device__ __forceinline__ int64_t row_at(int id, int h, int r, int Hkv, int shift) {
    return ((((int64_t)id * Hkv + h) << shift) + r) * kHeadDim;
}

// Warp-wide: the depths of nodes lane and lane + 32 of a tree of n <= 64 nodes, false if it is no tree.  Each
// round doubles how far up a node has looked.
__device__ __forceinline__ bool tree_depths(const int32_t* parent, int n, int (&depth)[2]) {
    const int lane = threadIdx.x & 31;
    int p[2];
    bool bad = false;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int i = lane + 32 * h;
        p[h] = i < n ? parent[i] : -1;
        bad |= i < n && (i == 0 ? p[h] != -1 : (p[h] < 0 || p[h] >= i));
        depth[h] = p[h] >= 0;
    }
    if (__any_sync(0xffffffffu, bad)) return false;
    for (int reach = 1; reach < n; reach <<= 1) {
        int d[2], q[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int s = max(p[h], 0);
            const int d0 = __shfl_sync(0xffffffffu, depth[0], s & 31), d1 = __shfl_sync(0xffffffffu, depth[1], s & 31);
            const int q0 = __shfl_sync(0xffffffffu, p[0], s & 31), q1 = __shfl_sync(0xffffffffu, p[1], s & 31);
            d[h] = p[h] < 0 ? 0 : (s < 32 ? d0 : d1);
            q[h] = p[h] < 0 ? -1 : (s < 32 ? q0 : q1);
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) { depth[h] += d[h]; p[h] = q[h]; }
    }
    return true;
}

}  // namespace paged
}  // namespace eagle
