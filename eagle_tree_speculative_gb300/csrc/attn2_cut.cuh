// How the two-slot attention kernels over a cache cut their work, and how cut units are merged.
//
// A unit is a (sequence, kv head, pair of row tiles).  All tiles of all units are laid out in a row, and each
// CTA takes an equal piece of it: sequence by sequence, head by head, row-tile pair by pair, tile by
// tile; a tile of a pair counts 2, of a single row tile 1, and a unit's first tile kUnitCost more (what
// its beginning and its output cost).  The host refuses sizes with 2^31 positions or more.
//
// A, the kernel's arguments, has B, Hkv, kUnitCost, kMinTiles (the least piece), tiles_of(b), row_tiles(),
// unit_rows(pair), out_row(b, head, pair, row) (-1: nobody's), out, and the parts: ws_o [grid][2][rows][128],
// ws_ml [grid][2][rows], rows.
#pragma once

#include "attn2_common.cuh"

namespace eagle {
namespace attn2 {

struct Cut {
    int total;                                    // positions
    int ctas;                                     // pieces
    __device__ int begin(int c) const { return total / ctas * c + total % ctas * c / ctas; }
};

// Warp-wide.
template <class A>
__device__ __forceinline__ Cut make_cut(const A& a, int grid) {
    int sum = 0;
    for (int b = threadIdx.x & 31; b < a.B; b += 32) sum += a.tiles_of(b) + A::kUnitCost;
    sum = __reduce_add_sync(0xffffffffu, sum);
    Cut c;
    const int rt = a.row_tiles();
    c.total = sum * rt * a.Hkv;
    c.ctas = max(1, min(grid, c.total / (A::kMinTiles * min(rt, 2))));
    return c;
}

// A unit and the tiles of it that lie in [pos, end).
struct Segment {
    int b, head, pair, T;                         // T tiles in all
    int weight;                                   // row tiles of the pair
    int start;                                    // position of its first tile
    int t0, t1;
};
// Tiles of a unit that begins at `start` whose own position lies before pos.
template <class A>
__device__ __forceinline__ int tiles_before(int start, int weight, int pos) {
    return pos <= start ? 0 : max(1, ((pos - start + weight - 1) >> (weight - 1)) - A::kUnitCost);
}

// Warp-wide: the unit at position pos; `b`, `base`: a sequence at or before it and its first
// position, moved on.
template <class A>
__device__ __forceinline__ Segment segment_at(const A& a, int pos, int end, int& b, int& base) {
    const int rt = a.row_tiles(), lane = threadIdx.x & 31;
    for (;;) {                                    // 32 sequences at a time
        const int mine = b + lane;
        const int w = mine < a.B ? (a.tiles_of(mine) + A::kUnitCost) * rt * a.Hkv : 0;
        int sum = w;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, sum, o);
            if (lane >= o) sum += y;
        }
        const unsigned past = __ballot_sync(0xffffffffu, base + sum > pos);
        if (past) {
            const int l = __ffs(past) - 1;
            base += __shfl_sync(0xffffffffu, sum - w, l);
            b += l;
            break;
        }
        base += __shfl_sync(0xffffffffu, sum, 31);
        b += 32;
        if (b >= a.B) { b = a.B - 1; break; }     // not reached: pos < total
    }
    Segment s;
    s.b = b;
    s.T = a.tiles_of(b);
    int off = pos - base;
    const int per_tile = s.T + A::kUnitCost, per_head = per_tile * rt;
    s.head = off / per_head;
    off -= s.head * per_head;
    s.pair = off / (2 * per_tile);
    off -= s.pair * 2 * per_tile;
    s.weight = min(2, rt - 2 * s.pair);
    s.start = pos - off;
    s.t0 = min(s.T, tiles_before<A>(s.start, s.weight, pos));
    s.t1 = min(s.T, tiles_before<A>(s.start, s.weight, end));
    return s;
}

// ---------------- merging of cut units ----------------
// Blocks (c, y): the unit whose first tile lies in piece c and whose last does not, one warp a row;
// its parts are piece c's second place and the first places of the pieces behind it.  m is in
// log2 units and a part's l and O share one factor, so a part weighs 2^(m - max m).  Lane p looks
// after part p (of up to 32 at a time), so that the parts' loads do not wait for one another.  The
// launch may begin while the attention kernel ends; the partials are awaited below.
constexpr int kMergeThreads = 256, kMergeWarps = kMergeThreads / 32;

template <class A>
__device__ __forceinline__ void merge_parts(const A& a, int grid) {
    const int lane = threadIdx.x & 31;
    const Cut cut = make_cut(a, grid);
    const int c = blockIdx.x;
    // A block that has nothing to merge awaits the attention kernel too: a kernel launched next
    // waits for this one alone.
    auto await = [] { asm volatile("griddepcontrol.wait;\n" ::: "memory"); };
    if (c + 1 >= cut.ctas) { await(); return; }           // the last piece ends with a whole unit
    const int begin = cut.begin(c), end = cut.begin(c + 1);
    int b = 0, base = 0;
    const Segment s = segment_at(a, end - 1, end, b, base);
    if (s.start < begin || s.t1 >= s.T) { await(); return; }   // it begins earlier, or is whole
    const int rows = a.unit_rows(s.pair);
    // lane's part: piece c + lane, and whether it holds tiles of the unit
    auto place_of = [&](int p) -> int {                   // -1: none, -2: none from here on
        if (p == c) return c * 2 + 1;
        if (p >= cut.ctas) return -2;
        const int t0 = tiles_before<A>(s.start, s.weight, cut.begin(p));
        const int t1 = p + 1 < cut.ctas ? tiles_before<A>(s.start, s.weight, cut.begin(p + 1)) : s.T;
        return t0 >= s.T ? -2 : t0 < t1 ? p * 2 : -1;
    };
    const int first = place_of(c + lane);
    await();
    for (int row = blockIdx.y * kMergeWarps + (threadIdx.x >> 5); row < rows; row += gridDim.y * kMergeWarps) {
        float m = -INFINITY, l = 0.f;
        float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int p0 = c;; p0 += 32) {
            const int place = p0 == c ? first : place_of(p0 + lane);
            const bool there = place >= 0;
            const float2 ml = there ? a.ws_ml[(int64_t)place * a.rows + row] : make_float2(-INFINITY, 0.f);
            float top = ml.x;
#pragma unroll
            for (int d = 16; d > 0; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
            const float mn = fmaxf(m, top), at = mn == -INFINITY ? 0.f : mn;
            const float w = exp2f(ml.x - at), wo = exp2f(m - at);
            m = mn;
            l = l * wo + warp_sum(ml.y * w);
            o.x *= wo; o.y *= wo; o.z *= wo; o.w *= wo;
            const unsigned live = __ballot_sync(0xffffffffu, there);
            const int parts = 32 - __clz(live);           // places up to the last one that is there
#pragma unroll 4
            for (int p = 0; p < parts; ++p) {
                const int at_p = max(__shfl_sync(0xffffffffu, place, p), 0);
                const float wp = __shfl_sync(0xffffffffu, w, p);
                const float4 x = *reinterpret_cast<const float4*>(a.ws_o + ((int64_t)at_p * a.rows + row) * kHeadDim + 4 * lane);
                if ((live >> p) & 1u) { o.x += x.x * wp; o.y += x.y * wp; o.z += x.z * wp; o.w += x.w * wp; }
            }
            if (__any_sync(0xffffffffu, place == -2)) break;
        }
        const float inv = l == 0.f ? 0.f : 1.f / l;
        const int64_t to = a.out_row(s.b, s.head, s.pair, row);
        if (to < 0) continue;                             // nobody's row
        reinterpret_cast<uint2*>(a.out + to * kHeadDim)[lane] = make_uint2(pack2(o.x * inv, o.y * inv), pack2(o.z * inv, o.w * inv));
    }
}

}  // namespace attn2
}  // namespace eagle
