// How the two-slot attention kernels over a cache cut their work, and how cut units are merged.
//
// A unit is a (sequence, kv head, pair of row tiles).  All tiles of all units are laid out in a row, and each
// CTA takes an equal piece of it: sequence by sequence, head by head, row-tile pair by pair, tile by
// tile; a tile of a pair counts 2, of a single row tile 1, and a unit's first tile kUnitCost more (what
// its beginning and its output cost).  The host refuses sizes with 2^31 positions or more.
//
// A, the kernel's arguments, has B, Hkv, kUnitCost, kMinTiles (the least piece), tiles_of(b), row_tiles(),
// unit_rows(pair), out_row(b, head, pair, row) (-1: nobody's), out, the parts: ws_o [grid][2][rows][128],
// ws_ml [grid][2][rows], rows, and how few rows are merged: kFewRows, kFewBatch.
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
// Blocks (c, y): the unit whose first tile lies in piece c and whose last does not; its parts are piece c's
// second place and the first places of the pieces behind it.  m is in log2 units and a part's l and O share one
// factor, so a part weighs 2^(m - max m).  A row's parts are looked after 32 at a time, so that their loads do not wait
// for one another: by a warp where rows are few (as a rule with many parts), else by eight lanes, 32 / 8 float4 of its O
// each, and as many blocks as registers leave room for (4 rows a warp: 151 units of 256 rows and two parts took 24 us
// with a warp a row, 10 with eight lanes, 6 less with 64 registers than with 74).  Few rows' parts have their places in
// registers, one a lane; many rows' are listed once a block (with that list for few rows too, 48 ragged sequences of one
// node over the 8-bit cache take 160.0 us instead of 158.4, one of 20 011 rows over pages 18.9 instead of 17.9).  The
// launch may begin while the attention kernel ends; the partials are awaited below.
constexpr int kMergeThreads = 256, kMergeWarps = kMergeThreads / 32;
constexpr int kMergeMaxParts = 1024;              // at most one per CTA of the attention kernel

// A warp a row.  place_of(p): piece p's part, -1: it has none, -2: none from there on; first: that of piece c + lane.
template <class A, class PlaceOf>
__device__ __forceinline__ void merge_few(const A& a, const Segment& s, int c, int first, PlaceOf place_of) {
    constexpr int kBatch = A::kFewBatch;          // parts on their way at a time
    static_assert(32 % kBatch == 0, "batches of 32 parts");
    const int lane = threadIdx.x & 31, rows = a.unit_rows(s.pair);
    for (int row = blockIdx.y * kMergeWarps + (threadIdx.x >> 5); row < rows; row += gridDim.y * kMergeWarps) {
        float m = -INFINITY, sum = 0.f;
        float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int p0 = c;; p0 += 32) {
            const int place = p0 == c ? first : place_of(p0 + lane);
            const float2 ml = place >= 0 ? a.ws_ml[(int64_t)place * a.rows + row] : make_float2(-INFINITY, 0.f);
            float top = ml.x;
#pragma unroll
            for (int d = 16; d > 0; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
            const float mn = fmaxf(m, top), at = mn == -INFINITY ? 0.f : mn;
            const float w = exp2f(ml.x - at), wo = exp2f(m - at);
            m = mn;
            sum = sum * wo + warp_sum(ml.y * w);
            o.x *= wo; o.y *= wo; o.z *= wo; o.w *= wo;
            const unsigned there = __ballot_sync(0xffffffffu, place >= 0);
            const int parts = 32 - __clz(there);          // up to the last one that is there
#pragma unroll 1
            for (int q0 = 0; q0 < parts; q0 += kBatch) {  // (of 32, so q0 + q stays below)
                float4 z[kBatch];
#pragma unroll
                for (int q = 0; q < kBatch; ++q) {
                    const int from = __shfl_sync(0xffffffffu, place, q0 + q);
                    if ((there >> (q0 + q)) & 1u)
                        z[q] = reinterpret_cast<const float4*>(a.ws_o + ((int64_t)from * a.rows + row) * kHeadDim)[lane];
                }
#pragma unroll
                for (int q = 0; q < kBatch; ++q) {
                    const float wp = __shfl_sync(0xffffffffu, w, q0 + q);
                    if ((there >> (q0 + q)) & 1u) { o.x += z[q].x * wp; o.y += z[q].y * wp; o.z += z[q].z * wp; o.w += z[q].w * wp; }
                }
            }
            if (__any_sync(0xffffffffu, place == -2)) break;
        }
        const float inv = sum == 0.f ? 0.f : 1.f / sum;
        const int64_t to = a.out_row(s.b, s.head, s.pair, row);
        if (to < 0) continue;                             // nobody's row
        reinterpret_cast<uint2*>(a.out + to * kHeadDim)[lane] = make_uint2(pack2(o.x * inv, o.y * inv), pack2(o.z * inv, o.w * inv));
    }
}

// Eight lanes a row; places: of the parts, -1: none.
template <class A>
__device__ __forceinline__ void merge_many(const A& a, const Segment& s, const int* places, int parts) {
    constexpr int kLanes = 8, kEach = 32 / kLanes;
    const int lane = threadIdx.x & 31, l = lane % kLanes;
    const int rows = a.unit_rows(s.pair), per_block = kMergeWarps * kEach;
    for (int row0 = blockIdx.y * per_block + (threadIdx.x >> 5) * kEach; row0 < rows; row0 += gridDim.y * per_block) {
        const int row = min(row0 + lane / kLanes, rows - 1);          // (the last row more than once)
        float m = -INFINITY, sum = 0.f;
        float4 o[kEach] = {};
        for (int p0 = 0; p0 < parts; p0 += 32) {
            float2 ml[kEach];
            float top = -INFINITY, w[kEach], y[kEach];
#pragma unroll
            for (int k = 0; k < kEach; ++k) {
                const int p = p0 + l + kLanes * k, place = p < parts ? places[p] : -1;
                ml[k] = place >= 0 ? a.ws_ml[(int64_t)place * a.rows + row] : make_float2(-INFINITY, 0.f);
            }
#pragma unroll
            for (int k = 0; k < kEach; ++k) top = fmaxf(top, ml[k].x);
#pragma unroll
            for (int d = kLanes / 2; d > 0; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
            const float mn = fmaxf(m, top), at = mn == -INFINITY ? 0.f : mn, wo = exp2f(m - at);
            m = mn;
#pragma unroll
            for (int k = 0; k < kEach; ++k) {
                w[k] = exp2f(ml[k].x - at);
                y[k] = ml[k].y * w[k];
            }
#pragma unroll
            for (int h = kEach / 2; h > 0; h >>= 1)
#pragma unroll
                for (int k = 0; k < h; ++k) y[k] += y[k + h];
#pragma unroll
            for (int d = kLanes / 2; d > 0; d >>= 1) y[0] += __shfl_xor_sync(0xffffffffu, y[0], d);
            sum = sum * wo + y[0];
#pragma unroll
            for (int c = 0; c < kEach; ++c) { o[c].x *= wo; o[c].y *= wo; o[c].z *= wo; o[c].w *= wo; }
#pragma unroll
            for (int k = 0; k < kEach; ++k) {
                const int first = p0 + k * kLanes, count = min(kLanes, parts - first);
#pragma unroll 1
                for (int q = 0; q < count; ++q) {
                    const int place = places[first + q];
                    const float4* x = reinterpret_cast<const float4*>(a.ws_o + ((int64_t)max(place, 0) * a.rows + row) * kHeadDim) + l;
                    const float wp = __shfl_sync(0xffffffffu, w[k], q, kLanes);
                    if (place < 0) continue;
                    float4 z[kEach];
#pragma unroll
                    for (int c = 0; c < kEach; ++c) z[c] = x[c * kLanes];
#pragma unroll
                    for (int c = 0; c < kEach; ++c) { o[c].x += z[c].x * wp; o[c].y += z[c].y * wp; o[c].z += z[c].z * wp; o[c].w += z[c].w * wp; }
                }
            }
        }
        const float inv = sum == 0.f ? 0.f : 1.f / sum;
        const int64_t to = a.out_row(s.b, s.head, s.pair, row);
        if (to < 0) continue;                             // nobody's row
#pragma unroll
        for (int c = 0; c < kEach; ++c)
            reinterpret_cast<uint2*>(a.out + to * kHeadDim)[l + c * kLanes] =
                make_uint2(pack2(o[c].x * inv, o[c].y * inv), pack2(o[c].z * inv, o[c].w * inv));
    }
}

template <bool kFew, class A>                     // rows of a part up to A::kFewRows
__device__ __forceinline__ void merge_parts(const A& a, int grid) {
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
    // piece p's part of the unit, whose first tile is piece c's; -1: it holds none of its tiles, -2: nor do those behind it
    auto place_of = [&](int p) {
        if (p >= cut.ctas) return -2;
        const int t0 = p == c ? 0 : tiles_before<A>(s.start, s.weight, cut.begin(p));
        const int t1 = p + 1 < cut.ctas ? tiles_before<A>(s.start, s.weight, cut.begin(p + 1)) : s.T;
        return t0 >= s.T ? -2 : t0 < min(t1, s.T) ? p * 2 + (p == c) : -1;
    };
    if constexpr (kFew) {
        const int first = place_of(c + (int)(threadIdx.x & 31));
        await();
        merge_few(a, s, c, first, place_of);
    } else {
        __shared__ int s_place[kMergeMaxParts];
        __shared__ int s_parts;
        if (threadIdx.x == 0) s_parts = cut.ctas - c;
        __syncthreads();
        for (int p = c + threadIdx.x; p < cut.ctas; p += kMergeThreads) {
            s_place[p - c] = place_of(p);
            if (s_place[p - c] == -2) atomicMin(&s_parts, p - c);
        }
        __syncthreads();
        await();
        merge_many(a, s, s_place, s_parts);
    }
}

// Launches the merging kernel of the rows' kind behind an attention kernel of `grid` CTAs.  Blocks a piece takes: a
// warp a row, or at most four, which fit on the device together with those of the other pieces (64 trees of 60
// nodes: 211.6 us with 4, 214.3 with 8 and the second half waiting).
template <class A>
inline cudaError_t launch_merge(void (*few)(A, int), void (*many)(A, int), const A& a, int grid, cudaStream_t stream) {
    const bool is_few = a.rows <= A::kFewRows;
    const int per = kMergeWarps * (is_few ? 1 : 4), y = (a.rows + per - 1) / per;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(grid - 1), (unsigned)(is_few || y < 4 ? y : 4));
    cfg.blockDim = dim3(kMergeThreads);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, is_few ? few : many, a, grid);
}

}  // namespace attn2
}  // namespace eagle
