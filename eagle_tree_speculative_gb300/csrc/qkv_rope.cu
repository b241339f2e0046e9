// Norms of the queries' and keys' heads, the rotation by position, and the rows into the cache's
// pages: one pass over what a layer's projections left.
//
// Mathematics.  y = w x / sqrt(mean x^2 + eps) over a head's 128 elements, then pairs (y_i, y_j) turned by
// position * f_i.  The angle is needed modulo a turn, at positions where a product in fp32 has lost
// it: f_i / 2 pi as a 64-bit fraction of a turn, times the position in integer arithmetic, whose
// overflow is whole turns; the upper 32 bits are the angle to 2^-32 of a turn (its fraction was rounded
// to 2^-53 of itself: 2^-29 of a turn at position 2^24).
//
// Layout.  Eight lanes a head, a group of four heads at once: a lane has two chunks of 8 elements (16 bytes) that
// hold both elements of its pairs, so nothing is exchanged for the rotation and three shuffles do the norm.  The
// token's 64 angles are computed by the warp once, two a lane, and go through shared memory.
// The last tokens' groups are shared out to the warps alike, so a single token is worked on by as many as it has
// groups and a call ends everywhere at once.  Each warp has kAhead - 1 groups on their way into shared memory, of this
// token and the next (cp.async; a lane reads only what it copied itself, so nothing waits for other lanes):
// registers would hold two.
//
// Measured: 24 ragged prompts, 16610 tokens of 32 / 8 heads with norms, rows packed and into pages, 75 us, 77 with other
// rows and pages in between: 5.7 TB/s, 85% of the measured copy; 64 trees of 60 nodes into pages 17.6 us where their 94 MB
// stay in L2, 22 from HBM (4.3 TB/s).  Bound: HBM; short calls, and those of a token or two a warp, the chain
// of dependent reads before a token's first output (place, page, angle).
#include <type_traits>

#include "attn2_common.cuh"
#include "paged_common.cuh"

namespace eagle {
namespace {

constexpr int kWarps = 4;
// Blocks of an SM: 16 warps for the calls that are over soon, 12 for those that stream (us with 12 / 16 / 20: 24 ragged
// prompts, 16610 tokens of 32 / 8 heads, 73.5 / 81.1 / 86.9; 64 trees of 60 nodes, in L2, 19.1 / 18.2 / 23.0).
constexpr int kBlocks = 4, kBlocksLong = 3;
constexpr int kLongTokens = 4;                    // tokens a warp from which a call is long
constexpr int kAhead = 8;                         // places of groups of four heads (1 KB); all but one on their way
constexpr int kRopeSmem = kWarps * (kAhead * 1024 + 64 * (int)sizeof(float2));
static_assert(kBlocks * (kRopeSmem + 1024) <= 233472, "shared memory of an SM");

struct RopeArgs {
    const uint16_t *q, *k, *v, *q_weight, *k_weight;
    const float* inv_freq;
    const int32_t *cu, *parent, *pos;
    uint16_t *q_out, *k_out, *k_pages, *v_pages;
    const int32_t* page_table;
    int T, B, n, Hq, Hkv, half;                   // half: rot_dim / 2 pairs
    int N, shift, P;
    float eps;
    int64_t q_stride, k_stride, v_stride;
    int32_t* dev_status;
};

// Two bf16 of a word, as floats.
__device__ __forceinline__ float lo_of(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float hi_of(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

__device__ __forceinline__ uint32_t pack_pair(uint64_t v) {
    float lo, hi;
    attn2::unf2(v, lo, hi);
    return pack2(lo, hi);
}

// The sum of squares of the eight lanes' 16 elements each.
__device__ __forceinline__ float sum_squares(const uint64_t (&x)[8]) {
    uint64_t s[2] = {0, 0};
#pragma unroll
    for (int e = 0; e < 8; ++e) s[e & 1] = attn2::fma2(x[e], x[e], s[e & 1]);
    float lo, hi;
    attn2::unf2(attn2::add2(s[0], s[1]), lo, hi);
    float t = lo + hi;
#pragma unroll
    for (int o = 4; o > 0; o >>= 1) t += __shfl_xor_sync(0xffffffffu, t, o);
    return t;
}

// 16 bytes of global into shared memory, behind this thread's back; kLeft: groups that may still be on their way.
__device__ __forceinline__ void copy16_async(uint32_t dst, const void* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;\n" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;\n" ::: "memory"); }
template <int kLeft>
__device__ __forceinline__ void copy_wait() {
    asm volatile("cp.async.wait_group %0;\n" ::"n"(kLeft) : "memory");
}

// kPairs2: pairs (2i, 2i + 1), else (i, i + rot_dim / 2).  kWhole: rot_dim is the head dimension
template <bool kPairs2, bool kWhole>
__global__ void __launch_bounds__(kWarps * 32, kBlocks) qkv_rope_kernel(RopeArgs a) {
    extern __shared__ uint4 s_all[];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    // a lane reads what it has copied itself: its two chunks of each of the warp's groups
    uint4* raw = s_all + warp * (kAhead * 64) + lane;                 // [kAhead][2][32]
    float2* turns = reinterpret_cast<float2*>(s_all + kWarps * (kAhead * 64)) + warp * 64;

    // ---- what is alike for all tokens: the lane's chunks, the angles a position turns by ----
    const int c = lane & 7;
    // Pairs of halves: the first m = half / 8 lanes have chunks c and c + m, the others those from 2 m on, in two runs.
    const int m = a.half >> 3;
    const bool pairs = c < m;
    const int p0 = kPairs2 || pairs ? c : c + m, p1 = !kPairs2 && pairs ? c + m : c + 8;
    const bool turned0 = kPairs2 ? p0 < (a.half >> 2) : pairs, turned1 = kPairs2 ? p1 < (a.half >> 2) : pairs;
    const int q_quads = (a.Hq + 3) >> 2, k_quads = (a.Hkv + 3) >> 2;
    const int total = q_quads + k_quads * (a.page_table ? 2 : 1);

    // ---- the warp's groups: every warps-th token, as long as there is one for each warp, then an equal share of
    // the groups that the last tokens have ----
    const int warps = gridDim.x * kWarps, w = blockIdx.x * kWarps + warp, rounds = a.T / warps;
    const int64_t rest = (int64_t)(a.T - rounds * warps) * total, begin = rest * w / warps;
    const int tail = (int)(rest * (w + 1) / warps - begin);
    const int tail_t = rounds * warps + (int)(begin / total), tail_y = (int)(begin % total);
    // a token's place in this order: which one, its first group here, rounds to come (it included; 0: in the tail)
    struct Place {
        int t, y, rounds;
    };
    auto start = [&] { return rounds > 0 ? Place{w, 0, rounds} : Place{tail_t, tail_y, 0}; };
    auto following = [&](const Place& p) {
        if (p.rounds > 1) return Place{p.t + warps, 0, p.rounds - 1};
        return p.rounds == 1 ? Place{tail_t, tail_y, 0} : Place{p.t + 1, 0, 0};
    };
    int left = rounds * total + tail;
    if (left == 0) return;
    // A token's groups are q's, then k's, then v's.  What is copied next: group next_y of a token, whose head for
    // this lane lies at `next` (a kind's last group may lack heads: those lanes copy its first one again)
    Place copy = start();
    int next_left = left, next_y = copy.y, next_end = next_y, next_h = 0, next_heads = 0;
    const uint16_t *next = nullptr, *next_base = nullptr;
    uint32_t copy_at = s32(raw), read_at = 0;     // places in the ring
    const uint32_t copy_begin = copy_at, copy_end = copy_at + kAhead * 1024;
    auto copy_next = [&] {
        if (next_left > 0) {
            --next_left;
            if (next_y == next_end) {             // a kind's first group
                if (next_y == total) {
                    copy = following(copy);
                    next_y = copy.y;
                }
                const int kind = next_y < q_quads ? 0 : next_y < q_quads + k_quads ? 1 : 2, y0 = kind == 0 ? 0 : kind == 1 ? q_quads : q_quads + k_quads;
                next_end = kind == 0 ? q_quads : y0 + k_quads;
                next_heads = kind == 0 ? a.Hq : a.Hkv;
                next_base = kind == 0 ? a.q + copy.t * a.q_stride : kind == 1 ? a.k + copy.t * a.k_stride : a.v + copy.t * a.v_stride;
                next_h = 4 * (next_y - y0) + (lane >> 3);
                next = next_base + next_h * kHeadDim;
            }
            const uint16_t* src = next_h < next_heads ? next : next_base;
            copy16_async(copy_at, src + 8 * p0);
            copy16_async(copy_at + 512, src + 8 * p1);
            next += 4 * kHeadDim;
            next_h += 4;
            ++next_y;
        }
        copy_commit();                            // (behind the last one: empty groups)
        copy_at += 1024;
        if (copy_at == copy_end) copy_at = copy_begin;
    };
#pragma unroll 1
    for (int i = 0; i < kAhead - 1; ++i) copy_next();

    unsigned long long frac[2];                   // of pairs lane and lane + 32, in turns
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int i = lane + 32 * h;
        const double f = i < a.half ? (double)a.inv_freq[i] * 0.15915494309189533577 : 0.0;
        frac[h] = (unsigned long long)((f - floor(f)) * 18446744073709551616.0);
    }
    // sequences, 32 at a time; the first ones stay in registers
    int c0 = 0, c1 = 0;
    if (a.cu) {
        bool bad = false;
        for (int b0 = 0; b0 < a.B; b0 += 32) {
            const int i = min(b0 + lane, a.B - 1), x0 = a.cu[i], x1 = a.cu[i + 1];
            bad |= x0 < 0 || x1 < x0 || x1 > a.T;
            if (b0 == 0) { c0 = x0; c1 = x1; }
        }
        if (__any_sync(0xffffffffu, bad)) {
            if (lane == 0) flag_error(a.dev_status, EAGLE_DEV_CAPACITY);
            copy_wait<0>();
            return;
        }
    }
    int tree_of = -1, depth[2] = {0, 0};
    bool tree_ok = false;

    for (Place at = start(); left > 0; at = following(at)) {
        const int t = at.t, first = at.y, end = min(total, first + left);
        left -= end - first;
        // ---- the token's sequence, its row there and its position ----
        int b = -1, row = 0, ahead = 0, rows = 0;
        bool skip = false;
        if (a.parent) {
            b = t / a.n;
            row = t - b * a.n;
            rows = a.n;
            if (b != tree_of) {
                tree_of = b;
                tree_ok = paged::tree_depths(a.parent + (int64_t)b * a.n, a.n, depth);
                if (!tree_ok && lane == 0) flag_error(a.dev_status, EAGLE_DEV_BAD_TREE);
            }
            skip = !tree_ok;
            const int d0 = __shfl_sync(0xffffffffu, depth[0], row & 31), d1 = __shfl_sync(0xffffffffu, depth[1], row & 31);
            ahead = row < 32 ? d0 : d1;
        } else {
            int x0 = c0, x1 = c1, b0 = 0;
            if (a.B > 32 && t >= __shfl_sync(0xffffffffu, c1, 31)) {
                // behind the first 32: the last place of cu with at most t, a 32nd of what is left each time
                int lo = 32, len = a.B - 31;      // in cu[lo .. lo + len), whose first is at most t
                while (len > 1) {
                    const int step = (len + 31) >> 5, x = lane * step;
                    const unsigned upto = __ballot_sync(0xffffffffu, x < len && a.cu[lo + min(x, len - 1)] <= t);
                    const int skipped = (31 - __clz(upto)) * step;
                    lo += skipped;
                    len = min(step, len - skipped);
                }
                b0 = lo;
                x0 = lo < a.B ? a.cu[lo] : 0;
                x1 = lo < a.B ? a.cu[lo + 1] : 0;
            }
            const unsigned in = __ballot_sync(0xffffffffu, x0 <= t && t < x1);
            if (in) {
                const int l = __ffs(in) - 1, begin = __shfl_sync(0xffffffffu, x0, l);
                b = b0 + l;                       // (one sequence's place in all lanes: l is 0)
                row = ahead = t - begin;
                rows = __shfl_sync(0xffffffffu, x1, l) - begin;
            }
            skip = b < 0;                         // a token of no sequence
        }
        int id = -1, in_page = 0, held = 0;
        if (!skip) {
            held = a.pos[b];
            const int64_t room = a.page_table ? (int64_t)a.P << a.shift : 0x7fffffffLL;
            if (held < 0 || held + (int64_t)rows > room) {
                if (lane == 0) flag_error(a.dev_status, EAGLE_DEV_CAPACITY);
                skip = true;
            } else if (a.page_table) {
                id = a.page_table[(int64_t)b * a.P + ((held + row) >> a.shift)];
                in_page = (held + row) & ((1 << a.shift) - 1);
                if (id < 0 || id >= a.N) {
                    if (lane == 0) flag_error(a.dev_status, EAGLE_DEV_CAPACITY);
                    id = -1;
                }
            }
        }

        // ---- the token's turns: two a lane, through shared memory ----
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int angle = (int)((frac[h] * (unsigned)(held + ahead)) >> 32);
            float2 turn;
            sincospif((float)angle * 0x1p-31f, &turn.y, &turn.x);
            turns[lane + 32 * h] = turn;
        }
        __syncwarp();
        float2 turn[8];
#pragma unroll
        for (int e = 0; e < 8; ++e)
            turn[e] = turns[kPairs2 ? (e < 4 ? 4 * c + e : 32 + 4 * c + e - 4) : 8 * c + e];
        __syncwarp();

        // ---- the heads, kind by kind ----
        for (int y = first; y < end;) {
            const int kind = y < q_quads ? 0 : y < q_quads + k_quads ? 1 : 2, y0 = kind == 0 ? 0 : kind == 1 ? q_quads : q_quads + k_quads;
            const int stop = min(end, kind == 0 ? q_quads : y0 + k_quads), heads = kind == 0 ? a.Hq : a.Hkv;
            int h = 4 * (y - y0) + (lane >> 3);
            uint16_t* packed = kind == 0 ? a.q_out + ((int64_t)t * a.Hq + h) * kHeadDim
                                         : kind == 1 && a.k_out ? a.k_out + ((int64_t)t * a.Hkv + h) * kHeadDim : nullptr;
            uint16_t* page = kind > 0 && id >= 0 ? (kind == 1 ? a.k_pages : a.v_pages) + paged::row_at(id, h, in_page, a.Hkv, a.shift) : nullptr;
            const uint16_t* weight = kind == 0 ? a.q_weight : kind == 1 ? a.k_weight : nullptr;
            uint4 w0, w1;
            if (weight) {
                w0 = reinterpret_cast<const uint4*>(weight)[p0];
                w1 = reinterpret_cast<const uint4*>(weight)[p1];
            }
#pragma unroll 1
            for (; y < stop; ++y, h += 4, packed += packed ? 4 * kHeadDim : 0, page += page ? (int64_t)(4 * kHeadDim) << a.shift : 0) {
                copy_wait<kAhead - 2>();
                const uint4 r0 = raw[read_at], r1 = raw[read_at + 32];
                read_at = read_at == (kAhead - 1) * 64 ? 0 : read_at + 64;
                uint32_t o[8] = {r0.x, r0.y, r0.z, r0.w, r1.x, r1.y, r1.z, r1.w};
                // The next copy goes into the place that was read a group ago: what came from there is in stores by now, or
                // nobody's.  What was read just now need not be in registers yet, and nothing orders a copy behind that.
                copy_next();
                if (skip) continue;
                if (kind < 2) {
                    uint64_t f[8];                // pairs of neighbours
#pragma unroll
                    for (int e = 0; e < 8; ++e) f[e] = attn2::f2(lo_of(o[e]), hi_of(o[e]));
                    if (weight) {
                        const float sum = sum_squares(f);
                        const float mean = fmaf(sum, 1.f / kHeadDim, a.eps);
                        float by = rsqrtf(mean);
                        const bool far = !(mean > 1e-30f && mean < 3e38f);
                        if (__any_sync(0xffffffffu, far)) {
                            // squares at the ends of fp32 or beyond: those heads once more, by 2^60 or 2^-80
                            const float to = mean < 1.f ? 0x1p60f : 0x1p-80f;
                            uint64_t g[8];
#pragma unroll
                            for (int e = 0; e < 8; ++e) g[e] = attn2::mul2(f[e], attn2::f2(to, to));
                            const float moved = sum_squares(g);
                            if (far) {
                                by = rsqrtf(fmaf(moved, 1.f / kHeadDim, a.eps * to * to));
#pragma unroll
                                for (int e = 0; e < 8; ++e) f[e] = g[e];
                            }
                        }
                        const uint32_t w[8] = {w0.x, w0.y, w0.z, w0.w, w1.x, w1.y, w1.z, w1.w};
                        const uint64_t by2 = attn2::f2(by, by);
#pragma unroll
                        for (int e = 0; e < 8; ++e)       // (w * by may leave fp32)
                            f[e] = attn2::mul2(attn2::mul2(f[e], by2), attn2::f2(lo_of(w[e]), hi_of(w[e])));
                    }
                    // (what is not turned does not meet its neighbour's infinities either)
                    if constexpr (kPairs2) {
#pragma unroll
                        for (int e = 0; e < 8; ++e) {
                            float x, z;
                            attn2::unf2(f[e], x, z);
                            const bool turned = kWhole || (e < 4 ? turned0 : turned1);
                            o[e] = turned ? pack2(x * turn[e].x - z * turn[e].y, z * turn[e].x + x * turn[e].y) : pack2(x, z);
                        }
                    } else {
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const float2 u = turn[2 * e], z = turn[2 * e + 1];
                            const uint64_t cs = attn2::f2(u.x, z.x), sn = attn2::f2(u.y, z.y), ns = attn2::f2(-u.y, -z.y);
                            const bool turned = kWhole || turned0;
                            o[e] = pack_pair(turned ? attn2::fma2(f[e], cs, attn2::mul2(f[4 + e], ns)) : f[e]);
                            o[4 + e] = pack_pair(turned ? attn2::fma2(f[4 + e], cs, attn2::mul2(f[e], sn)) : f[4 + e]);
                        }
                    }
                }
                if (h >= heads) continue;
                const uint4 o0 = make_uint4(o[0], o[1], o[2], o[3]), o1 = make_uint4(o[4], o[5], o[6], o[7]);
                if (packed) {
                    reinterpret_cast<uint4*>(packed)[p0] = o0;
                    reinterpret_cast<uint4*>(packed)[p1] = o1;
                }
                if (page) {
                    reinterpret_cast<uint4*>(page)[p0] = o0;
                    reinterpret_cast<uint4*>(page)[p1] = o1;
                }
            }
        }
    }
}

}  // namespace
}  // namespace eagle

using namespace eagle;

extern "C" eagle_status eagle_qkv_rope(const void* q, const void* k, const void* v, const void* q_weight,
                                       const void* k_weight, const float* inv_freq, const int32_t* cu,
                                       const int32_t* parent, const int32_t* pos, void* q_out, void* k_out,
                                       void* k_pages, void* v_pages, const int32_t* page_table, int T, int B,
                                       int n, int Hq, int Hkv, int head_dim, int rot_dim, int interleaved,
                                       float eps, int64_t q_stride, int64_t k_stride, int64_t v_stride, int N,
                                       int page, int P, int32_t* dev_status, eagle_stream_t stream) {
    const bool pages = k_pages || v_pages || page_table;
    if (T < 0 || B < 0 || Hq < 1 || Hkv < 1 || !(eps > 0.f) || !(eps <= 3.4e38f)) return EAGLE_ERR_INVALID_ARG;
    if (head_dim != kHeadDim || rot_dim < 16 || rot_dim > kHeadDim || rot_dim % 16 != 0 || Hq > 0xffff || Hkv > 0xffff)
        return EAGLE_ERR_SHAPE;
    if (q_stride < (int64_t)Hq * kHeadDim || k_stride < (int64_t)Hkv * kHeadDim || q_stride % 8 != 0 || k_stride % 8 != 0)
        return EAGLE_ERR_INVALID_ARG;
    if (pages) {
        if (N < 1 || P < 1 || v_stride < (int64_t)Hkv * kHeadDim || v_stride % 8 != 0) return EAGLE_ERR_INVALID_ARG;
        if (!paged::page_ok(page) || (int64_t)N * Hkv * page > paged::kMaxPool || (int64_t)P * page > paged::kMaxRows)
            return EAGLE_ERR_SHAPE;
    }
    if (T > 0x3fffffff) return EAGLE_ERR_SHAPE;         // 32-bit places
    if (B == 0 || T == 0) return EAGLE_OK;              // nothing read or written
    if (!q || !k || !inv_freq || !pos || !q_out || !cu == !parent) return EAGLE_ERR_INVALID_ARG;
    if (pages ? !(k_pages && v_pages && page_table && v) : !k_out) return EAGLE_ERR_INVALID_ARG;
    if (parent) {
        if (n < 1 || (int64_t)B * n != T) return EAGLE_ERR_INVALID_ARG;
        if (n > kMaxNodes) return EAGLE_ERR_SHAPE;
    }
    for (const void* p : {q, k, pages ? v : nullptr, q_weight, k_weight, (const void*)q_out, (const void*)k_out,
                          (const void*)k_pages, (const void*)v_pages})
        if (reinterpret_cast<uintptr_t>(p) & 15) return EAGLE_ERR_INVALID_ARG;
    RopeArgs a;
    a.q = static_cast<const uint16_t*>(q); a.k = static_cast<const uint16_t*>(k); a.v = static_cast<const uint16_t*>(v);
    a.q_weight = static_cast<const uint16_t*>(q_weight); a.k_weight = static_cast<const uint16_t*>(k_weight);
    a.inv_freq = inv_freq;
    a.cu = cu; a.parent = parent; a.pos = pos;
    a.q_out = static_cast<uint16_t*>(q_out); a.k_out = static_cast<uint16_t*>(k_out);
    a.k_pages = static_cast<uint16_t*>(k_pages); a.v_pages = static_cast<uint16_t*>(v_pages);
    a.page_table = page_table;
    a.T = T; a.B = B; a.n = n; a.Hq = Hq; a.Hkv = Hkv; a.half = rot_dim / 2;
    a.N = N; a.shift = pages ? paged::page_shift(page) : 0; a.P = P;
    a.eps = eps;
    a.q_stride = q_stride; a.k_stride = k_stride; a.v_stride = v_stride;
    a.dev_status = dev_status;
    const int sms = cached_sm_count();
    const bool is_long = T >= (int64_t)sms * kBlocksLong * kWarps * kLongTokens;
    const int64_t groups = ((Hq + 3) / 4 + (Hkv + 3) / 4 * (pages ? 2 : 1)) * (int64_t)T, most = (int64_t)sms * (is_long ? kBlocksLong : kBlocks);
    const int64_t need = (groups + kWarps - 1) / kWarps;
    const unsigned blocks = (unsigned)(need < most ? need : most);
    if (groups / (most * kWarps) > 0x3fffffff) return EAGLE_ERR_SHAPE;      // a warp counts its own
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    auto launch = [&](auto pairs2, auto whole) {
        constexpr auto kernel = qkv_rope_kernel<decltype(pairs2)::value, decltype(whole)::value>;
        if (!raise_smem_limit<kernel>(kRopeSmem)) return false;
        kernel<<<blocks, kWarps * 32, kRopeSmem, s>>>(a);
        return true;
    };
    const std::true_type yes;
    const std::false_type no;
    if (!(interleaved ? rot_dim == kHeadDim ? launch(yes, yes) : launch(yes, no) : rot_dim == kHeadDim ? launch(no, yes) : launch(no, no)))
        return EAGLE_ERR_CUDA;
    EAGLE_CHECK_LAUNCH();
    return EAGLE_OK;
}
