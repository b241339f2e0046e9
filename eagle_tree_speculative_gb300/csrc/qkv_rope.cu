// Norms of the queries' and keys' heads, the rotation by position, and the rows into the cache's
// pages: one pass over what a layer's projections left.
//
// Mathematics.  y = w x / sqrt(mean x^2 + eps) over a head's 128 elements, then pairs (y_i, y_j) turned by
// position * f_i.  The angle is needed modulo a turn, at positions where a product in fp32 has lost
// it: f_i / 2 pi as a 64-bit fraction of a turn, times the position in integer arithmetic, whose
// overflow is whole turns; the upper 32 bits are the angle to 2^-32 of a turn (its fraction was rounded
// to 2^-53 of itself: 2^-29 of a turn at position 2^24).
//
// Layout.  A task is a token, or a part of its heads where there are few tokens; a warp takes one at
// a time.  Eight lanes a head, four heads at once: a lane has two chunks of 8 elements (16 bytes)
// that hold both elements of its pairs, so nothing is exchanged for the rotation and three shuffles do the norm.
// The token's 64 angles are computed by the warp once, two a lane, and go through shared memory.
#include "paged_common.cuh"
#include "tc_common.cuh"

namespace eagle {
namespace {

constexpr int kWarps = 8;

struct RopeArgs {
    const uint16_t *q, *k, *v, *q_weight, *k_weight;
    const float* inv_freq;
    const int32_t *cu, *parent, *pos;
    uint16_t *q_out, *k_out, *k_pages, *v_pages;
    const int32_t* page_table;
    int T, B, n, Hq, Hkv, half;                   // half: rot_dim / 2 pairs
    int N, shift, P;
    int parts, quads;                             // tasks of a token, groups of four heads a task
    float eps;
    int64_t q_stride, k_stride, v_stride;
    int32_t* dev_status;
};

// Two bf16 of a word, as floats.
__device__ __forceinline__ float lo_of(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float hi_of(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

// The sum of squares of the eight lanes' 16 elements each.
__device__ __forceinline__ float sum_squares(const float (&x)[16], float by) {
    float s[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int e = 0; e < 16; ++e) {
        const float y = x[e] * by;
        s[e & 3] = fmaf(y, y, s[e & 3]);
    }
    float t = (s[0] + s[1]) + (s[2] + s[3]);
#pragma unroll
    for (int o = 4; o > 0; o >>= 1) t += __shfl_xor_sync(0xffffffffu, t, o);
    return t;
}

template <bool kPairs2>                           // pairs (2i, 2i + 1), else (i, i + rot_dim / 2)
__global__ void __launch_bounds__(kWarps * 32) qkv_rope_kernel(RopeArgs a) {
    __shared__ float2 s_turn[kWarps][64];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t task = (int64_t)blockIdx.x * kWarps + warp;
    const int t = (int)(task / a.parts), part = (int)(task - (int64_t)t * a.parts);
    if (t >= a.T) return;

    // ---- the token's sequence, its row there and its position ----
    int b = -1, row = 0, ahead = 0, rows = 0;
    if (a.parent) {
        b = t / a.n;
        row = t - b * a.n;
        rows = a.n;
        int depth[2];
        if (!paged::tree_depths(a.parent + (int64_t)b * a.n, a.n, depth)) {
            if (lane == 0) flag_error(a.dev_status, EAGLE_DEV_BAD_TREE);
            return;
        }
        const int d0 = __shfl_sync(0xffffffffu, depth[0], row & 31), d1 = __shfl_sync(0xffffffffu, depth[1], row & 31);
        ahead = row < 32 ? d0 : d1;
    } else {
        bool bad = false;
        for (int b0 = 0; b0 < a.B; b0 += 32) {
            const int i = min(b0 + lane, a.B - 1), c0 = a.cu[i], c1 = a.cu[i + 1];
            bad |= c0 < 0 || c1 < c0 || c1 > a.T;
            const unsigned in = __ballot_sync(0xffffffffu, c0 <= t && t < c1);
            if (b < 0 && in) {
                const int l = __ffs(in) - 1;
                b = b0 + l;
                const int first = __shfl_sync(0xffffffffu, c0, l);
                row = ahead = t - first;
                rows = __shfl_sync(0xffffffffu, c1, l) - first;
            }
        }
        if (__any_sync(0xffffffffu, bad)) {
            if (lane == 0) flag_error(a.dev_status, EAGLE_DEV_CAPACITY);
            return;
        }
        if (b < 0) return;                        // a token of no sequence
    }
    const int held = a.pos[b];
    const int64_t room = a.page_table ? (int64_t)a.P << a.shift : 0x7fffffffLL;
    if (held < 0 || held + (int64_t)rows > room) {
        if (lane == 0) flag_error(a.dev_status, EAGLE_DEV_CAPACITY);
        return;
    }
    int id = -1, in_page = 0;
    if (a.page_table) {
        const int at = held + row;
        id = a.page_table[(int64_t)b * a.P + (at >> a.shift)];
        in_page = at & ((1 << a.shift) - 1);
        if (id < 0 || id >= a.N) {
            if (lane == 0) flag_error(a.dev_status, EAGLE_DEV_CAPACITY);
            id = -1;
        }
    }

    // ---- the token's turns ----
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int i = lane + 32 * h;
        float2 turn = make_float2(1.f, 0.f);
        if (i < a.half) {
            const double f = (double)a.inv_freq[i] * 0.15915494309189533577;
            const unsigned long long frac = (unsigned long long)((f - floor(f)) * 18446744073709551616.0);
            const int angle = (int)((frac * (unsigned)(held + ahead)) >> 32);
            sincospif((float)angle * 0x1p-31f, &turn.y, &turn.x);
        }
        s_turn[warp][i] = turn;
    }
    __syncwarp();

    // ---- the lane's chunks, and its pairs' turns ----
    const int c = lane & 7;
    // pairs of halves: chunks c and c + half / 8; lanes without pairs share what lies behind rot_dim
    const bool pairs = c < (a.half >> 3);
    const int p0 = kPairs2 || pairs ? c : 2 * c, p1 = kPairs2 ? c + 8 : pairs ? c + (a.half >> 3) : 2 * c + 1;
    const bool turned0 = kPairs2 ? p0 < (a.half >> 2) : pairs, turned1 = kPairs2 ? p1 < (a.half >> 2) : pairs;
    float2 turn[8];
#pragma unroll
    for (int e = 0; e < 8; ++e)
        turn[e] = s_turn[warp][kPairs2 ? (e < 4 ? 4 * c + e : 32 + 4 * c + e - 4) : 8 * c + e];

    const int q_quads = (a.Hq + 3) >> 2, k_quads = (a.Hkv + 3) >> 2;
    const int total = q_quads + k_quads * (a.page_table ? 2 : 1);
    const int end = min(total, (part + 1) * a.quads);
    uint4 w0, w1;
    int kind = -1;
    for (int y = part * a.quads; y < end; ++y) {
        const int now = y < q_quads ? 0 : y < q_quads + k_quads ? 1 : 2;
        const int h = 4 * (y - (now > 0 ? q_quads : 0) - (now > 1 ? k_quads : 0)) + (lane >> 3);
        const bool on = h < (now == 0 ? a.Hq : a.Hkv);
        const uint16_t* src = now == 0 ? a.q + t * a.q_stride : now == 1 ? a.k + t * a.k_stride : a.v + t * a.v_stride;
        const uint4* x = reinterpret_cast<const uint4*>(src + (int64_t)(on ? h : 0) * kHeadDim);
        const uint4 r0 = x[p0], r1 = x[p1];
        if (now == 2) {
            if (on && id >= 0) {
                uint4* dst = reinterpret_cast<uint4*>(a.v_pages + paged::row_at(id, h, in_page, a.Hkv, a.shift));
                dst[p0] = r0;
                dst[p1] = r1;
            }
            continue;
        }
        const uint16_t* weight = now == 0 ? a.q_weight : a.k_weight;
        if (now != kind) {
            kind = now;
            if (weight) {
                w0 = reinterpret_cast<const uint4*>(weight)[p0];
                w1 = reinterpret_cast<const uint4*>(weight)[p1];
            }
        }
        const uint32_t in[8] = {r0.x, r0.y, r0.z, r0.w, r1.x, r1.y, r1.z, r1.w};
        float f[16];
#pragma unroll
        for (int e = 0; e < 8; ++e) { f[2 * e] = lo_of(in[e]); f[2 * e + 1] = hi_of(in[e]); }
        if (weight) {
            const float sum = sum_squares(f, 1.f);
            float r = rsqrtf(fmaf(sum, 1.f / kHeadDim, a.eps));
            if (__any_sync(0xffffffffu, !(sum < 3e38f))) {
                // squares beyond fp32: those heads once more, by 2^-80 (beside which eps is nothing)
                const float small = sum_squares(f, 0x1p-80f);
                if (!(sum < 3e38f)) {
                    r = rsqrtf(small * (1.f / kHeadDim));
#pragma unroll
                    for (int e = 0; e < 16; ++e) f[e] *= 0x1p-80f;
                }
            }
            const uint32_t w[8] = {w0.x, w0.y, w0.z, w0.w, w1.x, w1.y, w1.z, w1.w};
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                f[2 * e] *= r * lo_of(w[e]);
                f[2 * e + 1] *= r * hi_of(w[e]);
            }
        }
        uint32_t o[8];
        if constexpr (kPairs2) {
#pragma unroll
            for (int e = 0; e < 8; ++e)
                o[e] = pack2(f[2 * e] * turn[e].x - f[2 * e + 1] * turn[e].y, f[2 * e + 1] * turn[e].x + f[2 * e] * turn[e].y);
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float2 u = turn[2 * e], z = turn[2 * e + 1];
                o[e] = pack2(f[2 * e] * u.x - f[8 + 2 * e] * u.y, f[2 * e + 1] * z.x - f[9 + 2 * e] * z.y);
                o[4 + e] = pack2(f[8 + 2 * e] * u.x + f[2 * e] * u.y, f[9 + 2 * e] * z.x + f[2 * e + 1] * z.y);
            }
        }
        // what is not turned does not meet its neighbour's infinities either
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            if (!turned0) o[e] = pack2(f[2 * e], f[2 * e + 1]);
            if (!turned1) o[4 + e] = pack2(f[8 + 2 * e], f[9 + 2 * e]);
        }
        if (!on) continue;
        const uint4 o0 = make_uint4(o[0], o[1], o[2], o[3]), o1 = make_uint4(o[4], o[5], o[6], o[7]);
        uint16_t* packed = now == 0 ? a.q_out + ((int64_t)t * a.Hq + h) * kHeadDim
                                    : a.k_out ? a.k_out + ((int64_t)t * a.Hkv + h) * kHeadDim : nullptr;
        if (packed) {
            reinterpret_cast<uint4*>(packed)[p0] = o0;
            reinterpret_cast<uint4*>(packed)[p1] = o1;
        }
        if (now == 1 && id >= 0) {
            uint4* dst = reinterpret_cast<uint4*>(a.k_pages + paged::row_at(id, h, in_page, a.Hkv, a.shift));
            dst[p0] = o0;
            dst[p1] = o1;
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
    // few tokens: a token's heads are spread over as many warps as fill the device
    const int total = (Hq + 3) / 4 + (Hkv + 3) / 4 * (pages ? 2 : 1);
    const int64_t want = (int64_t)cached_sm_count() * 16 / T;
    a.parts = (int)(want < 1 ? 1 : want < total ? want : total);
    a.quads = (total + a.parts - 1) / a.parts;
    a.parts = (total + a.quads - 1) / a.quads;
    const int64_t blocks = ((int64_t)T * a.parts + kWarps - 1) / kWarps;
    if (blocks > 0x7fffffffLL) return EAGLE_ERR_SHAPE;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (interleaved) qkv_rope_kernel<true><<<(unsigned)blocks, kWarps * 32, 0, s>>>(a);
    else qkv_rope_kernel<false><<<(unsigned)blocks, kWarps * 32, 0, s>>>(a);
    EAGLE_CHECK_LAUNCH();
    return EAGLE_OK;
}
