// Tree attention over the 8-bit K/V cache on the tensor cores (tcgen05 kind::f8f6f4, TMEM, TMA).
//
// Digits.  The 8-bit MMA multiplies e4m3 by e4m3, and the cache's codes go into it as they lie in
// memory.  The other operand keeps bf16's precision as two e4m3 digits: x = hi + lo with hi the
// leading 4 bits of x's significand and lo the next 4.  Two passes over the 8-bit operand at twice
// the bf16 rate cost what one bf16 pass costs, without a conversion of K or V.
//   Q  per row times a power of two that brings its largest element to [128, 256): digits exact
//      for elements within 2^-9 of the largest, the rest to 2^-17 of it.
//   P  kept in [0, 256]: weights to 2^-8 of themselves (a bf16 P's rounding), or 2^-10 on that
//      scale for small ones, where the largest weight is at least 2^kOffset.
//   the tree's own rows (bf16, n <= 64): one 128-key tile with the hi digits in rows 0 .. 63 and
//      the lo digits in rows 64 .. 127, per-row powers of two; S of key j is S[j] + S[64 + j],
//      and both its rows get the same weight.
//
// Scales.  A block of 32 keys has K and V scales 2^ek and 2^ev.  2^ek joins the factor from S to
// the exponent.  2^ev joins the weight, P' = 2^(s + ev - m) with m the running maximum of s + ev:
// then O = sum P' code needs no scale, and l = sum P' 2^-ev is one factor per block.  m is the
// running maximum of what is multiplied with the codes, so P' uses e4m3's range whatever the
// blocks' scales are.
//
// Work.  A unit is one (sequence, kv head, pair of 128-row tiles), its keys in tiles of 128, the
// tree's tile last.  With two row tiles, each slot has one and both see every key tile; a
// single row tile (n G <= 128: decoding, small trees) has its key tiles dealt to the slots in
// turn, merged at the end, so that the tensor cores still have one slot's products to do during
// the other's softmax.  All tiles of all units are laid out in a row and cut into one equal
// piece per CTA (persistent, one per SM): ragged batches and few long sequences balance alike.
// A unit that is cut leaves partial (m, l, O) in the workspace, at most two per CTA; a second
// small kernel merges them.
//
// Roles: warp 0 loads K and V tiles (16 KB) through one ring, warp 1 issues the MMAs, warp 2 makes
// the K digits of the tree's rows and zeroes V rows behind the last key (whatever bits lie there:
// a zero weight does not cancel NaN), warp 3 cuts the work and makes the V digits, warps 4-11 are
// the softmax, which also makes the Q digits of the next unit before it writes this one's output.
#pragma once

#include "attn2_common.cuh"
#include "kv8_common.cuh"

namespace eagle {
namespace kv8_tc {

using attn2::kKeys;
using attn2::kRows;
using attn2::kSlots;
using kv8::kKv8Block;

constexpr int kStages = 7;
constexpr int kTile = 128 * 128;                  // 16 KB: a K or V tile, a digit plane of Q
constexpr int kInfo = 3;                          // units in flight between the roles
constexpr int kBlocks = kKeys / kKv8Block;        // scales per tile
constexpr float kOffset = 6.f, kRescale = 2.f;    // weights up to 2^(6 + 2) <= 448
constexpr int kMaxVExp = 44;                      // V scales up to 2^44, see below
constexpr int kMinTiles = 3;                      // a CTA's piece is at least so many tiles

struct Args {
    const uint16_t* q;
    const float* k_scale;
    const float* v_scale;
    const uint16_t* k_tree;
    const uint16_t* v_tree;
    const int32_t* kv_len;
    const int32_t* parent;
    uint16_t* out;
    float* ws_o;                                  // [grid][2][rows][128]
    float2* ws_ml;                                // [grid][2][rows]
    int B, n, Hq, Hkv, G, Lmax, NB;
    int rows;                                     // n G, at most 2 kRows of a unit are counted
    float scale_log2;
    int32_t* dev_status;
};

// ---------------- the cut: shared by the attention and the merging kernel ----------------
// Positions: sequence by sequence, head by head, row-tile pair by pair, tile by tile; a tile of a
// pair counts 2, of a single row tile 1.
struct Cut {
    int64_t total;                                // positions
    int ctas;                                     // pieces
    __device__ int64_t begin(int c) const { return total / ctas * c + total % ctas * c / ctas; }
};
__device__ __forceinline__ int tiles_of(const Args& a, int b) {
    const int L = a.kv_len[b];
    return (L < 0 || L > a.Lmax) ? 1 : (L + kKeys - 1) / kKeys + 1;
}
__device__ __forceinline__ int row_tiles(const Args& a) { return (a.n * a.G + kRows - 1) / kRows; }

// Warp-wide.
__device__ __forceinline__ Cut make_cut(const Args& a, int grid) {
    int64_t sum = 0;
    for (int b = threadIdx.x & 31; b < a.B; b += 32) sum += tiles_of(a, b);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    Cut c;
    const int rt = row_tiles(a);
    c.total = sum * rt * a.Hkv;
    const int64_t most = c.total / (kMinTiles * min(rt, 2));
    c.ctas = (int)max((int64_t)1, min((int64_t)grid, most));
    return c;
}

// A unit and the tiles of it that lie in [pos, end).
struct Segment {
    int b, head, pair, T;                         // T tiles in all, the last one the tree's
    int weight;                                   // row tiles of the pair
    int64_t start;                                // position of its first tile
    int t0, t1;
};
// Warp-wide: the unit at position pos; `b`, `base`: a sequence at or before it and its first
// position, moved on.
__device__ __forceinline__ Segment segment_at(const Args& a, int64_t pos, int64_t end, int& b, int64_t& base) {
    const int rt = row_tiles(a), lane = threadIdx.x & 31;
    for (;;) {                                    // 32 sequences at a time; the last one holds what is left
        const int mine = b + lane;
        const int64_t w = mine < a.B ? (int64_t)tiles_of(a, mine) * rt * a.Hkv : 0;
        int64_t sum = w;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t y = __shfl_up_sync(0xffffffffu, sum, o);
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
    s.T = tiles_of(a, b);
    int64_t off = pos - base;
    const int64_t per_head = (int64_t)s.T * rt;
    s.head = (int)(off / per_head);
    off -= s.head * per_head;
    s.pair = (int)(off / (2 * s.T));
    off -= (int64_t)s.pair * 2 * s.T;
    s.weight = min(2, rt - 2 * s.pair);
    s.start = pos - off;
    s.t0 = (int)((off + s.weight - 1) / s.weight);
    s.t1 = (int)min((int64_t)s.T, (end - s.start + s.weight - 1) / s.weight);
    return s;
}

// ---------------- the attention kernel ----------------
struct Unit {
    int b, head, pair;
    int t0, n;                                    // first tile, number of tiles (0: write zeros)
    int tree;                                     // the last of them is the tree's
    int L;
    int split_keys;                               // one row tile: its key tiles alternate between the slots
    int part;                                     // -1: whole, else the partial's place
    int pad;
    unsigned long long anc[kMaxNodes];            // node i and its ancestors
};

struct Shared {
    uint64_t full[kStages], empty[kStages], v_last[kStages];
    uint64_t q_full[kSlots], s_full[kSlots], p_full[kSlots], o_full[kSlots];
    uint64_t tree_full, tree_empty, merge_in, merge_out;
    uint64_t info_full[kInfo], info_empty[kInfo];
    uint64_t drain;
    uint32_t tmem;
    int abort_flag;
    float2 ml[kSlots][kRows];
    float k_fac[kMaxNodes];                       // of the tree's rows: 2^ek
    float v_exp[kMaxNodes];                       // ev
    Unit info[kInfo];
};

constexpr int kSmem = kSlots * 2 * kTile + 2 * kTile + kStages * kTile + (int)sizeof(Shared) + 1024;
static_assert(kSmem <= 232448, "shared memory of a CTA");

// tcgen05.mma kind::f8f6f4, A and B e4m3 (format 0), D fp32.
__host__ __device__ constexpr uint32_t idesc_e4m3(int M, int N, int b_mn_major) {
    return (1u << 4) | ((uint32_t)b_mn_major << 16) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}
constexpr uint32_t kIdescQK = idesc_e4m3(128, kKeys, 0);
constexpr uint32_t kIdescPV = idesc_e4m3(128, kHeadDim, 1);

__device__ __forceinline__ void umma_f8(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                        uint32_t accumulate) {
    asm volatile(
        "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
        " tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n}\n" ::"r"(d_tmem),
        "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
        : "memory");
}
__device__ __forceinline__ void umma_f8_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t bdesc, uint32_t idesc,
                                           uint32_t accumulate) {
    asm volatile(
        "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
        " tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], [%1], %2, %3, p;\n}\n" ::"r"(d_tmem),
        "r"(a_tmem), "l"(bdesc), "r"(idesc), "r"(accumulate)
        : "memory");
}

// The leading digit of x: its significand cut to 4 bits, a value that e4m3 holds exactly (for
// |x| in [2^-6, 448]; smaller ones are rounded to its 2^-9 grid when they are converted).
__device__ __forceinline__ float lead(float x) { return __uint_as_float(__float_as_uint(x) & 0xfff00000u); }

// Exponent e that brings a row with the given largest magnitude to [128, 256), within [lo, 120].
__device__ __forceinline__ int digit_exp(float amax, int lo) {
    const int E = (int)(__float_as_uint(amax) >> 23) - 127;
    return amax > 0.f ? min(max(E - 7, lo), 120) : lo;
}

// Byte offset of (row, column byte) in a tile of 128-byte rows with the 128-byte swizzle.
__device__ __forceinline__ int swz(int row, int byte) { return row * 128 + ((((byte >> 4) ^ (row & 7)) << 4) | (byte & 15)); }

// Digits of 8 bf16 elements (x * by): hi and lo, 4 codes a word.
__device__ __forceinline__ void digits8(const uint4& x, float by, uint32_t (&hi)[2], uint32_t (&lo)[2]) {
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        float f[4], h[4];
#pragma unroll
        for (int c = 0; c < 2; ++c) {
            f[2 * c] = __uint_as_float(w[2 * i + c] << 16) * by;
            f[2 * c + 1] = __uint_as_float(w[2 * i + c] & 0xffff0000u) * by;
        }
#pragma unroll
        for (int c = 0; c < 4; ++c) h[c] = lead(f[c]);
        hi[i] = kv8::e4m3x4(h[0], h[1], h[2], h[3]);
        lo[i] = kv8::e4m3x4(f[0] - h[0], f[1] - h[1], f[2] - h[2], f[3] - h[3]);
    }
}
__device__ __forceinline__ float amax8(const uint4& x) {
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
    uint32_t m = 0u;
#pragma unroll
    for (int i = 0; i < 4; ++i) m = max(m, max(w[i] & 0x7fffu, (w[i] >> 16) & 0x7fffu));
    return __uint_as_float(m << 16);
}

// Warp-wide: the digits of the tree's rows of one head into a tile (rows 0 .. 63 hi, 64 .. 127 lo;
// rows from n on zero), sixteen lanes a row.  Returns the OR of status bits.
template <class Put>
__device__ __forceinline__ int tree_digits(const uint16_t* x, int64_t stride, int n, uint8_t* tile, int lo_exp,
                                           int max_exp, Put put) {
    const int lane = threadIdx.x & 31, half = lane >> 4, c = lane & 15;
    int bits = 0;
    for (int r0 = 0; r0 < kMaxNodes; r0 += 8) {
        uint4 v[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int r = r0 + 2 * i + half;
            v[i] = r < n ? __ldg(reinterpret_cast<const uint4*>(x + r * stride) + c) : make_uint4(0u, 0u, 0u, 0u);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int r = r0 + 2 * i + half;
            float m = amax8(v[i]);
#pragma unroll
            for (int o = 8; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
            const int e = digit_exp(m, lo_exp);
            if (e > max_exp) bits = EAGLE_DEV_NONFINITE;
            uint32_t hi[2], lo[2];
            digits8(v[i], kv8::exp2i(-e), hi, lo);
            *reinterpret_cast<uint2*>(tile + swz(r, 8 * c)) = make_uint2(hi[0], hi[1]);
            *reinterpret_cast<uint2*>(tile + swz(kMaxNodes + r, 8 * c)) = make_uint2(lo[0], lo[1]);
            if (c == 0) put(r, e);
        }
    }
    return bits;
}

__global__ void __launch_bounds__(attn2::kThreads, 1)
tree_attn_kv8_kernel(const __grid_constant__ CUtensorMap map_k, const __grid_constant__ CUtensorMap map_v, Args a) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                               ~static_cast<uintptr_t>(1023));
    uint8_t* sQ = smem;                                   // [slot][hi, lo][16 KB]
    uint8_t* sT = sQ + kSlots * 2 * kTile;                // the tree's K tile, V tile
    uint8_t* sR = sT + 2 * kTile;                         // [kStages][16 KB]
    Shared* sh = reinterpret_cast<Shared*>(sR + kStages * kTile);
    volatile int* abort_flag = &sh->abort_flag;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

    if (tid == 0) {
        for (int i = 0; i < kStages; ++i) {
            mbar_init(s32(&sh->full[i]), 1);
            mbar_init(s32(&sh->empty[i]), 1);
            mbar_init(s32(&sh->v_last[i]), 1);
        }
        for (int s = 0; s < kSlots; ++s) {
            mbar_init(s32(&sh->q_full[s]), 4);
            mbar_init(s32(&sh->s_full[s]), 1);
            mbar_init(s32(&sh->p_full[s]), 4);
            mbar_init(s32(&sh->o_full[s]), 1);
        }
        mbar_init(s32(&sh->tree_full), 2);
        mbar_init(s32(&sh->tree_empty), 1);
        mbar_init(s32(&sh->merge_in), 8);
        mbar_init(s32(&sh->merge_out), 8);
        // read by the loader, the MMA thread, warp 2 and the eight softmax warps
        for (int i = 0; i < kInfo; ++i) { mbar_init(s32(&sh->info_full[i]), 1); mbar_init(s32(&sh->info_empty[i]), 11); }
        mbar_init(s32(&sh->drain), 1);
        sh->abort_flag = 0;
        asm volatile("fence.mbarrier_init.release.cluster;\n" ::: "memory");
    }
    if (warp == 1) tmem_alloc(s32(&sh->tmem), attn2::kTmemCols);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = sh->tmem;

    // the i-th unit of this CTA; nullptr at the end (or on abort)
    auto next_unit = [&](int i) -> const Unit* {
        if (!mbar_wait(s32(&sh->info_full[i % kInfo]), ((uint32_t)i / kInfo) & 1u, abort_flag)) return nullptr;
        const Unit* u = &sh->info[i % kInfo];
        return u->head >= 0 ? u : nullptr;
    };
    auto unit_read = [&](int i) { mbar_arrive(s32(&sh->info_empty[i % kInfo])); };

    if (warp < 4) {
        attn2::regs_dec<attn2::kRegsRole>();
        if (warp == 0 && lane == 0) {
            // ---------------- loads ----------------
            uint32_t r = 0;
            bool ok = true;
            for (int i = 0; ok; ++i) {
                const Unit* up = next_unit(i);
                if (!up) break;
                const int t0 = up->t0, nc = up->n - up->tree, z = up->b * a.Hkv + up->head, L = up->L;
                unit_read(i);
                for (int j = 0; ok && j < nc; ++j) {
                    const int key0 = (t0 + j) * kKeys;
                    for (int v = 0; v < 2; ++v, ++r) {
                        const int st = r % kStages;
                        ok = ok && mbar_wait(s32(&sh->empty[st]), ((r / kStages) & 1u) ^ 1u, abort_flag);
                        if (!ok) break;
                        // a V tile with rows behind the last key goes through warp 2 first
                        const uint32_t bar = s32(v && key0 + kKeys > L ? &sh->v_last[st] : &sh->full[st]);
                        mbar_expect_tx(bar, kTile);
                        tma_load_3d(s32(sR + st * kTile), v ? &map_v : &map_k, bar, 0, key0, z);
                    }
                }
            }
        } else if (warp == 1 && lane == 0) {
            // ---------------- MMA issue ----------------
            const uint64_t dq0 = sw128_desc(s32(sQ)), dk0 = sw128_desc(s32(sR)), dkt = sw128_desc(s32(sT));
            const uint64_t dv0 = sw128_desc_mn(s32(sR), kTile, 1024), dvt = sw128_desc_mn(s32(sT + kTile), kTile, 1024);
            uint32_t r = 0, trees = 0, nqs[kSlots] = {0, 0}, nps[kSlots] = {0, 0};
            bool ok = true;
            auto wait = [&](uint64_t* bar, uint32_t parity) {
                ok = ok && mbar_wait(s32(bar), parity & 1u, abort_flag);
                if (ok) tc_fence_after();
                return ok;
            };
            for (int i = 0; ok; ++i) {
                const Unit* up = next_unit(i);
                if (!up) break;
                const int n = up->n, tree = up->tree, nc = n - tree;
                const bool alt = up->split_keys != 0;
                unit_read(i);
                bool q_there[kSlots] = {false, false};
                // S of slot s = Q K(t)^T, both digits of Q
                auto qk = [&](int s, int t) {
                    if (!q_there[s]) {
                        if (!wait(&sh->q_full[s], nqs[s]++)) return;
                        q_there[s] = true;
                    }
                    const uint32_t use = r + 2 * t;
                    if (t < nc ? !wait(&sh->full[use % kStages], use / kStages) : !wait(&sh->tree_full, trees)) return;
                    const uint64_t dk = t < nc ? dk0 + (uint64_t)(((use % kStages) * kTile) >> 4) : dkt;
#pragma unroll
                    for (int d = 0; d < 2; ++d) {
                        const uint64_t dq = dq0 + (uint64_t)(((2 * s + d) * kTile) >> 4);
#pragma unroll
                        for (int k = 0; k < kHeadDim / 32; ++k)
                            umma_f8(tmem + attn2::s_col(s), dq + 2 * k, dk + 2 * k, kIdescQK, (d | k) ? 1u : 0u);
                    }
                    umma_commit(s32(&sh->s_full[s]));
                };
                // O of slot s += P V(t), both digits of P
                auto pv = [&](int s, int t, bool first, bool last) {
                    const uint32_t use = r + 2 * t + 1;
                    if (t < nc && !wait(&sh->full[use % kStages], use / kStages)) return;
                    if (!wait(&sh->p_full[s], nps[s]++)) return;
                    const uint64_t dv = t < nc ? dv0 + (uint64_t)(((use % kStages) * kTile) >> 4) : dvt;
#pragma unroll
                    for (int d = 0; d < 2; ++d)
#pragma unroll
                        for (int k = 0; k < kKeys / 32; ++k)
                            umma_f8_ts(tmem + attn2::o_col(s), tmem + attn2::s_col(s) + 32 * d + 8 * k,
                                       dv + (uint64_t)((k * 32 * 128) >> 4), kIdescPV, (!first || d || k) ? 1u : 0u);
                    if (last) umma_commit(s32(&sh->o_full[s]));
                };
                auto k_done = [&](int t) { if (t < nc) umma_commit(s32(&sh->empty[(r + 2 * t) % kStages])); };
                auto v_done = [&](int t) {
                    umma_commit(s32(t < nc ? &sh->empty[(r + 2 * t + 1) % kStages] : &sh->tree_empty));
                };
                if (alt) {                                // tile t is slot t & 1's
                    for (int t = 0; ok && t < n + 2; ++t) {
                        if (t >= 2) {
                            pv(t & 1, t - 2, t < 4, t >= n);
                            if (ok) v_done(t - 2);
                        }
                        if (ok && t < n) {
                            qk(t & 1, t);
                            if (ok) k_done(t);
                        }
                    }
                } else {
                    for (int t = 0; ok && t <= n; ++t) {
                        for (int s = 0; ok && s < kSlots; ++s) {
                            if (t > 0) pv(s, t - 1, t == 1, t == n);
                            if (ok && t < n) qk(s, t);
                        }
                        if (ok && t > 0) v_done(t - 1);
                        if (ok && t < n) k_done(t);
                    }
                }
                r += 2 * nc;
                trees += tree;
            }
            umma_commit(s32(&sh->drain));
            mbar_wait(s32(&sh->drain), 0u, abort_flag, /*honour_abort=*/false);
        } else if (warp == 2) {
            // ---------------- K digits of the tree's rows; V rows behind the last key ----------------
            uint32_t r = 0, phases = 0, trees = 0;
            int bits = 0;
            for (int i = 0;; ++i) {
                const Unit* up = next_unit(i);
                if (!__all_sync(0xffffffffu, up != nullptr)) break;
                const int b = up->b, head = up->head, t0 = up->t0, nc = up->n - up->tree, tree = up->tree, L = up->L;
                __syncwarp();
                if (lane == 0) unit_read(i);
                if (tree) {
                    const bool got = mbar_wait(s32(&sh->tree_empty), (trees++ & 1u) ^ 1u, abort_flag);
                    if (!__all_sync(0xffffffffu, got)) break;
                    bits |= tree_digits(a.k_tree + ((int64_t)b * a.n * a.Hkv + head) * kHeadDim, (int64_t)a.Hkv * kHeadDim,
                                        a.n, sT, -40, 120, [&](int row, int e) { sh->k_fac[row] = kv8::exp2i(e); });
                    attn2::fence_async_shared();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(s32(&sh->tree_full));
                }
                r += 2 * nc;
                if (nc > 0 && (t0 + nc) * kKeys > L) {
                    const uint32_t st = (r - 1) % kStages;
                    const bool got = mbar_wait(s32(&sh->v_last[st]), (phases >> st) & 1u, abort_flag);
                    phases ^= 1u << st;
                    if (!__all_sync(0xffffffffu, got)) break;
                    uint8_t* v = sR + st * kTile;
                    for (int row = L - (t0 + nc - 1) * kKeys + (lane >> 3); row < kKeys; row += 4)
                        *reinterpret_cast<uint4*>(v + row * 128 + (lane & 7) * 16) = make_uint4(0u, 0u, 0u, 0u);
                    attn2::fence_async_shared();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(s32(&sh->full[st]));
                }
            }
            if (bits) flag_error(a.dev_status, bits);
        } else if (warp == 3) {
            // ---------------- the cut; V digits of the tree's rows ----------------
            const Cut cut = make_cut(a, gridDim.x);
            const bool mine = (int)blockIdx.x < cut.ctas;
            int64_t pos = mine ? cut.begin(blockIdx.x) : 0, base = 0;
            const int64_t end = mine ? cut.begin(blockIdx.x + 1) : 0;
            int b = 0, anc_of = -1, bits = 0;
            uint32_t trees = 0;
            unsigned long long anc[2] = {0, 0};           // of nodes lane and lane + 32
            bool bad_tree = false;
            // publishes the next unit as entry i; 0: stop, 1: published (head -1: there is none)
            auto publish = [&](int i, int& tree_b, int& tree_head) {
                Segment s;
                bool have = false;
                while (!have && pos < end) {
                    s = segment_at(a, pos, end, b, base);
                    pos = s.start + (int64_t)s.weight * s.T;
                    have = s.t0 < s.t1;
                }
                const bool got = mbar_wait(s32(&sh->info_empty[i % kInfo]), (((uint32_t)i / kInfo) & 1u) ^ 1u, abort_flag);
                if (!__all_sync(0xffffffffu, got)) return false;
                Unit* u = &sh->info[i % kInfo];
                tree_head = -1;
                if (!have) {
                    if (lane == 0) u->head = -1;
                } else {
                    if (s.b != anc_of) {
                        // anc: each round doubles how far up a node's set reaches
                        anc_of = s.b;
                        int p[2];
                        bool bad = false;
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            const int i2 = lane + 32 * h;
                            p[h] = i2 < a.n ? a.parent[(int64_t)s.b * a.n + i2] : -1;
                            if (i2 < a.n && (i2 == 0 ? p[h] != -1 : (p[h] < 0 || p[h] >= i2))) bad = true;
                            anc[h] = 1ull << i2;
                        }
                        bad_tree = __any_sync(0xffffffffu, bad);
                        for (int round = 0; !bad_tree && round < 6; ++round) {
                            unsigned long long add[2];
                            int up[2];
#pragma unroll
                            for (int h = 0; h < 2; ++h) {
                                const int src = p[h] < 0 ? 0 : p[h];
                                const unsigned long long x0 = __shfl_sync(0xffffffffu, anc[0], src & 31);
                                const unsigned long long x1 = __shfl_sync(0xffffffffu, anc[1], src & 31);
                                const int y0 = __shfl_sync(0xffffffffu, p[0], src & 31);
                                const int y1 = __shfl_sync(0xffffffffu, p[1], src & 31);
                                add[h] = p[h] < 0 ? 0ull : (src < 32 ? x0 : x1);
                                up[h] = p[h] < 0 ? -1 : (src < 32 ? y0 : y1);
                            }
#pragma unroll
                            for (int h = 0; h < 2; ++h) { anc[h] |= add[h]; p[h] = up[h]; }
                        }
                    }
                    const int L = a.kv_len[s.b];
                    const bool bad_len = L < 0 || L > a.Lmax;
                    if ((bad_len || bad_tree) && s.head == 0 && s.pair == 0 && s.t0 == 0)
                        bits |= (bad_len ? EAGLE_DEV_CAPACITY : 0) | (bad_tree ? EAGLE_DEV_BAD_TREE : 0);
                    const bool zero = bad_len || bad_tree;
                    u->anc[lane] = anc[0];
                    u->anc[lane + 32] = anc[1];
                    if (lane == 0) {
                        u->b = s.b; u->head = s.head; u->pair = s.pair;
                        u->t0 = s.t0;
                        u->n = zero ? 0 : s.t1 - s.t0;
                        u->tree = !zero && s.t1 == s.T;
                        u->L = zero ? 0 : L;
                        u->split_keys = s.weight == 1;
                        u->part = s.t0 == 0 && s.t1 == s.T ? -1 : (int)blockIdx.x * 2 + (s.t0 == 0);
                    }
                    if (!zero && s.t1 == s.T) { tree_b = s.b; tree_head = s.head; }
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(s32(&sh->info_full[i % kInfo]));
                return have;
            };
            int tb = 0, th = -1;
            bool more = publish(0, tb, th);
            for (int i = 1; more; ++i) {                  // one unit ahead of the digits
                int tb1 = 0, th1 = -1;
                const bool next = publish(i, tb1, th1);
                if (th >= 0) {
                    const bool got = mbar_wait(s32(&sh->tree_empty), (trees++ & 1u) ^ 1u, abort_flag);
                    if (!__all_sync(0xffffffffu, got)) break;
                    bits |= tree_digits(a.v_tree + ((int64_t)tb * a.n * a.Hkv + th) * kHeadDim, (int64_t)a.Hkv * kHeadDim,
                                        a.n, sT + kTile, kv8::kMinExp, kMaxVExp,
                                        [&](int row, int e) { sh->v_exp[row] = (float)e; });
                    attn2::fence_async_shared();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(s32(&sh->tree_full));
                }
                more = next;
                tb = tb1;
                th = th1;
            }
            if (bits) flag_error(a.dev_status, bits);
        }
    } else {
        // ---------------- softmax: one thread per query row ----------------
        attn2::regs_inc<attn2::kRegsSoftmax>();
        const int slot = (warp - 4) >> 2;
        const int row = (warp & 3) * 32 + lane;
        const uint32_t lane_base = (uint32_t)((warp & 3) * 32) << 16;
        const uint32_t s_addr = tmem + lane_base + attn2::s_col(slot);
        const uint32_t o_addr = tmem + lane_base + attn2::o_col(slot);
        uint32_t tiles_done = 0, units_done = 0, merges = 0, trees = 0;
        int bits = 0;

        struct Row {                                      // this thread's row of a unit
            int b, head, pair, t0, n, tree, L, alt, part;
            int r;                                        // row of the (sequence, head), node * G + g; -1: nobody's
            unsigned long long anc;
            float sc;                                     // S to log2 units, without the key's scale
        };
        // the i-th unit, its Q digits written; false at the end
        auto begin_unit = [&](int i, Row& w) {
            const Unit* up = next_unit(i);
            if (!__all_sync(0xffffffffu, up != nullptr)) return false;
            w.b = up->b; w.head = up->head; w.pair = up->pair; w.t0 = up->t0; w.n = up->n; w.tree = up->tree;
            w.L = up->L; w.alt = up->split_keys; w.part = up->part;
            const int r = w.pair * 2 * kRows + (w.alt ? 0 : slot * kRows) + row;
            w.r = r < a.n * a.G ? r : -1;
            const int node = w.r < 0 ? 0 : r / a.G;
            w.anc = up->anc[node];
            __syncwarp();
            if (lane == 0) unit_read(i);
            // a slot without a tile leaves Q (and its barrier) alone: it could be units ahead
            if (w.n <= (w.alt ? slot : 0)) return true;
            uint4 q[16];
            if (w.r >= 0) {
                const uint4* src = reinterpret_cast<const uint4*>(
                    a.q + (((int64_t)w.b * a.n + node) * a.Hq + w.head * a.G + r % a.G) * kHeadDim);
#pragma unroll
                for (int c = 0; c < 16; ++c) q[c] = __ldg(src + c);
            } else {
#pragma unroll
                for (int c = 0; c < 16; ++c) q[c] = make_uint4(0u, 0u, 0u, 0u);
            }
            float m = 0.f;
#pragma unroll
            for (int c = 0; c < 16; ++c) m = fmaxf(m, amax8(q[c]));
            const int e = digit_exp(m, -40);
            w.sc = a.scale_log2 * kv8::exp2i(e);
            const float by = kv8::exp2i(-e);
            // every QK of this slot's last unit has completed (its S was read): Q may be replaced
            uint8_t* dst = sQ + slot * 2 * kTile;
#pragma unroll
            for (int c = 0; c < 8; ++c) {
                uint32_t h0[2], l0[2], h1[2], l1[2];
                digits8(q[2 * c], by, h0, l0);
                digits8(q[2 * c + 1], by, h1, l1);
                *reinterpret_cast<uint4*>(dst + swz(row, 16 * c)) = make_uint4(h0[0], h0[1], h1[0], h1[1]);
                *reinterpret_cast<uint4*>(dst + kTile + swz(row, 16 * c)) = make_uint4(l0[0], l0[1], l1[0], l1[1]);
            }
            attn2::fence_async_shared();
            __syncwarp();
            if (lane == 0) mbar_arrive(s32(&sh->q_full[slot]));
            return true;
        };

        Row w;
        bool have = begin_unit(0, w), ok = true;
        for (int i = 0; have; ++i) {
            const bool idle = !__any_sync(0xffffffffu, w.r >= 0);        // rows are independent: leave P as it is
            const int64_t sc_at = ((int64_t)w.b * a.Hkv + w.head) * a.NB;
            const int nc = w.n - w.tree, step = w.alt ? 2 : 1;
            float mref = -INFINITY;
            uint64_t l2 = 0;                                             // two partial sums
            float ks[kBlocks], vs[kBlocks];
            // scales of blocks with a key before L; others have no key and are not read
            auto load_scales = [&](int t) {
#pragma unroll
                for (int c = 0; c < kBlocks; ++c) {
                    const int blk = (w.t0 + t) * kBlocks + c;
                    const bool there = t < nc && blk * kKv8Block < w.L;
                    ks[c] = there ? __ldg(a.k_scale + sc_at + blk) : 1.f;
                    vs[c] = there ? __ldg(a.v_scale + sc_at + blk) : 1.f;
                }
            };
            const int first = w.alt ? slot : 0;
            int mine = 0;                                                // tiles of this slot
            load_scales(first);
            for (int t = first; t < w.n; t += step, ++mine) {
                const bool got = mbar_wait(s32(&sh->s_full[slot]), tiles_done & 1u, abort_flag);
                if (!__all_sync(0xffffffffu, got)) { ok = false; break; }
                ++tiles_done;
                tc_fence_after();
                if (!idle) {
                    float x[kKeys];
                    attn2::load_row(s_addr, x);
                    uint32_t hi[32], lo[32];
                    float mx, alpha = 1.f;
                    auto raise = [&]() {                                 // the reference maximum, if mx is far above it
                        if (mx > mref + kRescale || (mref == -INFINITY && mx > -INFINITY)) {
                            alpha = exp2f(mref - mx);                    // 0 for the first maximum
                            mref = mx;
                            l2 = attn2::mul2(l2, attn2::f2(alpha, alpha));
                        }
                        // the commit behind this QK covers every PV before it: O is complete
                        if (mine > 0 && __any_sync(0xffffffffu, alpha != 1.f)) attn2::rescale_row(o_addr, alpha);
                    };
                    if (t < nc) {
                        const int left = w.L - (w.t0 + t) * kKeys;
                        if (left < kKeys) {
#pragma unroll
                            for (int c = 0; c < kKeys; ++c) x[c] = c < left ? x[c] : -INFINITY;
                        }
                        float f[kBlocks], ev[kBlocks], inv[kBlocks];
#pragma unroll
                        for (int c = 0; c < kBlocks; ++c) {
                            f[c] = fmaxf(ks[c] * w.sc, 1.17549435e-38f); // above 0: a masked block stays -inf
                            const int e = (int)(__float_as_uint(vs[c]) >> 23) - 127;
                            if (e > kMaxVExp) bits = EAGLE_DEV_NONFINITE;
                            ev[c] = (float)e;
                            inv[c] = kv8::exp2i(min(-e, 127));
                        }
                        load_scales(t + step);
                        float mb[kBlocks];
#pragma unroll
                        for (int c = 0; c < kBlocks; ++c) mb[c] = fmaf(attn2::max_of<kKv8Block>(x + kKv8Block * c), f[c], ev[c]);
                        mx = fmaxf(attn2::max3(mb[0], mb[1], mb[2]), mb[3]);
                        raise();
#pragma unroll
                        for (int c = 0; c < kBlocks; ++c) {
                            const float off = ev[c] - mref + kOffset;
                            const uint64_t f_2 = attn2::f2(f[c], f[c]), off2 = attn2::f2(off, off);
                            uint64_t acc[2] = {0, 0};
#pragma unroll
                            for (int d = 0; d < 8; ++d) {
                                float p[4], h[4];
#pragma unroll
                                for (int y = 0; y < 2; ++y) {
                                    const int at = 32 * c + 4 * d + 2 * y;
                                    float s0, s1;
                                    attn2::unf2(attn2::fma2(attn2::f2(x[at], x[at + 1]), f_2, off2), s0, s1);
                                    p[2 * y] = ex2_approx(s0);
                                    p[2 * y + 1] = ex2_approx(s1);
                                    acc[y] = attn2::add2(acc[y], attn2::f2(p[2 * y], p[2 * y + 1]));
                                }
#pragma unroll
                                for (int y = 0; y < 4; ++y) h[y] = lead(p[y]);
                                hi[8 * c + d] = kv8::e4m3x4(h[0], h[1], h[2], h[3]);
                                lo[8 * c + d] = kv8::e4m3x4(p[0] - h[0], p[1] - h[1], p[2] - h[2], p[3] - h[3]);
                            }
                            l2 = attn2::fma2(attn2::add2(acc[0], acc[1]), attn2::f2(inv[c], inv[c]), l2);
                        }
                    } else {
                        // the tree's tile: key j's score is the sum of its digits' columns
                        // its factors are there: the MMA thread has seen this barrier, now this one does
                        const bool seen = mbar_wait(s32(&sh->tree_full), trees & 1u, abort_flag);
                        if (!__all_sync(0xffffffffu, seen)) { ok = false; break; }
                        mx = -INFINITY;
#pragma unroll
                        for (int j = 0; j < kMaxNodes; ++j) {
                            const float f = fmaxf(sh->k_fac[j] * w.sc, 1.17549435e-38f);
                            const bool sees = (w.anc >> j) & 1ull;
                            x[j] = sees ? fmaf(x[j] + x[kMaxNodes + j], f, sh->v_exp[j]) : -INFINITY;
                            mx = fmaxf(mx, x[j]);
                        }
                        raise();
                        float sum = 0.f;
#pragma unroll
                        for (int d = 0; d < 16; ++d) {
                            float p[4], h[4];
#pragma unroll
                            for (int y = 0; y < 4; ++y) {
                                const int j = 4 * d + y;
                                p[y] = ex2_approx(x[j] - mref + kOffset);
                                sum = fmaf(p[y], kv8::exp2i(-(int)sh->v_exp[j]), sum);
                                h[y] = lead(p[y]);
                            }
                            hi[d] = hi[16 + d] = kv8::e4m3x4(h[0], h[1], h[2], h[3]);
                            lo[d] = lo[16 + d] = kv8::e4m3x4(p[0] - h[0], p[1] - h[1], p[2] - h[2], p[3] - h[3]);
                        }
                        l2 = attn2::add2(l2, attn2::f2(sum, 0.f));
                    }
                    attn2::tmem_st32_nowait(s_addr, hi);                 // P's digits over S
                    attn2::tmem_st32_nowait(s_addr + 32, lo);
                    attn2::tmem_wait_st();
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(s32(&sh->p_full[slot]));
            }
            if (!ok) break;
            trees += w.tree;
            // the next unit's Q goes in now: its first products can run during this one's output
            Row next;
            have = begin_unit(i + 1, next);
            if (mine > 0) {
                const bool got = mbar_wait(s32(&sh->o_full[slot]), units_done & 1u, abort_flag);
                if (!__all_sync(0xffffffffu, got)) break;
                ++units_done;
                tc_fence_after();
            }
            float la, lb;
            attn2::unf2(l2, la, lb);
            float l = la + lb, m = mref, w0 = 1.f, w1 = 0.f;             // weights of the slots' O
            bool use0 = mine > 0, use1 = false;
            const int c0 = w.alt ? 64 * slot : 0, c1 = w.alt ? c0 + 64 : kHeadDim;
            uint32_t a0 = o_addr, a1 = o_addr;
            if (w.alt) {
                // both slots hold this row: (m, l) change hands, each slot writes half of the columns
                sh->ml[slot][row] = make_float2(mref, l);
                __syncwarp();
                if (lane == 0) mbar_arrive(s32(&sh->merge_in));
                const bool got = mbar_wait(s32(&sh->merge_in), merges & 1u, abort_flag);
                if (!__all_sync(0xffffffffu, got)) break;
                tc_fence_after();
                const float2 x0 = sh->ml[0][row], x1 = sh->ml[1][row];
                m = fmaxf(x0.x, x1.x);
                w0 = x0.x == -INFINITY ? 0.f : exp2f(x0.x - m);
                w1 = x1.x == -INFINITY ? 0.f : exp2f(x1.x - m);
                l = x0.y * w0 + x1.y * w1;
                use0 = w.n > 0;
                use1 = w.n > 1;
                a0 = tmem + lane_base + attn2::o_col(0);
                a1 = tmem + lane_base + attn2::o_col(1);
            }
            if (!idle) {
                const float inv = w.n == 0 || l == 0.f ? 0.f : 1.f / l;
                const int node = w.r < 0 ? 0 : w.r / a.G, g = w.r < 0 ? 0 : w.r % a.G;
                uint16_t* out = a.out + (((int64_t)w.b * a.n + node) * a.Hq + w.head * a.G + g) * kHeadDim;
                const int64_t place = (int64_t)w.part * a.rows + (w.r - w.pair * 2 * kRows);
                for (int c = c0; c < c1; c += 32) {
                    uint32_t o[32];
                    if (use0) tmem_ld32(a0 + c, o);
                    if (use1) {
                        uint32_t o1[32];
                        tmem_ld32(a1 + c, o1);
#pragma unroll
                        for (int e = 0; e < 32; ++e)
                            o[e] = __float_as_uint(__uint_as_float(o[e]) * w0 + __uint_as_float(o1[e]) * w1);
                    }
                    if (w.r < 0) continue;
                    if (w.part < 0) {
#pragma unroll
                        for (int e = 0; e < 32; e += 8) {
                            uint32_t y[4];
#pragma unroll
                            for (int d = 0; d < 4; ++d)
                                y[d] = use0 ? pack2(__uint_as_float(o[e + 2 * d]) * inv, __uint_as_float(o[e + 2 * d + 1]) * inv) : 0u;
                            *reinterpret_cast<uint4*>(out + c + e) = make_uint4(y[0], y[1], y[2], y[3]);
                        }
                    } else {
#pragma unroll
                        for (int e = 0; e < 32; e += 4)
                            *reinterpret_cast<uint4*>(a.ws_o + place * kHeadDim + c + e) =
                                use0 ? make_uint4(o[e], o[e + 1], o[e + 2], o[e + 3]) : make_uint4(0u, 0u, 0u, 0u);
                    }
                }
                if (w.r >= 0 && w.part >= 0 && (!w.alt || slot == 0))
                    a.ws_ml[place] = use0 ? make_float2(m, l) : make_float2(-INFINITY, 0.f);
            }
            if (w.alt) {                                                 // O and ml are free again
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(s32(&sh->merge_out));
                const bool got = mbar_wait(s32(&sh->merge_out), merges & 1u, abort_flag);
                if (!__all_sync(0xffffffffu, got)) break;
                ++merges;
            }
            w = next;
        }
        if (bits) flag_error(a.dev_status, bits);
    }
    __syncthreads();
    if (tid == 0 && *abort_flag) flag_error(a.dev_status, EAGLE_DEV_TIMEOUT);
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, attn2::kTmemCols);
    }
}

// ---------------- merging of cut units ----------------
// Block (c, y): the unit whose first tile lies in piece c and whose last does not, rows y, y + 8,
// .. one warp each; its parts are piece c's second place and the first places of the pieces
// behind it.  m is in log2 units and a part's l and O share one factor, so a part weighs
// 2^(m - max m).
constexpr int kMergeThreads = 256, kMergeWarps = kMergeThreads / 32;

__global__ void __launch_bounds__(kMergeThreads) tree_attn_kv8_merge_kernel(Args a, int grid) {
    const int lane = threadIdx.x & 31;
    const Cut cut = make_cut(a, grid);
    const int c = blockIdx.x;
    if (c + 1 >= cut.ctas) return;                        // the last piece ends with a whole unit
    const int64_t begin = cut.begin(c), end = cut.begin(c + 1);
    int b = 0;
    int64_t base = 0;
    const Segment s = segment_at(a, end - 1, end, b, base);
    if (s.start < begin || s.t1 >= s.T) return;           // it begins earlier, or is whole
    const int rows = min(a.n * a.G - s.pair * 2 * kRows, 2 * kRows);
    int last = c;                                         // the piece with the unit's last tile
    while (last + 1 < cut.ctas && (cut.begin(last + 1) - s.start + s.weight - 1) / s.weight < s.T) ++last;
    for (int row = blockIdx.y * kMergeWarps + (threadIdx.x >> 5); row < rows; row += gridDim.y * kMergeWarps) {
        // part p of pieces c .. last; a piece may hold no tile of the unit
        auto place = [&](int p) -> int64_t {
            if (p == c) return ((int64_t)c * 2 + 1) * a.rows + row;
            const int64_t t0 = (cut.begin(p) - s.start + s.weight - 1) / s.weight;
            const int64_t t1 = p + 1 < cut.ctas ? (cut.begin(p + 1) - s.start + s.weight - 1) / s.weight : s.T;
            return t0 < s.T && t0 < t1 ? (int64_t)p * 2 * a.rows + row : -1;
        };
        float m = -INFINITY, l = 0.f;
        float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int p = c; p <= last; ++p) {
            const int64_t at = place(p);
            if (at < 0) continue;
            const float2 ml = a.ws_ml[at];
            const float4 x = *reinterpret_cast<const float4*>(a.ws_o + at * kHeadDim + 4 * lane);
            const float mn = fmaxf(m, ml.x);
            if (mn == -INFINITY) continue;
            const float wo = exp2f(m - mn), wx = exp2f(ml.x - mn);
            m = mn;
            l = l * wo + ml.y * wx;
            o.x = o.x * wo + x.x * wx; o.y = o.y * wo + x.y * wx;
            o.z = o.z * wo + x.z * wx; o.w = o.w * wo + x.w * wx;
        }
        const float inv = l == 0.f ? 0.f : 1.f / l;
        const int r = s.pair * 2 * kRows + row;
        uint16_t* out = a.out + (((int64_t)s.b * a.n + r / a.G) * a.Hq + s.head * a.G + r % a.G) * kHeadDim;
        reinterpret_cast<uint2*>(out)[lane] = make_uint2(pack2(o.x * inv, o.y * inv), pack2(o.z * inv, o.w * inv));
    }
}

}  // namespace kv8_tc
}  // namespace eagle
