// Tree attention over the 8-bit K/V cache on the tensor cores (tcgen05, TMEM, TMA).
//
// QK in 8 bits, PV in 16.  The cache's K codes go into kind::f8f6f4 as they lie in memory; the
// query keeps bf16's precision as two e4m3 digits, q = hi + lo with hi the leading 4 bits of the
// significand and lo the next 4: two passes at twice the bf16 rate, no conversion of K.  The
// weights change per tile and thread, so splitting them as well costs more instructions than the
// whole softmax (0.56 ms against 0.275 ms at the first shape below); V is widened to fp16 once per tile
// instead (every e4m3 value is a half), for both slots, and PV runs in kind::f16.
//   Q  per row times a power of two that brings its largest element to [128, 256): digits exact
//      for elements within 2^-9 of the largest, the rest to 2^-16 of it.
//   P  fp16, between 2^-24 and 2^14: a rounding of 2^-11 on a weight, where the largest weight is
//      at least 2^kOffset (or bf16, see Scales).
//   the tree's own rows (bf16, n <= 64): K as one 128-key tile with the hi digits in rows 0 .. 63
//      and the lo digits in rows 64 .. 127 (S of key j is S[j] + S[64 + j]), V in fp16, with a
//      power of two per row that brings its largest element to [128, 256).
//
// Scales.  A block of 32 keys has K and V scales 2^ek and 2^ev.  2^ek joins the factor from S to
// the exponent.  2^ev joins the weight, P' = 2^(s + ev - m) with m the running maximum of s + ev:
// then O = sum P' code needs no scale, and l = sum P' 2^-ev is one factor per block.  m is the
// running maximum of what is multiplied with the codes, so P' uses fp16's range whatever the
// blocks' scales have in common.  What it does not hold is a wide spread: beside a block of far larger
// scale, whose codes may well be zero in most columns, the other blocks' weights would be subnormal
// halves or zero.  A CTA that finds the exponents of a unit's V rows spread over more than kSpread
// goes through these units a second time, with P and V in bf16 (a rounding of 2^-8; the tree's P with
// its remainder, its V as it is), which replaces what the first pass wrote.  Only the second
// pass pays for that: bf16 as a case in the loops cost 5 to 10% of every call, and a copy of
// the loops that shared values with the first ones 1 to 8%.
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
// Roles: warp 0 loads K and V tiles, warp 1 issues the MMAs, warp 2 looks for wide spreads, warp 3 cuts
// the work, warps 4-11 are the softmax, which also makes the Q digits of the next unit before it
// writes this one's output, warps 12-15 widen V into two tiles (of two halves of 64 keys) and make the K
// digits of the tree's rows; V rows behind the last key become zeros there (whatever bits lie in them: a zero weight
// does not cancel NaN).
//
// Measured: 64 trees of 60 nodes over 4096 rows, 32 / 8 heads, 0.263 ms (the bf16 cache's kernel:
// 0.296 ms from twice the bytes); tensor pipe 50% active, 646 MB read.  48 sequences of one node over
// 100 .. 30 000 rows, 64 / 8 heads: 158.5 us, 3.8 TB/s.  With a second pass over every unit 0.58 ms and 350 us.
// Bound: the chain of QK, softmax and PV per slot and the MMA warp's control, about 3 800 cycles per 256
// rows x 128 keys, and 20 to 30 thousand cycles at a unit's ends; neither HBM nor the tensor pipe is full.
// ptxas: 616 bytes of spill stores, 700 of loads, 200 bytes of stack, most of them in the warps of 64
// registers and in the second pass.
#pragma once

#include <cstddef>
#include <type_traits>

#include "attn2_common.cuh"
#include "attn2_cut.cuh"
#include "kv8_common.cuh"

namespace eagle {
namespace kv8_tc {

using attn2::kKeys;
using attn2::kRows;
using attn2::kSlots;
using kv8::kKv8Block;

constexpr int kThreads = 512;
// 4 warpgroups x 128 registers at launch; 64 + 2 x 192 + 64 = 4 x 128
constexpr int kRegsOther = 64, kRegsSoftmax = 192;
constexpr int kKStages = 3, kVStages = 2;         // rings of raw tiles
constexpr int kWide = 2;                          // V tiles in fp16, two halves of 64 keys each
constexpr int kTile = 128 * 128;                  // 16 KB: a K or V tile, a digit plane of Q, half a V tile in fp16
constexpr int kHalfKeys = 64, kHalfBox = kHalfKeys * 128;     // 64 keys x 64 dims of fp16
constexpr int kInfo = 3;                          // units in flight between the roles
constexpr int kTrees = 8;                         // trees in flight, see Shared
constexpr int kBlocks = kKeys / kKv8Block;        // scales per tile
// What a unit costs beside its tiles (digits, the tree, its output), in tiles.  us with 3 / 6 / 8 / 12: 48
// ragged sequences of one node 183 / 150 / 139 / 139, 16 ragged trees of 48 nodes 109 / 108 / 109 / 106, 64 equal
// trees 270 / 271 / 273 / 274; few units: one sequence of 40 heads 28.3 / 29.8 / 29.3 / 29.3, 4 trees of 60 nodes
// 51.9 / 51.9 / 51.9 / 53.9.
constexpr int kUnitCost = 8;
constexpr float kOffset = 6.f, kRescale = 8.f;    // weights up to 2^14
constexpr int kMaxVExp = 44;                      // V scales up to 2^44, see below
// The spread of a unit's V exponents up to which its weights are fp16.  A weight that is 2^-x of the
// largest in the product with its block's scale is off by 2^(x - 31) of itself at most, so 2^8 leaves a
// weight of 2^-15 (one of 32k equal ones) 8 bits.
constexpr int kSpread = 8;
// A CTA's piece is at least so many tiles (and fixed costs in tiles).  us with 1 / 2 / 3 / 4 / 6: one sequence,
// 8 heads, 2048 rows 22.7 / 23.7 / 23.2 / 25.2 / 27.8; one head, 30 000 rows 41.6 / 37 / 35.5 / 31.4 / 31; two trees of
// 12 nodes 23.2 / 27.3 / 25.7 / 26.2 / 29.3; large batches alike.
constexpr int kMinTiles = 3;
// Merging: a warp takes a row up to so many rows of a part, with so many parts on their way, in so many blocks an SM.  us
// with a warp / eight lanes a row: 48 sequences of 100 .. 30 000 rows, G = 8, 32 rows of a part 170.2 / 171.4, 48 182.4 /
// 180.2, 64 180.9 / 179.4, 96 209 / 205; one sequence alike.  With 8 parts on their way in 3 blocks 32 rows take 171.5 us,
// in 2 (no limit on registers) 172.7.
constexpr int kFewRows = 32, kFewBatch = 4, kFewBlocks = 4;

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

    // what the cut and the merging kernel ask for
    static constexpr int kUnitCost = kv8_tc::kUnitCost, kMinTiles = kv8_tc::kMinTiles;
    static constexpr int kFewRows = kv8_tc::kFewRows, kFewBatch = kv8_tc::kFewBatch;
    __device__ int tiles_of(int b) const {        // key tiles of a sequence, the tree's the last
        const int L = kv_len[b];
        return (L < 0 || L > Lmax) ? 1 : (L + kKeys - 1) / kKeys + 1;
    }
    __device__ int row_tiles() const { return (n * G + kRows - 1) / kRows; }
    __device__ int unit_rows(int pair) const { return min(n * G - pair * 2 * kRows, 2 * kRows); }
    __device__ int64_t out_row(int b, int head, int pair, int row) const {
        const int r = pair * 2 * kRows + row;
        return ((int64_t)b * n + r / G) * Hq + head * G + r % G;
    }
};

using attn2::Cut;
using attn2::make_cut;
using attn2::Segment;
using attn2::segment_at;

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

struct Barriers {
    uint64_t k_full[kKStages], k_empty[kKStages], k_grant[kKStages], v_full[kVStages], v_empty[kVStages];
    uint64_t h_full[kWide], h_empty[kWide];
    uint64_t q_full[kSlots], s_full[kSlots], p_full[kSlots], o_full[kSlots];
    uint64_t tree_full[kTrees], merge_in, merge_out;
    uint64_t info_full[kInfo], info_empty[kInfo];
    uint64_t drain;
};
struct Shared {
    Barriers bars[2];                             // of the first and the second pass
    uint32_t tmem;
    int abort_flag;
    int wide;                                     // a unit of this CTA has a wide spread
    float2 ml[kSlots][kRows];
    // factors of the tree's rows.  Their writers run ahead of the softmax by what the K ring and S
    // hold: at most kKStages + kSlots trees, fewer than kTrees
    float k_fac[kTrees][kMaxNodes];               // 2^ek
    float v_exp[kTrees][kMaxNodes];               // ev
    float v_inv[kTrees][kMaxNodes];               // 2^-ev
    Unit info[kInfo];
};
static_assert(kKStages + kSlots < kTrees && kWide < kTrees, "trees in flight");

constexpr int kSmem = kSlots * 2 * kTile + (kKStages + kVStages + 2 * kWide) * kTile + (int)sizeof(Shared) + 1024;
static_assert(kSmem <= 232448, "shared memory of a CTA");

// tcgen05.mma kind::f8f6f4, A and B e4m3 (format 0), both K-major, D fp32.
__host__ __device__ constexpr uint32_t idesc_e4m3(int M, int N) {
    return (1u << 4) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}
constexpr uint32_t kIdescQK = idesc_e4m3(128, kKeys);
// kind::f16 with A and B fp16 (format 0), B MN-major, D fp32
constexpr uint32_t kIdescPV = (1u << 4) | (1u << 16) | ((uint32_t)(kHeadDim >> 3) << 17) | ((128u >> 4) << 24);
constexpr uint32_t kIdescPVbf = idesc_bf16(128, kHeadDim, 0, 1);         // the same in bf16

// Two floats as an fp16 pair (round to nearest even), lo in the low half.
__device__ __forceinline__ uint32_t pack_half2(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;\n" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

// Two halves that hold e4m3 values as a bf16 pair (exact).
__device__ __forceinline__ uint32_t half2_bf162(uint32_t h) {
    const float2 f = kv8::half2_float(h);
    return pack2(f.x, f.y);
}

// The leading digit of x: its significand cut to 4 bits, a value that e4m3 holds exactly (for
// |x| in [2^-6, 448]; smaller ones are rounded to its 2^-9 grid when they are converted).
__device__ __forceinline__ float lead(float x) { return __uint_as_float(__float_as_uint(x) & 0xfff00000u); }

// The least exponent of a row's digits.  Their factor with the softmax's, scale log2 e 2^e, keeps 16 bits
// and more down to 2^-133, and a key's scale joins it afterwards: small queries may meet keys as large
// as bf16 and the cache hold them.
constexpr int kLowExp = -126;

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

// The 256 bytes of a row, asked into L2.
__device__ __forceinline__ void prefetch_l2(const void* p) {
    asm volatile("prefetch.global.L2 [%0];\n prefetch.global.L2 [%0 + 128];\n" ::"l"(p) : "memory");
}

// Warp-wide: of two rows at once, sixteen lanes a row, the exponent of each lane's row.
__device__ __forceinline__ int row_exp(const uint4& v, int lo_exp) {
    float m = amax8(v);
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    return digit_exp(m, lo_exp);
}

// Warp-wide: whether the exponents of the V rows in tiles [t0, t1) of a (sequence, kv head) spread over more
// than kSpread, or one is below the least of the cache.  Scales are loaded 512 at a time, so that a long
// piece waits for few loads: in fours of 32, one sequence of 30 000 rows and one head took 36.5 us instead
// of 33.4.
__device__ __forceinline__ bool wide_spread(const Args& a, int b, int head, int t0, int t1, bool tree, int L) {
    const int lane = threadIdx.x & 31;
    int top = 0, low = 255;                       // exponents as stored
    const int end = min((L + kKv8Block - 1) / kKv8Block, t1 * kBlocks);
    const float* scales = a.v_scale + ((int64_t)b * a.Hkv + head) * a.NB;
    for (int y = t0 * kBlocks; y < end; y += 512)
#pragma unroll
        for (int k = 0; k < 16; ++k) {
            const int e = (int)(__float_as_uint(__ldg(scales + min(y + 32 * k + lane, end - 1))) >> 23);
            top = max(top, e);
            low = min(low, e);
        }
    const uint16_t* x = a.v_tree + ((int64_t)b * a.n * a.Hkv + head) * kHeadDim + (lane & 15) * 8;
    for (int r0 = lane >> 4; tree && r0 - (lane >> 4) < a.n; r0 += 4) {
        uint4 v[2];
#pragma unroll
        for (int k = 0; k < 2; ++k)
            v[k] = __ldg(reinterpret_cast<const uint4*>(x + (int64_t)min(r0 + 2 * k, a.n - 1) * a.Hkv * kHeadDim));
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const int e = row_exp(v[k], -127) + 127;
            if (e == 0) continue;                 // below 2^-120: a row of zeros, or as good as one
            top = max(top, e);
            low = min(low, e);
        }
    }
    top = __reduce_max_sync(0xffffffffu, top);
    low = __reduce_min_sync(0xffffffffu, low);
    return top - low > kSpread || low < kv8::kMinExp + 127;
}

// All threads of the CTA, wherever in the roles' code they are.
__device__ __forceinline__ void all_sync() { asm volatile("bar.sync 1, %0;\n" ::"n"(kThreads) : "memory"); }

__global__ void __launch_bounds__(kThreads, 1)
tree_attn_kv8_kernel(const __grid_constant__ CUtensorMap map_k, const __grid_constant__ CUtensorMap map_v, Args a) {
    extern __shared__ uint8_t smem_raw[];
    uint32_t at = (0u - s32(smem_raw)) & 1023u;           // tiles begin at a multiple of 1024
    uint8_t *sQ, *sK, *sV, *sH;
    Shared* sh;
    auto place = [&]() {
        sQ = smem_raw + at;                               // [slot][hi, lo][16 KB]
        sK = sQ + kSlots * 2 * kTile;                     // [kKStages][16 KB]
        sV = sK + kKStages * kTile;                       // [kVStages][16 KB]
        sH = sV + kVStages * kTile;                       // [kWide][2 halves][2 boxes of 64 dims][64 keys][128 B]
        sh = reinterpret_cast<Shared*>(sH + 2 * kWide * kTile);
    };
    place();
    volatile int* abort_flag = &sh->abort_flag;
    // barriers by their 32-bit shared addresses: 64-bit pointer arithmetic in the control of the MMA
    // warp is time that the tensor cores wait
    uint32_t sb = s32(&sh->bars[0]);
#define BAR(name) (sb + (uint32_t)offsetof(Barriers, name))
#define BAR_AT(name, i) (sb + (uint32_t)offsetof(Barriers, name) + 8u * (uint32_t)(i))
    const int tid = threadIdx.x, warp = tid >> 5;
    int lane = tid & 31;

    auto init_barriers = [&]() {
        for (int i = 0; i < kKStages; ++i) { mbar_init(BAR_AT(k_full, i), 4); mbar_init(BAR_AT(k_empty, i), 1); mbar_init(BAR_AT(k_grant, i), 1); }
        for (int i = 0; i < kVStages; ++i) { mbar_init(BAR_AT(v_full, i), 1); mbar_init(BAR_AT(v_empty, i), 4); }
        for (int i = 0; i < kWide; ++i) { mbar_init(BAR_AT(h_full, i), 4); mbar_init(BAR_AT(h_empty, i), 1); }
        for (int s = 0; s < kSlots; ++s) {
            mbar_init(BAR_AT(q_full, s), 4);
            mbar_init(BAR_AT(s_full, s), 1);
            mbar_init(BAR_AT(p_full, s), 4);
            mbar_init(BAR_AT(o_full, s), 1);
        }
        for (int i = 0; i < kTrees; ++i) mbar_init(BAR_AT(tree_full, i), 4);
        mbar_init(BAR(merge_in), 8);
        mbar_init(BAR(merge_out), 8);
        // read by warps 0, 1 and 2, the eight softmax and the four widening warps
        for (int i = 0; i < kInfo; ++i) { mbar_init(BAR_AT(info_full, i), 1); mbar_init(BAR_AT(info_empty, i), 15); }
        mbar_init(BAR(drain), 1);
        asm volatile("fence.mbarrier_init.release.cluster;\n" ::: "memory");
    };
    if (tid == 0) {
        sh->abort_flag = 0;
        sh->wide = 0;
        init_barriers();
    }
    if (warp == 1) tmem_alloc(s32(&sh->tmem), attn2::kTmemCols);
    // the merging kernel may be launched as CTAs of this one end; it waits for all of them itself
    asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    uint32_t tmem = sh->tmem;

    // the i-th unit of this CTA; nullptr at the end (or on abort)
    auto next_unit = [&](int i) -> const Unit* {
        if (!attn2::wait_for(BAR_AT(info_full, i % kInfo), ((uint32_t)i / kInfo) & 1u, abort_flag)) return nullptr;
        const Unit* u = &sh->info[i % kInfo];
        return u->head >= 0 ? u : nullptr;
    };
    // Every role's end of the first pass over this CTA's units: whether a second one follows.  It has
    // barriers of its own: arrivals that nobody awaited may still be on their way to the first ones.
    auto again = [&]() {
        __syncwarp();
        tc_fence_before();
        all_sync();
        tc_fence_after();
        if (!sh->wide || *abort_flag) return false;
        sb += (uint32_t)sizeof(Barriers);
        // values that the compiler is not to take from the first pass: it would compute there what
        // only the second one needs, and keep it
        asm volatile("" : "+r"(lane), "+r"(sb), "+r"(tmem), "+r"(at));
        place();
        if (tid == 0) init_barriers();
        all_sync();
        return true;
    };
    auto unit_read = [&](int i) { attn2::arrive_if(lane == 0, BAR_AT(info_empty, i % kInfo)); };

    if (warp < 4) {
        attn2::regs_dec<kRegsOther>();
        if (warp == 0) {
            // ---------------- K and V tiles ----------------
            for (int pass = 0;; ++pass) {
                uint32_t ks = 0, kp = 1, vs = 0, vp = 1;
                bool ok = true;
                for (int i = 0; ok; ++i) {
                    const Unit* up = next_unit(i);
                    if (!__all_sync(0xffffffffu, up != nullptr)) break;
                    const int t0 = up->t0, nc = up->n - up->tree, tree = up->tree, z = up->b * a.Hkv + up->head;
                    __syncwarp();
                    unit_read(i);
#pragma unroll 1
                    for (int j = 0; ok && j < nc; ++j) {
                        const bool k_free = attn2::wait_for(BAR_AT(k_empty, ks), kp, abort_flag);
                        ok = __all_sync(0xffffffffu, k_free);
                        attn2::arrive_if(ok && lane > 0 && lane < 4, BAR_AT(k_full, ks));     // four arrivals, as for the tree's
                        if (ok && lane == 0) {
                            mbar_expect_tx(BAR_AT(k_full, ks), kTile);
                            tma_load_3d(s32(sK + ks * kTile), &map_k, BAR_AT(k_full, ks), 0, (t0 + j) * kKeys, z);
                        }
                        if (++ks == kKStages) { ks = 0; kp ^= 1u; }
                        const bool v_free = ok && attn2::wait_for(BAR_AT(v_empty, vs), vp, abort_flag);
                        ok = __all_sync(0xffffffffu, v_free);
                        if (ok && lane == 0) {
                            mbar_expect_tx(BAR_AT(v_full, vs), kTile);
                            tma_load_3d(s32(sV + vs * kTile), &map_v, BAR_AT(v_full, vs), 0, (t0 + j) * kKeys, z);
                        }
                        if (++vs == kVStages) { vs = 0; vp ^= 1u; }
                    }
                    if (ok && tree) {
                        // the tree's stage is the widening warps' to fill.  They do not follow this
                        // ring, and a parity names a phase only to a waiter that is at most one
                        // behind, so the stage is handed over when it is free
                        const bool free = attn2::wait_for(BAR_AT(k_empty, ks), kp, abort_flag);
                        ok = __all_sync(0xffffffffu, free);
                        attn2::arrive_if(ok && lane == 0, BAR_AT(k_grant, ks));
                        if (++ks == kKStages) { ks = 0; kp ^= 1u; }
                    }
                }
                if (pass > 0 || !again()) break;
            }
        } else if (warp == 1) {
            // ---------------- MMA issue ----------------
            // One warp for both slots, whose products then stay together in the tensor pipe (with a
            // warp per slot they interleave, and both slots wait for both).  This warp's control
            // is what the tensor pipe waits for: steps have their slot as a template argument, loads
            // are waited for before P is, and no lane's instruction stands in a branch.
            auto pass = [&](auto wide) {
                constexpr bool kBf = decltype(wide)::value;
                const bool leader = attn2::elect_lane();
                const uint32_t on = leader;
                const uint32_t tm = (uint32_t)attn2::uniform_of((int)tmem);
                const uint32_t dq0 = attn2::desc_lo(s32(sQ)), dk0 = attn2::desc_lo(s32(sK)), dh0 = attn2::desc_lo_mn(s32(sH), kHalfBox);
                uint32_t ks = 0, kp = 0, hs = 0, hp = 0, qph = 0, pph = 0;    // ring places, phases
                bool ok = true;
                // (a wait that gives up lets the step run on, on data that nobody will use)
                auto wait = [&](uint32_t bar, uint32_t parity) { ok &= attn2::wait_for(bar, parity, abort_flag); };
                // O of slot s += P V of the tile at the ring's place, then S = Q K^T of the next tile there.
                // two: a tile of 128 keys (the tree's is one half; in bf16 its weights are two parts of 64
                // keys, both on that half's rows).  opens, closes: the tiles' first, last use
                auto step = [&](auto slot_c, bool pv, bool pv_first, bool pv_last, bool two, bool qk, bool qk_first, bool opens, bool closes) {
                    constexpr int s = decltype(slot_c)::value;
                    const uint32_t scol = tm + attn2::s_col(s), ocol = tm + attn2::o_col(s);
                    if (opens && pv) wait(BAR_AT(h_full, hs), hp);
                    if (opens && qk) wait(BAR_AT(k_full, ks), kp);
                    if (qk && qk_first) {
                        wait(BAR_AT(q_full, s), qph >> s);
                        qph ^= 1u << s;
                    }
                    if (pv) {
                        wait(BAR_AT(p_full, s), pph >> s);
                        pph ^= 1u << s;
                        tc_fence_after();
                        constexpr uint32_t id = kBf ? kIdescPVbf : kIdescPV;
                        const uint32_t dv = dh0 + ((hs * 2 * kTile) >> 4), dv2 = dv + (kBf && !two ? 0 : kTile >> 4);
                        attn2::mma_ts(on, ocol, scol, dv, id, pv_first ? 0u : 1u);
#pragma unroll
                        for (int k = 1; k < kHalfKeys / 16; ++k)
                            attn2::mma_ts(on, ocol, scol + 8 * k, dv + ((k * 16 * 128) >> 4), id, 1u);
                        const uint32_t on2 = leader && (kBf || two);
#pragma unroll
                        for (int k = 0; k < kHalfKeys / 16; ++k)
                            attn2::mma_ts(on2, ocol, scol + 32 + 8 * k, dv2 + ((k * 16 * 128) >> 4), id, 1u);
                    }
                    if (qk) {
                        tc_fence_after();
                        const uint32_t dk = dk0 + ((ks * kTile) >> 4), dq = dq0 + ((2 * s * kTile) >> 4);
#pragma unroll
                        for (int d = 0; d < 2; ++d)                           // both digits of Q
#pragma unroll
                            for (int k = 0; k < kHeadDim / 32; ++k)
                                attn2::mma_ss<true>(on, scol, dq + ((d * kTile) >> 4) + 2 * k, dk + 2 * k, kIdescQK, (d | k) ? 1u : 0u);
                        attn2::commit_if(leader, BAR_AT(s_full, s));
                    }
                    attn2::commit_if(leader && pv && pv_last, BAR_AT(o_full, s));
                    if (closes && pv) {
                        attn2::commit_if(leader, BAR_AT(h_empty, hs));
                        hs ^= 1u;
                        hp ^= hs == 0;
                    }
                    if (closes && qk) {
                        attn2::commit_if(leader, BAR_AT(k_empty, ks));
                        if (++ks == kKStages) { ks = 0; kp ^= 1u; }
                    }
                };
                const std::integral_constant<int, 0> s0;
                const std::integral_constant<int, 1> s1;
                for (int i = 0; ok; ++i) {
                    const Unit* up = next_unit(i);
                    if (!__all_sync(0xffffffffu, up != nullptr)) break;
                    const int n = attn2::uniform_of(up->n), nc = n - attn2::uniform_of(up->tree);     // the tree's tile is one half
                    const int alt = attn2::uniform_of(up->split_keys);
                    __syncwarp();
                    unit_read(i);
                    if (n == 0) continue;
                    if (alt) {                                // tile t is slot t & 1's
#pragma unroll 1
                        for (int t = 0; t < n + 2 && __all_sync(0xffffffffu, ok); t += 2) {
                            step(s0, t >= 2, t == 2, t >= n, t - 2 < nc, t < n, t == 0, true, true);
                            step(s1, t >= 2 && t - 1 < n, t == 2, t + 1 >= n, t - 1 < nc, t + 1 < n, t == 0, true, true);
                        }
                    } else {                                  // every tile is both slots'
#pragma unroll 1
                        for (int t = 0; t <= n && __all_sync(0xffffffffu, ok); ++t) {
                            step(s0, t > 0, t == 1, t == n, t - 1 < nc, t < n, t == 0, true, false);
                            step(s1, t > 0, t == 1, t == n, t - 1 < nc, t < n, t == 0, false, true);
                        }
                    }
                    ok = __all_sync(0xffffffffu, ok);
                }
                if (leader) {
                    umma_commit(BAR(drain));
                    attn2::wait_drain(BAR(drain));
                }
            };
            pass(std::false_type{});
            if (again()) pass(std::true_type{});
        } else if (warp == 2) {
            // ---------------- which units have a wide spread ----------------
            for (int pass = 0;; ++pass) {
                for (int i = 0;; ++i) {
                    const Unit* u = next_unit(i);
                    if (!__all_sync(0xffffffffu, u != nullptr)) break;
                    if (pass == 0 && wide_spread(a, u->b, u->head, u->t0, u->t0 + u->n, u->tree, u->L) && lane == 0) sh->wide = 1;
                    __syncwarp();
                    unit_read(i);
                }
                if (pass > 0 || !again()) break;
            }
        } else if (warp == 3) {
            // ---------------- the cut ----------------
            for (int pass = 0;; ++pass) {
                const Cut cut = make_cut(a, gridDim.x);
                const bool mine = (int)blockIdx.x < cut.ctas;
                int pos = mine ? cut.begin(blockIdx.x) : 0, base = 0;
                const int end = mine ? cut.begin(blockIdx.x + 1) : 0;
                int b = 0, anc_of = -1, bits = 0;
                unsigned long long anc[2] = {0, 0};           // of nodes lane and lane + 32
                bool bad_tree = false;
                bool have = true;
                for (int i = 0; have; ++i) {
                    Segment s;
                    have = false;
                    while (!have && pos < end) {
                        s = segment_at(a, pos, end, b, base);
                        pos = s.start + s.weight * (s.T + kUnitCost);
                        have = s.t0 < s.t1;
                        if (pass > 0 && have) {           // the second pass: units of a wide spread alone
                            const int L = a.kv_len[s.b];
                            have = L >= 0 && L <= a.Lmax && wide_spread(a, s.b, s.head, s.t0, s.t1, s.t1 == s.T, L);
                        }
                    }
                    const bool got = attn2::wait_for(BAR_AT(info_empty, i % kInfo), (((uint32_t)i / kInfo) & 1u) ^ 1u, abort_flag);
                    if (!__all_sync(0xffffffffu, got)) break;
                    Unit* u = &sh->info[i % kInfo];
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
#pragma unroll 1
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
                    }
                    __syncwarp();
                    attn2::arrive_if(lane == 0, BAR_AT(info_full, i % kInfo));
                    if (have) {
                        // the unit's rows of Q and of the tree go into L2 meanwhile
                        const char* qr = reinterpret_cast<const char*>(a.q + ((int64_t)s.b * a.n * a.Hq + s.head * a.G) * kHeadDim);
                        const int64_t tree_at = ((int64_t)s.b * a.n * a.Hkv + s.head) * kHeadDim;
                        for (int y = lane; y < a.n; y += 32) {
                            prefetch_l2(a.k_tree + tree_at + (int64_t)y * a.Hkv * kHeadDim);
                            prefetch_l2(a.v_tree + tree_at + (int64_t)y * a.Hkv * kHeadDim);
                            for (int g = 0; g < a.G; ++g) prefetch_l2(qr + ((int64_t)y * a.Hq + g) * kHeadDim * 2);
                        }
                    }
                }
                if (bits) flag_error(a.dev_status, bits);
                if (pass > 0 || !again()) break;
            }
        }
    } else if (warp < 12) {
        // ---------------- softmax: one thread per query row ----------------
        attn2::regs_inc<kRegsSoftmax>();
        auto pass = [&](auto wide) {
            constexpr bool kBf = decltype(wide)::value;
            const int slot = (warp - 4) >> 2;
            const int row = (warp & 3) * 32 + lane;
            const uint32_t lane_base = (uint32_t)((warp & 3) * 32) << 16;
            const uint32_t s_addr = tmem + lane_base + attn2::s_col(slot);
            const uint32_t o_addr = tmem + lane_base + attn2::o_col(slot);
            uint32_t tiles_done = 0, units_done = 0, merges = 0, trees = 0;
            int bits = 0;

            // Everything that a unit is stays in shared memory until its output is written; this thread
            // keeps its row (node * G + g, -1: nobody's), the row's ancestors and its factor from S to
            // log2 units, without the key's scale.
            int row_of = -1, alt = 0;
            unsigned long long anc = 0;
            float sc = 0.f;
            // the i-th unit: its Q digits; false at the end
            auto begin_unit = [&](int i, int& row_next, unsigned long long& anc_next, float& sc_next) {
                const Unit* up = next_unit(i);
                if (!__all_sync(0xffffffffu, up != nullptr)) return false;
                const int r = up->pair * 2 * kRows + (up->split_keys ? 0 : slot * kRows) + row;
                row_next = r < a.n * a.G ? r : -1;
                const int node = row_next < 0 ? 0 : r / a.G;
                anc_next = up->anc[node];
                // a slot without a tile leaves Q (and its barrier) alone: it could be units ahead
                if (up->n <= (up->split_keys ? slot : 0)) return true;
                // every QK of this slot's last unit has completed (its S was read): Q may be replaced.
                // The warp makes its 32 rows' digits together, two rows at once, sixteen lanes a row.
                const int my_off = row_next < 0 ? -1 : node * a.Hq + (r - node * a.G);
                const uint16_t* src = a.q + ((int64_t)up->b * a.n * a.Hq + up->head * a.G) * kHeadDim + (lane & 15) * 8;
                uint8_t* dst = sQ + slot * 2 * kTile;
                int e_mine = 0;
                const int count = __popc(__ballot_sync(0xffffffffu, row_next >= 0));   // rows of this warp that exist, its first ones
#pragma unroll 1
                for (int r0 = 0; r0 < count; r0 += 16) {
                    uint4 v[8];
#pragma unroll
                    for (int k = 0; k < 8; ++k) {
                        // a row that does not exist takes the first one's place in the load: loads
                        // under a condition each wait for the one before
                        const int off = max(__shfl_sync(0xffffffffu, my_off, r0 + 2 * k + (lane >> 4)), 0);
                        v[k] = __ldg(reinterpret_cast<const uint4*>(src + (int64_t)off * kHeadDim));
                    }
#pragma unroll 1
                    for (int k = 0; k < 8; k += 4) {                         // four row pairs at once, to hide their latencies
                        int e[4];
#pragma unroll
                        for (int y = 0; y < 4; ++y) e[y] = row_exp(v[y], kLowExp);
#pragma unroll
                        for (int y = 0; y < 4; ++y) {
                            const int rr = r0 + 2 * (k + y) + (lane >> 4), at = (warp & 3) * 32 + rr;
                            uint32_t hi[2], lo[2];
                            digits8(v[y], kv8::exp2i(-e[y]), hi, lo);
                            *reinterpret_cast<uint2*>(dst + swz(at, 8 * (lane & 15))) = make_uint2(hi[0], hi[1]);
                            *reinterpret_cast<uint2*>(dst + kTile + swz(at, 8 * (lane & 15))) = make_uint2(lo[0], lo[1]);
                            const int e_of = __shfl_sync(0xffffffffu, e[y], (lane & 1) << 4);   // of row r0 + 2 (k + y) + (lane & 1)
                            if ((lane >> 1) == (r0 >> 1) + k + y) e_mine = e_of;
                        }
#pragma unroll
                        for (int y = 0; y < 4; ++y) v[y] = v[y + 4];         // the loop's body exists once
                    }
                }
                sc_next = a.scale_log2 * kv8::exp2i(e_mine);
                attn2::fence_async_shared();
                __syncwarp();
                attn2::arrive_if(lane == 0, BAR_AT(q_full, slot));
                return true;
            };

            // Per unit: the Q digits of the next one go in, so that its first products can run during
            // this one's output; then this one's output; then the next one's tiles.
            bool have = true, ok = true, idle = true;
            float mref = 0.f;
            uint64_t l2 = 0;                                                 // two partial sums of the weights
            int mine = 0;                                                    // tiles of this slot
            for (int i = 0; have && ok; ++i) {
                int row_next = -1;
                unsigned long long anc_next = 0;
                float sc_next = 0.f;
                have = begin_unit(i, row_next, anc_next, sc_next);
                if (i > 0) {
                    const Unit* u = &sh->info[(i - 1) % kInfo];
                    if (mine > 0) {
                        const bool got = attn2::wait_for(BAR_AT(o_full, slot), units_done & 1u, abort_flag);
                        if (!__all_sync(0xffffffffu, got)) break;
                        ++units_done;
                        tc_fence_after();
                    }
                    float la, lb;
                    attn2::unf2(l2, la, lb);
                    float l = la + lb, m = mref, w0 = 1.f, w1 = 0.f;             // weights of the slots' O
                    bool use0 = mine > 0, use1 = false;
                    const int c0 = alt ? 64 * slot : 0, c1 = alt ? c0 + 64 : kHeadDim;
                    uint32_t a0 = o_addr, a1 = o_addr;
                    if (alt) {
                        // both slots hold this row: (m, l) change hands, each slot writes half of the columns
                        sh->ml[slot][row] = make_float2(mref, l);
                        __syncwarp();
                        attn2::arrive_if(lane == 0, BAR(merge_in));
                        const bool got = attn2::wait_for(BAR(merge_in), merges & 1u, abort_flag);
                        if (!__all_sync(0xffffffffu, got)) break;
                        tc_fence_after();
                        const float2 x0 = sh->ml[0][row], x1 = sh->ml[1][row];
                        m = fmaxf(x0.x, x1.x);
                        w0 = x0.x == -INFINITY ? 0.f : exp2f(x0.x - m);
                        w1 = x1.x == -INFINITY ? 0.f : exp2f(x1.x - m);
                        l = x0.y * w0 + x1.y * w1;
                        use0 = u->n > 0;
                        use1 = u->n > 1;
                        a0 = tmem + lane_base + attn2::o_col(0);
                        a1 = tmem + lane_base + attn2::o_col(1);
                    }
                    if (!idle) {
                        const float inv = u->n == 0 || l == 0.f ? 0.f : 1.f / l;
                        const int node = row_of < 0 ? 0 : row_of / a.G, g = row_of < 0 ? 0 : row_of - node * a.G, part = u->part;
                        uint16_t* out = a.out + (((int64_t)u->b * a.n + node) * a.Hq + u->head * a.G + g) * kHeadDim;
                        const int64_t place = (int64_t)part * a.rows + (row_of - u->pair * 2 * kRows);
#pragma unroll 1
                        for (int c = c0; c < c1; c += 16) {
                            uint32_t o[16], o1[16];
                            if (use0) attn2::load16(a0 + c, o);
                            if (use1) attn2::load16(a1 + c, o1);
#pragma unroll
                            for (int e = 0; e < 16; ++e) {
                                const float x0 = use0 ? __uint_as_float(o[e]) : 0.f, x1 = use1 ? __uint_as_float(o1[e]) : 0.f;
                                o[e] = __float_as_uint(fmaf(x0, w0, x1 * w1));
                            }
                            if (row_of < 0) continue;
                            if (part < 0) {
                                uint32_t y[8];
#pragma unroll
                                for (int e = 0; e < 8; ++e)
                                    y[e] = pack2(__uint_as_float(o[2 * e]) * inv, __uint_as_float(o[2 * e + 1]) * inv);
                                *reinterpret_cast<uint4*>(out + c) = make_uint4(y[0], y[1], y[2], y[3]);
                                *reinterpret_cast<uint4*>(out + c + 8) = make_uint4(y[4], y[5], y[6], y[7]);
                            } else {
#pragma unroll
                                for (int e = 0; e < 16; e += 4)
                                    *reinterpret_cast<uint4*>(a.ws_o + place * kHeadDim + c + e) = make_uint4(o[e], o[e + 1], o[e + 2], o[e + 3]);
                            }
                        }
                        if (row_of >= 0 && part >= 0 && (!alt || slot == 0))
                            a.ws_ml[place] = use0 ? make_float2(m, l) : make_float2(-INFINITY, 0.f);
                    }
                    if (alt) {                                                   // O and ml are free again
                        tc_fence_before();
                        __syncwarp();
                        attn2::arrive_if(lane == 0, BAR(merge_out));
                        const bool got = attn2::wait_for(BAR(merge_out), merges & 1u, abort_flag);
                        if (!__all_sync(0xffffffffu, got)) break;
                        ++merges;
                    }
                }
                if (i > 0) {
                    __syncwarp();
                    unit_read(i - 1);
                }
                if (!have) break;
                row_of = row_next;
                anc = anc_next;
                sc = sc_next;
                idle = !__any_sync(0xffffffffu, row_of >= 0);     // rows are independent: leave P as it is
                const Unit* u = &sh->info[i % kInfo];
                const int n = u->n, nc = n - u->tree, left0 = u->L - u->t0 * kKeys;     // keys from the unit's first tile on
                alt = u->split_keys;
                mref = -INFINITY;
                l2 = 0;
                mine = 0;
                // lanes 0 .. 3 (and every lane alike mod 8) hold the K scales of a tile's blocks, lanes
                // 4 .. 7 the V scales, loaded a tile ahead; blocks without a key take the last one's
                const float* scales = ((lane & 4) ? a.v_scale : a.k_scale) + ((int64_t)u->b * a.Hkv + u->head) * a.NB + u->t0 * kBlocks;
                const int last_block = max(u->L - 1, 0) / kKv8Block - u->t0 * kBlocks;
                auto load_scale = [&](int t) { return __ldg(scales + min(t * kBlocks + (lane & 3), last_block)); };
                const int first = alt ? slot : 0, step = alt ? 2 : 1;
                float scale = load_scale(first);
                for (int t = first; t < n; t += step, ++mine) {
                    const bool got = attn2::wait_for(BAR_AT(s_full, slot), tiles_done & 1u, abort_flag);
                    if (!__all_sync(0xffffffffu, got)) { ok = false; break; }
                    ++tiles_done;
                    tc_fence_after();
                    if (!idle) {
                        float mx = -INFINITY, alpha = 1.f;
                        // raises the reference maximum where mx is far above it (every tile has a visible
                        // key: mx is finite, and the first one always is above), without branches of a lane
                        auto raise = [&]() {
                            const bool up = mx > mref + kRescale;
                            alpha = up ? ex2_approx(mref - mx) : 1.f;        // 0 for the first maximum
                            mref = up ? mx : mref;
                            l2 = attn2::mul2(l2, attn2::f2(alpha, alpha));
                            // the commit behind this QK covers every PV before it: O is complete
                            if (mine > 0 && __any_sync(0xffffffffu, up)) attn2::rescale_row(o_addr, alpha);
                        };
                        if (t < nc) {
                            const int left = left0 - t * kKeys;
                            uint32_t x[kKeys];
                            float mb[kBlocks];
                            attn2::load_row_nowait(s_addr, x, mb);
                            // a block's factor (above 0, so that a masked block stays -inf) and exponent
                            float f[kBlocks];
                            int ev[kBlocks];
#pragma unroll
                            for (int c = 0; c < kBlocks; ++c) {
                                f[c] = fmaxf(__shfl_sync(0xffffffffu, scale, c) * sc, 1.17549435e-38f);
                                ev[c] = (int)(__float_as_uint(__shfl_sync(0xffffffffu, scale, kBlocks + c)) >> 23) - 127;
                                if (ev[c] > kMaxVExp) bits = EAGLE_DEV_NONFINITE;
                            }
                            scale = load_scale(t + step);
                            attn2::tmem_wait_ld();
                            if (left < kKeys) {
#pragma unroll
                                for (int c = 0; c < kBlocks; ++c) {
                                    float y[kKv8Block];
#pragma unroll
                                    for (int e = 0; e < kKv8Block; ++e) {
                                        y[e] = kKv8Block * c + e < left ? __uint_as_float(x[kKv8Block * c + e]) : -INFINITY;
                                        x[kKv8Block * c + e] = __float_as_uint(y[e]);
                                    }
                                    mb[c] = attn2::max_of<kKv8Block>(y);
                                }
                            }
#pragma unroll
                            for (int c = 0; c < kBlocks; ++c) mx = fmaxf(mx, fmaf(mb[c], f[c], (float)ev[c]));
                            raise();
#pragma unroll
                            for (int c = 0; c < kBlocks; ++c) {
                                const float off = (float)ev[c] - mref + kOffset, inv = kv8::exp2i(min(-ev[c], 127));
                                const uint64_t f_2 = attn2::f2(f[c], f[c]), off2 = attn2::f2(off, off);
                                uint64_t acc[2] = {0, 0};
                                uint32_t pk[16];
#pragma unroll
                                for (int d = 0; d < 16; ++d) {
                                    float s0, s1;
                                    attn2::unf2(attn2::fma2(attn2::f2(__uint_as_float(x[32 * c + 2 * d]), __uint_as_float(x[32 * c + 2 * d + 1])), f_2, off2), s0, s1);
                                    const float p0 = ex2_approx(s0), p1 = ex2_approx(s1);
                                    acc[d & 1] = attn2::add2(acc[d & 1], attn2::f2(p0, p1));
                                    pk[d] = kBf ? pack2(p0, p1) : pack_half2(p0, p1);
                                }
                                attn2::tmem_st16_nowait(s_addr + 16 * c, pk);        // P over S
                                l2 = attn2::fma2(attn2::add2(acc[0], acc[1]), attn2::f2(inv, inv), l2);
                            }
                        } else {
                            // the tree's tile, 32 keys at a time: key j's score is the sum of its digits'
                            // columns j and 64 + j; its factors have a barrier per tree in flight
                            const int tr = trees % kTrees;
                            const bool seen = attn2::wait_for(BAR_AT(tree_full, tr), (trees / kTrees) & 1u, abort_flag);
                            if (!__all_sync(0xffffffffu, seen)) { ok = false; break; }
                            // first pass: scores, back into TMEM; second pass: weights.  In bf16 (V as it is):
                            // a weight and its remainder, the scores meanwhile where the lo digits' were.
                            constexpr int kAt = kBf ? kMaxNodes : 0;
                            uint32_t x[16], y[16];
#pragma unroll 1
                            for (int c = 0; c < kMaxNodes; c += 16) {
                                attn2::load16(s_addr + c, x);
                                attn2::load16(s_addr + kMaxNodes + c, y);
                                const uint32_t sees = (uint32_t)(anc >> c);
                                float s[16];
#pragma unroll
                                for (int j = 0; j < 16; ++j) {
                                    const float f = fmaxf(sh->k_fac[tr][c + j] * sc, 1.17549435e-38f);
                                    s[j] = (sees >> j) & 1u ? fmaf(__uint_as_float(x[j]) + __uint_as_float(y[j]), f, kBf ? 0.f : sh->v_exp[tr][c + j])
                                                           : -INFINITY;
                                    x[j] = __float_as_uint(s[j]);
                                }
                                mx = fmaxf(mx, attn2::max_of<16>(s));
                                attn2::tmem_st16_nowait(s_addr + kAt + c, x);
                            }
                            attn2::tmem_wait_st();
                            raise();
                            float sum = 0.f;
                            const float off = kOffset - mref;
#pragma unroll 1
                            for (int c = 0; c < kMaxNodes; c += 16) {
                                attn2::load16(s_addr + kAt + c, x);
                                uint32_t pk[8], lo[8];
#pragma unroll
                                for (int d = 0; d < 8; ++d) {
                                    const float p0 = ex2_approx(__uint_as_float(x[2 * d]) + off);
                                    const float p1 = ex2_approx(__uint_as_float(x[2 * d + 1]) + off);
                                    if constexpr (kBf) {
                                        sum += p0 + p1;
                                        pk[d] = pack2(p0, p1);
                                        lo[d] = pack2(p0 - __uint_as_float(pk[d] << 16), p1 - __uint_as_float(pk[d] & 0xffff0000u));
                                    } else {
                                        sum = fmaf(p0, sh->v_inv[tr][c + 2 * d], fmaf(p1, sh->v_inv[tr][c + 2 * d + 1], sum));
                                        pk[d] = pack_half2(p0, p1);
                                    }
                                }
                                attn2::tmem_st8_nowait(s_addr + c / 2, pk);      // over scores that have been read
                                if constexpr (kBf) attn2::tmem_st8_nowait(s_addr + kMaxNodes / 2 + c / 2, lo);
                            }
                            l2 = attn2::add2(l2, attn2::f2(sum, 0.f));
                        }
                        attn2::tmem_wait_st();
                    }
                    tc_fence_before();
                    __syncwarp();
                    attn2::arrive_if(lane == 0, BAR_AT(p_full, slot));
                }
                trees += n - nc;
            }
            if (bits) flag_error(a.dev_status, bits);
        };
        pass(std::false_type{});
        if (again()) pass(std::true_type{});
    } else {
        // ---------------- V in fp16 ----------------
        attn2::regs_dec<kRegsOther>();
        auto pass = [&](auto wide) {
            constexpr bool kBf = decltype(wide)::value;
            const int cw = warp - 12;
            // this lane's key of a group of eight and 16-byte chunk of four: the eight lanes of a
            // shared-memory phase read and write all 32 banks, under both tiles' swizzles
            const int key8 = (lane >> 3) ^ ((lane & 4) ? 5 : 0), c4 = lane & 3;
            uint32_t r = 0, rh = 0, rk = 0, trees = 0, grants = 0;   // uses of the rings; a phase bit per K stage
            int bits = 0;
            bool ok = true;
            auto ready = [&](uint32_t bar, uint32_t parity) {
                const bool got = attn2::wait_for(bar, parity, abort_flag);
                ok = ok && __all_sync(0xffffffffu, got);
                return ok;
            };
            auto tile_done = [&]() {
                attn2::fence_async_shared();
                __syncwarp();
                attn2::arrive_if(lane == 0, BAR_AT(h_full, rh % kWide));
                ++rh;
            };
            for (int i = 0; ok; ++i) {
                const Unit* up = next_unit(i);
                if (!__all_sync(0xffffffffu, up != nullptr)) break;
                const int b = up->b, head = up->head, t0 = up->t0, nc = up->n - up->tree, tree = up->tree, L = up->L;
                __syncwarp();
                unit_read(i);
                for (int j = 0; j < nc; ++j, ++r) {
                    const int st = r % kVStages, left = L - (t0 + j) * kKeys;
                    if (!ready(BAR_AT(v_full, st), r / kVStages)) break;
                    if (!ready(BAR_AT(h_empty, rh % kWide), (rh / kWide) ^ 1u)) break;
#pragma unroll 1
                    for (int h = 0; h < 2; ++h) {
                        const uint8_t* src = sV + st * kTile + h * kHalfKeys * 128;
                        uint8_t* dst = sH + (rh % kWide * 2 + h) * kTile;
                        uint4 x[4];
#pragma unroll
                        for (int y = 0; y < 4; ++y)
                            x[y] = *reinterpret_cast<const uint4*>(src + swz((cw * 2 + (y >> 1)) * 8 + key8, (4 * (y & 1) + c4) * 16));
#pragma unroll
                        for (int y = 0; y < 4; ++y) {
                            const int key = (cw * 2 + (y >> 1)) * 8 + key8, box = y & 1;
                            const bool there = h * kHalfKeys + key < left;
                            const uint32_t w[4] = {there ? x[y].x : 0u, there ? x[y].y : 0u, there ? x[y].z : 0u, there ? x[y].w : 0u};
                            uint32_t o[8];
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                o[2 * e] = kv8::e4m3x2_half2((uint16_t)w[e]);
                                o[2 * e + 1] = kv8::e4m3x2_half2((uint16_t)(w[e] >> 16));
                            }
                            if constexpr (kBf)
#pragma unroll
                                for (int e = 0; e < 8; ++e) o[e] = half2_bf162(o[e]);
                            *reinterpret_cast<uint4*>(dst + box * kHalfBox + swz(key, 32 * c4)) = make_uint4(o[0], o[1], o[2], o[3]);
                            *reinterpret_cast<uint4*>(dst + box * kHalfBox + swz(key, 32 * c4 + 16)) = make_uint4(o[4], o[5], o[6], o[7]);
                        }
                    }
                    tile_done();
                    attn2::arrive_if(lane == 0, BAR_AT(v_empty, st));
                }
                rk += nc;
                if (ok && tree) {
                    const uint32_t ks = rk++ % kKStages;
                    {
                        // K: digits.  Rows from n on are left as they are: no key of theirs is ever seen.
                        uint8_t* tile = sK + ks * kTile;
                        const uint16_t* x = a.k_tree + ((int64_t)b * a.n * a.Hkv + head) * kHeadDim + (lane & 15) * 8;
                        const int r0 = cw * 16 + (lane >> 4);
                        uint4 v[8];
#pragma unroll
                        for (int k = 0; k < 8; ++k)
                            v[k] = __ldg(reinterpret_cast<const uint4*>(x + (int64_t)min(r0 + 2 * k, a.n - 1) * a.Hkv * kHeadDim));
                        if (!ready(BAR_AT(k_grant, ks), grants >> ks)) break;
                        grants ^= 1u << ks;
                        const int pairs = min(8, (a.n - cw * 16 + 1) >> 1);
#pragma unroll 1
                        for (int k = 0; k < pairs; k += 4) {                     // four row pairs at once, to hide their latencies
                            int e[4];
#pragma unroll
                            for (int y = 0; y < 4; ++y) e[y] = row_exp(v[y], kLowExp);
#pragma unroll
                            for (int y = 0; y < 4; ++y) {
                                const int row = r0 + 2 * (k + y), c = lane & 15;
                                uint32_t hi[2], lo[2];
                                digits8(v[y], kv8::exp2i(-e[y]), hi, lo);
                                if (row < a.n) {
                                    *reinterpret_cast<uint2*>(tile + swz(row, 8 * c)) = make_uint2(hi[0], hi[1]);
                                    *reinterpret_cast<uint2*>(tile + swz(kMaxNodes + row, 8 * c)) = make_uint2(lo[0], lo[1]);
                                    if (c == 0) sh->k_fac[trees % kTrees][row] = kv8::exp2i(e[y]);
                                }
                            }
#pragma unroll
                            for (int y = 0; y < 4; ++y) v[y] = v[y + 4];     // the loop's body exists once
                        }
                        attn2::fence_async_shared();
                        __syncwarp();
                        attn2::arrive_if(lane == 0, BAR_AT(k_full, ks));
                    }
                    // V
                    if (!ready(BAR_AT(h_empty, rh % kWide), (rh / kWide) ^ 1u)) break;
                    uint8_t* dst = sH + rh % kWide * 2 * kTile;
                    const uint16_t* x = a.v_tree + ((int64_t)b * a.n * a.Hkv + head) * kHeadDim;
#pragma unroll 1
                    for (int r0 = cw * 16 + (lane >> 4); r0 < cw * 16 + 16; r0 += 8) {
                        if (r0 - (lane >> 4) >= a.n) {        // no row of the tree
#pragma unroll
                            for (int k = 0; k < 4; ++k) {
                                *reinterpret_cast<uint4*>(dst + ((lane & 15) >> 3) * kHalfBox + swz(r0 + 2 * k, (lane & 7) * 16)) =
                                    make_uint4(0u, 0u, 0u, 0u);
                                // the sum multiplies it with a weight of zero, which does not cancel NaN
                                if ((lane & 15) == 0) sh->v_inv[trees % kTrees][r0 + 2 * k] = 0.f;
                            }
                            continue;
                        }
                        uint4 v[4];
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            v[k] = __ldg(reinterpret_cast<const uint4*>(x + (int64_t)min(r0 + 2 * k, a.n - 1) * a.Hkv * kHeadDim) + (lane & 15));
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            const int row = r0 + 2 * k, c = lane & 15;
                            const bool there = row < a.n;                    // zeros behind the tree's rows
                            if constexpr (kBf) {
                                *reinterpret_cast<uint4*>(dst + (c >> 3) * kHalfBox + swz(row, (c & 7) * 16)) =
                                    there ? v[k] : make_uint4(0u, 0u, 0u, 0u);
                                continue;
                            }
                            const int e = row_exp(v[k], kv8::kMinExp);
                            const float by = kv8::exp2i(-e);
                            if (there && e > kMaxVExp) bits = EAGLE_DEV_NONFINITE;
                            const uint32_t w[4] = {there ? v[k].x : 0u, there ? v[k].y : 0u, there ? v[k].z : 0u, there ? v[k].w : 0u};
                            uint32_t o[4];
#pragma unroll
                            for (int y = 0; y < 4; ++y)
                                o[y] = pack_half2(__uint_as_float(w[y] << 16) * by, __uint_as_float(w[y] & 0xffff0000u) * by);
                            *reinterpret_cast<uint4*>(dst + (c >> 3) * kHalfBox + swz(row, (c & 7) * 16)) = make_uint4(o[0], o[1], o[2], o[3]);
                            if (c == 0) {
                                sh->v_exp[trees % kTrees][row] = (float)e;
                                sh->v_inv[trees % kTrees][row] = by;
                            }
                        }
                    }
                    __syncwarp();
                    attn2::arrive_if(lane == 0, BAR_AT(tree_full, trees % kTrees));
                    ++trees;
                    tile_done();
                }
            }
            if (bits) flag_error(a.dev_status, bits);
        };
        pass(std::false_type{});
        if (again()) pass(std::true_type{});
    }
    __syncthreads();
    if (tid == 0 && *abort_flag) report_timeout(a.dev_status);
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, attn2::kTmemCols);
    }
#undef BAR
#undef BAR_AT
}

template <bool kFew>
__global__ void __launch_bounds__(attn2::kMergeThreads, kFew ? kFewBlocks : 4) tree_attn_kv8_merge_kernel(Args a, int grid) {
    attn2::merge_parts<kFew>(a, grid);
}

}  // namespace kv8_tc
}  // namespace eagle
