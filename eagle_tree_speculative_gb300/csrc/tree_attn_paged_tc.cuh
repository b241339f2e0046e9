// Tree attention over the paged K/V cache on the tensor cores (tcgen05, TMEM, TMA).
//
// Mathematics: out = softmax(scale q k^T) v per row with the running maximum and sum of the softmax in
// fp32, in the exp2 domain; P is rounded to bf16 for the PV product (2^-8 of each weight, as the output's
// own rounding), sums use the unrounded weights.
//
// Rows.  A row tile is P = 128 / G nodes x G query heads that share a kv head (row p * G + g), so a
// kv head's K/V tile serves the whole group.  A unit is one (sequence, kv head, pair of row tiles), its
// keys in tiles of 128 rows, 128 / page pages each.  With two row tiles each softmax slot has one and both
// see every key tile: its bytes cross into the SM once for 256 rows.  A single row tile (decoding,
// small trees) has its key tiles dealt to the slots in turn, merged at the end.
// All tiles of all units are cut into one equal piece per CTA (attn2_cut.cuh): ragged batches and few long
// sequences balance alike.
//
// Roles: warp 0 loads Q and K, warp 2 V (tiles through one ring of 32 KB stages, page numbers a tile ahead; a
// page of 16 rows is a box of 2 KB, 32 of them a tile of K and V), warp 1 issues the MMAs, warp 3 cuts the work
// and zeroes V rows behind the tree's last (never written: a zero weight does not cancel NaN), warps 4-11
// are the softmax.
//
// MMA order: PV of a slot's last tile, then its next QK, whose commit also says that O holds that PV.
//
// Measured (with the merging kernel): 48 sequences of one node over 100 .. 30 000 rows, 64 / 8 heads, 209 .. 215 us: 6.9 ..
// 6.7 TB/s; 64 trees of 60 nodes over 4096 rows, 32 / 8 heads, 196 .. 210 us replayed one behind the other (5.9 .. 5.5 TB/s,
// 1.31 .. 1.23 PFLOP/s; the slab's kernel 296), 207 .. 221 with other caches read in between, up to 237 (4.9 TB/s, 1.09
// PFLOP/s) in turn with other work; tensor pipe 70% active; from pages that stay in L2 187 .. 191, so the chain of QK, softmax
// and PV per slot (3 000 cycles a tile of 256 rows) and HBM bind the trees together.  Tried, us of these trees: loads
// without the L2 policy 5 more; one loading warp for K and V 4 more; L2 prefetches two to six tiles ahead 10 to 75
// more; P handed over in halves no change; merging by the warp that comes last, in this kernel, 40 more (its
// code and registers).  With five stages instead of six the ragged sequences take 248 us.
#pragma once

#include <cstddef>
#include <type_traits>

#include "attn2_common.cuh"
#include "attn2_cut.cuh"
#include "paged_common.cuh"

namespace eagle {
namespace paged_tc {

using attn2::kKeys;
using attn2::kRows;
using attn2::kSlots;

constexpr int kThreads = 384;
// 3 warpgroups x 168 registers at launch; 72 + 2 x 216 = 3 x 168
constexpr int kRegsRole = 72, kRegsSoftmax = 216;
// Tiles in shared memory: Q, and the stages of the ring.  A launch whose units are single row tiles has Q once.
constexpr int kTiles = 7, kMaxStages = kTiles - 1;
template <bool kSingle> constexpr int kQTiles = kSingle ? 1 : kSlots;
constexpr int kBox = 128 * 64 * 2;                // 16 KB: 128 rows x 64 dims
constexpr int kTile = 2 * kBox;                   // 32 KB: Q of a slot, or a K or V tile
constexpr int kInfo = 3;                          // units in flight between the roles
// What a unit costs beside its tiles, in tiles.  us with 1 / 2 / 3: 16 ragged trees of 48 nodes 63 / 55 / 58, of 16 nodes 32 /
// 30 / 30, 48 ragged sequences of one node 214 / 210 / 211, 64 equal trees alike.
constexpr int kUnitCost = 2;
// A CTA's piece is at least so many tiles (and unit costs).  us with 3 / 4 / 5 / 6, few units only: one tree of 60 nodes over
// 4096 rows 26.5 / 25.6 / 23.0 / 25.9, two 27.9 / 27.7 / 25.7 / 27.2, eight over 500 .. 1000 rows 25.2 / 24.6 / 26.0 / 26.4;
// one sequence of one node over 4000 rows 13.6 / 13.1 / 14.7 / 15.0; large batches alike.
constexpr int kMinTiles = 5;
// Merging: a warp takes a row up to so many rows of a part, with so many parts on their way, in so many blocks an SM.  us
// with a warp / eight lanes a row, G = 4 or 8: one sequence of 20 011 rows, 32 rows of a part 22.2 / 25.0, 48 23.2 / 25.8,
// 64 24.1 / 25.2, 96 28.4 / 26.6; 48 sequences of 100 .. 30 000 rows, 32 rows 217 / 216, 48 218 / 216, 64 222 / 218, 96
// 232 / 218.  With 4 parts on their way one sequence of one node takes 18.9 us, with 8 18.2; with 2 blocks an SM (no
// limit on registers) the ragged sequences of 64 rows take 225 us, with 3 222.
constexpr int kFewRows = 64, kFewBatch = 8, kFewBlocks = 3;
constexpr float kRescale = 8.f;                   // log2 units the maximum may grow by

struct Args {
    const int32_t* table;
    const int32_t* kv_len;
    const int32_t* parent;
    uint16_t* out;
    float* ws_o;                                  // [grid][2][rows][128], at a multiple of 32 bytes
    float2* ws_ml;                                // [grid][2][rows]
    int B, n, Hq, Hkv, G, P;                      // P: nodes of a row tile
    int N, shift, width;                          // pages; log2 of a page's rows; entries of a table row
    int rows;                                     // rows of a part
    bool out_whole;                               // out at a multiple of 32 bytes
    float scale_log2;
    int32_t* dev_status;

    // what the cut and the merging kernel ask for
    static constexpr int kUnitCost = paged_tc::kUnitCost, kMinTiles = paged_tc::kMinTiles;
    static constexpr int kFewRows = paged_tc::kFewRows, kFewBatch = paged_tc::kFewBatch;
    __device__ bool bad_length(int L) const { return L < 0 || L + (int64_t)n > (int64_t)width << shift; }
    __device__ int tiles_of(int b) const {        // a sequence that is refused has one, of zeros
        const int L = kv_len[b];
        return bad_length(L) ? 1 : (L + n + kKeys - 1) / kKeys;
    }
    // a pair's missing row tile counts too: its key tiles take as long as two row tiles' (a tile's bytes, not its
    // products, are what a single row tile waits for; three draws of 16 ragged trees of 48 nodes, 64 / 8 heads, 54 / 89 / 73
    // us, counted by its rows 60 / 104 / 81)
    __device__ int row_tiles() const { return n <= P ? 1 : (n + 2 * P - 1) / (2 * P) * 2; }
    __device__ int unit_rows(int pair) const {
        const int left = n - pair * 2 * P;        // nodes from the pair's first on
        return left > P ? kRows + min(left - P, P) * G : left * G;
    }
    __device__ int64_t out_row(int b, int head, int pair, int row) const {
        const int slot = row >= kRows, r = row - slot * kRows, p = r / G;
        if (p >= P) return -1;
        return ((int64_t)b * n + (pair * 2 + slot) * P + p) * Hq + head * G + (r - p * G);
    }
};

struct Unit {
    int b, head, pair;                            // head -1: no more units
    int t0, n;                                    // first tile, number of tiles (0: write zeros)
    int L;
    int split;                                    // one row tile: its key tiles alternate between the slots
    int part;                                     // -1: whole, else the part's place
    uint8_t parent[kMaxNodes];
};

struct Shared {
    uint64_t full[kMaxStages], empty[kMaxStages]; // K/V ring
    uint64_t v_last[kMaxStages];                  // a V tile that needs repair has landed
    uint64_t q_full[kSlots], q_empty[kSlots];
    uint64_t s_full[kSlots], p_full[kSlots], o_full[kSlots];
    uint64_t merge_in, merge_out;
    uint64_t info_full[kInfo], info_empty[kInfo];
    uint64_t drain;
    uint32_t tmem;
    int abort_flag;
    float2 ml[kRows];                             // slot 1's maximum and sum of each row
    Unit info[kInfo];
};

constexpr int kSmem = kTiles * kTile + (int)sizeof(Shared) + 1024;
static_assert(kSmem <= 232448, "shared memory of a CTA");

constexpr uint32_t kIdescQK = idesc_bf16(128, kKeys, 0, 0);
constexpr uint32_t kIdescPV = idesc_bf16(128, kHeadDim, 0, 1);

// Whether a unit's last tile of the cut reaches behind the last row.  Its V tile then lands on the
// stage's v_last, and the repair warp completes the stage's own barrier once the rows are zero.
__device__ __forceinline__ bool needs_fix(const Unit& u, int n) { return u.n > 0 && (u.t0 + u.n) * kKeys > u.L + n; }

// What a row with ancestors `anc` sees of 32 keys from the one `at` rows behind L on (at < 0: before L).
__device__ __forceinline__ uint32_t sees32(unsigned long long anc, int at) {
    if (at <= -32) return 0xffffffffu;
    if (at < 0) return ((1u << -at) - 1u) | ((uint32_t)anc << -at);
    return at < kMaxNodes ? (uint32_t)(anc >> at) : 0u;
}

template <bool kSingle>                           // every unit is a single row tile
__global__ void __launch_bounds__(kThreads, 1)
tree_attn_paged_kernel(const __grid_constant__ CUtensorMap map_q, const __grid_constant__ CUtensorMap map_k,
                       const __grid_constant__ CUtensorMap map_v, Args a) {
    constexpr int kStages = kTiles - kQTiles<kSingle>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = smem_raw + ((0u - s32(smem_raw)) & 1023u);
    uint8_t* sQ = smem;                                   // [kQTiles][32 KB]
    uint8_t* sR = sQ + kQTiles<kSingle> * kTile;          // [kStages][32 KB]
    Shared* sh = reinterpret_cast<Shared*>(sR + kStages * kTile);
    volatile int* abort_flag = &sh->abort_flag;
    const uint32_t sb = s32(sh);
#define BAR(name) (sb + (uint32_t)offsetof(Shared, name))
#define BAR_AT(name, i) (sb + (uint32_t)offsetof(Shared, name) + 8u * (uint32_t)(i))
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

    if (tid == 0) {
        for (int i = 0; i < kStages; ++i) {
            mbar_init(BAR_AT(full, i), 1);
            mbar_init(BAR_AT(empty, i), 1);
            mbar_init(BAR_AT(v_last, i), 1);
        }
        for (int s = 0; s < kSlots; ++s) {
            mbar_init(BAR_AT(q_full, s), 1);
            mbar_init(BAR_AT(q_empty, s), 1);
            mbar_init(BAR_AT(s_full, s), 1);
            mbar_init(BAR_AT(p_full, s), 4);
            mbar_init(BAR_AT(o_full, s), 1);
        }
        mbar_init(BAR(merge_in), 4);
        mbar_init(BAR(merge_out), 4);
        // read by the four single warps and the eight softmax warps
        for (int i = 0; i < kInfo; ++i) { mbar_init(BAR_AT(info_full, i), 1); mbar_init(BAR_AT(info_empty, i), 12); }
        mbar_init(BAR(drain), 1);
        sh->abort_flag = 0;
        asm volatile("fence.mbarrier_init.release.cluster;\n" ::: "memory");
    }
    if (warp == 1) tmem_alloc(s32(&sh->tmem), attn2::kTmemCols);
    if (warp == 2 && lane == 0) {
        prefetch_map(&map_q);
        prefetch_map(&map_k);
        prefetch_map(&map_v);
    }
    // the merging kernel may be launched as CTAs of this one end; it waits for all of them itself
    asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = sh->tmem;

    // the i-th unit of this CTA; nullptr at the end (or on abort).  Warp-wide.
    auto next_unit = [&](int i) -> const Unit* {
        const bool got = attn2::wait_for(BAR_AT(info_full, i % kInfo), ((uint32_t)i / kInfo) & 1u, abort_flag);
        const Unit* u = &sh->info[i % kInfo];
        return __all_sync(0xffffffffu, got) && u->head >= 0 ? u : nullptr;
    };
    auto unit_read = [&](int i) {
        __syncwarp();
        attn2::arrive_if(lane == 0, BAR_AT(info_empty, i % kInfo));
    };

    if (warp < 4) {
        attn2::regs_dec<kRegsRole>();
        if (warp == 0 || warp == 2) {
            // ---------------- loads: warp 0 Q and K, warp 2 V ----------------
            // K and V tiles take turns in the ring: K's at even places, V's at odd ones.  (A stage's uses may alternate
            // between the warps.  Neither can be two uses ahead on one, which its parity would not show: a
            // place two before has been waited for, and the products that freed it come behind the older use's.)
            const bool is_v = warp == 2;
            const uint64_t policy = l2_policy_evict_first();
            const CUtensorMap* map = is_v ? &map_v : &map_k;
            const int per = kKeys >> a.shift;             // pages of a tile
            const uint32_t on = attn2::elect_lane();
            const uint32_t page_bytes = 128u << a.shift;  // of half the head dimension
            uint32_t st = is_v, ph = 1;                   // place in the ring, its phase
            uint32_t qph = 3;                             // a bit per slot
            int bits = 0;
            bool ok = true;
            const Unit* u;
            for (int i = 0; ok && (u = next_unit(i)); ++i) {
                const int b = u->b, head = u->head, pair = u->pair, t0 = u->t0, end = u->L + a.n;
                const int n = attn2::uniform_of(u->n);
                const bool split = kSingle || u->split, fix = is_v && needs_fix(*u, a.n);
                unit_read(i);
                if (n == 0) continue;
                auto load_q = [&](int s) {
                    const bool free = attn2::wait_for(BAR_AT(q_empty, s), qph >> s, abort_flag);
                    ok = ok && __all_sync(0xffffffffu, free);
                    qph ^= 1u << s;
                    if (!ok || lane != 0) return;
                    mbar_expect_tx(BAR_AT(q_full, s), (uint32_t)(2 * a.P * a.G * 128));
                    for (int x = 0; x < 2; ++x)
                        tma_load_4d(s32(sQ + s * kTile + x * kBox), &map_q, BAR_AT(q_full, s), 64 * x, 0, head,
                                    b * a.n + (pair * 2 + s) * a.P);
                };
                const int32_t* ids = a.table + (int64_t)b * a.width;
                const int pages = (end + (1 << a.shift) - 1) >> a.shift;
                auto load_id = [&](int j) {               // lane x: of page x of tile j
                    const int x = (t0 + j) * per + lane;
                    return lane < per && x < pages ? __ldg(ids + x) : -1;
                };
                int id = load_id(0);
                if (!is_v) load_q(0);
                for (int j = 0; ok && j < n; ++j) {
                    const int count = attn2::uniform_of(min(per, pages - (t0 + j) * per));
                    const bool bad = id < 0 || id >= a.N;
                    if (bad && lane < count) bits = EAGLE_DEV_CAPACITY;
                    // a page that does not exist: the place behind a page's last row, which reads as zeros
                    const int z = bad ? 0 : id * a.Hkv + head, y = bad ? 1 << a.shift : 0;
                    if (j + 1 < n) id = load_id(j + 1);
                    const bool free = attn2::wait_for(BAR_AT(empty, st), ph, abort_flag);
                    ok = __all_sync(0xffffffffu, free);
                    if (ok) {
                        const uint32_t bar = fix && j == n - 1 ? BAR_AT(v_last, st) : BAR_AT(full, st);
                        const uint32_t to = s32(sR) + st * kTile;
                        if (on) mbar_expect_tx(bar, 2u * page_bytes * (uint32_t)count);
                        __syncwarp();
#pragma unroll
                        for (int x = 0; x < kKeys / 16; ++x) {
                            if (x >= count) break;
                            const int zx = __shfl_sync(0xffffffffu, z, x), yx = __shfl_sync(0xffffffffu, y, x);
                            tma_load_3d_hint_if(on, to + x * page_bytes, map, bar, 0, yx, zx, policy);
                            tma_load_3d_hint_if(on, to + x * page_bytes + kBox, map, bar, 64, yx, zx, policy);
                        }
                    }
                    st += 2;
                    if (st >= kStages) { st -= kStages; ph ^= 1u; }
                    if (!is_v && j == 0 && !split) load_q(1);
                }
            }
            if (bits) flag_error(a.dev_status, bits);
        } else if (warp == 1) {
            // ---------------- MMA issue ----------------
            const bool leader = attn2::elect_lane();
            const uint32_t on = leader;
            const uint32_t tm = (uint32_t)attn2::uniform_of((int)tmem);
            const uint32_t dq0 = attn2::desc_lo(s32(sQ)), dk0 = attn2::desc_lo(s32(sR)), dv0 = attn2::desc_lo_mn(s32(sR), kBox);
            uint32_t qph = 0, pph = 0;
            uint32_t ks = 0, kp = 0, vs = 1, vp = 0;      // places of the next K and V tile
            bool ok = true;
            // (a wait that gives up lets the step run on, on data that nobody will use)
            auto wait = [&](uint32_t bar, uint32_t parity) { ok &= attn2::wait_for(bar, parity, abort_flag); };
            auto advance = [&](uint32_t& st, uint32_t& ph) {      // K and V tiles take turns in the ring
                st += 2;
                if (st >= kStages) { st -= kStages; ph ^= 1u; }
            };
            // O of slot s += P V of the next V tile, then S = Q K^T of the next K tile.  qs: the slot whose Q it is;
            // first, last: of the unit's tiles in the slot (PV), of its Q (QK); opens, closes: the tile's first, last use
            struct Use {
                bool on, first, last, opens, closes;
            };
            auto step = [&](int s, int qs, Use pv, Use qk) {
                const uint32_t scol = tm + (uint32_t)(s << 7), ocol = scol + 256;
                if (pv.on) {
                    if (pv.opens) wait(BAR_AT(full, vs), vp);
                    wait(BAR_AT(p_full, s), pph >> s);
                    pph ^= 1u << s;
                    tc_fence_after();
                    const uint32_t dv = dv0 + ((vs * kTile) >> 4);
                    uint32_t acc = pv.first ? 0u : 1u;
#pragma unroll
                    for (int k = 0; k < kKeys / 16; ++k) {
                        attn2::mma_ts(on, ocol, scol + 8 * k, dv + ((k * 16 * 128) >> 4), kIdescPV, acc);
                        acc = 1u;
                    }
                    // (the unit's result must not wait for the next one's Q)
                    if (pv.last) attn2::commit_if(leader, BAR_AT(o_full, s));
                    // The V tile's place: behind PV where pairs of row tiles read it (16 ragged trees of 48 nodes 60 to
                    // 55 us, longer ones 122 to 101), else behind QK (48 ragged sequences of one node 210 to 208 us).
                    if (!kSingle) attn2::commit_if(leader && pv.closes, BAR_AT(empty, vs));
                }
                if (qk.on) {
                    if (qk.opens) wait(BAR_AT(full, ks), kp);
                    if (qk.first) {
                        wait(BAR_AT(q_full, qs), qph >> qs);
                        qph ^= 1u << qs;
                    }
                    tc_fence_after();
                    const uint32_t dk = dk0 + ((ks * kTile) >> 4), dq = dq0 + ((qs * kTile) >> 4);
#pragma unroll
                    for (int k = 0; k < kHeadDim / 16; ++k) {
                        const uint32_t at = ((k >> 2) * kBox + (k & 3) * 32) >> 4;
                        attn2::mma_ss<false>(on, scol, dq + at, dk + at, kIdescQK, k > 0 ? 1u : 0u);
                    }
                    attn2::commit_if(leader, BAR_AT(s_full, s));
                }
                attn2::commit_if(leader && qk.on && qk.last, BAR_AT(q_empty, qs));
                if (kSingle) attn2::commit_if(leader && pv.on && pv.closes, BAR_AT(empty, vs));
                attn2::commit_if(leader && qk.on && qk.closes, BAR_AT(empty, ks));
                if (pv.on && pv.closes) advance(vs, vp);
                if (qk.on && qk.closes) advance(ks, kp);
            };
            // A unit of a single tile leaves its PV to the steps of the next ones, in which the slots go on taking turns,
            // so that such units follow one another without a gap (64 / 8 heads: 1024 sequences of one node over 1 .. 100
            // rows 194 to 128 us, 256 over 100 .. 400 rows 78 to 72); behind longer ones that gained nothing.  The last
            // units' PV, and that before a unit without tiles (whose rows the softmax cannot write before), have steps of
            // their own.
            int turn = 0, owed = 0;                       // the slot that is next; a bit per slot that owes PV
            for (int i = 0;; ++i) {
                const Unit* u = ok ? next_unit(i) : nullptr;
                int n = 0;
                bool split = kSingle;
                if (u) {
                    n = attn2::uniform_of(u->n);
                    split = kSingle || attn2::uniform_of(u->split);
                    unit_read(i);
                }
                const bool one = split && n == 1;
                turn = attn2::uniform_of(turn);
                owed = attn2::uniform_of(owed);
                // step x.  Both slots see every tile: PV of tile x / 2 - 1, QK of tile x / 2.  Tiles in turn: PV of
                // tile x - 2, QK of tile x.  The first two: what is owed.
                const int steps = one ? 1 : n == 0 ? 2 : split ? n + 2 : 2 * n + 2;
#pragma unroll 1
                for (int x = 0; x < steps && __all_sync(0xffffffffu, ok); ++x) {
                    const int s = (turn + x) & 1, j = split ? x : x >> 1, back = split ? 2 : 1;
                    const bool early = x < 2, opens = split || !(x & 1), closes = split || (x & 1);
                    step(s, split ? 0 : s, Use{!early || ((owed >> s) & 1), early || j < 2 * back, early || j >= n, early || opens, early || closes},
                         Use{j < n, j == 0, j == n - 1, opens, closes});
                }
                owed = one ? owed | 1 << turn : 0;
                turn = one ? turn ^ 1 : 0;
                ok = __all_sync(0xffffffffu, ok);
                if (!u) break;
            }
            if (leader) {
                umma_commit(BAR(drain));
                attn2::wait_drain(BAR(drain));
            }
        } else {
            // ---------------- the cut; V rows behind the tree's last ----------------
            const attn2::Cut cut = attn2::make_cut(a, gridDim.x);
            const bool mine = (int)blockIdx.x < cut.ctas;
            int pos = mine ? cut.begin(blockIdx.x) : 0, base = 0, b = 0;
            const int end = mine ? cut.begin(blockIdx.x + 1) : 0;
            const int pairs = (a.row_tiles() + 1) / 2;
            attn2::Segment s;
            int told_of = -1, L = 0, bits = 0, parent[2] = {-1, -1};  // of nodes lane and lane + 32
            bool zero = false;
            // tells the roles unit i, or that there is none: then false
            auto tell = [&](int i) {
                bool have = false;
                while (!have && pos < end) {
                    if (told_of >= 0 && (s.pair + 1 < pairs || s.head + 1 < a.Hkv)) {
                        // the sequence's next unit: nothing has to be looked up, which would take longer than a tile
                        s.head += s.pair + 1 == pairs;
                        s.pair = s.pair + 1 == pairs ? 0 : s.pair + 1;
                        s.start = pos;
                        s.t0 = 0;
                        s.t1 = min(s.T, attn2::tiles_before<Args>(pos, s.weight, end));
                    } else {
                        s = attn2::segment_at(a, pos, end, b, base);
                    }
                    pos = s.start + s.weight * (s.T + kUnitCost);
                    have = s.t0 < s.t1;
                }
                if (have && s.b != told_of) {
                    told_of = s.b;
                    L = a.kv_len[s.b];
                    bool bad = false;
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const int x = lane + 32 * h;
                        parent[h] = x < a.n ? a.parent[(int64_t)s.b * a.n + x] : 0;
                        bad |= x < a.n && (x == 0 ? parent[h] != -1 : (parent[h] < 0 || parent[h] >= x));
                    }
                    const bool bad_len = a.bad_length(L), bad_tree = __any_sync(0xffffffffu, bad);
                    zero = bad_len || bad_tree;
                    bits |= (bad_len ? EAGLE_DEV_CAPACITY : 0) | (bad_tree ? EAGLE_DEV_BAD_TREE : 0);
                }
                const bool got = attn2::wait_for(BAR_AT(info_empty, i % kInfo), (((uint32_t)i / kInfo) & 1u) ^ 1u, abort_flag);
                if (!__all_sync(0xffffffffu, got)) return false;
                Unit* u = &sh->info[i % kInfo];
                if (!have) {
                    if (lane == 0) u->head = -1;
                } else {
                    u->parent[lane] = (uint8_t)parent[0];
                    u->parent[lane + 32] = (uint8_t)parent[1];
                    if (lane == 0) {
                        u->b = s.b; u->head = s.head; u->pair = s.pair;
                        u->t0 = s.t0;
                        u->n = zero ? 0 : s.t1 - s.t0;
                        u->L = zero ? 0 : L;
                        u->split = s.pair * 2 * a.P + a.P >= a.n;
                        u->part = s.t0 == 0 && s.t1 == s.T ? -1 : (int)blockIdx.x * 2 + (s.t0 == 0);
                    }
                }
                __syncwarp();
                attn2::arrive_if(lane == 0, BAR_AT(info_full, i % kInfo));
                return have;
            };
            // units are told kInfo - 1 ahead of the one whose V tile is looked after
            bool more = tell(0);
            if (more) more = tell(1);
            uint32_t r = 0, phases = 0;                   // places in the ring so far; a bit per stage
            const Unit* u;
            for (int i = 0; (u = next_unit(i)); ++i) {
                const int n = u->n, first = u->L + a.n - (u->t0 + n - 1) * kKeys;
                const bool fix = needs_fix(*u, a.n);
                unit_read(i);
                if (more) more = tell(i + 2);
                r += 2 * n;
                if (!fix) continue;
                const uint32_t st = (r - 1) % kStages;
                const bool got = attn2::wait_for(BAR_AT(v_last, st), (phases >> st) & 1u, abort_flag);
                phases ^= 1u << st;
                if (!__all_sync(0xffffffffu, got)) break;
                uint8_t* v = sR + st * kTile;
                for (int row = first + (lane >> 4); row < kKeys; row += 2)
                    *reinterpret_cast<uint4*>(v + ((lane >> 3) & 1) * kBox + row * 128 + (lane & 7) * 16) = make_uint4(0u, 0u, 0u, 0u);
                attn2::fence_async_shared();
                __syncwarp();
                attn2::arrive_if(lane == 0, BAR_AT(full, st));
            }
            if (bits && lane == 0) flag_error(a.dev_status, bits);
        }
    } else {
        // ---------------- softmax: one thread per query row ----------------
        attn2::regs_inc<kRegsSoftmax>();
        const int slot = (warp - 4) >> 2;
        const int row = (warp & 3) * 32 + lane;
        const uint32_t lane_base = (uint32_t)((warp & 3) * 32) << 16;
        const uint32_t s_addr = tmem + lane_base + attn2::s_col(slot);
        const uint32_t o_addr = tmem + lane_base + attn2::o_col(slot);
        const int p = row / a.G, g = row % a.G;
        const float sc = a.scale_log2;
        const uint64_t sc2 = attn2::f2(sc, sc);
        uint32_t tiles_done = 0, units_done = 0, merges = 0;
        int turn = 0;                                     // the slot that has a unit's first tile
        bool ok = true;
        const Unit* u;
        for (int i = 0; ok && (u = next_unit(i)); ++i) {
            const int n = u->n, t0 = u->t0, part = u->part, L = u->L;
            const bool split = kSingle || u->split;
            const int row_tile = u->pair * 2 + (split ? 0 : slot), node = row_tile * a.P + p;
            const bool valid = p < a.P && node < a.n;
            unsigned long long anc = 0;                   // the node and its ancestors
            if (valid && n > 0)
                for (int x = node;; x = u->parent[x]) {
                    anc |= 1ull << x;
                    if (x == 0) break;
                }
            const int64_t at = ((int64_t)u->b * a.n + node) * a.Hq + u->head * a.G + g;
            const int64_t place = (int64_t)part * a.rows + (split ? 0 : slot * kRows) + row;
            unit_read(i);
            const bool idle = !__any_sync(0xffffffffu, valid);       // rows are independent: leave P as it is
            float mref = -INFINITY;
            uint64_t l2 = 0;                              // two partial sums
            int mine = 0;                                 // tiles of this slot
            for (int t = split ? slot ^ turn : 0; t < n; t += split ? 2 : 1, ++mine) {
                const bool got = attn2::wait_for(BAR_AT(s_full, slot), tiles_done & 1u, abort_flag);
                if (!__all_sync(0xffffffffu, got)) { ok = false; break; }
                ++tiles_done;
                tc_fence_after();
                if (!idle) {
                    uint32_t x[kKeys];
                    float m4[4];
                    attn2::load_row_nowait(s_addr, x, m4);
                    const int first = (t0 + t) * kKeys - L;          // rows from L on to the tile's first key
                    attn2::tmem_wait_ld();
                    if (first > -kKeys) {
                        float y[kKeys];
#pragma unroll
                        for (int w = 0; w < 4; ++w) {
                            const uint32_t sees = sees32(anc, first + 32 * w);
#pragma unroll
                            for (int c = 0; c < 32; ++c) {
                                y[32 * w + c] = (sees >> c) & 1u ? __uint_as_float(x[32 * w + c]) : -INFINITY;
                                x[32 * w + c] = __float_as_uint(y[32 * w + c]);
                            }
                        }
                        m4[0] = attn2::max_of<kKeys>(y);
                        m4[1] = m4[2] = m4[3] = m4[0];
                    }
                    const float mx = fmaxf(attn2::max3(m4[0], m4[1], m4[2]), m4[3]) * sc;    // scale > 0 commutes with max
                    // no branches of a lane; the first finite maximum is always above the reference
                    const bool up = mx > mref + kRescale;
                    const float alpha = up ? ex2_approx(mref - mx) : 1.f;            // 0 for the first one
                    mref = up ? mx : mref;
                    l2 = attn2::mul2(l2, attn2::f2(alpha, alpha));
                    // this QK was committed after the slot's last PV: O is complete
                    if (mine > 0 && __any_sync(0xffffffffu, up)) attn2::rescale_row(o_addr, alpha);
                    const float base = mref == -INFINITY ? 0.f : mref;
                    const uint64_t nb2 = attn2::f2(-base, -base);
                    uint64_t acc[4] = {l2, 0, 0, 0};
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        uint32_t pk[32];
#pragma unroll
                        for (int e = 0; e < 32; ++e) {
                            float s0, s1;
                            attn2::unf2(attn2::fma2(attn2::f2(__uint_as_float(x[64 * h + 2 * e]), __uint_as_float(x[64 * h + 2 * e + 1])), sc2, nb2), s0, s1);
                            const float p0 = ex2_approx(s0), p1 = ex2_approx(s1);
                            acc[e & 3] = attn2::add2(acc[e & 3], attn2::f2(p0, p1));
                            pk[e] = pack2(p0, p1);
                        }
                        attn2::tmem_st32_nowait(s_addr + 32 * h, pk);    // P over S
                    }
                    l2 = attn2::add2(attn2::add2(acc[0], acc[1]), attn2::add2(acc[2], acc[3]));
                    attn2::tmem_wait_st();
                }
                tc_fence_before();
                __syncwarp();
                attn2::arrive_if(lane == 0, BAR_AT(p_full, slot));
            }
            if (!ok) break;
            if (mine > 0) {
                const bool got = attn2::wait_for(BAR_AT(o_full, slot), units_done & 1u, abort_flag);
                if (!__all_sync(0xffffffffu, got)) break;
                ++units_done;
                tc_fence_after();
            }
            const bool one = split && n == 1;
            const int writer = one ? turn : 0;            // who writes a single row tile
            turn = one ? turn ^ 1 : 0;
            float la, lb;
            attn2::unf2(l2, la, lb);
            float l = la + lb, m = mref, w0 = 1.f, w1 = 0.f;             // weights of the slots' O
            if (split && n > 1) {
                // the row's other tiles are slot 1's: (m, l) go to slot 0, which writes both
                if (slot == 1) {
                    sh->ml[row] = make_float2(m, l);
                    tc_fence_before();
                    __syncwarp();
                    attn2::arrive_if(lane == 0, BAR(merge_in));
                    const bool got = attn2::wait_for(BAR(merge_out), merges & 1u, abort_flag);
                    if (!__all_sync(0xffffffffu, got)) break;
                    ++merges;
                    continue;
                }
                const bool got = attn2::wait_for(BAR(merge_in), merges & 1u, abort_flag);
                if (!__all_sync(0xffffffffu, got)) break;
                ++merges;
                tc_fence_after();
                const float2 other = sh->ml[row];
                m = fmaxf(mref, other.x);
                const float mb = m == -INFINITY ? 0.f : m;
                w0 = exp2f(mref - mb);
                w1 = exp2f(other.x - mb);
                l = l * w0 + other.y * w1;
            } else if (split && slot != writer) {
                continue;
            }
            if (!idle) {
                const float inv = l == 0.f ? 0.f : 1.f / l;
                // 32 columns of O, both slots' where the row's tiles were dealt to them
                auto load_o = [&](int c, uint32_t (&o)[32]) {
                    if (n > 0) tmem_ld32(o_addr + c, o);
                    else
#pragma unroll
                        for (int e = 0; e < 32; ++e) o[e] = 0u;
                    if (split && n > 1) {
                        uint32_t o1[32];
                        tmem_ld32(o_addr + 128 + c, o1);
#pragma unroll
                        for (int e = 0; e < 32; ++e)
                            o[e] = __float_as_uint(fmaf(__uint_as_float(o[e]), w0, __uint_as_float(o1[e]) * w1));
                    }
                };
                // Four lanes exchange what they have of their rows, so that they store 128 bytes of one of them at a time
                const unsigned rows4 = __ballot_sync(0xffffffffu, valid) >> (lane & 28);
                if (part < 0) {
                    uint16_t* to[4];
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        to[k] = a.out + __shfl_sync(0xffffffffu, at, (lane & 28) + k) * kHeadDim + 16 * (lane & 3);
#pragma unroll 1
                    for (int c = 0; c < kHeadDim; c += 64) {
                        uint32_t o[32], w[32];
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            load_o(c + 32 * h, o);
#pragma unroll
                            for (int e = 0; e < 16; ++e) w[16 * h + e] = pack2(__uint_as_float(o[2 * e]) * inv, __uint_as_float(o[2 * e + 1]) * inv);
                        }
                        attn2::transpose4(w, lane);
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            if ((rows4 >> k) & 1u) attn2::store32(to[k] + c, w + 8 * k, a.out_whole);
                        __syncwarp();
                    }
                } else {
                    float* to = a.ws_o + (place - (lane & 3)) * kHeadDim + 8 * (lane & 3);
#pragma unroll 1
                    for (int c = 0; c < kHeadDim; c += 32) {
                        uint32_t o[32];
                        load_o(c, o);
                        attn2::transpose4(o, lane);
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            if ((rows4 >> k) & 1u) attn2::store32(to + k * kHeadDim + c, o + 8 * k, true);
                        __syncwarp();
                    }
                }
                if (valid && part >= 0) a.ws_ml[place] = make_float2(m, l);
            }
            if (split && n > 1) {                         // O of slot 1 and ml are free again
                tc_fence_before();
                __syncwarp();
                attn2::arrive_if(lane == 0, BAR(merge_out));
            }
        }
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
__global__ void __launch_bounds__(attn2::kMergeThreads, kFew ? kFewBlocks : 4) tree_attn_paged_merge_kernel(Args a, int grid) {
    attn2::merge_parts<kFew>(a, grid);
}

}  // namespace paged_tc
}  // namespace eagle
