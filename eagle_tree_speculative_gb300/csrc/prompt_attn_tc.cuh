// Causal attention of packed prompts on the tensor cores (tcgen05, TMEM, TMA).
//
// Mathematics: out = softmax(scale q k^T) v per row with the running maximum and sum of the
// softmax in fp32, in the exp2 domain; P is rounded to bf16 for the PV product (one rounding of
// 2^-8 on each weight, the same as the output's), sums use the unrounded weights.
//
// Rows.  A row tile is P = 128 / G positions x G query heads that share a kv head (G = Hq /
// Hkv; row p * G + g), so a kv head's K/V tile serves the whole group and the causal edge of a
// tile is only P positions deep.  A unit is two consecutive row tiles (slots) of one sequence
// and kv head: while the tensor cores work for one slot, the other slot's softmax runs.
//
// Persistent CTAs, one per SM.  Units are dealt from the one with most keys to the one with
// fewest, in alternating direction from round to round, so CTAs end together; nothing is shared
// between them.  Barriers run on through units (a phase bit each), so the next unit's loads and
// first products overlap this unit's last softmax and output.
//
// Roles: warp 0 loads (Q per slot, then K and V tiles of 128 keys through one ring of 32 KB
// stages), warp 1 issues the MMAs, warp 2 zeroes V rows behind a sequence's last key (they are
// the next sequence's, or nobody's: a zero weight does not cancel NaN), warp 3 finds the units,
// warps 4-11 are the softmax.
//
// MMA order: PV of slot s and tile j - 1, then QK of slot s and tile j, slots in turn.  The
// tensor pipe runs MMAs of one thread in order, so QK(j) overwrites S (and the P in it) only
// after PV(j - 1) has read it, and the commit behind QK(j) also says that O holds PV(j - 1):
// the softmax warps may then rescale O without a wait of its own.  P of the next unit's first
// tile is written only after the same warps have read O of this one, which keeps O safe.
//
// Measured: one prompt of 16384 tokens, 32 / 8 heads, 1.50 ms = 1.47 PFLOP/s over the visible keys
// (79% of the library GEMM's burst, 87% of its sustained rate); 8 prompts of 2048, 0.239 ms, tensor
// pipe 53% active.  Bound: the tensor pipe and the softmax in turn (about 1450 cycles a tile), and
// the MMA warp's control; short prompts: the ends of their units.  An MMA warp per slot took 1.72
// against 1.61 ms: their products interleave, and both slots wait for both.
#pragma once

#include <cstddef>

#include "attn2_common.cuh"

namespace eagle {
namespace prompt_tc {

using attn2::kKeys;
using attn2::kRows;
using attn2::kSlots;

constexpr int kThreads = 384;
// 3 warpgroups x 168 registers at launch; 72 + 2 x 216 = 3 x 168
constexpr int kRegsRole = 72, kRegsSoftmax = 216;
constexpr int kStages = 5;
constexpr int kBox = 128 * 64 * 2;                // 16 KB: 128 rows x 64 dims
constexpr int kTile = 2 * kBox;                   // 32 KB: Q of a slot, or a K or V tile
constexpr int kInfo = 3;                          // units in flight between the roles
constexpr float kRescale = 8.f;                   // log2 units the maximum may grow by
// Keys of a sequence: a unit goes through them in 2^20 tiles of 3 300 cycles at most, during which the
// roles that are done with it wait for the next one.  Waits give up from 2^32 cycles on.
constexpr int kMaxKeys = 1 << 27;

struct Args {
    const int32_t* cu_q;
    const int32_t* cu_k;
    uint16_t* out;
    float* lse;
    int Tq, Tk, B, Hq, Hkv, G, P;
    float scale_log2;
    int32_t* dev_status;
};

// One unit: rows of positions pos .. pos + 2P - 1 of a sequence and kv head.
struct Unit {
    int q0, nq;                                   // first token and number of queries
    int k0, nk;                                   // first token and number of keys
    int pos;                                      // first position of slot 0
    int head;                                     // kv head, -1: no more units
    int tiles[kSlots];                            // key tiles of each slot
};

struct Shared {
    uint64_t full[kStages], empty[kStages];       // K/V ring
    uint64_t q_full[kSlots], q_empty[kSlots];
    uint64_t s_full[kSlots], p_full[kSlots], o_full[kSlots];
    uint64_t v_last[kStages];                     // a V tile that needs repair has landed
    uint64_t info_full[kInfo], info_empty[kInfo];
    uint64_t drain;
    uint32_t tmem;
    int abort_flag;
    Unit info[kInfo];
};

constexpr int kSmem = kSlots * kTile + kStages * kTile + (int)sizeof(Shared) + 1024;
static_assert(kSmem <= 232448, "shared memory of a CTA");

constexpr uint32_t kIdescQK = idesc_bf16(128, kKeys, 0, 0);
constexpr uint32_t kIdescPV = idesc_bf16(128, kHeadDim, 0, 1);

// Whether the unit's last tile reaches behind the sequence's last key.  Its V tile then lands on
// the stage's v_last, and the repair warp completes the stage's own barrier once the rows are zero.
__device__ __forceinline__ bool needs_fix(const Unit& u, int tiles) {
    return tiles > 0 && tiles * kKeys > u.nk;
}

// Key tiles that a row tile beginning at position p sees: keys up to nk - nq + its last position.
__device__ __forceinline__ int tiles_of(int nq, int nk, int p, int P) {
    if (p >= nq) return 0;
    const int end = nk - nq + min(p + P, nq);
    return end <= 0 ? 0 : (end + kKeys - 1) / kKeys;
}

// Units of a sequence with more than t key tiles in their second slot's place: units are ranked
// by the last key that their 2P positions can see, unclipped at the sequence's end.
__device__ __forceinline__ int units_above(int nq, int nk, int t, int W) {
    const int units = (nq + W - 1) / W;
    // unit u reaches key nk - nq + (u + 1) W; > t * kKeys  <=>  u + 1 > (t kKeys - (nk - nq)) / W
    const int x = t * kKeys - (nk - nq);
    return units - min(units, x < 0 ? 0 : x / W);
}

// Warp-wide: the unit of rank i in order of falling key count, over all sequences.  `top`: no
// unit has more than top tiles; nq0, nk0: the counts of sequence `lane`, if there is one.
__device__ __forceinline__ void find_unit(const Args& a, int i, int top, int nq0, int nk0, Unit& u) {
    const int lane = threadIdx.x & 31, W = 2 * a.P;
    const int rank = i / a.Hkv, head = i - rank * a.Hkv;
    auto queries = [&](int b) { return b < 32 ? nq0 : a.cu_q[b + 1] - a.cu_q[b]; };      // b = lane mod 32
    auto keys = [&](int b) { return b < 32 ? nk0 : a.cu_k[b + 1] - a.cu_k[b]; };
    auto count = [&](int t) {                     // units with more than t tiles
        int c = 0;
        for (int b = lane; b < a.B; b += 32) {
            const int nq = queries(b);
            if (nq > 0) c += units_above(nq, keys(b), t, W);
        }
        return __reduce_add_sync(0xffffffffu, c);
    };
    // the least t with count(t) <= rank: the unit has exactly t tiles (or t = 0: at most none)
    int lo = 0, hi = top;
    while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (count(mid) <= rank) hi = mid;
        else lo = mid + 1;
    }
    // among the units of exactly lo tiles (for lo = 0 all that is left): by sequence
    int left = rank - count(lo);
    u.head = -1;
    for (int b0 = 0; b0 < a.B; b0 += 32) {
        const int b = b0 + lane;
        int nq = 0, nk = 0, n = 0, above = 0;
        if (b < a.B) {
            nq = queries(b);
            nk = keys(b);
            if (nq > 0) {
                above = units_above(nq, nk, lo, W);
                n = (lo == 0 ? (nq + W - 1) / W : units_above(nq, nk, lo - 1, W)) - above;
            }
        }
        int sum = n;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, sum, o);
            if (lane >= o) sum += y;
        }
        const unsigned past = __ballot_sync(0xffffffffu, sum > left);
        if (past) {
            const int l = __ffs(past) - 1;
            const int at = left - __shfl_sync(0xffffffffu, sum - n, l);
            const int units = (__shfl_sync(0xffffffffu, nq, l) + W - 1) / W;
            u.nq = __shfl_sync(0xffffffffu, nq, l);
            u.nk = __shfl_sync(0xffffffffu, nk, l);
            u.pos = (units - 1 - __shfl_sync(0xffffffffu, above, l) - at) * W;
            u.q0 = a.cu_q[b0 + l];
            u.k0 = a.cu_k[b0 + l];
            u.head = head;
            break;
        }
        left -= __shfl_sync(0xffffffffu, sum, 31);
    }
    u.tiles[0] = tiles_of(u.nq, u.nk, u.pos, a.P);
    u.tiles[1] = tiles_of(u.nq, u.nk, u.pos + a.P, a.P);
}

__global__ void __launch_bounds__(kThreads, 1)
prompt_attn_kernel(const __grid_constant__ CUtensorMap map_q, const __grid_constant__ CUtensorMap map_k,
                   const __grid_constant__ CUtensorMap map_v, Args a) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                               ~static_cast<uintptr_t>(1023));
    uint8_t* sQ = smem;                                   // [kSlots][32 KB]
    uint8_t* sR = sQ + kSlots * kTile;                    // [kStages][32 KB]
    Shared* sh = reinterpret_cast<Shared*>(sR + kStages * kTile);
    volatile int* abort_flag = &sh->abort_flag;
    // barriers by their 32-bit shared addresses: 64-bit pointer arithmetic in the control of the MMA
    // warp is time that the tensor cores wait
    const uint32_t sb = s32(sh);
#define BAR(name) (sb + (uint32_t)offsetof(Shared, name))
#define BAR_AT(name, i) (sb + (uint32_t)offsetof(Shared, name) + 8u * (uint32_t)(i))
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

    if (tid == 0) {
        for (int i = 0; i < kStages; ++i) {
            mbar_init(s32(&sh->full[i]), 1);
            mbar_init(s32(&sh->empty[i]), 1);
            mbar_init(s32(&sh->v_last[i]), 1);
        }
        for (int s = 0; s < kSlots; ++s) {
            mbar_init(s32(&sh->q_full[s]), 1);
            mbar_init(s32(&sh->q_empty[s]), 1);
            mbar_init(s32(&sh->s_full[s]), 1);
            mbar_init(s32(&sh->p_full[s]), 4);
            mbar_init(s32(&sh->o_full[s]), 1);
        }
        // read by the loader, the MMA thread, the repair warp and the eight softmax warps
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

    // the i-th unit of this CTA, as the reading roles see it; false at the end (or on abort)
    auto next_unit = [&](int i, Unit& u) {
        if (!attn2::wait_for(BAR_AT(info_full, i % kInfo), ((uint32_t)i / kInfo) & 1u, abort_flag)) return false;
        u = sh->info[i % kInfo];
        return u.head >= 0;
    };
    auto unit_read = [&](int i) { attn2::arrive_if(lane == 0, BAR_AT(info_empty, i % kInfo)); };

    if (warp < 4) {
        attn2::regs_dec<kRegsRole>();
        if (warp == 0 && lane == 0) {
            // ---------------- loads ----------------
            uint32_t r = 0;                               // ring stages used so far
            uint32_t nqs[kSlots] = {0, 0};                // Q tiles loaded so far
            bool ok = true;
            Unit u;
            for (int i = 0; ok && next_unit(i, u); ++i) {
                unit_read(i);
                auto load_q = [&](int s) {
                    if (u.tiles[s] == 0) return;
                    ok = ok && attn2::wait_for(BAR_AT(q_empty, s), (nqs[s] & 1u) ^ 1u, abort_flag);
                    if (!ok) return;
                    const uint32_t bar = s32(&sh->q_full[s]);
                    mbar_expect_tx(bar, (uint32_t)(2 * a.P * a.G * 128));
                    for (int x = 0; x < 2; ++x)
                        tma_load_4d(s32(sQ + s * kTile + x * kBox), &map_q, bar, 64 * x, 0, u.head,
                                    u.q0 + u.pos + s * a.P);
                    ++nqs[s];
                };
                auto load_kv = [&](const CUtensorMap* map, int j, bool repair) {
                    const int st = r % kStages;
                    ok = ok && attn2::wait_for(BAR_AT(empty, st), ((r / kStages) & 1u) ^ 1u, abort_flag);
                    if (!ok) return;
                    const uint32_t bar = s32(repair ? &sh->v_last[st] : &sh->full[st]);
                    mbar_expect_tx(bar, kTile);
                    for (int x = 0; x < 2; ++x)
                        tma_load_3d(s32(sR + st * kTile + x * kBox), map, bar, 64 * x, u.head, u.k0 + j * kKeys);
                    ++r;
                };
                const int n = max(u.tiles[0], u.tiles[1]);
                const bool fix = needs_fix(u, n);
                load_q(0);
                for (int j = 0; ok && j < n; ++j) {
                    load_kv(&map_k, j, false);
                    if (j == 0) load_q(1);
                    load_kv(&map_v, j, fix && j == n - 1);
                }
            }
        } else if (warp == 1) {
            // ---------------- MMA issue ----------------
            // One copy of each product's code for both slots; the ring's place is kept as (stage,
            // phase), barrier phases as bits: nothing here may live in local memory, which has next
            // to no L1 beside this much shared memory.  (The kernel's 32 bytes of stack are the softmax
            // warps' unit, whose tiles they take by slot, once a unit; there are no spills.)
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
            for (int i = 0; ok; ++i) {
                Unit u;
                if (!__all_sync(0xffffffffu, next_unit(i, u))) break;
                unit_read(i);
                const int n0 = attn2::uniform_of(u.tiles[0]), n1 = attn2::uniform_of(u.tiles[1]), n = max(n0, n1);
                // step x: slot s = x & 1, O += P V of tile j - 1, then S = Q K^T of tile j = x / 2
                const int steps = n > 0 ? 2 * n + 2 : 0;
#pragma unroll 1
                for (int x = 0; x < steps && __all_sync(0xffffffffu, ok); ++x) {
                    const int s = x & 1, j = x >> 1, ns = s ? n1 : n0;
                    const bool pv = j > 0 && j <= ns, qk = j < ns;
                    const uint32_t scol = tm + (uint32_t)(s << 7), ocol = scol + 256;
                    if (s == 0 && j > 0) wait(BAR_AT(full, vs), vp);
                    if (pv) {
                        wait(BAR_AT(p_full, s), pph >> s);
                        pph ^= 1u << s;
                        tc_fence_after();
                        const uint32_t dv = dv0 + ((vs * kTile) >> 4);
                        uint32_t acc = j > 1 ? 1u : 0u;
#pragma unroll
                        for (int k = 0; k < kKeys / 16; ++k) {
                            attn2::mma_ts(on, ocol, scol + 8 * k, dv + ((k * 16 * 128) >> 4), kIdescPV, acc);
                            acc = 1u;
                        }
                    }
                    if (s == 0 && j < n) wait(BAR_AT(full, ks), kp);
                    if (qk) {
                        if (j == 0) {
                            wait(BAR_AT(q_full, s), qph >> s);
                            qph ^= 1u << s;
                        }
                        tc_fence_after();
                        const uint32_t dk = dk0 + ((ks * kTile) >> 4), dq = dq0 + ((s * kTile) >> 4);
#pragma unroll
                        for (int k = 0; k < kHeadDim / 16; ++k) {
                            const uint32_t at = ((k >> 2) * kBox + (k & 3) * 32) >> 4;
                            attn2::mma_ss<false>(on, scol, dq + at, dk + at, kIdescQK, k > 0 ? 1u : 0u);
                        }
                        attn2::commit_if(leader, BAR_AT(s_full, s));
                    }
                    attn2::commit_if(leader && pv && j == ns, BAR_AT(o_full, s));
                    attn2::commit_if(leader && qk && j == ns - 1, BAR_AT(q_empty, s));
                    attn2::commit_if(leader && s && j > 0, BAR_AT(empty, vs));
                    attn2::commit_if(leader && s && j < n, BAR_AT(empty, ks));
                    if (s) {
                        if (j > 0) advance(vs, vp);
                        if (j < n) advance(ks, kp);
                    }
                }
            }
            if (leader) {
                umma_commit(s32(&sh->drain));
                mbar_wait(s32(&sh->drain), 0u, abort_flag, /*honour_abort=*/false);
            }
        } else if (warp == 2) {
            // ---------------- V rows behind the sequence's last key ----------------
            uint32_t r = 0, phases = 0;                   // phases: a bit per stage
            Unit u;
            for (int i = 0;; ++i) {
                if (!__all_sync(0xffffffffu, next_unit(i, u))) break;
                unit_read(i);
                const int n = max(u.tiles[0], u.tiles[1]);
                r += 2 * n;
                if (!needs_fix(u, n)) continue;
                const uint32_t st = (r - 1) % kStages;
                const bool got = attn2::wait_for(BAR_AT(v_last, st), (phases >> st) & 1u, abort_flag);
                phases ^= 1u << st;
                if (!__all_sync(0xffffffffu, got)) break;
                uint8_t* v = sR + st * kTile;
                for (int row = u.nk - (n - 1) * kKeys + (lane >> 4); row < kKeys; row += 2)
                    *reinterpret_cast<uint4*>(v + ((lane >> 3) & 1) * kBox + row * 128 + (lane & 7) * 16) =
                        make_uint4(0u, 0u, 0u, 0u);
                attn2::fence_async_shared();
                __syncwarp();
                attn2::arrive_if(lane == 0, BAR_AT(full, st));
            }
        } else if (warp == 3) {
            // ---------------- which units ----------------
            bool bad = false;
            int top = 0, units = 0, nq0 = 0, nk0 = 0;
            for (int b = lane; b < a.B; b += 32) {
                const int q0 = a.cu_q[b], q1 = a.cu_q[b + 1], k0 = a.cu_k[b], k1 = a.cu_k[b + 1];
                if (q0 < 0 || q1 < q0 || q1 > a.Tq || k0 < 0 || k1 < k0 || k1 > a.Tk || k1 - k0 > kMaxKeys) bad = true;
                else if (q1 > q0) {
                    if (b < 32) { nq0 = q1 - q0; nk0 = k1 - k0; }
                    units += (q1 - q0 + 2 * a.P - 1) / (2 * a.P);
                    top = max(top, (k1 - k0) / kKeys + 2 * a.P / kKeys + 2);
                }
            }
            bad = __any_sync(0xffffffffu, bad);
            const int64_t total = bad ? 0 : (int64_t)__reduce_add_sync(0xffffffffu, units) * a.Hkv;
            top = __reduce_max_sync(0xffffffffu, top);
            if (bad && blockIdx.x == 0 && lane == 0) flag_error(a.dev_status, EAGLE_DEV_CAPACITY);
            for (int i = 0;; ++i) {
                // rounds of gridDim.x units, every second one dealt in the other direction
                const int64_t at = (int64_t)i * gridDim.x + ((i & 1) ? gridDim.x - 1 - blockIdx.x : blockIdx.x);
                Unit u{};
                u.head = -1;
                if (at < total) find_unit(a, (int)at, top, nq0, nk0, u);
                const bool got = attn2::wait_for(BAR_AT(info_empty, i % kInfo), (((uint32_t)i / kInfo) & 1u) ^ 1u, abort_flag);
                if (!__all_sync(0xffffffffu, got)) break;
                if (lane == 0) {
                    sh->info[i % kInfo] = u;
                    mbar_arrive(s32(&sh->info_full[i % kInfo]));
                }
                if (u.head < 0) break;                    // places of later rounds lie further on
            }
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
        const bool in_tile = p < a.P;
        const float sc = a.scale_log2;
        const uint64_t sc2 = attn2::f2(sc, sc);
        uint32_t tiles_done = 0, units_done = 0;
        bool ok = true;
        Unit u;
        for (int i = 0; ok; ++i) {
            if (!__all_sync(0xffffffffu, next_unit(i, u))) break;
            unit_read(i);
            const int pos = u.pos + slot * a.P + p;
            const bool valid = in_tile && pos < u.nq;
            // keys 0 .. seen - 1 are visible; a row of nobody sees all, its result is not used
            const int seen = valid ? min(u.nk, max(0, u.nk - u.nq + pos + 1)) : 0x7fffffff;
            const int n = u.tiles[slot];
            const bool idle = !__any_sync(0xffffffffu, valid);   // rows are independent: leave P as it is
            float mref = -INFINITY;
            uint64_t l2 = 0;                              // two partial sums
            for (int j = 0; j < n; ++j) {
                const bool got = attn2::wait_for(BAR_AT(s_full, slot), tiles_done & 1u, abort_flag);
                if (!__all_sync(0xffffffffu, got)) { ok = false; break; }
                ++tiles_done;
                tc_fence_after();
                if (!idle) {
                    uint32_t x[kKeys];
                    float m4[4];
                    attn2::load_row_nowait(s_addr, x, m4);
                    const int left = seen - j * kKeys;
                    attn2::tmem_wait_ld();
                    if (__any_sync(0xffffffffu, left < kKeys)) {
                        float y[kKeys];
#pragma unroll
                        for (int c = 0; c < kKeys; ++c) {
                            y[c] = c < left ? __uint_as_float(x[c]) : -INFINITY;
                            x[c] = __float_as_uint(y[c]);
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
                    // QK(j) was committed after PV(j - 1): O is complete up to tile j - 1
                    if (j > 0 && __any_sync(0xffffffffu, up)) attn2::rescale_row(o_addr, alpha);
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
            if (n > 0) {
                const bool got = attn2::wait_for(BAR_AT(o_full, slot), units_done & 1u, abort_flag);
                if (!__all_sync(0xffffffffu, got)) break;
                ++units_done;
                tc_fence_after();
            }
            if (idle) continue;
            float la, lb;
            attn2::unf2(l2, la, lb);
            const float l = la + lb;
            const bool none = n == 0 || l == 0.f;                        // sees no key (NaN goes through)
            const float inv = none ? 0.f : 1.f / l;
            const int64_t at = (int64_t)(u.q0 + pos) * a.Hq + u.head * a.G + g;
#pragma unroll
            for (int h = 0; h < 4; ++h) {
                uint32_t o[32];
                if (n > 0) tmem_ld32(o_addr + 32 * h, o);
                if (valid) {
                    uint4* dst = reinterpret_cast<uint4*>(a.out + at * kHeadDim + 32 * h);
#pragma unroll
                    for (int e = 0; e < 32; e += 8) {
                        uint32_t w[4];
#pragma unroll
                        for (int c = 0; c < 4; ++c)
                            w[c] = none ? 0u : pack2(__uint_as_float(o[e + 2 * c]) * inv, __uint_as_float(o[e + 2 * c + 1]) * inv);
                        dst[e / 8] = make_uint4(w[0], w[1], w[2], w[3]);
                    }
                }
            }
            if (valid && a.lse) a.lse[at] = none ? -INFINITY : (mref + log2f(l)) * 0.69314718055994531f;
        }
    }
    __syncthreads();
    if (tid == 0 && *abort_flag) flag_error(a.dev_status, EAGLE_DEV_TIMEOUT);
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, attn2::kTmemCols);
    }
#undef BAR
#undef BAR_AT
}

}  // namespace prompt_tc
}  // namespace eagle
