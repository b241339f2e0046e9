// The pages of the K/V cache: which pages a sequence holds (eagle_pages_assign), and the accepted
// path's rows brought behind the committed ones (eagle_pages_commit).
//
// Assignment.  Everything is decided from the state before the call and nothing is written until it is
// known that the call can be carried out, in three steps of one cluster with a barrier between
// them: (1) per slot, a warp each: what it keeps, how many fresh pages it needs, whether all numbers
// are in range; per part of refs: how many pages are free; (2) the free pages that are needed, by
// number; (3) per slot: its table, and the differences in refs (integer atomics: their order does
// not matter).  A fresh page had refs = 0, so no slot that is still being read holds it, and what a call
// gives back is free for the next one only: no copy's source is another's destination.
// A second kernel copies the rows of pages that sequences share no longer, in every layer.
//
// Commit.  The path is strictly increasing from 0, so path[t] >= t: rows are moved in rounds of rising t, a
// round's rows all read before any of it is written.  A write to row t of one round is below every
// path[t'] of the rounds after it, and no earlier round wrote a row of this one's sources.
#include "paged_common.cuh"

namespace eagle {
namespace {

// ---------------- assignment ----------------
// Threads of a CTA: a warp a slot in calls of up to kPlanFew / 32 * kCluster slots, whose barriers cost less (us with
// 256 / 512 / 1024, growing: 64 slots 6.6 / 7.1 / 8.4, 96 8.4 / 7.1 / 8.4, 256 13.7 / 9.8 / 9.0, 1024 39.5 / 24.5 / 20.8).
// Growing takes 21 us more for every 1024 slots (8192 175 us, 65 536 1.4 ms).  A reorder in which most slots are the only
// ones to go on with their source looks through src, up to the slot, for each: 1024 32 us, 4096 148, 8192 410, 16 384
// 1.3 ms, 65 536 20 ms.
constexpr int kPlanFew = 256, kPlanMany = 512;

// The workspace: what is known of each slot, the copies, the number of copies, the free pages in each CTA's part of
// refs, fresh page numbers, and a table of what slots keep.
struct Slot {
    int fresh;                                    // pages it needs
    int from, rows;                               // a page to copy, how many rows of it; rows = 0: none
    int length;                                   // its rows
    int bad;
};
struct Copy {
    int from, to, rows, pad;
};
constexpr int kCluster = 8;
constexpr int kMaxSlots = 1 << 16;                // a slot may look through those before it

struct AssignArgs {
    int32_t *table, *held, *refs, *kv_len;
    const int32_t *grow, *src;
    Copy* copies;                                 // [B]
    Slot* slots;                                  // [B]
    int32_t* copy_count;
    int32_t* free_count;                          // [kCluster]
    int32_t* free_ids;                            // [min(N, B P)]
    int32_t* kept;                                // [B][P]
    int B, N, P, shift;
    int32_t* dev_status;
};

size_t assign_words(int B, int N, int P) {
    const int64_t cells = (int64_t)B * P;
    return (size_t)B * ((sizeof(Copy) + sizeof(Slot)) / 4) + 1 + kCluster + (size_t)(N < cells ? N : cells) + (size_t)cells;
}

// Warp-wide: the slot that goes on in the page in which s's rows end: s itself, else the first of those that
// go on with s.
__device__ __forceinline__ bool goes_on(const AssignArgs& a, int b, int s) {
    if (!a.src || b == s) return true;
    const int lane = threadIdx.x & 31;
    if (a.src[s] == s) return false;
    for (int x0 = 0; x0 < b; x0 += 128) {         // four loads on their way at a time
        bool other = false;
#pragma unroll
        for (int y = 0; y < 4; ++y) {
            const int x = x0 + 32 * y + lane;
            other |= x < b && a.src[x] == s;
        }
        if (__any_sync(0xffffffffu, other)) return false;
    }
    return true;
}

template <int kPlanThreads>
__global__ void __launch_bounds__(kPlanThreads) pages_plan_kernel(AssignArgs a) {
    constexpr int kPlanWarps = kPlanThreads / 32;
    __shared__ int s_sum[kPlanWarps];
    // the copying kernel may be launched meanwhile; it waits for this one itself
    asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int rank = (int)cg::this_cluster().block_rank();
    const int page = 1 << a.shift;
    auto all_sync = [] { cg::this_cluster().sync(); };
    auto block_sum = [&](int x) {                 // of every thread; for every thread
        x = __reduce_add_sync(0xffffffffu, x);
        __syncthreads();
        if (lane == 0) s_sum[warp] = x;
        __syncthreads();
        int t = 0;
        for (int w = 0; w < kPlanWarps; ++w) t += s_sum[w];
        return t;
    };

    // ---- (1) what each slot keeps and needs; how many pages are free ----
    for (int b = rank * kPlanWarps + warp; b < a.B; b += kCluster * kPlanWarps) {
        const int s = a.src ? a.src[b] : b;
        Slot y = {};
        const int had = a.held[b], grow = a.grow[b];
        bool bad = s < -1 || s >= a.B || had < 0 || had > a.P || grow < 0;
        int theirs = 0;
        if (!bad && s >= 0) {
            y.length = a.kv_len[s];
            theirs = a.held[s];
            bad = y.length < 0 || theirs < 0 || theirs > a.P || (int64_t)y.length > (int64_t)theirs << a.shift;
        }
        const int full = y.length >> a.shift, part = y.length & (page - 1);
        const int64_t need64 = ((int64_t)y.length + grow + page - 1) >> a.shift;
        bad = bad || need64 > a.P;
        if (!bad) {
            const int need = (int)need64;
            const int32_t* old = a.table + (int64_t)b * a.P;
            const int32_t* from = a.table + (int64_t)max(s, 0) * a.P;
            int32_t* kept = a.kept + (int64_t)b * a.P;
            if (s != b) {
                // its own pages are all given back or found again; those of s up to the full ones are shared
                for (int t = lane; t < had; t += 32) {
                    const int id = old[t];
                    bad |= id < 0 || id >= a.N;
                }
                for (int t = lane; t < full; t += 32) {
                    const int id = from[t];
                    bad |= id < 0 || id >= a.N;
                    kept[t] = id;
                }
                y.fresh = need - full;
            } else {
                for (int t0 = full; t0 < max(need, had); t0 += 32) {
                    const int t = t0 + lane;
                    int id = -1;
                    if (t < had) {
                        id = old[t];
                        bad |= id < 0 || id >= a.N;
                        if (id >= 0 && id < a.N && a.refs[id] > 1) id = -1;
                    }
                    if (t < need) kept[t] = id;
                    y.fresh += __popc(__ballot_sync(0xffffffffu, t < need && id < 0));
                }
                // full pages that stay are not looked at
            }
            if (part) {
                const int id = from[full];
                bad |= id < 0 || id >= a.N;
                const bool alone = !bad && a.refs[id] <= 1;
                const bool goes = goes_on(a, b, s);
                if (alone && goes) {
                    if (s != b) {
                        if (lane == 0) kept[full] = id;
                        --y.fresh;
                    }
                } else {
                    if (s != b && lane == 0) kept[full] = -1;
                    y.from = id;
                    y.rows = part;
                }
            }
        }
        y.bad = __any_sync(0xffffffffu, bad);
        if (lane == 0) a.slots[b] = y;
    }
    const int per = (a.N + kCluster - 1) / kCluster, r0 = min(a.N, rank * per), r1 = min(a.N, r0 + per);
    int mine = 0;
    for (int p = r0 + tid; p < r1; p += kPlanThreads) mine += a.refs[p] == 0;
    const int frees = block_sum(mine);
    if (tid == 0) a.free_count[rank] = frees;
    all_sync();

    // ---- can it be done? ----
    bool bad = false;
    int fresh = 0, copies = 0;                    // fresh: at most B * P < 2^30
    for (int b = tid; b < a.B; b += kPlanThreads) {
        bad |= __ldcg(&a.slots[b].bad) != 0;
        fresh += __ldcg(&a.slots[b].fresh);
        copies += __ldcg(&a.slots[b].rows) != 0;
    }
    const int total = block_sum(fresh);
    if (rank == 0) copies = block_sum(copies);
    int before = 0, there = 0;                    // free pages of lower parts, of all
    for (int r = 0; r < kCluster; ++r) {
        const int x = __ldcg(a.free_count + r);
        before += r < rank ? x : 0;
        there += x;
    }
    if (__syncthreads_or(bad) || total > there) {       // alike in every CTA
        if (rank == 0 && tid == 0) {
            flag_error(a.dev_status, EAGLE_DEV_CAPACITY);
            *a.copy_count = 0;
        }
        return;
    }
    if (rank == 0 && tid == 0) *a.copy_count = copies;

    // ---- (2) the first `total` free pages ----
    for (int p0 = r0; p0 < r1 && before < total; p0 += kPlanThreads) {
        const int p = p0 + tid;
        const bool is = p < r1 && a.refs[p] == 0;
        const unsigned who = __ballot_sync(0xffffffffu, is);
        __syncthreads();
        if (lane == 0) s_sum[warp] = __popc(who);
        __syncthreads();
        int at = before + __popc(who & ((1u << lane) - 1u)), all = 0;
        for (int w = 0; w < kPlanWarps; ++w) {
            at += w < warp ? s_sum[w] : 0;
            all += s_sum[w];
        }
        if (is && at < total) a.free_ids[at] = p;
        before += all;
    }
    all_sync();

    // ---- (3) tables and counts ----
    int seen = 0, fresh_seen = 0, copies_seen = 0;    // fresh pages and copies of the slots before `seen`
    for (int b = rank * kPlanWarps + warp; b < a.B; b += kCluster * kPlanWarps) {
        int f = 0, c = 0;
        for (int x = seen + lane; x < b; x += 32) {
            f += __ldcg(&a.slots[x].fresh);
            c += __ldcg(&a.slots[x].rows) != 0;
        }
        fresh_seen += __reduce_add_sync(0xffffffffu, f);
        copies_seen += __reduce_add_sync(0xffffffffu, c);
        seen = b;
        int at = fresh_seen;
        const int copy = copies_seen;
        const int rows = __ldcg(&a.slots[b].rows), from = __ldcg(&a.slots[b].from);
        const int s = a.src ? a.src[b] : b;
        const int length = __ldcg(&a.slots[b].length), had = a.held[b], full = length >> a.shift;
        const int need = (int)(((int64_t)length + a.grow[b] + page - 1) >> a.shift);
        // (the pages of s from full on are this slot's only where `kept` says so)
        const int known = s == b ? need : min(need, full + ((length & (page - 1)) != 0));
        const int32_t* kept = a.kept + (int64_t)b * a.P;
        int32_t* row = a.table + (int64_t)b * a.P;
        for (int t0 = s == b ? full : 0; t0 < max(need, had); t0 += 32) {
            const int t = t0 + lane;
            int id = t < known ? __ldcg(kept + t) : -1;
            const bool fresh_page = t < need && id < 0;
            const unsigned who = __ballot_sync(0xffffffffu, fresh_page);
            if (fresh_page) id = __ldcg(a.free_ids + at + __popc(who & ((1u << lane) - 1u)));
            at += __popc(who);
            const int was = t < had ? row[t] : -1;
            if (t < max(need, had) && id != was) {
                row[t] = id;
                if (id >= 0) atomicAdd(a.refs + id, 1);
                if (was >= 0) atomicAdd(a.refs + was, -1);
            }
            if (t == full && t < need && rows) a.copies[copy] = Copy{from, id, rows, 0};
        }
        __syncwarp();
        if (lane == 0) {
            a.held[b] = need;
            a.kv_len[b] = length;
        }
    }
}

constexpr int kCopyThreads = 256, kCopyWarps = kCopyThreads / 32;
constexpr int kCopyBlocks = 4;                    // of an SM
constexpr int kCopyAhead = 8;                     // 16-byte loads of a lane on their way

// A warp takes a copy's rows of one layer, K or V, and head at a time: they lie in one piece.
__global__ void __launch_bounds__(kCopyThreads, kCopyBlocks)
pages_copy_kernel(uint16_t* k, uint16_t* v, const Copy* copies, const int32_t* count, int n_layers, int N, int Hkv, int shift) {
    asm volatile("griddepcontrol.wait;\n" ::: "memory");
    const int lane = threadIdx.x & 31, per = n_layers * 2 * Hkv;
    const int64_t units = (int64_t)__ldcg(count) * per;
    for (int64_t u = (int64_t)blockIdx.x * kCopyWarps + (threadIdx.x >> 5); u < units; u += (int64_t)gridDim.x * kCopyWarps) {
        const int i = (int)(u / per), part = (int)(u - (int64_t)i * per), h = part % Hkv, layer = part / (2 * Hkv);
        const int4 c = __ldcg(reinterpret_cast<const int4*>(copies + i));
        uint16_t* base = ((part / Hkv) & 1 ? v : k) + (((int64_t)layer * N * Hkv) << shift) * kHeadDim;
        const uint4* src = reinterpret_cast<const uint4*>(base + paged::row_at(c.x, h, 0, Hkv, shift)) + lane;
        uint4* dst = reinterpret_cast<uint4*>(base + paged::row_at(c.y, h, 0, Hkv, shift)) + lane;
        const int chunks = c.z * (kHeadDim / 8);
        for (int x0 = 0; x0 < chunks; x0 += 32 * kCopyAhead) {
            uint4 x[kCopyAhead];
#pragma unroll
            for (int y = 0; y < kCopyAhead; ++y)
                if (x0 + 32 * y + lane < chunks) x[y] = src[x0 + 32 * y];
#pragma unroll
            for (int y = 0; y < kCopyAhead; ++y)
                if (x0 + 32 * y + lane < chunks) dst[x0 + 32 * y] = x[y];
        }
    }
}

// ---------------- commit ----------------
// Threads of a CTA, eight of which look after a sequence: what is waited for is memory, so many warps, as long as all
// CTAs have an SM of their own (64 sequences, 32 layers: 12.1 us with 256, 21.1 with 512; one: 5.2 with 512, 6.1 with 256).
// A warp has the rows of kCommitUnits (layer, K or V, kv head)s on their way at once (1 / 2 / 4 / 8: 64 sequences that
// are in HBM 23 / 21 / 25 / 35 us, 16 sequences of 60 moved rows 25.4 / 22.8 / 24.4 / 48.8).
constexpr int kCommitFew = 512, kCommitMany = 256, kCommitCluster = 8;
constexpr int kCommitUnits = 2;

struct CommitArgs {
    uint16_t *k, *v;
    const int32_t *table, *kv_len, *path, *accept_len;
    int32_t* kv_len_out;
    int n_layers, B, N, Hkv, shift, P, D;
    int32_t* dev_status;
};

__global__ void __launch_bounds__(kCommitFew) pages_commit_kernel(CommitArgs a) {
    __shared__ int s_from[kMaxNodes + 1], s_to[kMaxNodes + 1];      // row of a head's slab, all pages one behind the other
    __shared__ int s_moves, s_ok;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int rank = (int)cg::this_cluster().block_rank(), b = blockIdx.x / kCommitCluster, warps = blockDim.x >> 5;
    const int32_t* path = a.path + (int64_t)b * (a.D + 1);
    const int acc = a.accept_len[b], L = a.kv_len[b];
    if (warp == 0) {
        const int ahead = path[min(lane, a.D)];   // on its way together with the lengths
        int err = 0, moves = 0;
        if (acc >= 0) {
            if (acc > a.D || L < 0 || (int64_t)L + acc + 1 > (int64_t)a.P << a.shift) err = EAGLE_DEV_CAPACITY;
            for (int t0 = 0; err == 0 && t0 <= acc; t0 += 32) {
                const int t = t0 + lane;
                const bool on = t <= acc;
                const int p = !on ? 0 : t0 == 0 ? ahead : path[t], before = __shfl_up_sync(0xffffffffu, p, 1);
                const int q = lane > 0 ? before : t0 > 0 ? path[t0 - 1] : -1;
                int e = 0, from = 0, to = 0;
                if (on && (t == 0 ? p != 0 : p <= q)) e = EAGLE_DEV_BAD_TREE;
                else if (on && (int64_t)L + p >= (int64_t)a.P << a.shift) e = EAGLE_DEV_CAPACITY;
                else if (on && p != t) {
                    from = a.table[(int64_t)b * a.P + ((L + p) >> a.shift)];
                    to = a.table[(int64_t)b * a.P + ((L + t) >> a.shift)];
                    if (from < 0 || from >= a.N || to < 0 || to >= a.N) e = EAGLE_DEV_CAPACITY;
                }
                err = __reduce_or_sync(0xffffffffu, e);
                // the rows that move, in order
                const unsigned who = __ballot_sync(0xffffffffu, on && p != t);
                if (on && p != t) {
                    const int at = moves + __popc(who & ((1u << lane) - 1u)), mask = (1 << a.shift) - 1;
                    s_from[at] = ((from * a.Hkv) << a.shift) + ((L + p) & mask);
                    s_to[at] = ((to * a.Hkv) << a.shift) + ((L + t) & mask);
                }
                moves += __popc(who);
            }
        }
        if (lane == 0) {
            if (err && rank == 0) flag_error(a.dev_status, err);
            s_moves = err ? 0 : moves;
            s_ok = acc >= 0 && err == 0;
        }
    }
    __syncthreads();
    const int moves = s_moves;
    const int units = moves ? a.n_layers * 2 * a.Hkv : 0;            // (layer, K|V, kv head)
    const int stride = kCommitCluster * warps;
    for (int u0 = rank * warps + warp; u0 < units; u0 += kCommitUnits * stride) {
        uint4* base[kCommitUnits];
#pragma unroll
        for (int i = 0; i < kCommitUnits; ++i) {
            const int u = min(u0 + i * stride, units - 1), h = u % a.Hkv, layer = u / (2 * a.Hkv);
            base[i] = reinterpret_cast<uint4*>(((u / a.Hkv) & 1 ? a.v : a.k)) +
                      ((((int64_t)layer * a.N * a.Hkv + h) << a.shift) * (kHeadDim / 8)) + (lane & 15);
        }
        for (int m0 = 0; m0 < moves; m0 += 8) {                      // four pairs of rows a round
            uint4 x[kCommitUnits][4];
#pragma unroll
            for (int y = 0; y < 4; ++y) {
                const int m = m0 + 2 * y + (lane >> 4);
                const int64_t from = m < moves ? (int64_t)s_from[m] * (kHeadDim / 8) : -1;
#pragma unroll
                for (int i = 0; i < kCommitUnits; ++i)
                    if (from >= 0 && u0 + i * stride < units) x[i][y] = base[i][from];
            }
            __syncwarp();
#pragma unroll
            for (int y = 0; y < 4; ++y) {
                const int m = m0 + 2 * y + (lane >> 4);
                const int64_t to = m < moves ? (int64_t)s_to[m] * (kHeadDim / 8) : -1;
#pragma unroll
                for (int i = 0; i < kCommitUnits; ++i)
                    if (to >= 0 && u0 + i * stride < units) base[i][to] = x[i][y];
            }
            __syncwarp();
        }
    }
    // every CTA has read kv_len[b] before it changes
    cg::this_cluster().sync();
    if (rank == 0 && tid == 0) a.kv_len_out[b] = s_ok ? L + acc + 1 : L;
}

eagle_status check_pages(int n_layers, int B, int N, int Hkv, int page, int head_dim, int P) {
    if (n_layers < 0 || B < 0 || N < 1 || Hkv < 1 || P < 1) return EAGLE_ERR_INVALID_ARG;
    if (head_dim != kHeadDim || B > kMaxSlots || !paged::page_ok(page) || (int64_t)N * Hkv * page > paged::kMaxPool ||
        (int64_t)P * page > paged::kMaxRows || (int64_t)B * P > 0x3fffffff || (int64_t)n_layers * Hkv > 0x3fffffff)
        return EAGLE_ERR_SHAPE;
    return EAGLE_OK;
}

}  // namespace
}  // namespace eagle

using namespace eagle;

extern "C" size_t eagle_pages_workspace_size(int B, int N, int P) {
    if (B < 1 || B > kMaxSlots || N < 1 || P < 1 || (int64_t)B * P > 0x3fffffff) return 0;
    return assign_words(B, N, P) * 4;
}

extern "C" eagle_status eagle_pages_assign(void* k_pages, void* v_pages, int32_t* page_table, int32_t* held,
                                           int32_t* refs, int32_t* kv_len, const int32_t* grow,
                                           const int32_t* src, int n_layers, int B, int N, int Hkv, int page,
                                           int head_dim, int P, void* workspace, size_t ws_bytes,
                                           int32_t* dev_status, eagle_stream_t stream) {
    const eagle_status ok = check_pages(n_layers, B, N, Hkv, page, head_dim, P);
    if (ok != EAGLE_OK || B == 0) return ok;
    if (!page_table || !held || !refs || !kv_len || !grow || (n_layers > 0 && (!k_pages || !v_pages)))
        return EAGLE_ERR_INVALID_ARG;
    for (const void* p : {(const void*)k_pages, (const void*)v_pages, (const void*)workspace})
        if (reinterpret_cast<uintptr_t>(p) & 15) return EAGLE_ERR_INVALID_ARG;
    if (!workspace || ws_bytes < assign_words(B, N, P) * 4) return EAGLE_ERR_CAPACITY;
    AssignArgs a;
    a.table = page_table; a.held = held; a.refs = refs; a.kv_len = kv_len;
    a.grow = grow; a.src = src;
    a.copies = static_cast<Copy*>(workspace);
    a.slots = reinterpret_cast<Slot*>(a.copies + B);
    a.copy_count = reinterpret_cast<int32_t*>(a.slots + B);
    a.free_count = a.copy_count + 1;
    a.free_ids = a.free_count + kCluster;
    a.kept = a.free_ids + (N < (int64_t)B * P ? N : (int64_t)B * P);
    a.B = B; a.N = N; a.P = P; a.shift = paged::page_shift(page);
    a.dev_status = dev_status;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    const cudaError_t e = B <= kCluster * (kPlanFew / 32) ? launch_clustered(pages_plan_kernel<kPlanFew>, 1, kCluster, kPlanFew, 0, s, a)
                                                          : launch_clustered(pages_plan_kernel<kPlanMany>, 1, kCluster, kPlanMany, 0, s, a);
    if (e != cudaSuccess) return EAGLE_ERR_CUDA;
    if (n_layers > 0) {
        const int64_t blocks = ((int64_t)B * n_layers * 2 * Hkv + kCopyWarps - 1) / kCopyWarps, most = (int64_t)kCopyBlocks * cached_sm_count();
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3((unsigned)(blocks < most ? blocks : most));
        cfg.blockDim = dim3(kCopyThreads);
        cfg.stream = s;
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[0].val.programmaticStreamSerializationAllowed = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        if (cudaLaunchKernelEx(&cfg, pages_copy_kernel, static_cast<uint16_t*>(k_pages), static_cast<uint16_t*>(v_pages),
                               (const Copy*)a.copies, (const int32_t*)a.copy_count, n_layers, N, Hkv, a.shift) != cudaSuccess)
            return EAGLE_ERR_CUDA;
    }
    return EAGLE_OK;
}

extern "C" eagle_status eagle_pages_commit(void* k_pages, void* v_pages, const int32_t* page_table,
                                           const int32_t* kv_len, int32_t* kv_len_out, const int32_t* path,
                                           const int32_t* accept_len, int n_layers, int B, int N, int Hkv,
                                           int page, int head_dim, int P, int max_depth, int32_t* dev_status,
                                           eagle_stream_t stream) {
    const eagle_status ok = check_pages(n_layers, B, N, Hkv, page, head_dim, P);
    if (ok != EAGLE_OK) return ok;
    if (max_depth < 0) return EAGLE_ERR_INVALID_ARG;
    if (max_depth > kMaxNodes) return EAGLE_ERR_SHAPE;
    if (B == 0 || n_layers == 0) return EAGLE_OK;       // nothing read or written
    if (!k_pages || !v_pages || !page_table || !kv_len || !kv_len_out || !path || !accept_len) return EAGLE_ERR_INVALID_ARG;
    for (const void* p : {(const void*)k_pages, (const void*)v_pages})
        if (reinterpret_cast<uintptr_t>(p) & 15) return EAGLE_ERR_INVALID_ARG;
    CommitArgs a;
    a.k = static_cast<uint16_t*>(k_pages); a.v = static_cast<uint16_t*>(v_pages);
    a.table = page_table; a.kv_len = kv_len; a.path = path; a.accept_len = accept_len;
    a.kv_len_out = kv_len_out;
    a.n_layers = n_layers; a.B = B; a.N = N; a.Hkv = Hkv; a.shift = paged::page_shift(page); a.P = P; a.D = max_depth;
    a.dev_status = dev_status;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    const int threads = B * (int64_t)kCommitCluster <= cached_sm_count() ? kCommitFew : kCommitMany;
    return launch_clustered(pages_commit_kernel, B, kCommitCluster, threads, 0, s, a) == cudaSuccess ? EAGLE_OK : EAGLE_ERR_CUDA;
}
