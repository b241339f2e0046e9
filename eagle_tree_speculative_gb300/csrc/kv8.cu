// Writers of the 8-bit K/V cache: eagle_kv8_append (one layer's new rows, packed by
// sequence) and eagle_kv8_commit (the accepted path's rows of every layer).
//
// Method.  The unit of work is one scale: the new rows of one block of 32 cache rows, for one
// (layer, sequence, kv head, K or V).  One warp owns it, so nothing is shared and no atomics
// order anything: it takes the rows' largest magnitude, the least power of two 2^e with amax <=
// 448 * 2^e, raises it to the block's present scale if the block holds rows already, and writes
// x * 2^-e as e4m3.  Where the scale rose, the rows held are read back, multiplied by old / new and
// rounded again: a power of two, so a code changes only where it becomes subnormal.  Scaling by
// a power of two is exact in fp32, so each value is rounded once, by the conversion.
// Up to 2 R rows stay in registers (16 bytes a lane and load, two rows at a time) between the
// maximum and the conversion; more are read twice, the second time from L2.
//
// Bound: HBM, 2 bytes read and 1 written per value; in practice the latency of a warp's few dependent
// accesses, so what counts is warps in flight.  Append, 8 x 2048 rows of 8 heads: 18.4 us, 5.5 TB/s (81% of
// a copy's rate); commit, 32 layers: 4 sequences 15.1 us, 64 sequences 35 us (its floor is 10 us).
#include "common.cuh"
#include "kv8_common.cuh"

namespace eagle {
namespace {

using kv8::kKv8Block;

constexpr unsigned kFull = 0xffffffffu;

struct Cache {
    uint8_t* k;
    uint8_t* v;
    float* k_scale;
    float* v_scale;
    int Lmax, NB;
};

// Magnitudes of bf16 order like integers: the larger ones of 8, as two packed halves, two elements
// an instruction.
__device__ __forceinline__ uint32_t top8(const uint4& x, uint32_t top) {
    top = __vmaxu2(top, x.x & 0x7fff7fffu);
    top = __vmaxu2(top, x.y & 0x7fff7fffu);
    top = __vmaxu2(top, x.z & 0x7fff7fffu);
    return __vmaxu2(top, x.w & 0x7fff7fffu);
}
// The same where infinities and NaN (exponents of all ones) do not count.
__device__ __forceinline__ uint32_t top8_finite(const uint4& x, uint32_t top) {
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t lo = w[i] & 0x7fffu, hi = (w[i] >> 16) & 0x7fffu;
        top = __vmaxu2(top, (lo < 0x7f80u ? lo : 0u) | ((hi < 0x7f80u ? hi : 0u) << 16));
    }
    return top;
}
__device__ __forceinline__ uint2 codes8(const uint4& x, float inv) {
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
    float f[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        f[2 * i] = __uint_as_float(w[i] << 16) * inv;
        f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u) * inv;
    }
    return make_uint2(kv8::e4m3x4(f[0], f[1], f[2], f[3]), kv8::e4m3x4(f[4], f[5], f[6], f[7]));
}

// Writes rows first .. first + m - 1 (all within one block) of the head slab `slab`; `src(t)`
// is the address of the row that becomes row first + t.
template <int R, class Src>
__device__ __forceinline__ int write_block(const Cache& c, int kv, int64_t slab, int first, int m, Src src) {
    const int lane = threadIdx.x & 31, half = lane >> 4, col = lane & 15;
    const int blk = first / kKv8Block, r0 = blk * kKv8Block;
    float* sp = (kv ? c.v_scale : c.k_scale) + slab * c.NB + blk;
    uint8_t* rows = (kv ? c.v : c.k) + (slab * c.Lmax + r0) * kHeadDim;
    const bool held = first > r0;         // the block holds rows r0 .. first - 1
    const float old = held ? *sp : 0.f;
    // a row behind the last is the last one again: its magnitudes count once more, which changes
    // nothing, and the loads need no condition (under one each waits for the one before)
    uint4 x[R];
    auto load = [&](int t0) {
#pragma unroll
        for (int s = 0; s < R; ++s)
            x[s] = __ldg(reinterpret_cast<const uint4*>(src(min(t0 + 2 * s + half, m - 1))) + col);
    };
    uint32_t top = 0u;
    for (int t0 = 0; t0 < m; t0 += 2 * R) {
        load(t0);
#pragma unroll
        for (int s = 0; s < R; ++s) top = top8(x[s], top);
    }
    top = __reduce_max_sync(kFull, max(top & 0xffffu, top >> 16));
    const bool odd = top >= 0x7f80u;      // an infinity or a NaN: the finite ones again
    if (odd) {
        top = 0u;
        for (int t0 = 0; t0 < m; t0 += 2 * R) {
            if (m > 2 * R) load(t0);
#pragma unroll
            for (int s = 0; s < R; ++s) top = top8_finite(x[s], top);
        }
        top = __reduce_max_sync(kFull, max(top & 0xffffu, top >> 16));
    }
    float scale = kv8::exp2i(kv8::scale_exp(__uint_as_float(top << 16)));
    if (held) {
        __syncwarp();                     // every lane has read the scale before it is replaced
        if (old >= scale) {
            scale = old;
        } else {
            const float by = old / scale;
            for (int t = lane >> 3; t < first - r0; t += 4) {        // 8 lanes x 16 bytes a row
                uint4* p = reinterpret_cast<uint4*>(rows + (int64_t)t * kHeadDim) + (lane & 7);
                const uint4 v = *p;
                uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float2 a = kv8::e4m3x2_float((uint16_t)w[i]);
                    const float2 b = kv8::e4m3x2_float((uint16_t)(w[i] >> 16));
                    w[i] = kv8::e4m3x4(a.x * by, a.y * by, b.x * by, b.y * by);
                }
                *p = make_uint4(w[0], w[1], w[2], w[3]);
            }
        }
    }
    if (lane == 0) *sp = scale;
    const float inv = 1.f / scale;        // exact: a power of two
    for (int t0 = 0; t0 < m; t0 += 2 * R) {
        if (m > 2 * R) load(t0);
#pragma unroll
        for (int s = 0; s < R; ++s) {
            const int t = t0 + 2 * s + half;
            const uint2 y = codes8(x[s], inv);
            if (t < m) *reinterpret_cast<uint2*>(rows + (int64_t)(first - r0 + t) * kHeadDim + col * 8) = y;
        }
    }
    return odd ? EAGLE_DEV_NONFINITE : 0;
}

// ---------------------------------------------------------------- append
constexpr int kAppendWarps = 4;

struct AppendArgs {
    const uint16_t* k;
    const uint16_t* v;
    int64_t k_stride, v_stride;
    const int32_t* cu;
    const int32_t* pos;
    Cache c;
    int T, B, Hkv;
    int32_t* dev_status;
};

// Blocks that sequence b's new rows touch; 0 for one that is skipped (flagged in err).
__device__ __forceinline__ int blocks_of(const AppendArgs& a, int b, int& err, bool& bad_cu) {
    if (b >= a.B) return 0;
    const int c0 = a.cu[b], c1 = a.cu[b + 1], p = a.pos[b];
    if (c0 < 0 || c1 < c0 || c1 > a.T) {
        bad_cu = true;
        return 0;
    }
    if (c1 == c0) return 0;
    if (p < 0 || (int64_t)p + (c1 - c0) > a.c.Lmax) {
        err |= EAGLE_DEV_CAPACITY;
        return 0;
    }
    return (p + (c1 - c0) + kKv8Block - 1) / kKv8Block - p / kKv8Block;
}

// grid (touched blocks, an upper bound; groups of kAppendWarps (head, K|V) units).  Five CTAs per SM:
// see the bound above
__global__ void __launch_bounds__(kAppendWarps * 32, 5) kv8_append_kernel(AppendArgs a) {
    const int lane = threadIdx.x & 31, unit = blockIdx.y * kAppendWarps + (threadIdx.x >> 5);
    // which (sequence, block) this is: the touched blocks counted along the sequences
    int left = (int)blockIdx.x, b = -1, at = 0, err = 0;
    bool bad_cu = false;
    for (int b0 = 0; b0 < a.B; b0 += 32) {
        const int n = blocks_of(a, b0 + lane, err, bad_cu);
        int sum = n;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(kFull, sum, o);
            if (lane >= o) sum += y;
        }
        const unsigned past = __ballot_sync(kFull, sum > left);
        if (past && b < 0) {
            const int l = __ffs(past) - 1;
            b = b0 + l;
            at = left - __shfl_sync(kFull, sum - n, l);
        }
        left -= __shfl_sync(kFull, sum, 31);
    }
    const bool first_warp = blockIdx.x == 0 && unit == 0;
    if (__any_sync(kFull, bad_cu)) {
        if (first_warp && lane == 0) flag_error(a.dev_status, EAGLE_DEV_CAPACITY);
        return;
    }
    if (first_warp && err) flag_error(a.dev_status, err);
    if (b < 0 || unit >= 2 * a.Hkv) return;
    const int kv = unit / a.Hkv, h = unit % a.Hkv;
    const int c0 = a.cu[b], end = a.pos[b] + (a.cu[b + 1] - c0), p = a.pos[b];
    const int blk = p / kKv8Block + at;
    const int lo = max(p, blk * kKv8Block), hi = min(end, (blk + 1) * kKv8Block);
    const int64_t stride = kv ? a.v_stride : a.k_stride;
    const uint16_t* x = (kv ? a.v : a.k) + (int64_t)(c0 + lo - p) * stride + h * kHeadDim;
    const int odd = write_block<kKv8Block / 2>(a.c, kv, (int64_t)b * a.Hkv + h, lo, hi - lo,
                                               [&](int t) { return x + t * stride; });
    if (odd) flag_error(a.dev_status, odd);
}

// ---------------------------------------------------------------- commit
constexpr int kCommitWarps = 16;

struct CommitArgs {
    const uint16_t* k;                    // of the tree, [n_layers, B, n, Hkv, 128]
    const uint16_t* v;
    Cache c;
    const int32_t* kv_len;
    int32_t* kv_len_out;
    const int32_t* path;
    const int32_t* accept_len;
    int n_layers, B, n, Hkv, D;
    int32_t* dev_status;
};

// One cluster of CS CTAs per sequence; its warps walk the (layer, K|V, head) units, each a few
// rows in one to three blocks.  The cluster barrier at the end orders every CTA's read of
// kv_len[b] before its update.
template <int CS>
__global__ void __launch_bounds__(kCommitWarps * 32, 2) kv8_commit_kernel(CommitArgs a) {
    __shared__ int s_path[kMaxNodes + 1];
    __shared__ int s_ok;
    const int tid = threadIdx.x, warp = tid >> 5;
    const int rank = (int)cg::this_cluster().block_rank();
    const int b = blockIdx.x / CS;
    const int acc = a.accept_len[b];
    const int L = a.kv_len[b];
    if (tid == 0) {
        int ok = acc >= 0, err = 0;
        if (ok) {
            if (acc > a.D || L < 0 || (int64_t)L + acc + 1 > a.c.Lmax) { ok = 0; err = EAGLE_DEV_CAPACITY; }
            for (int t = 0; ok && t <= acc; ++t) {
                const int p = a.path[(int64_t)b * (a.D + 1) + t];
                s_path[t] = p;
                if ((t == 0 && p != 0) || (t > 0 && p <= s_path[t - 1]) || p >= a.n) { ok = 0; err = EAGLE_DEV_BAD_TREE; }
            }
        }
        if (err && rank == 0) flag_error(a.dev_status, err);
        s_ok = ok;
    }
    __syncthreads();
    const bool ok = s_ok != 0;
    if (ok) {
        const int units = a.n_layers * 2 * a.Hkv;
        int odd = 0;
        for (int u = rank * kCommitWarps + warp; u < units; u += CS * kCommitWarps) {
            const int h = u % a.Hkv, kv = (u / a.Hkv) & 1;
            const int64_t seq = (int64_t)(u / (2 * a.Hkv)) * a.B + b;          // (layer, sequence)
            const uint16_t* x = (kv ? a.v : a.k) + (seq * a.n * a.Hkv + h) * kHeadDim;
            for (int lo = L; lo <= L + acc;) {
                const int hi = min(L + acc + 1, (lo / kKv8Block + 1) * kKv8Block);
                odd |= write_block<4>(a.c, kv, seq * a.Hkv + h, lo, hi - lo, [&](int t) {
                    return x + (int64_t)s_path[lo - L + t] * a.Hkv * kHeadDim;
                });
                lo = hi;
            }
        }
        if (odd) flag_error(a.dev_status, odd);
    }
    cg::this_cluster().sync();
    if (rank == 0 && tid == 0) a.kv_len_out[b] = ok ? L + acc + 1 : L;
}

bool misaligned(std::initializer_list<const void*> ps) {
    for (const void* p : ps)
        if (reinterpret_cast<uintptr_t>(p) & 15) return true;
    return false;
}

}  // namespace
}  // namespace eagle

using namespace eagle;

extern "C" eagle_status eagle_kv8_append(const void* k, const void* v, const int32_t* cu,
                                         const int32_t* pos, void* k8, void* v8, float* k_scale,
                                         float* v_scale, int T, int B, int Hkv, int head_dim,
                                         int Lmax, int64_t k_stride, int64_t v_stride,
                                         int32_t* dev_status, eagle_stream_t stream) {
    if (T < 0 || B < 0 || Hkv < 1 || Lmax < 1) return EAGLE_ERR_INVALID_ARG;
    if (head_dim != kHeadDim || Hkv > 65535 || Lmax > kv8::kMaxRows) return EAGLE_ERR_SHAPE;
    const int64_t row = (int64_t)Hkv * kHeadDim;
    if (k_stride < row || v_stride < row || k_stride % 8 != 0 || v_stride % 8 != 0)
        return EAGLE_ERR_INVALID_ARG;
    // a sequence's m rows touch at most m / 32 + 2 blocks
    const int64_t blocks = T / kKv8Block + 2LL * B;
    if (blocks > 0x7fffffffLL) return EAGLE_ERR_SHAPE;
    if (B == 0 || T == 0) return EAGLE_OK;              // nothing read or written
    if (!k || !v || !cu || !pos || !k8 || !v8 || !k_scale || !v_scale) return EAGLE_ERR_INVALID_ARG;
    if (misaligned({k, v, k8, v8})) return EAGLE_ERR_INVALID_ARG;
    AppendArgs a{};
    a.k = static_cast<const uint16_t*>(k);
    a.v = static_cast<const uint16_t*>(v);
    a.k_stride = k_stride; a.v_stride = v_stride;
    a.cu = cu; a.pos = pos;
    a.c = Cache{static_cast<uint8_t*>(k8), static_cast<uint8_t*>(v8), k_scale, v_scale, Lmax,
                (Lmax + kKv8Block - 1) / kKv8Block};
    a.T = T; a.B = B; a.Hkv = Hkv;
    a.dev_status = dev_status;
    const dim3 grid((unsigned)blocks, (unsigned)((2 * Hkv + kAppendWarps - 1) / kAppendWarps));
    kv8_append_kernel<<<grid, kAppendWarps * 32, 0, reinterpret_cast<cudaStream_t>(stream)>>>(a);
    EAGLE_CHECK_LAUNCH();
    return EAGLE_OK;
}

extern "C" eagle_status eagle_kv8_commit(const void* k_tree, const void* v_tree, void* k8, void* v8,
                                         float* k_scale, float* v_scale, const int32_t* kv_len,
                                         int32_t* kv_len_out, const int32_t* path,
                                         const int32_t* accept_len, int n_layers, int B, int n,
                                         int Hkv, int head_dim, int Lmax, int max_depth,
                                         int32_t* dev_status, eagle_stream_t stream) {
    if (n_layers < 0 || B < 0 || n < 1 || Hkv < 1 || Lmax < 1 || max_depth < 0)
        return EAGLE_ERR_INVALID_ARG;
    if (head_dim != kHeadDim || n > kMaxNodes || max_depth > kMaxNodes || Lmax > kv8::kMaxRows ||
        (int64_t)n_layers * 2 * Hkv > 0x3fffffffLL)
        return EAGLE_ERR_SHAPE;
    if (B == 0 || n_layers == 0) return EAGLE_OK;       // nothing read or written
    if (!k_tree || !v_tree || !k8 || !v8 || !k_scale || !v_scale || !kv_len || !kv_len_out || !path ||
        !accept_len)
        return EAGLE_ERR_INVALID_ARG;
    if (misaligned({k_tree, v_tree, k8, v8})) return EAGLE_ERR_INVALID_ARG;
    CommitArgs a{};
    a.k = static_cast<const uint16_t*>(k_tree);
    a.v = static_cast<const uint16_t*>(v_tree);
    a.c = Cache{static_cast<uint8_t*>(k8), static_cast<uint8_t*>(v8), k_scale, v_scale, Lmax,
                (Lmax + kKv8Block - 1) / kKv8Block};
    a.kv_len = kv_len; a.kv_len_out = kv_len_out; a.path = path; a.accept_len = accept_len;
    a.n_layers = n_layers; a.B = B; a.n = n; a.Hkv = Hkv; a.D = max_depth;
    a.dev_status = dev_status;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    // Clusters of 8 for up to a sequence an SM, of 4 for more.  us with 8 / 4 / 2 / 1, 32 layers: 1 sequence
    // 16 / 23 / 39 / 53, 64: 35 / 37 / 57 / 86, 100: 51 / 57 / 72 / 90, 153: 70 / 68 / 76 / 92, 305: 127 / 117 /
    // 127 / 137, 400: 160 / 148 / 156 / 166.
    const cudaError_t e = B <= cached_sm_count() ? launch_clustered(kv8_commit_kernel<8>, B, 8, kCommitWarps * 32, 0, s, a)
                                                 : launch_clustered(kv8_commit_kernel<4>, B, 4, kCommitWarps * 32, 0, s, a);
    return e == cudaSuccess ? EAGLE_OK : EAGLE_ERR_CUDA;
}
