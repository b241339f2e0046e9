// Writers of the 8-bit K/V cache: eagle_kv8_append (one layer's new rows, packed by
// sequence) and eagle_kv8_commit (the accepted path's rows of every layer).
//
// Method.  The unit of work is one scale: the new rows of one block of 32 cache rows, for one
// (layer, sequence, kv head, K or V).  One warp owns it, so nothing is shared and no atomics
// order anything: it holds the block's new rows in registers (up to 32 rows of 256 bytes, 16
// bytes a lane and load, two rows at a time), takes their largest magnitude, the least power
// of two 2^e with amax <= 448 * 2^e, raises it to the block's present scale if the block holds
// rows already, and writes x * 2^-e as e4m3.  Where the scale rose, the rows held are read
// back, multiplied by old / new and rounded again: a power of two, so a code changes only
// where it becomes subnormal.  Scaling by a power of two is exact in fp32, so each value is
// rounded once, by the conversion.
//
// Bound: HBM, 2 bytes read and 1 written per value.
#include "common.cuh"
#include "kv8_common.cuh"

namespace eagle {
namespace {

using kv8::kKv8Block;

constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
constexpr unsigned kFull = 0xffffffffu;

struct Cache {
    uint8_t* code[2];                     // K, V
    float* scale[2];
    int Lmax, NB;
};

// Writes rows first .. first + m - 1 (all within one block) of the head slab `slab`; `src(t)`
// is the address of the row that becomes row first + t, 32 lanes x 16 bytes being two rows.
template <class Src>
__device__ __forceinline__ int write_block(const Cache& c, int kv, int64_t slab, int first, int m,
                                           Src src) {
    const int lane = threadIdx.x & 31, half = lane >> 4, col = lane & 15;
    uint4 x[kKv8Block / 2];
#pragma unroll
    for (int s = 0; s < kKv8Block / 2; ++s) {
        // a row behind the last is the last one again: its magnitudes count once more, which changes
        // nothing, and the loads need no condition (under one each waits for the one before)
        x[s] = __ldg(reinterpret_cast<const uint4*>(src(min(2 * s + half, m - 1))) + col);
    }
    // the largest finite magnitude, as the bits of a bf16 (magnitudes order like integers);
    // an exponent of all ones is an infinity or a NaN and does not count
    uint32_t top = 0u;
    bool odd = false;
#pragma unroll
    for (int s = 0; s < kKv8Block / 2; ++s) {
        const uint32_t w[4] = {x[s].x, x[s].y, x[s].z, x[s].w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t lo = w[i] & 0x7fffu, hi = (w[i] >> 16) & 0x7fffu;
            if (lo >= 0x7f80u) odd = true; else top = max(top, lo);
            if (hi >= 0x7f80u) odd = true; else top = max(top, hi);
        }
    }
    top = __reduce_max_sync(kFull, top);
    int e = kv8::scale_exp(__uint_as_float(top << 16));

    const int blk = first / kKv8Block, r0 = blk * kKv8Block;
    float* sp = c.scale[kv] + slab * c.NB + blk;
    uint8_t* rows = c.code[kv] + (slab * c.Lmax + r0) * kHeadDim;
    float scale = kv8::exp2i(e);
    if (first > r0) {                     // the block holds rows r0 .. first - 1
        const float old = *sp;
        __syncwarp();                     // every lane has read it before it is replaced
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
#pragma unroll
    for (int s = 0; s < kKv8Block / 2; ++s) {
        const int t = 2 * s + half;
        if (t < m) {
            const uint32_t w[4] = {x[s].x, x[s].y, x[s].z, x[s].w};
            float f[8];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                f[2 * i] = __uint_as_float(w[i] << 16) * inv;
                f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u) * inv;
            }
            *reinterpret_cast<uint2*>(rows + (int64_t)(first - r0 + t) * kHeadDim + col * 8) =
                make_uint2(kv8::e4m3x4(f[0], f[1], f[2], f[3]), kv8::e4m3x4(f[4], f[5], f[6], f[7]));
        }
    }
    return odd ? EAGLE_DEV_NONFINITE : 0;
}

// ---------------------------------------------------------------- append
struct AppendArgs {
    const uint16_t* x[2];                 // K, V rows
    int64_t stride[2];
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

// grid (touched blocks, an upper bound; groups of kWarps (head, K|V) units)
__global__ void __launch_bounds__(kThreads) kv8_append_kernel(AppendArgs a) {
    const int lane = threadIdx.x & 31, unit = blockIdx.y * kWarps + (threadIdx.x >> 5);
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
    const uint16_t* x = a.x[kv] + (int64_t)(c0 + lo - p) * a.stride[kv] + h * kHeadDim;
    const int odd = write_block(a.c, kv, (int64_t)b * a.Hkv + h, lo, hi - lo,
                                [&](int t) { return x + (int64_t)t * a.stride[kv]; });
    if (odd) flag_error(a.dev_status, odd);
}

// ---------------------------------------------------------------- commit
struct CommitArgs {
    const uint16_t* x[2];                 // K, V of the tree, [n_layers, B, n, Hkv, 128]
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
__global__ void __launch_bounds__(kThreads) kv8_commit_kernel(CommitArgs a) {
    __shared__ int s_path[kMaxNodes + 1];
    __shared__ int s_ok;
    const int tid = threadIdx.x, warp = tid >> 5;
    const int rank = CS > 1 ? (int)cg::this_cluster().block_rank() : 0;
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
        for (int u = rank * kWarps + warp; u < units; u += CS * kWarps) {
            const int h = u % a.Hkv, kv = (u / a.Hkv) & 1;
            const int64_t seq = (int64_t)(u / (2 * a.Hkv)) * a.B + b;          // (layer, sequence)
            const uint16_t* x = a.x[kv] + (seq * a.n * a.Hkv + h) * kHeadDim;
            for (int lo = L; lo <= L + acc;) {
                const int hi = min(L + acc + 1, (lo / kKv8Block + 1) * kKv8Block);
                odd |= write_block(a.c, kv, seq * a.Hkv + h, lo, hi - lo, [&](int t) {
                    return x + (int64_t)s_path[lo - L + t] * a.Hkv * kHeadDim;
                });
                lo = hi;
            }
        }
        if (odd) flag_error(a.dev_status, odd);
    }
    if constexpr (CS > 1) cg::this_cluster().sync();
    else __syncthreads();
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
    if (head_dim != kHeadDim || Hkv > 65535) return EAGLE_ERR_SHAPE;
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
    a.x[0] = static_cast<const uint16_t*>(k);
    a.x[1] = static_cast<const uint16_t*>(v);
    a.stride[0] = k_stride; a.stride[1] = v_stride;
    a.cu = cu; a.pos = pos;
    a.c = Cache{{static_cast<uint8_t*>(k8), static_cast<uint8_t*>(v8)}, {k_scale, v_scale}, Lmax,
                (Lmax + kKv8Block - 1) / kKv8Block};
    a.T = T; a.B = B; a.Hkv = Hkv;
    a.dev_status = dev_status;
    const dim3 grid((unsigned)blocks, (unsigned)((2 * Hkv + kWarps - 1) / kWarps));
    kv8_append_kernel<<<grid, kThreads, 0, reinterpret_cast<cudaStream_t>(stream)>>>(a);
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
    if (head_dim != kHeadDim || n > kMaxNodes || max_depth > kMaxNodes ||
        (int64_t)n_layers * 2 * Hkv > 0x3fffffffLL)
        return EAGLE_ERR_SHAPE;
    if (B == 0 || n_layers == 0) return EAGLE_OK;       // nothing read or written
    if (!k_tree || !v_tree || !k8 || !v8 || !k_scale || !v_scale || !kv_len || !kv_len_out || !path ||
        !accept_len)
        return EAGLE_ERR_INVALID_ARG;
    if (misaligned({k_tree, v_tree, k8, v8})) return EAGLE_ERR_INVALID_ARG;
    CommitArgs a{};
    a.x[0] = static_cast<const uint16_t*>(k_tree);
    a.x[1] = static_cast<const uint16_t*>(v_tree);
    a.c = Cache{{static_cast<uint8_t*>(k8), static_cast<uint8_t*>(v8)}, {k_scale, v_scale}, Lmax,
                (Lmax + kKv8Block - 1) / kKv8Block};
    a.kv_len = kv_len; a.kv_len_out = kv_len_out; a.path = path; a.accept_len = accept_len;
    a.n_layers = n_layers; a.B = B; a.n = n; a.Hkv = Hkv; a.D = max_depth;
    a.dev_status = dev_status;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    // clusters of 8 while every CTA is resident at once, fewer for large batches
    const int sms = device_sm_count();
    int cs = 8;
    while (cs > 1 && (int64_t)B * cs > 4LL * sms) cs >>= 1;
    cudaError_t e;
    switch (cs) {
        case 8: e = launch_clustered(kv8_commit_kernel<8>, B, 8, kThreads, 0, s, a); break;
        case 4: e = launch_clustered(kv8_commit_kernel<4>, B, 4, kThreads, 0, s, a); break;
        case 2: e = launch_clustered(kv8_commit_kernel<2>, B, 2, kThreads, 0, s, a); break;
        default: e = launch_clustered(kv8_commit_kernel<1>, B, 1, kThreads, 0, s, a); break;
    }
    return e == cudaSuccess ? EAGLE_OK : EAGLE_ERR_CUDA;
}
