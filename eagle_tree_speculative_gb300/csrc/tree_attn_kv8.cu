// Tree attention over the 8-bit K/V cache.
//
// Method: one warp per (sequence, node, query head); lane l holds dims 4l .. 4l + 3, the cache
// rows and then the node's ancestors' own rows are walked one by one with the running maximum
// and sum of the softmax.
#include "common.cuh"
#include "kv8_common.cuh"

#include <cuda_bf16.h>

namespace eagle {
namespace {

struct Args {
    const uint16_t* q;
    const uint8_t* k8;
    const uint8_t* v8;
    const float* ks;
    const float* vs;
    const uint16_t* kt;
    const uint16_t* vt;
    const int32_t* kv_len;
    const int32_t* parent;
    uint16_t* out;
    int B, n, Hq, Hkv, Lmax, NB;
    float scale;
    int32_t* dev_status;
};

__device__ __forceinline__ float4 load4(const uint16_t* p, int lane) {
    const uint2 w = __ldg(reinterpret_cast<const uint2*>(p) + lane);
    return make_float4(__uint_as_float(w.x << 16), __uint_as_float(w.x & 0xffff0000u),
                       __uint_as_float(w.y << 16), __uint_as_float(w.y & 0xffff0000u));
}
__device__ __forceinline__ float4 load4(const uint8_t* p, int lane, float s) {
    const uint32_t w = __ldg(reinterpret_cast<const uint32_t*>(p) + lane);
    const float2 a = kv8::e4m3x2_float((uint16_t)w), b = kv8::e4m3x2_float((uint16_t)(w >> 16));
    return make_float4(a.x * s, a.y * s, b.x * s, b.y * s);
}

__global__ void __launch_bounds__(128) tree_attn_kv8_kernel(Args a) {
    const int lane = threadIdx.x & 31;
    const int64_t unit = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 5);
    if (unit >= (int64_t)a.B * a.n * a.Hq) return;
    const int h = (int)(unit % a.Hq), i = (int)(unit / a.Hq % a.n), b = (int)(unit / a.Hq / a.n);
    const int L = a.kv_len[b], hk = h / (a.Hq / a.Hkv);
    int err = (L < 0 || L > a.Lmax) ? EAGLE_DEV_CAPACITY : 0;
    const int32_t* par = a.parent + (int64_t)b * a.n;
    for (int j = lane; j < a.n; j += 32)
        if (j == 0 ? par[0] != -1 : (par[j] < 0 || par[j] >= j)) err |= EAGLE_DEV_BAD_TREE;
    err = __reduce_or_sync(0xffffffffu, err);
    if (err && i == 0 && h == 0 && lane == 0) flag_error(a.dev_status, err);
    float m = -INFINITY, l = 0.f;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    const float4 q = load4(a.q + unit * kHeadDim, lane);
    auto key = [&](float4 k, float4 v) {
        const float s = warp_sum(q.x * k.x + q.y * k.y + q.z * k.z + q.w * k.w) * a.scale;
        if (s > m) {
            const float w = expf(m - s);
            l *= w; o.x *= w; o.y *= w; o.z *= w; o.w *= w;
            m = s;
        }
        const float p = expf(s - m);
        l += p;
        o.x += p * v.x; o.y += p * v.y; o.z += p * v.z; o.w += p * v.w;
    };
    if (!err) {
        const int64_t slab = (int64_t)b * a.Hkv + hk;
        for (int j = 0; j < L; ++j) {
            const int64_t row = (slab * a.Lmax + j) * kHeadDim, sc = slab * a.NB + j / kv8::kKv8Block;
            key(load4(a.k8 + row, lane, a.ks[sc]), load4(a.v8 + row, lane, a.vs[sc]));
        }
        for (int j = i; j >= 0; j = par[j]) {
            const int64_t row = (((int64_t)b * a.n + j) * a.Hkv + hk) * kHeadDim;
            key(load4(a.kt + row, lane), load4(a.vt + row, lane));
        }
    }
    const float inv = l > 0.f ? 1.f / l : 0.f;
    __nv_bfloat162 lo = __floats2bfloat162_rn(o.x * inv, o.y * inv);
    __nv_bfloat162 hi = __floats2bfloat162_rn(o.z * inv, o.w * inv);
    reinterpret_cast<uint2*>(a.out + unit * kHeadDim)[lane] =
        make_uint2(*reinterpret_cast<uint32_t*>(&lo), *reinterpret_cast<uint32_t*>(&hi));
}

}  // namespace
}  // namespace eagle

using namespace eagle;

extern "C" size_t eagle_tree_attn_kv8_workspace_size(int B, int n, int Hq, int Hkv, int head_dim,
                                                     int Lmax) {
    return 0;
}

extern "C" eagle_status eagle_tree_attn_kv8(const void* q, const void* k8, const void* v8,
                                            const float* k_scale, const float* v_scale,
                                            const void* k_tree, const void* v_tree,
                                            const int32_t* kv_len, const int32_t* parent, void* out,
                                            int B, int n, int Hq, int Hkv, int head_dim, int Lmax,
                                            float scale, void* workspace, size_t ws_bytes,
                                            int32_t* dev_status, eagle_stream_t stream) {
    if (B < 0 || n < 1 || Hq < 1 || Hkv < 1 || Lmax < 1 || !(scale > 0.f) || !(scale <= 3.4e38f))
        return EAGLE_ERR_INVALID_ARG;
    if (n > kMaxNodes || head_dim != kHeadDim || Hq % Hkv != 0) return EAGLE_ERR_SHAPE;
    if (B == 0) return EAGLE_OK;                        // nothing read or written
    if (!q || !k8 || !v8 || !k_scale || !v_scale || !k_tree || !v_tree || !kv_len || !parent || !out)
        return EAGLE_ERR_INVALID_ARG;
    for (const void* p : {q, k8, v8, k_tree, v_tree, (const void*)out})
        if (reinterpret_cast<uintptr_t>(p) & 15) return EAGLE_ERR_INVALID_ARG;
    Args a{static_cast<const uint16_t*>(q), static_cast<const uint8_t*>(k8),
           static_cast<const uint8_t*>(v8), k_scale, v_scale, static_cast<const uint16_t*>(k_tree),
           static_cast<const uint16_t*>(v_tree), kv_len, parent, static_cast<uint16_t*>(out), B, n, Hq,
           Hkv, Lmax, (Lmax + kv8::kKv8Block - 1) / kv8::kKv8Block, scale, dev_status};
    const int64_t blocks = ((int64_t)B * n * Hq + 3) / 4;
    if (blocks > 0x7fffffffLL) return EAGLE_ERR_SHAPE;
    tree_attn_kv8_kernel<<<(unsigned)blocks, 128, 0, reinterpret_cast<cudaStream_t>(stream)>>>(a);
    EAGLE_CHECK_LAUNCH();
    return EAGLE_OK;
}
