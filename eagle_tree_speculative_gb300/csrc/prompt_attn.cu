// Causal attention of packed prompts.
//
// Method: one warp per (token, query head); lane l holds dims 4l .. 4l + 3 of the query, the
// keys are walked one by one with the running maximum m and sum l of the softmax, and the
// output is rescaled when the maximum grows.
#include "common.cuh"

#include <cuda_bf16.h>

namespace eagle {
namespace {

constexpr unsigned kFull = 0xffffffffu;

struct PromptArgs {
    const uint16_t* q;
    const uint16_t* k;
    const uint16_t* v;
    const int32_t* cu_q;
    const int32_t* cu_k;
    uint16_t* out;
    float* lse;
    int Tq, Tk, B, Hq, Hkv;
    int64_t qs, ks, vs;
    float scale;
    int32_t* dev_status;
};

__device__ __forceinline__ float4 load4(const uint16_t* p, int lane) {
    const uint2 w = __ldg(reinterpret_cast<const uint2*>(p) + lane);
    return make_float4(__uint_as_float(w.x << 16), __uint_as_float(w.x & 0xffff0000u),
                       __uint_as_float(w.y << 16), __uint_as_float(w.y & 0xffff0000u));
}

__global__ void __launch_bounds__(128) prompt_attn_kernel(PromptArgs a) {
    const int lane = threadIdx.x & 31;
    const int64_t unit = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 5);
    const int t = (int)(unit / a.Hq), h = (int)(unit % a.Hq);
    bool bad = false;
    int b = -1;
    for (int i = lane; i < a.B; i += 32) {
        const int q0 = a.cu_q[i], q1 = a.cu_q[i + 1], k0 = a.cu_k[i], k1 = a.cu_k[i + 1];
        if (q0 < 0 || q1 < q0 || q1 > a.Tq || k0 < 0 || k1 < k0 || k1 > a.Tk) bad = true;
        else if (t >= q0 && t < q1) b = i;
    }
    if (__any_sync(kFull, bad)) {
        if (unit == 0 && lane == 0) flag_error(a.dev_status, EAGLE_DEV_CAPACITY);
        return;
    }
    b = __reduce_max_sync(kFull, b);
    if (b < 0 || t >= a.Tq) return;
    const int q0 = a.cu_q[b], nq = a.cu_q[b + 1] - q0, k0 = a.cu_k[b], nk = a.cu_k[b + 1] - k0;
    const int end = nk - nq + (t - q0) + 1;
    const int64_t hk = (int64_t)(h / (a.Hq / a.Hkv)) * kHeadDim;
    const float4 q = load4(a.q + (int64_t)t * a.qs + (int64_t)h * kHeadDim, lane);
    float m = -INFINITY, l = 0.f;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int j = 0; j < end; ++j) {
        const float4 k = load4(a.k + (int64_t)(k0 + j) * a.ks + hk, lane);
        const float s = warp_sum(q.x * k.x + q.y * k.y + q.z * k.z + q.w * k.w) * a.scale;
        if (s > m) {
            const float w = expf(m - s);
            l *= w; o.x *= w; o.y *= w; o.z *= w; o.w *= w;
            m = s;
        }
        const float p = expf(s - m);
        const float4 v = load4(a.v + (int64_t)(k0 + j) * a.vs + hk, lane);
        l += p;
        o.x += p * v.x; o.y += p * v.y; o.z += p * v.z; o.w += p * v.w;
    }
    const float inv = l > 0.f ? 1.f / l : 0.f;
    __nv_bfloat162 lo = __floats2bfloat162_rn(o.x * inv, o.y * inv);
    __nv_bfloat162 hi = __floats2bfloat162_rn(o.z * inv, o.w * inv);
    reinterpret_cast<uint2*>(a.out + ((int64_t)t * a.Hq + h) * kHeadDim)[lane] =
        make_uint2(*reinterpret_cast<uint32_t*>(&lo), *reinterpret_cast<uint32_t*>(&hi));
    if (a.lse && lane == 0) a.lse[(int64_t)t * a.Hq + h] = l > 0.f ? m + logf(l) : -INFINITY;
}

}  // namespace
}  // namespace eagle

using namespace eagle;

extern "C" eagle_status eagle_prompt_attn(const void* q, const void* k, const void* v,
                                          const int32_t* cu_q, const int32_t* cu_k, void* out,
                                          float* lse, int Tq, int Tk, int B, int Hq, int Hkv,
                                          int head_dim, int64_t q_stride, int64_t k_stride,
                                          int64_t v_stride, float scale, int32_t* dev_status,
                                          eagle_stream_t stream) {
    if (Tq < 0 || Tk < 0 || B < 0 || Hq < 1 || Hkv < 1 || !(scale > 0.f) || !(scale <= 3.4e38f))
        return EAGLE_ERR_INVALID_ARG;
    if (head_dim != kHeadDim || Hq % Hkv != 0 || Hq / Hkv > 128) return EAGLE_ERR_SHAPE;
    if (q_stride < (int64_t)Hq * kHeadDim || k_stride < (int64_t)Hkv * kHeadDim ||
        v_stride < (int64_t)Hkv * kHeadDim || q_stride % 8 != 0 || k_stride % 8 != 0 ||
        v_stride % 8 != 0)
        return EAGLE_ERR_INVALID_ARG;
    if (B == 0 || Tq == 0) return EAGLE_OK;             // nothing read or written
    if (!q || !cu_q || !cu_k || !out || (Tk > 0 && (!k || !v))) return EAGLE_ERR_INVALID_ARG;
    for (const void* p : {q, k, v, (const void*)out})
        if (reinterpret_cast<uintptr_t>(p) & 15) return EAGLE_ERR_INVALID_ARG;
    PromptArgs a{static_cast<const uint16_t*>(q), static_cast<const uint16_t*>(k),
                 static_cast<const uint16_t*>(v), cu_q, cu_k, static_cast<uint16_t*>(out), lse, Tq, Tk,
                 B, Hq, Hkv, q_stride, k_stride, v_stride, scale, dev_status};
    const int64_t blocks = ((int64_t)Tq * Hq + 3) / 4;
    if (blocks > 0x7fffffffLL) return EAGLE_ERR_SHAPE;
    prompt_attn_kernel<<<(unsigned)blocks, 128, 0, reinterpret_cast<cudaStream_t>(stream)>>>(a);
    EAGLE_CHECK_LAUNCH();
    return EAGLE_OK;
}
