// Causal attention of packed prompts: host side (argument checks, TMA tensor maps).  The method
// and the kernel are in prompt_attn_tc.cuh.
#include <cuda.h>
#include <cudaTypedefs.h>

#include "common.cuh"
#include "prompt_attn_tc.cuh"

namespace eagle {
namespace {

// Q as (128 dims, G heads of the group, Hkv groups, Tq tokens): boxes of 64 dims x G heads x P
// tokens, the rows of a row tile in order.  Tokens from Tq on read as zeros.
bool q_map(CUtensorMap* map, const void* q, int G, int P, int Hkv, int Tq, int64_t stride) {
    auto fn = tensor_map_encoder();
    if (!fn) return false;
    cuuint64_t dims[4] = {(cuuint64_t)kHeadDim, (cuuint64_t)G, (cuuint64_t)Hkv, (cuuint64_t)Tq};
    cuuint64_t strides[3] = {(cuuint64_t)kHeadDim * 2, (cuuint64_t)G * kHeadDim * 2, (cuuint64_t)stride * 2};
    cuuint32_t box[4] = {64, (cuuint32_t)G, 1, (cuuint32_t)P};
    cuuint32_t estr[4] = {1, 1, 1, 1};
    return fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(q), dims, strides, box, estr,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
              CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// K or V as (128 dims, Hkv heads, Tk tokens): boxes of 64 dims x 128 tokens of one head.
bool kv_map(CUtensorMap* map, const void* x, int Hkv, int Tk, int64_t stride) {
    auto fn = tensor_map_encoder();
    if (!fn) return false;
    cuuint64_t dims[3] = {(cuuint64_t)kHeadDim, (cuuint64_t)Hkv, (cuuint64_t)Tk};
    cuuint64_t strides[2] = {(cuuint64_t)kHeadDim * 2, (cuuint64_t)stride * 2};
    cuuint32_t box[3] = {64, 1, (cuuint32_t)prompt_tc::kKeys};
    cuuint32_t estr[3] = {1, 1, 1};
    return fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(x), dims, strides, box, estr,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
              CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
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
    prompt_tc::Args a;
    a.cu_q = cu_q; a.cu_k = cu_k;
    a.out = static_cast<uint16_t*>(out);
    a.lse = lse;
    a.Tq = Tq; a.Tk = Tk; a.B = B; a.Hq = Hq; a.Hkv = Hkv;
    a.G = Hq / Hkv;
    a.P = prompt_tc::kRows / a.G;
    a.scale_log2 = scale * 1.4426950408889634f;
    a.dev_status = dev_status;
    // without keys nothing is loaded through the K and V maps: any valid address will do
    CUtensorMap mq, mk, mv;
    if (!q_map(&mq, q, a.G, a.P, Hkv, Tq, q_stride) ||
        !kv_map(&mk, Tk > 0 ? k : q, Hkv, Tk > 0 ? Tk : 1, Tk > 0 ? k_stride : q_stride) ||
        !kv_map(&mv, Tk > 0 ? v : q, Hkv, Tk > 0 ? Tk : 1, Tk > 0 ? v_stride : q_stride))
        return EAGLE_ERR_CUDA;
    // a sequence of m queries has at most m / 2P + 1 units
    const int64_t units = ((int64_t)Tq / (2 * a.P) + B) * Hkv;
    if (units > 0x3fffffffLL || Tq > 0x3fffffff || Tk > 0x3fffffff) return EAGLE_ERR_SHAPE;      // 32-bit places
    const int sms = cached_sm_count();
    const unsigned grid = (unsigned)(units < sms ? units : sms);
    if (!raise_smem_limit<prompt_tc::prompt_attn_kernel>(prompt_tc::kSmem))
        return EAGLE_ERR_CUDA;
    prompt_tc::prompt_attn_kernel<<<grid, prompt_tc::kThreads, prompt_tc::kSmem,
                                    reinterpret_cast<cudaStream_t>(stream)>>>(mq, mk, mv, a);
    EAGLE_CHECK_LAUNCH();
    return EAGLE_OK;
}
