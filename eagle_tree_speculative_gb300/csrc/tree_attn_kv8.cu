// Tree attention over the 8-bit K/V cache: host side (argument checks, TMA tensor maps, the
// workspace).  The method and the kernels are in tree_attn_kv8_tc.cuh.
#include <cuda.h>
#include <cudaTypedefs.h>

#include "common.cuh"
#include "tree_attn_kv8_tc.cuh"

namespace eagle {
namespace {

// Codes of K or V as (128 bytes, Lmax rows, B * Hkv slabs): boxes of 128 rows of one slab.  Rows
// from Lmax on read as zeros.
bool code_map(CUtensorMap* map, const void* x, int Lmax, int64_t slabs) {
    auto fn = tensor_map_encoder();
    if (!fn) return false;
    cuuint64_t dims[3] = {(cuuint64_t)kHeadDim, (cuuint64_t)Lmax, (cuuint64_t)slabs};
    cuuint64_t strides[2] = {(cuuint64_t)kHeadDim, (cuuint64_t)Lmax * kHeadDim};
    cuuint32_t box[3] = {(cuuint32_t)kHeadDim, (cuuint32_t)kv8_tc::kKeys, 1};
    cuuint32_t estr[3] = {1, 1, 1};
    return fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<void*>(x), dims, strides, box, estr,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
              CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// The most positions that the cut can have, or -1 from 2^31 on.
int64_t kv8_positions(int B, int rows, int Hkv, int Lmax) {
    const int64_t rt = (rows + kv8_tc::kRows - 1) / kv8_tc::kRows, tiles = (Lmax + kv8_tc::kKeys - 1) / kv8_tc::kKeys + 1 + kv8_tc::kUnitCost;
    const int64_t units = (int64_t)B * Hkv;
    if (units > 0x7fffffffLL || units * rt > 0x7fffffffLL || units * rt * tiles > 0x7fffffffLL) return -1;
    return units * rt * tiles;
}
// CTAs: one per SM, and no more than there can be pieces.
int kv8_grid(int64_t positions, int rows) {
    const int rt = (rows + kv8_tc::kRows - 1) / kv8_tc::kRows;
    const int64_t pieces = positions / (kv8_tc::kMinTiles * (rt < 2 ? rt : 2));
    const int sms = cached_sm_count();
    return (int)(pieces < 1 ? 1 : pieces < sms ? pieces : sms);
}
// Rows of a partial: those of a unit.
int kv8_part_rows(int rows) { return rows < 2 * kv8_tc::kRows ? rows : 2 * kv8_tc::kRows; }

size_t kv8_workspace(int grid, int rows) {
    return (size_t)grid * 2 * kv8_part_rows(rows) * (kHeadDim * sizeof(float) + sizeof(float2));
}

}  // namespace
}  // namespace eagle

using namespace eagle;

extern "C" size_t eagle_tree_attn_kv8_workspace_size(int B, int n, int Hq, int Hkv, int head_dim,
                                                     int Lmax) {
    if (B < 1 || n < 1 || n > kMaxNodes || Hq < 1 || Hkv < 1 || Hq % Hkv != 0 || head_dim != kHeadDim ||
        Lmax < 1 || Lmax > kv8::kMaxRows || (int64_t)n * (Hq / Hkv) > 0x3fffffffLL)
        return 0;
    const int rows = n * (Hq / Hkv);
    const int64_t positions = kv8_positions(B, rows, Hkv, Lmax);
    if (positions < 0) return 0;
    const int grid = kv8_grid(positions, rows);
    return grid > 1 ? kv8_workspace(grid, rows) : 0;
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
    if (n > kMaxNodes || head_dim != kHeadDim || Hq % Hkv != 0 || Lmax > kv8::kMaxRows) return EAGLE_ERR_SHAPE;
    if ((int64_t)n * (Hq / Hkv) > 0x3fffffffLL) return EAGLE_ERR_SHAPE;
    const int rows = n * (Hq / Hkv);
    const int64_t positions = kv8_positions(B, rows, Hkv, Lmax);
    if (positions < 0) return EAGLE_ERR_SHAPE;
    if (B == 0) return EAGLE_OK;                        // nothing read or written
    if (!q || !k8 || !v8 || !k_scale || !v_scale || !k_tree || !v_tree || !kv_len || !parent || !out)
        return EAGLE_ERR_INVALID_ARG;
    for (const void* p : {q, k8, v8, k_tree, v_tree, (const void*)out, (const void*)workspace})
        if (reinterpret_cast<uintptr_t>(p) & 15) return EAGLE_ERR_INVALID_ARG;
    const int grid = kv8_grid(positions, rows);
    if (grid > 1 && (!workspace || ws_bytes < kv8_workspace(grid, rows))) return EAGLE_ERR_CAPACITY;
    kv8_tc::Args a;
    a.q = static_cast<const uint16_t*>(q);
    a.k_scale = k_scale; a.v_scale = v_scale;
    a.k_tree = static_cast<const uint16_t*>(k_tree);
    a.v_tree = static_cast<const uint16_t*>(v_tree);
    a.kv_len = kv_len; a.parent = parent;
    a.out = static_cast<uint16_t*>(out);
    a.rows = kv8_part_rows(rows);
    a.ws_o = static_cast<float*>(workspace);
    a.ws_ml = reinterpret_cast<float2*>(a.ws_o + (size_t)grid * 2 * a.rows * kHeadDim);
    a.B = B; a.n = n; a.Hq = Hq; a.Hkv = Hkv; a.G = Hq / Hkv; a.Lmax = Lmax;
    a.NB = (Lmax + kv8::kKv8Block - 1) / kv8::kKv8Block;
    a.scale_log2 = scale * 1.4426950408889634f;
    a.dev_status = dev_status;
    CUtensorMap mk, mv;
    if (!code_map(&mk, k8, Lmax, (int64_t)B * Hkv) || !code_map(&mv, v8, Lmax, (int64_t)B * Hkv))
        return EAGLE_ERR_CUDA;
    if (!raise_smem_limit<kv8_tc::tree_attn_kv8_kernel>(kv8_tc::kSmem))
        return EAGLE_ERR_CUDA;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    kv8_tc::tree_attn_kv8_kernel<<<grid, kv8_tc::kThreads, kv8_tc::kSmem, s>>>(mk, mv, a);
    EAGLE_CHECK_LAUNCH();
    if (grid > 1 && attn2::launch_merge(kv8_tc::tree_attn_kv8_merge_kernel<true>, kv8_tc::tree_attn_kv8_merge_kernel<false>, a, grid, s) != cudaSuccess)
        return EAGLE_ERR_CUDA;
    return EAGLE_OK;
}
