// Tree attention over the paged K/V cache: host side (argument checks, TMA tensor maps, the workspace).  The
// method and the kernels are in tree_attn_paged_tc.cuh.
#include <cuda.h>
#include <cudaTypedefs.h>

#include "common.cuh"
#include "tree_attn_paged_tc.cuh"

namespace eagle {
namespace {

// Q as (128 dims, G heads of the group, Hkv groups, B n nodes): boxes of 64 dims x G heads x P nodes, the
// rows of a row tile in order.  Nodes from B n on read as zeros.
bool paged_q_map(CUtensorMap* map, const void* q, int G, int P, int Hkv, int64_t nodes) {
    auto fn = tensor_map_encoder();
    if (!fn) return false;
    cuuint64_t dims[4] = {(cuuint64_t)kHeadDim, (cuuint64_t)G, (cuuint64_t)Hkv, (cuuint64_t)nodes};
    cuuint64_t strides[3] = {(cuuint64_t)kHeadDim * 2, (cuuint64_t)G * kHeadDim * 2, (cuuint64_t)G * Hkv * kHeadDim * 2};
    cuuint32_t box[4] = {64, (cuuint32_t)G, 1, (cuuint32_t)P};
    cuuint32_t estr[4] = {1, 1, 1, 1};
    return fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(q), dims, strides, box, estr,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
              CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// K or V as (128 dims, a page's rows, N * Hkv slabs): boxes of 64 dims x one page of one head.
bool page_map(CUtensorMap* map, const void* x, int page, int64_t slabs) {
    auto fn = tensor_map_encoder();
    if (!fn) return false;
    cuuint64_t dims[3] = {(cuuint64_t)kHeadDim, (cuuint64_t)page, (cuuint64_t)slabs};
    cuuint64_t strides[2] = {(cuuint64_t)kHeadDim * 2, (cuuint64_t)page * kHeadDim * 2};
    cuuint32_t box[3] = {64, (cuuint32_t)page, 1};
    cuuint32_t estr[3] = {1, 1, 1};
    return fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(x), dims, strides, box, estr,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
              CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Row tiles of a sequence and kv head; rows of a part: those of a unit.
int paged_row_tiles(int n, int G) {
    const int P = paged_tc::kRows / G;
    return n <= P ? 1 : (n + 2 * P - 1) / (2 * P) * 2;    // as the cut counts them
}
int paged_part_rows(int n, int G) {
    const int rt = paged_row_tiles(n, G);
    return rt > 1 ? 2 * paged_tc::kRows : n * G;
}
// The most positions that the cut can have, or -1 from 2^31 on.
int64_t paged_positions(int B, int n, int G, int Hkv, int64_t rows) {
    const int64_t tiles = (rows + paged_tc::kKeys - 1) / paged_tc::kKeys + paged_tc::kUnitCost;
    const int64_t units = (int64_t)B * Hkv, rt = paged_row_tiles(n, G);
    if (units > 0x7fffffffLL || units * rt > 0x7fffffffLL || units * rt * tiles > 0x7fffffffLL) return -1;
    return units * rt * tiles;
}
// CTAs: one per SM, and no more than there can be pieces.
int paged_grid(int64_t positions, int n, int G) {
    const int rt = paged_row_tiles(n, G);
    const int64_t pieces = positions / (paged_tc::kMinTiles * (rt < 2 ? rt : 2));
    const int sms = cached_sm_count();
    return (int)(pieces < 1 ? 1 : pieces < sms ? pieces : sms);
}
size_t paged_workspace(int grid, int rows) {
    return (size_t)grid * 2 * rows * (kHeadDim * sizeof(float) + sizeof(float2)) + 16;      // 16: a workspace at an odd multiple
}

bool paged_shape_ok(int n, int Hq, int Hkv, int head_dim, int page, int P) {
    return n <= kMaxNodes && head_dim == kHeadDim && Hq % Hkv == 0 && Hq / Hkv <= paged_tc::kRows && paged::page_ok(page) &&
           (int64_t)P * page <= paged::kMaxRows;
}

}  // namespace
}  // namespace eagle

using namespace eagle;

extern "C" size_t eagle_tree_attn_paged_workspace_size(int B, int n, int Hq, int Hkv, int head_dim, int page, int P) {
    if (B < 1 || n < 1 || Hq < 1 || Hkv < 1 || P < 1 || !paged_shape_ok(n, Hq, Hkv, head_dim, page, P)) return 0;
    const int64_t positions = paged_positions(B, n, Hq / Hkv, Hkv, (int64_t)P * page);
    if (positions < 0) return 0;
    const int grid = paged_grid(positions, n, Hq / Hkv);
    return grid > 1 ? paged_workspace(grid, paged_part_rows(n, Hq / Hkv)) : 0;
}

extern "C" eagle_status eagle_tree_attn_paged(const void* q, const void* k_pages, const void* v_pages,
                                              const int32_t* page_table, const int32_t* kv_len,
                                              const int32_t* parent, void* out, int B, int n, int Hq, int Hkv,
                                              int head_dim, int N, int page, int P, float scale,
                                              void* workspace, size_t ws_bytes, int32_t* dev_status,
                                              eagle_stream_t stream) {
    if (B < 0 || n < 1 || Hq < 1 || Hkv < 1 || N < 1 || P < 1 || !(scale > 0.f) || !(scale <= 3.4e38f))
        return EAGLE_ERR_INVALID_ARG;
    if (!paged_shape_ok(n, Hq, Hkv, head_dim, page, P) || (int64_t)N * Hkv * page > paged::kMaxPool || (int64_t)B * n > 0x3fffffff)
        return EAGLE_ERR_SHAPE;
    const int G = Hq / Hkv;
    const int64_t positions = paged_positions(B, n, G, Hkv, (int64_t)P * page);
    if (positions < 0) return EAGLE_ERR_SHAPE;
    if (B == 0) return EAGLE_OK;                        // nothing read or written
    if (!q || !k_pages || !v_pages || !page_table || !kv_len || !parent || !out) return EAGLE_ERR_INVALID_ARG;
    for (const void* p : {q, k_pages, v_pages, (const void*)out, (const void*)workspace})
        if (reinterpret_cast<uintptr_t>(p) & 15) return EAGLE_ERR_INVALID_ARG;
    const int grid = paged_grid(positions, n, G);
    paged_tc::Args a;
    a.rows = paged_part_rows(n, G);
    if (grid > 1 && (!workspace || ws_bytes < paged_workspace(grid, a.rows))) return EAGLE_ERR_CAPACITY;
    a.table = page_table; a.kv_len = kv_len; a.parent = parent;
    a.out = static_cast<uint16_t*>(out);
    a.ws_o = reinterpret_cast<float*>((reinterpret_cast<uintptr_t>(workspace) + 31) & ~static_cast<uintptr_t>(31));
    a.out_whole = (reinterpret_cast<uintptr_t>(out) & 31) == 0;
    a.ws_ml = reinterpret_cast<float2*>(a.ws_o + (size_t)grid * 2 * a.rows * kHeadDim);
    a.B = B; a.n = n; a.Hq = Hq; a.Hkv = Hkv; a.G = G; a.P = paged_tc::kRows / G;
    a.N = N; a.shift = paged::page_shift(page); a.width = P;
    a.scale_log2 = scale * 1.4426950408889634f;
    a.dev_status = dev_status;
    CUtensorMap mq, mk, mv;
    if (!paged_q_map(&mq, q, G, a.P, Hkv, (int64_t)B * n) || !page_map(&mk, k_pages, page, (int64_t)N * Hkv) ||
        !page_map(&mv, v_pages, page, (int64_t)N * Hkv))
        return EAGLE_ERR_CUDA;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (n <= a.P) {
        if (!raise_smem_limit<paged_tc::tree_attn_paged_kernel<true>>(paged_tc::kSmem)) return EAGLE_ERR_CUDA;
        paged_tc::tree_attn_paged_kernel<true><<<grid, paged_tc::kThreads, paged_tc::kSmem, s>>>(mq, mk, mv, a);
    } else {
        if (!raise_smem_limit<paged_tc::tree_attn_paged_kernel<false>>(paged_tc::kSmem)) return EAGLE_ERR_CUDA;
        paged_tc::tree_attn_paged_kernel<false><<<grid, paged_tc::kThreads, paged_tc::kSmem, s>>>(mq, mk, mv, a);
    }
    EAGLE_CHECK_LAUNCH();
    if (grid > 1 && attn2::launch_merge(paged_tc::tree_attn_paged_merge_kernel<true>, paged_tc::tree_attn_paged_merge_kernel<false>, a, grid, s) != cudaSuccess)
        return EAGLE_ERR_CUDA;
    return EAGLE_OK;
}
