// Pieces of the two-slot attention kernels (prompt attention and tree attention over the
// 8-bit cache): one CTA holds two softmax slots of 128 query rows each, so that the tensor
// cores work for one slot while the other slot's softmax runs.
//
// TMEM (512 columns): S of slot s at s * 128 (its P is written over the first 64 columns),
// O of slot s at 256 + s * 128.  Warps 0-3 have single roles (loads, MMA issue, scheduling),
// warps 4-7 and 8-11 are the softmax of slots 0 and 1, one thread per query row.  The other warps
// give registers up to the softmax warps.
#pragma once

#include "common.cuh"
#include "tc_common.cuh"

namespace eagle {
namespace attn2 {

constexpr int kRows = 128;                        // query rows of a slot
constexpr int kKeys = 128;                        // keys of a tile
constexpr int kSlots = 2;
constexpr uint32_t kTmemCols = 512;

__device__ __forceinline__ uint32_t s_col(int slot) { return (uint32_t)(slot * 128); }
__device__ __forceinline__ uint32_t o_col(int slot) { return (uint32_t)(256 + slot * 128); }

template <int N>
__device__ __forceinline__ void regs_inc() {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;\n" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void regs_dec() {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;\n" ::"n"(N));
}

// Two floats in a 64-bit register pair, and the packed operations on them.
__device__ __forceinline__ uint64_t f2(float lo, float hi) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};\n" : "=l"(r) : "f"(lo), "f"(hi));
    return r;
}
__device__ __forceinline__ void unf2(uint64_t v, float& lo, float& hi) {
    asm("mov.b64 {%0, %1}, %2;\n" : "=f"(lo), "=f"(hi) : "l"(v));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;\n" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;\n" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;\n" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
    float r;
    asm("max.f32 %0, %1, %2, %3;\n" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}

// The maximum of N values: four chains of three-input maxima.
template <int N>
__device__ __forceinline__ float max_of(const float* x) {
    static_assert(N % 8 == 0, "pairs for four chains");
    float m[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) m[e] = fmaxf(x[2 * e], x[2 * e + 1]);
#pragma unroll
    for (int c = 8; c < N; c += 8)
#pragma unroll
        for (int e = 0; e < 4; ++e) m[e] = max3(m[e], x[c + 2 * e], x[c + 2 * e + 1]);
    return fmaxf(max3(m[0], m[1], m[2]), m[3]);
}

// 32 columns of this thread's TMEM lane, to be waited for with tmem_wait_ld.
__device__ __forceinline__ void load32_nowait(uint32_t addr, float (&x)[32]) {
    uint32_t u[32];
    tmem_ld32_nowait(addr, u);
#pragma unroll
    for (int c = 0; c < 32; ++c) x[c] = __uint_as_float(u[c]);
}
__device__ __forceinline__ void tmem_wait_ld() {
    asm volatile("tcgen05.wait::ld.sync.aligned;\n" ::: "memory");
}

// 128 columns of this thread's TMEM lane.
__device__ __forceinline__ void load_row(uint32_t addr, float (&x)[128]) {
    uint32_t u[4][32];
#pragma unroll
    for (int h = 0; h < 4; ++h) tmem_ld32_nowait(addr + 32 * h, u[h]);
    asm volatile("tcgen05.wait::ld.sync.aligned;\n" ::: "memory");
#pragma unroll
    for (int h = 0; h < 4; ++h)
#pragma unroll
        for (int c = 0; c < 32; ++c) x[32 * h + c] = __uint_as_float(u[h][c]);
}

__device__ __forceinline__ void tmem_st32_nowait(uint32_t taddr, const uint32_t (&r)[32]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,"
        "%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};\n" ::"r"(taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
        "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]),
        "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]),
        "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]),
        "r"(r[29]), "r"(r[30]), "r"(r[31])
        : "memory");
}
__device__ __forceinline__ void tmem_st16_nowait(uint32_t taddr, const uint32_t (&o)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,"
        "%14,%15,%16};\n" ::"r"(taddr),
        "r"(o[0]), "r"(o[1]), "r"(o[2]), "r"(o[3]), "r"(o[4]), "r"(o[5]), "r"(o[6]), "r"(o[7]),
        "r"(o[8]), "r"(o[9]), "r"(o[10]), "r"(o[11]), "r"(o[12]), "r"(o[13]), "r"(o[14]), "r"(o[15])
        : "memory");
}
__device__ __forceinline__ void tmem_wait_st() {
    asm volatile("tcgen05.wait::st.sync.aligned;\n" ::: "memory");
}

// O (128 columns of this thread's lane) *= alpha.  Sixteen columns at a time in a loop that stays
// a loop: the caller holds a row of scores in registers meanwhile, and this is rare.
__device__ __forceinline__ void rescale_row(uint32_t addr, float alpha) {
#pragma unroll 1
    for (int h = 0; h < 8; ++h) {
        uint32_t o[16];
        asm volatile(
            "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,"
            "%15}, [%16];\n"
            "tcgen05.wait::ld.sync.aligned;\n"
            : "=r"(o[0]), "=r"(o[1]), "=r"(o[2]), "=r"(o[3]), "=r"(o[4]), "=r"(o[5]), "=r"(o[6]),
              "=r"(o[7]), "=r"(o[8]), "=r"(o[9]), "=r"(o[10]), "=r"(o[11]), "=r"(o[12]), "=r"(o[13]),
              "=r"(o[14]), "=r"(o[15])
            : "r"(addr + 16 * h)
            : "memory");
#pragma unroll
        for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha);
        tmem_st16_nowait(addr + 16 * h, o);
    }
    tmem_wait_st();
}

// Shared-memory writes become visible to the tensor cores and TMA.
__device__ __forceinline__ void fence_async_shared() {
    asm volatile("fence.proxy.async.shared::cta;\n" ::: "memory");
}

}  // namespace attn2
}  // namespace eagle
