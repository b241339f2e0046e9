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

// Bounded wait, in as little code as it can be: these kernels wait in many places, and their
// speed depends on how much code goes round.  False when the abort flag is up, or after `limit`
// ticks of the clock, which raises the flag.  wait_for: two ticks of the clock's upper word (2^32 to
// 2^33 cycles, two to four seconds).
__device__ __forceinline__ uint32_t clock_hi() {
    uint32_t x;
    asm volatile("mov.u32 %0, %%clock_hi;\n" : "=r"(x));
    return x;
}
template <class Clock>
__device__ __forceinline__ bool wait_until(uint32_t bar, uint32_t parity, volatile int* abort_flag, Clock clock, uint32_t limit) {
    if (mbar_try_wait(bar, parity & 1u)) return true;
    const uint32_t t0 = clock();
#pragma unroll 1
    while (!mbar_try_wait(bar, parity & 1u)) {
        if (*abort_flag) return false;
        if (clock() - t0 >= limit) {
            *abort_flag = 1;
            return false;
        }
    }
    return true;
}
__device__ __forceinline__ bool wait_for(uint32_t bar, uint32_t parity, volatile int* abort_flag) {
    return wait_until(bar, parity, abort_flag, [] { return clock_hi(); }, 2u);
}

// Arrival and commit of one lane, `on`, without a branch: warps that part for a lane's instruction
// and meet again lose 200 to 300 cycles here.
__device__ __forceinline__ void arrive_if(bool on, uint32_t bar) {
    asm volatile("{\n .reg .pred q;\n setp.ne.b32 q, %1, 0;\n @q mbarrier.arrive.shared::cta.b64 _, [%0];\n}\n" ::"r"(bar),
                 "r"((uint32_t)on)
                 : "memory");
}
__device__ __forceinline__ void commit_if(bool on, uint32_t bar) {
    asm volatile(
        "{\n .reg .pred q;\n setp.ne.b32 q, %1, 0;\n"
        " @q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n}\n" ::"r"(bar),
        "r"((uint32_t)on)
        : "memory");
}

// The end of an MMA thread: its own products, which always end, have left the tensor cores.
__device__ __forceinline__ void wait_drain(uint32_t bar) {
    int never = 0;
    mbar_wait(bar, 0u, &never, /*honour_abort=*/false);
}

// MMA issue.  One elected lane issues, but the whole warp walks the loop, and what the loop
// depends on is broadcast (uniform_of): the instruction takes its descriptors from uniform
// registers, and from values that only one lane computes each of them costs a move across, 130 to
// 160 cycles an MMA instead of 64.  A descriptor is a constant upper word and the lower word, which
// holds the start address / 16 in its low 14 bits.
__device__ __forceinline__ bool elect_lane() {
    uint32_t p;
    asm volatile("{\n .reg .pred P;\n elect.sync _|P, 0xffffffff;\n selp.u32 %0, 1, 0, P;\n}\n" : "=r"(p));
    return p != 0;
}
__device__ __forceinline__ int uniform_of(int x) { return __shfl_sync(0xffffffffu, x, 0); }

// Upper words: stride between 8-row groups 1024 bytes, version 1, 128-byte swizzle.
constexpr uint32_t kDescHi = (1024u >> 4) | (1u << 14) | (2u << 29);
// Lower words: K-major (leading offset unused), and MN-major with `lbo` between 64-element atoms.
__device__ __forceinline__ uint32_t desc_lo(uint32_t saddr) { return ((saddr >> 4) & 0x3fffu) | (1u << 16); }
__device__ __forceinline__ uint32_t desc_lo_mn(uint32_t saddr, uint32_t lbo) {
    return ((saddr >> 4) & 0x3fffu) | (((lbo >> 4) & 0x3fffu) << 16);
}

// D (+)= A B with A and B in shared memory (SS) or A in TMEM (TS); kind::f16 or kind::f8f6f4.  Issued
// by the lane that is `on`, without a branch.
template <bool F8>
__device__ __forceinline__ void mma_ss(uint32_t on, uint32_t d, uint32_t a_lo, uint32_t b_lo, uint32_t idesc, uint32_t accumulate) {
    if constexpr (F8)
        asm volatile(
            "{\n .reg .pred p, q;\n .reg .b64 a, b;\n setp.ne.b32 p, %5, 0;\n setp.ne.b32 q, %6, 0;\n"
            " mov.b64 a, {%1, %3};\n mov.b64 b, {%2, %3};\n"
            " @q tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], a, b, %4, p;\n}\n" ::"r"(d),
            "r"(a_lo), "r"(b_lo), "n"(kDescHi), "r"(idesc), "r"(accumulate), "r"(on)
            : "memory");
    else
        asm volatile(
            "{\n .reg .pred p, q;\n .reg .b64 a, b;\n setp.ne.b32 p, %5, 0;\n setp.ne.b32 q, %6, 0;\n"
            " mov.b64 a, {%1, %3};\n mov.b64 b, {%2, %3};\n"
            " @q tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %4, p;\n}\n" ::"r"(d),
            "r"(a_lo), "r"(b_lo), "n"(kDescHi), "r"(idesc), "r"(accumulate), "r"(on)
            : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t on, uint32_t d, uint32_t a_tmem, uint32_t b_lo, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n .reg .pred p, q;\n .reg .b64 b;\n setp.ne.b32 p, %5, 0;\n setp.ne.b32 q, %6, 0;\n mov.b64 b, {%2, %3};\n"
        " @q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], b, %4, p;\n}\n" ::"r"(d),
        "r"(a_tmem), "r"(b_lo), "n"(kDescHi), "r"(idesc), "r"(accumulate), "r"(on)
        : "memory");
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

__device__ __forceinline__ void tmem_wait_ld() {
    asm volatile("tcgen05.wait::ld.sync.aligned;\n" ::: "memory");
}
// 32 columns of this thread's TMEM lane and their maximum, which the load itself takes (NaN does not
// count); both are there after tmem_wait_ld.
__device__ __forceinline__ void load32_max_nowait(uint32_t addr, uint32_t* r, float& mx) {
    asm volatile(
        "tcgen05.ld.red.sync.aligned.32x32b.x32.max.f32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,"
        "%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, %32, [%33];\n"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
          "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
          "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]),
          "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]),
          "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31]), "=f"(mx)
        : "r"(addr));
}

// 128 columns of this thread's TMEM lane, and the maximum of each 32; there after tmem_wait_ld.
__device__ __forceinline__ void load_row_nowait(uint32_t addr, uint32_t (&u)[128], float (&mx)[4]) {
#pragma unroll
    for (int h = 0; h < 4; ++h) load32_max_nowait(addr + 32 * h, u + 32 * h, mx[h]);
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
__device__ __forceinline__ void tmem_st8_nowait(uint32_t taddr, const uint32_t (&o)[8]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};\n" ::"r"(taddr), "r"(o[0]),
        "r"(o[1]), "r"(o[2]), "r"(o[3]), "r"(o[4]), "r"(o[5]), "r"(o[6]), "r"(o[7])
        : "memory");
}
__device__ __forceinline__ void tmem_wait_st() {
    asm volatile("tcgen05.wait::st.sync.aligned;\n" ::: "memory");
}

// 16 columns of this thread's TMEM lane, waited for.
__device__ __forceinline__ void load16(uint32_t addr, uint32_t (&o)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,"
        "%15}, [%16];\n"
        "tcgen05.wait::ld.sync.aligned;\n"
        : "=r"(o[0]), "=r"(o[1]), "=r"(o[2]), "=r"(o[3]), "=r"(o[4]), "=r"(o[5]), "=r"(o[6]),
          "=r"(o[7]), "=r"(o[8]), "=r"(o[9]), "=r"(o[10]), "=r"(o[11]), "=r"(o[12]), "=r"(o[13]),
          "=r"(o[14]), "=r"(o[15])
        : "r"(addr)
        : "memory");
}

// O (128 columns of this thread's lane) *= alpha.  Sixteen columns at a time in a loop that stays
// a loop: the caller may hold a row of scores in registers meanwhile, and this is rare.
__device__ __forceinline__ void rescale_row(uint32_t addr, float alpha) {
#pragma unroll 1
    for (int h = 0; h < 8; ++h) {
        uint32_t o[16];
        load16(addr + 16 * h, o);
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
