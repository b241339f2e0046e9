// The 8-bit K/V cache: e4m3 codes with one power-of-two scale per kKv8Block rows and kv
// head, and the conversions between codes and floats.
#pragma once

#include "common.cuh"

namespace eagle {
namespace kv8 {

constexpr int kKv8Block = EAGLE_KV8_BLOCK;
constexpr int kMinExp = -64;              // the smallest scale is 2^-64
constexpr int kMaxRows = 0x7fffffff - 127;  // of a cache: its last tile of 128 ends within 32 bits

// Two floats as e4m3 codes (nearest, ties to even, saturating; NaN stays NaN), lo in the
// low byte.
__device__ __forceinline__ uint16_t e4m3x2(float lo, float hi) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;\n" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}
// Four floats, the first in the lowest byte.
__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d) {
    return (uint32_t)e4m3x2(a, b) | ((uint32_t)e4m3x2(c, d) << 16);
}
// Two codes as halves (every e4m3 value is one), and as floats.
__device__ __forceinline__ uint32_t e4m3x2_half2(uint16_t c) {
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;\n" : "=r"(h) : "h"(c));
    return h;
}
__device__ __forceinline__ float2 half2_float(uint32_t h) {
    float2 f;
    asm("{\n .reg .b16 l, u;\n mov.b32 {l, u}, %2;\n cvt.f32.f16 %0, l;\n cvt.f32.f16 %1, u;\n}\n"
        : "=f"(f.x), "=f"(f.y)
        : "r"(h));
    return f;
}
__device__ __forceinline__ float2 e4m3x2_float(uint16_t c) { return half2_float(e4m3x2_half2(c)); }

// 2^e as a float, -126 <= e <= 127.
__device__ __forceinline__ float exp2i(int e) { return __int_as_float((e + 127) << 23); }

// The least e >= kMinExp with amax <= 448 * 2^e, for finite amax >= 0.  448 = 1.75 * 2^8: of
// amax = m 2^E, 1 <= m < 2, only m > 1.75 needs E - 7.  A subnormal amax has E = -127 here and
// ends at kMinExp, as it should.  At most 2^120 (the largest float is below 2 * 2^127).
__device__ __forceinline__ int scale_exp(float amax) {
    const uint32_t u = __float_as_uint(amax);
    const int E = (int)(u >> 23) - 127;
    const int e = E - 8 + ((u & 0x7fffffu) > 0x600000u ? 1 : 0);
    return e < kMinExp ? kMinExp : e;
}

}  // namespace kv8
}  // namespace eagle
