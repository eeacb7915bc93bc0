// e4m3.cuh -- 8-bit values with power-of-two scales, shared by the kernels that write or read them.
//
// A group of values x is held as e4m3 codes c and one scale s = 2^e, x = c s, with
// e the smallest exponent in [-100, 120] for which amax <= 448 * 2^e (448 is the
// largest e4m3 value).  e4m3 is a floating-point type, so a power-of-two scale costs no
// precision against an arbitrary one, it only moves the range (at most one binade of
// subnormals); in return c s is exact in bf16 and fp32, and moving codes to a larger
// scale is exact apart from underflow.  A NaN stays a NaN code (0x7f), an infinity
// becomes +-448.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

namespace rglru {
namespace e4m3 {

constexpr int kMinExp = -100, kMaxExp = 120;

// 2^e for a non-negative amax (an infinity counts as the largest exponent)
__device__ __forceinline__ float scale_of(float amax)
{
    const uint32_t b = __float_as_uint(amax);
    // amax = 1.m 2^x <= 1.75 2^(e + 8)  <=>  e >= x - 8, one more when 1.m > 1.75
    int e = (int)(b >> 23) - 127 - 8 + ((b & 0x7fffffu) > 0x600000u ? 1 : 0);
    e = max(kMinExp, min(kMaxExp, e));
    return __uint_as_float((uint32_t)(e + 127) << 23);
}
// 1 / s of a scale from scale_of, exact
__device__ __forceinline__ float inverse(float s) { return __uint_as_float((254u << 23) - __float_as_uint(s)); }

// codes of (lo, hi), lo in the low byte; to nearest, ties to even, saturating
__device__ __forceinline__ uint32_t pack2(float lo, float hi)
{
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}
__device__ __forceinline__ uint32_t pack4(float a, float b, float c, float d) { return pack2(a, b) | (pack2(c, d) << 16); }

// two codes to f16x2, exact (every e4m3 value is an f16 value)
__device__ __forceinline__ uint32_t to_f16x2(uint32_t codes)
{
    uint32_t r;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"((uint16_t)codes));
    return r;
}
// four codes (the low two, the high two)
__device__ __forceinline__ void to_f16x2x2(uint32_t codes, uint32_t &lo, uint32_t &hi)
{
    asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
        : "=r"(lo), "=r"(hi)
        : "r"(codes));
}
// Two f16 values as two e4m3 terms each, x = hi + lo: hi the nearest code, lo that of the rest.  hi keeps 4 significant
// bits, lo 4 more of a rest of at most half hi's step: a bf16 x (8 bits) is exact while |x| >= 2^-2; below
// that the error is at most 2^-10 absolutely (half of lo's smallest step).
__device__ __forceinline__ void split2(uint32_t x, uint32_t &hi, uint32_t &lo)
{
    asm("{\n\t.reg .b16 h, l;\n\t.reg .b32 f, r;\n\t"
        "cvt.rn.satfinite.e4m3x2.f16x2 h, %2;\n\tcvt.rn.f16x2.e4m3x2 f, h;\n\t"
        "sub.rn.f16x2 r, %2, f;\n\tcvt.rn.satfinite.e4m3x2.f16x2 l, r;\n\t"
        "cvt.u32.u16 %0, h;\n\tcvt.u32.u16 %1, l;\n\t}"
        : "=r"(hi), "=r"(lo)
        : "r"(x));
}
__device__ __forceinline__ void to_f32x2(uint32_t codes, float &lo, float &hi)
{
    const uint32_t h = to_f16x2(codes);
    asm("{\n\t.reg .f16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.f32.f16 %0, a;\n\tcvt.f32.f16 %1, b;\n\t}"
        : "=f"(lo), "=f"(hi)
        : "r"(h));
}

}  // namespace e4m3
}  // namespace rglru
