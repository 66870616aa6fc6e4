// 8-bit caches: e4m3 codes (sign, four bits of exponent with bias 7, three of mantissa, 0x7f NaN)
// and the scales of their blocks, which are powers of two.
#pragma once

#include "tv_device.cuh"

namespace tv {

// Of a scale that is no power of two the exponent counts.
__device__ __forceinline__ uint32_t exponent_byte(float scale) { return (__float_as_uint(scale) >> 23) & 0xffu; }
__device__ __forceinline__ float scale_of(uint32_t exponent) { return __uint_as_float(exponent << 23); }

// The smallest power of two, from 2^-100 on, times which 448 reaches a (finite, not negative): with
// a = m 2^E, m in [1, 2), 448 = 1.75 2^8 does at 2^(E - 8) for m <= 1.75.
__device__ __forceinline__ float scale_needed(float a) {
    const uint32_t b = __float_as_uint(a);
    const int e = (int)(b >> 23) - 8 + ((b & 0x7fffffu) > 0x600000u ? 1 : 0);
    return scale_of((uint32_t)max(e, 127 - 100));
}
// 1 / scale for a power of two of [2^-126, 2^126].
__device__ __forceinline__ float scale_inverse(float scale) {
    return __uint_as_float((254u << 23) - (__float_as_uint(scale) & 0x7f800000u));
}

__device__ __forceinline__ float e4m3_float(uint32_t c) {
    const float x = __uint_as_float(((c & 0x80u) << 24) | ((c & 0x7fu) << 20)) * 1.329227995784916e36f;  // 2^120
    return (c & 0x7fu) == 0x7fu ? __uint_as_float(0x7fc00000u) : x;
}
// Two float32 to codes (lo in the low byte), to the nearest, ties to even; NaN to NaN.
__device__ __forceinline__ uint32_t e4m3_pair(float lo, float hi) {
    uint16_t d;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(d) : "f"(hi), "f"(lo));
    return d;
}
// The same of and to pairs of float16.
__device__ __forceinline__ uint32_t e4m3_of_half2(uint32_t h) {
    uint16_t d;
    asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(d) : "r"(h));
    return d;
}
__device__ __forceinline__ uint32_t half2_of_e4m3(uint32_t c) {
    uint32_t d;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(d) : "h"((uint16_t)c));
    return d;
}
__device__ __forceinline__ uint32_t half2_of(float lo, float hi) {
    uint32_t d;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
    return d;
}
__device__ __forceinline__ uint32_t half2_sub(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}
__device__ __forceinline__ uint32_t max_u16x2(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("max.u16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}
// Four codes times a power of two, rounded again.
__device__ __forceinline__ uint32_t e4m3_scaled(uint32_t w, float by) {
    const uint32_t lo = e4m3_pair(e4m3_float(w & 0xffu) * by, e4m3_float((w >> 8) & 0xffu) * by);
    return lo | e4m3_pair(e4m3_float((w >> 16) & 0xffu) * by, e4m3_float(w >> 24) * by) << 16;
}

}  // namespace tv
