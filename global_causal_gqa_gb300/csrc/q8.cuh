// q8.cuh -- the numbers of the 8-bit paged cache.
//
// A vector x of one token and KV head is kept as d e4m3 numbers y and one power of two 2^e, e the
// smallest integer in [-126, 119] with max |x| <= 448 * 2^e (448 is e4m3's largest number):
//   y_i = x_i / 2^e rounded to the nearest e4m3 number (ties to even; at most 448 in magnitude),
// the byte e + 127 beside it (E8M0).  A power of two keeps everything but that one rounding exact:
// the division, the values read back in bf16 (4 significant bits), and, in attention, the
// factor's way out of the products.  e4m3 loses nothing to a factor of 448 / max |x| that is up to
// 2 off, since its step is relative down to 2^-6.  A vector with an infinity or a NaN gets the byte
// 255 and reads back as NaN.  Byte b stands for 2^(b - 127), whoever wrote it.
#pragma once
#include <cuda_fp16.h>

#include <cstdint>

#include "ptx.cuh"

namespace gqa {

constexpr uint32_t kScaleNan = 255;

// |a| or |b|, the larger; NaN if one is.
__device__ __forceinline__ float amax_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(fabsf(a)), "f"(fabsf(b)));
    return r;
}

// The byte of a vector whose largest magnitude is `most`: with most = 1.m * 2^E, e = E - 8, or
// E - 7 where 1.m > 1.75.
__device__ __forceinline__ uint32_t scale_byte(float most) {
    const uint32_t bits = __float_as_uint(most);
    if (bits >= 0x7f800000u) return kScaleNan;
    const int b = static_cast<int>(bits >> 23) - 8 + ((bits & 0x7fffffu) > 0x600000u ? 1 : 0);
    return b < 1 ? 1u : b > 246 ? 246u : static_cast<uint32_t>(b);
}

// 2^(byte - 127)
__device__ __forceinline__ float scale_of(uint32_t byte) {
    return byte == 0 ? __uint_as_float(0x00400000u)
                     : __uint_as_float(byte == kScaleNan ? 0x7fffffffu : byte << 23);
}
// byte - 127, the exponent that a scale byte stands for; NaN for 255.
__device__ __forceinline__ float exponent_of(uint32_t byte) {
    return byte == kScaleNan ? __uint_as_float(0x7fffffffu)
                             : __uint_as_float(0x4b000000u | byte) - 8388735.0f;
}
// 2^(127 - byte) for a byte that scale_byte gives to finite vectors; 0 for the others
__device__ __forceinline__ float inverse_scale(uint32_t byte) {
    return byte == kScaleNan ? 0.f : __uint_as_float((254u - byte) << 23);
}

// Two numbers as e4m3, lo in the low byte.
__device__ __forceinline__ uint32_t to_e4m3x2(float lo, float hi) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}
// Two e4m3 numbers (the low 16 bits of w) as f16, exactly.
__device__ __forceinline__ uint32_t e4m3x2_f16x2(uint32_t w) {
    uint32_t r;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(static_cast<uint16_t>(w)));
    return r;
}
// Two f16 numbers as e5m2, rounded to nearest, the first in the low byte.
__device__ __forceinline__ uint32_t to_e5m2x2(__half2 x) {
    uint16_t r;
    asm("cvt.rn.satfinite.e5m2x2.f16x2 %0, %1;"
        : "=h"(r)
        : "r"(*reinterpret_cast<const uint32_t *>(&x)));
    return r;
}
// Four e4m3 numbers times f, as bf16.
__device__ __forceinline__ uint2 e4m3x4_bf16(uint32_t w, float f) {
    const uint32_t a = e4m3x2_f16x2(w & 0xffffu), b = e4m3x2_f16x2(w >> 16);
    const float2 x = __half22float2(*reinterpret_cast<const __half2 *>(&a));
    const float2 y = __half22float2(*reinterpret_cast<const __half2 *>(&b));
    return make_uint2(pack_bf16x2(x.x * f, x.y * f), pack_bf16x2(y.x * f, y.y * f));
}

}  // namespace gqa
