// The 4-bit values of a paged cache.
//
// 16 columns of a row share a scale of 8 bits: five exponent bits and three
// fraction bits, the bits 14 .. 7 of a float16 (2^-17 .. 10240; what is more would
// overflow a float16 with the largest code).  A code is sign, two exponent bits
// and a fraction bit: 0, 0.5, 1, 1.5, 2, 3, 4, 6.  A value is code times scale:
// at most 6 significant bits, so it is exact in float16 and in bf16.
//
//   scale = round(amax / 6), to nearest, ties to even, at most 10240;
//   code  = round(x / scale), to nearest, ties to even, at most 6 (0 where the scale is 0).
// A scale is off by 1/16 of itself, a code below 4 by 1/2 and above by 1: a value by
// 17/16 amax / 6 at most.  A group with a NaN or an infinity has scale byte 255, a float16 NaN.
#pragma once

#include <cuda_fp16.h>

#include "ptx.cuh"

namespace eta {

constexpr int kE2m1TopScale = 0xE2;   // 10240
constexpr int kE2m1NanScale = 0xFF;

// The largest magnitude of 8 values, as float bits (a NaN above all).
__device__ __forceinline__ uint32_t e2m1_amax(const float (&x)[8]) {
    uint32_t m = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e) m = max(m, __float_as_uint(x[e]) & 0x7fffffffu);
    return m;
}

// The scale byte of a group whose largest magnitude has these bits.
__device__ __forceinline__ int e2m1_scale(uint32_t amax) {
    if (amax >= 0x7f800000u) return kE2m1NanScale;
    const float t = __fdiv_rn(__uint_as_float(amax), 6.f);
    if (t < 6.103515625e-05f) return static_cast<int>(rintf(t * 131072.f));   // below 2^-14: multiples of 2^-17
    uint32_t b = __float_as_uint(t);
    b = (b + 0x7ffffu + ((b >> 20) & 1u)) >> 20;   // four significant bits
    return min(static_cast<int>(b) - ((127 - 15) << 3), kE2m1TopScale);
}

// Two copies of a scale, as float16.
__device__ __forceinline__ uint32_t e2m1_scale_h2(uint32_t byte) { return byte * 0x00800080u; }

// 8 values as codes, the first in the lowest four bits.  x / scale is rounded
// to float32 first: the quotient of a float by a number of 4 bits lies further
// from a border between two codes than that rounding moves it, unless it is on
// the border.  (Markstein's correction of x times the rounded reciprocal: with
// it the quotient is the correctly rounded one.)
__device__ __forceinline__ uint32_t e2m1_pack(const float (&x)[8], int byte) {
    if (byte == 0 || byte == kE2m1NanScale) return 0u;
    const float s = __half2float(__ushort_as_half(static_cast<unsigned short>(byte << 7)));
    const float inv = __frcp_rn(s);
    float q[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const float y = __fmul_rn(x[e], inv);
        q[e] = copysignf(__fmaf_rn(__fmaf_rn(-y, s, x[e]), inv, y), x[e]);   // (-0 keeps its sign)
    }
    uint32_t r;
    asm("{\n\t.reg .b8 a, b, c, d;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
        "mov.b32 %0, {a, b, c, d};\n\t}"
        : "=r"(r)
        : "f"(q[0]), "f"(q[1]), "f"(q[2]), "f"(q[3]), "f"(q[4]), "f"(q[5]), "f"(q[6]), "f"(q[7]));
    return r;
}

// The float16 pairs that the four bytes of a word stand for, unscaled.
__device__ __forceinline__ void e2m1_halves(uint32_t w, uint32_t (&r)[4]) {
    asm("{\n\t.reg .b8 a, b, c, d;\n\t"
        "mov.b32 {a, b, c, d}, %4;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, a;\n\t"
        "cvt.rn.f16x2.e2m1x2 %1, b;\n\t"
        "cvt.rn.f16x2.e2m1x2 %2, c;\n\t"
        "cvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
        : "r"(w));
}
__device__ __forceinline__ uint32_t h2_mul(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
__device__ __forceinline__ void e2m1_values(uint32_t w, uint32_t scale2, uint32_t *out) {
    uint32_t r[4];
    e2m1_halves(w, r);
#pragma unroll
    for (int e = 0; e < 4; ++e) out[e] = h2_mul(r[e], scale2);
}

// bf16 rows beside 4-bit values become float16 (which holds those values exactly):
// the power of two that brings a row's largest magnitude (float bits) to 2^14 ..
// 2^15.  A column then keeps its 8 bits down to 2^-29 of the largest, and is off by
// 2^-39 of that at most below (half of 2^-24, beside 2^14 at least).  -114 .. 126.
__device__ __forceinline__ int f16_shift(uint32_t top) {
    return top == 0u ? 0 : min(14 + 127 - static_cast<int>(top >> 23), 126);
}
// What turns a product with such a row back into a score; a number, or a score of 0 would be NaN.
__device__ __forceinline__ float f16_back(float scale, int up) {
    return fminf(scale * __uint_as_float(static_cast<uint32_t>(127 - up) << 23), 3.402823466e+38f);
}

}  // namespace eta
