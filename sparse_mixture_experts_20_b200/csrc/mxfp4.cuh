// MXFP4: blocks of 32 consecutive columns of a row, each an E8M0 scale byte
// s (the value 2^(s - 127); 255 is NaN) and 32 E2M1 codes (sign, two exponent
// bits, one mantissa bit: 0, 0.5, 1, 1.5, 2, 3, 4, 6), two codes per byte with
// the even column in the low nibble.
#pragma once

#include "common.cuh"

namespace moe {

// The scale byte of a block whose largest magnitude has the fp32 bits `bits`:
// the smallest k with amax <= 6 * 2^k as k + 127 (6 = 1.5 * 2^2; k >= -126, so
// that a scale is a normal fp32 number; 2^0 for a block of zeros), or 255 when
// the block holds an infinity or a NaN.
__device__ __forceinline__ uint32_t mxfp4_scale_byte(uint32_t bits) {
    const int e = static_cast<int>(bits >> 23);
    if (e == 255) return 255u;
    if (bits == 0) return 127u;
    // amax = (1 + m / 2^23) 2^(e - 127) <= 1.5 * 2^(2 + k)  <=>  k >= e - 129
    // for m <= 0.5, k >= e - 128 above; a subnormal amax clamps anyway
    const int k = e - 129 + ((bits & 0x7FFFFFu) > 0x400000u ? 1 : 0);
    return static_cast<uint32_t>(max(k, -126) + 127);
}

// 2^(127 - b) for a scale byte b of mxfp4_scale_byte (1 <= b <= 253), exactly.
__device__ __forceinline__ float mxfp4_inv_scale(uint32_t b) { return __uint_as_float((254u - b) << 23); }

// The value of any scale byte as fp32 (0: 2^-127, subnormal; 255: NaN).
__device__ __forceinline__ float e8m0_value(uint32_t b) {
    return __uint_as_float(b == 0u ? 0x00400000u : b == 255u ? 0x7FC00000u : b << 23);
}

// Eight fp32 values to eight codes, column i in nibble i, round to nearest
// even, saturating at +-6.
__device__ __forceinline__ uint32_t f32x8_to_e2m1x8(const float (&v)[8]) {
    uint32_t r;
    asm("{\n\t.reg .b8 a, b, c, d;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
        "mov.b32 %0, {a, b, c, d};\n\t}"
        : "=r"(r)
        : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]));
    return r;
}

// Eight codes to four pairs of fp16 (exact): pair i holds columns 2i (low
// half) and 2i + 1.
__device__ __forceinline__ void e2m1x8_to_f16x2(uint32_t codes, uint32_t (&h)[4]) {
    asm("{\n\t.reg .b8 a, b, c, d;\n\t"
        "mov.b32 {a, b, c, d}, %4;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, a;\n\t"
        "cvt.rn.f16x2.e2m1x2 %1, b;\n\t"
        "cvt.rn.f16x2.e2m1x2 %2, c;\n\t"
        "cvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
        : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3]) : "r"(codes));
}

}  // namespace moe
