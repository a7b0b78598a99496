// MXFP4: blocks of 32 consecutive columns of a row, each an E8M0 scale byte
// s (the value 2^(s - 127); 255 is NaN) and 32 E2M1 codes (sign, two exponent
// bits, one mantissa bit: 0, 0.5, 1, 1.5, 2, 3, 4, 6), two codes per byte with
// the even column in the low nibble.
#pragma once

#include <cuda_fp16.h>
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

// Four fp32 values to four codes, column i in nibble i, and back.
__device__ __forceinline__ uint32_t f32x4_to_e2m1x4(float v0, float v1, float v2, float v3) {
    uint16_t r;
    asm("{\n\t.reg .b8 a, b;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
        "mov.b16 %0, {a, b};\n\t}"
        : "=h"(r) : "f"(v0), "f"(v1), "f"(v2), "f"(v3));
    return r;
}

__device__ __forceinline__ void e2m1x4_to_f32(uint32_t codes, float (&v)[4]) {
    uint32_t lo, hi;
    asm("{\n\t.reg .b8 a, b;\n\t"
        "mov.b16 {a, b}, %2;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, a;\n\t"
        "cvt.rn.f16x2.e2m1x2 %1, b;\n\t}"
        : "=r"(lo), "=r"(hi) : "h"(static_cast<uint16_t>(codes)));
    const float2 a = __half22float2(*reinterpret_cast<const __half2*>(&lo));
    const float2 b = __half22float2(*reinterpret_cast<const __half2*>(&hi));
    v[0] = a.x; v[1] = a.y; v[2] = b.x; v[3] = b.y;
}

// Instruction descriptor of kind::mxf4.block_scale for 128 rows x n columns:
// E2M1 A and B (format 1, bits 7-9 and 10-11), N >> 3 (17-22), UE8M0 scales
// (bit 23), M >> 7 (27-28), and the byte offset (0 or 2) of the two scales of
// an MMA in its columns' words (bits 4-5 for B, 29-30 for A).
__host__ __device__ constexpr uint32_t make_idesc_mxf4(uint32_t n, uint32_t sf_byte) {
    return (sf_byte << 4) | (1u << 7) | (1u << 10) | ((n >> 3) << 17) | (1u << 23) | (1u << 27) | (sf_byte << 29);
}

// D[tmem] (+)= (SFA x A[smem]) * (SFB x B[smem])^T: packed E2M1 operands, 64
// elements of K, one UE8M0 scale per row per 32 of them from tensor memory.
__device__ __forceinline__ void umma_mxf4_bs(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                             uint32_t sfa_tmem, uint32_t sfb_tmem, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%5], [%6], p;\n\t}"
        :: "r"(d_tmem), "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate), "r"(sfa_tmem), "r"(sfb_tmem)
        : "memory");
}

// 32 rows x 16 bytes (512 contiguous bytes of shared memory, groups of 8 rows
// 128 bytes apart) to 4 columns of tensor memory, the same in every lane
// quadrant: the scales of 128 rows for 128 elements of K (UE8M0 bytes, row r's
// four at 16 (r mod 32) + 4 (r div 32)).
__device__ __forceinline__ void tmem_cp_scales(uint32_t taddr, const void* src) {
    uint64_t d = 0;
    d |= static_cast<uint64_t>((smem_u32(src) & 0x3FFFFu) >> 4);
    d |= static_cast<uint64_t>(128u >> 4) << 16;
    d |= static_cast<uint64_t>(128u >> 4) << 32;
    d |= static_cast<uint64_t>(1u) << 46;
    asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" :: "r"(taddr), "l"(d) : "memory");
}

}  // namespace moe
