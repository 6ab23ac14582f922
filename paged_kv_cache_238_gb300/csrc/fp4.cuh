// The 4-bit pool: its layout, and the conversions between codes and values.
//
// A value is code * scale * factor: the code in e2m1 (0, 0.5, 1, 1.5, 2, 3, 4, 6 and their
// negatives), the scale in e4m3 shared by 16 consecutive dims of a token's head row, and the pool's
// factor, a power of two that the caller passes. code * scale has 6 significant bits between 2^-10
// and 2688, so fp16, bf16 and fp32 hold it exactly.
//
// A page of 16 tokens of one kv head is 9 D contiguous bytes: 16 rows of D / 2 bytes of codes (the
// even dim in the low half of its byte), then 16 rows of D / 16 scales. Codes and scales lie apart so
// that 16-byte loads of codes are aligned, and a warp that reads 16 bytes a lane of consecutive keys
// reads consecutive addresses.
#pragma once

#include <cuda_fp16.h>

#include "pa_device.cuh"

namespace pa {

constexpr int kFp4Group = 16;  // dims that share a scale

__host__ __device__ constexpr int fp4_page_bytes(int D) { return 9 * D; }
__host__ __device__ constexpr int fp4_scales_at(int D) { return 8 * D; }  // within a page

// Byte offset of a page in a pool: page `sub` of (block, kv head).
__device__ __forceinline__ int64_t fp4_page_at(int32_t block, int32_t num_kv_heads, int32_t h, int32_t sub_log2,
                                               int32_t sub, int D) {
    return (((static_cast<int64_t>(block) * num_kv_heads + h) << sub_log2) + sub) * fp4_page_bytes(D);
}

// Eight codes -> eight halves, in order; the hardware conversion costs about 1.5 issue slots for two values
// (shifts and masks: 4).
__device__ __forceinline__ void fp4_halves(uint32_t w, uint32_t (&h)[4]) {
    asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
        "mov.b32 {b0, b1, b2, b3}, %4;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, b0;\n\t"
        "cvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
        "cvt.rn.f16x2.e2m1x2 %2, b2;\n\t"
        "cvt.rn.f16x2.e2m1x2 %3, b3;\n\t}"
        : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
        : "r"(w));
}

// Two e4m3 scales -> two halves (low byte first). e4m3 lies within fp16's normal range and its subnormals are exact.
__device__ __forceinline__ uint32_t e4m3x2_halves(uint16_t s) {
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(s));
    return h;
}

__device__ __forceinline__ uint32_t hmul2(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}

__device__ __forceinline__ float2 halves_to_floats(uint32_t h) {
    return __half22float2(*reinterpret_cast<const __half2*>(&h));
}

// Four values -> two bytes of codes, nearest with ties to the even code, saturated to +-6.
__device__ __forceinline__ uint32_t fp4_codes4(float x0, float x1, float x2, float x3) {
    uint32_t r;
    asm("{\n\t.reg .b8 b0, b1;\n\t.reg .b32 lo, hi;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n\t"
        "cvt.u32.u8 lo, b0;\n\t"
        "cvt.u32.u8 hi, b1;\n\t"
        "shl.b32 hi, hi, 8;\n\t"
        "or.b32 %0, lo, hi;\n\t}"
        : "=r"(r)
        : "f"(x0), "f"(x1), "f"(x2), "f"(x3));
    return r;
}

// A scale in e4m3, nearest with ties to even, saturated to 448.
__device__ __forceinline__ uint32_t e4m3_byte(float x) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(0.f), "f"(x));
    return r & 0xffu;
}

// 16 values that share a scale -> 8 bytes of codes, and the scale: s = e4m3(max |y| / 6), code = e2m1(y / s).
// Every border is decided exactly. A border is t s (t halfway between two codes) or 6 t (halfway between two
// scales), which fp32 holds exactly; a different fp32 number divided by s (or 6) is more than 0.53 steps of t away from
// t, as s has 4 bits. So the quotient must be exact where it is representable and within 0.53 steps elsewhere: y / s is
// the product with 1 / s, corrected once by its exact residual. A scale of 0 makes all codes 0. A NaN takes no part in
// the maximum; its code is some number's.
__device__ __forceinline__ uint2 fp4_pack16(const float (&y)[16], uint32_t* scale_byte) {
    float top = 0.f;
#pragma unroll
    for (int i = 0; i < 16; ++i) top = fmaxf(top, fabsf(y[i]));
    const uint32_t byte = e4m3_byte(__fdiv_rn(top, 6.f));
    *scale_byte = byte;
    if (byte == 0u) return make_uint2(0u, 0u);
    const float s = halves_to_floats(e4m3x2_halves(static_cast<uint16_t>(byte))).x;
    const float inv = __frcp_rn(s);
    float z[16];
    if (top < 1e30f) {
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            const float q = __fmul_rn(y[i], inv);
            z[i] = __fmaf_rn(__fmaf_rn(-q, s, y[i]), inv, q);
        }
    } else {  // the residual would overflow; s is 448
#pragma unroll
        for (int i = 0; i < 16; ++i) z[i] = __fdiv_rn(y[i], s);
    }
    return make_uint2(fp4_codes4(z[0], z[1], z[2], z[3]) | fp4_codes4(z[4], z[5], z[6], z[7]) << 16,
                      fp4_codes4(z[8], z[9], z[10], z[11]) | fp4_codes4(z[12], z[13], z[14], z[15]) << 16);
}

}  // namespace pa
