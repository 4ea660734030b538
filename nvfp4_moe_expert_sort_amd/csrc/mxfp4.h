// mxfp4.h -- the microscaled 4-bit format (OCP MX: blocks of 32 elements along
// the row, one E8M0 power-of-two scale each, E2M1 elements) and the operand
// layouts of its products.
//
// v_mfma_scale_f32_16x16x128_f8f6f4 takes both operands as they are stored:
// lane q*16 + r supplies row r's 32 codes of columns [32 q, 32 q + 32) of a
// 128-column chunk (16 bytes, element 2i in the low nibble of byte i) and one
// scale byte, picked from a 32-bit register by an immediate.  Every layout
// below therefore keeps the scales of four consecutive chunks in one word.
#pragma once

#include "nvfp4_device.h"

namespace nvfp4 {

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));
typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

constexpr uint32_t kMxNan = 255;  // E8M0 NaN: the scale of a block that holds an Inf or NaN

// Larger of two words' 16-bit halves, each a BF16 magnitude.
__device__ __forceinline__ uint32_t mx_max2(uint32_t a, uint32_t b) {
    return __builtin_bit_cast(uint32_t, __builtin_elementwise_max(__builtin_bit_cast(u16x2, a), __builtin_bit_cast(u16x2, b)));
}
__device__ __forceinline__ uint32_t mx_abs(uint32_t w) { return w & 0x7FFF7FFFu; }

// Largest magnitude (BF16 bits) of a block whose elements four neighbouring lanes hold, eight each.
__device__ __forceinline__ uint32_t mx_block_max(u32x4 v) {
    uint32_t m = mx_max2(mx_max2(mx_abs(v[0]), mx_abs(v[1])), mx_max2(mx_abs(v[2]), mx_abs(v[3])));
    m = max(m & 0xFFFFu, m >> 16);
    m = max(m, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)m, 0xB1, 0xF, 0xF, true));         // lanes 1 0 3 2
    return max(m, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)m, 0x4E, 0xF, 0xF, true));  // lanes 2 3 0 1
}

// Scale byte k + 127 of a block whose largest magnitude has the BF16 bits m
// (15 bits): with m = 1.f x 2^e, k = e - 2 (floor), or e - 1 where 1.f > 1.5
// and the scale is rounded up so that m <= 6 x 2^k.  Scales end at 2^-127,
// below which a BF16 magnitude lies under 2^-124.
__device__ __forceinline__ uint32_t mx_scale_byte(uint32_t m, bool up) {
    const int e = (int)(m >> 7);
    if (e == 255) return kMxNan;
    return (uint32_t)max(e - 2 + ((up && (m & 127u) > 64u) ? 1 : 0), 0);
}

// Codes of 8 BF16 elements (4 words) under a scale byte: the hardware divides
// by the power of two and rounds to the nearest E2M1 value, ties to the even
// code, saturating at 6 and keeping the sign.
__device__ __forceinline__ uint32_t mx_encode8(u32x4 w, uint32_t byte) {
    const float s = __uint_as_float(byte << 23);
    const uint32_t w0 = w[0], w1 = w[1], w2 = w[2], w3 = w[3];  // (a bit cast of a vector element itself reads element 0)
    uint32_t r = 0;
    r = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(r, __builtin_bit_cast(bf16x2, w0), s, 0);
    r = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(r, __builtin_bit_cast(bf16x2, w1), s, 1);
    r = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(r, __builtin_bit_cast(bf16x2, w2), s, 2);
    r = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(r, __builtin_bit_cast(bf16x2, w3), s, 3);
    return byte == kMxNan ? 0u : r;
}

// The 8 BF16 values of a word of codes.
__device__ __forceinline__ u32x4 mx_decode8(uint32_t codes, uint32_t byte) {
    const float s = __uint_as_float(byte << 23);
    u32x4 w;
    w[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, s, 0));
    w[1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, s, 1));
    w[2] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, s, 2));
    w[3] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, s, 3));
    return byte == kMxNan ? u32x4{0x7FC07FC0u, 0x7FC07FC0u, 0x7FC07FC0u, 0x7FC07FC0u} : w;
}

// acc += W A^T over one 128-column chunk: register j of lane q*16 + r holds
// weight row 4 q + j of the tile and activation row r.  SEL: byte of the scale words.
template <int SEL>
__device__ __forceinline__ f32x4 mx_mfma(u32x4 w, u32x4 a, f32x4 acc, uint32_t ws, uint32_t as) {
    const i32x8 wv = {(int)w[0], (int)w[1], (int)w[2], (int)w[3], 0, 0, 0, 0};
    const i32x8 av = {(int)a[0], (int)a[1], (int)a[2], (int)a[3], 0, 0, 0, 0};
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(wv, av, acc, 4, 4, SEL, (int)ws, SEL, (int)as);
}

}  // namespace nvfp4
