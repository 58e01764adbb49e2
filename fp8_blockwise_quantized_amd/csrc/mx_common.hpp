// Microscaled 4-bit operands (MXFP4) on the device: blocks of 32 values along the contraction, E2M1 codes
// (0, .5, 1, 1.5, 2, 3, 4, 6 and negatives; two per byte, the even element in the low half) and one E8M0
// scale byte b per block, 2^(b - 127).
//
// Scales of four consecutive blocks (128 values) share a 32-bit word, block j in byte j; the words of a
// 128-long stretch are contiguous over the rows: s[(k / 128) * lds + row].  A lane that owns block j of a row
// shifts the word by 8 j and the MFMA's byte select picks the rest.
//
// Quantization of a block: e = max(floor(log2 amax) - 2, -127), the largest power of two that puts amax
// below 8 (E2M1's largest binade is [4, 8)); codes are x 2^-e rounded to the nearest, ties to even, values
// past 6 to 6.  With amax's bits this is b = max(exponent field - 2, 0), exact and free of logarithms.  A block
// with a NaN or an infinity (exponent field 255) gets b = 255, E8M0's NaN, which makes every product that
// reads it NaN.  x 2^-e is exact (a power of two; 2^127 at most, so no scale is subnormal: the converter
// flushes subnormal scales, which is why the product is taken first and the converter's scale is 1).
#pragma once

#include "device_common.hpp"

namespace fp8bq {

constexpr int kMxBlock = 32;

typedef float v16f __attribute__((ext_vector_type(16)));

// Scale byte of a block whose largest magnitude has the float bits amax (NaN and infinity included: as
// unsigned integers the bits of magnitudes are ordered, infinities and NaNs last).
__device__ __forceinline__ uint32_t mx_scale_byte(uint32_t amax) {
  const uint32_t ex = amax >> 23;
  return ex == 255u ? 255u : (ex > 2u ? ex - 2u : 0u);
}
// 2^-e for that byte (1 for the NaN byte, whose codes do not matter).
__device__ __forceinline__ float mx_inverse(uint32_t b) {
  return __uint_as_float(b == 255u ? 0x3F800000u : (254u - b) << 23);
}
// Eight scaled values -> eight codes, the first in the lowest half byte.
__device__ __forceinline__ uint32_t mx_pack8(const float (&y)[8]) {
  uint32_t w = 0;
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, y[0], y[1], 1.0f, 0);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, y[2], y[3], 1.0f, 1);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, y[4], y[5], 1.0f, 2);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, y[6], y[7], 1.0f, 3);
  return w;
}
__device__ __forceinline__ uint32_t mx_abs_bits(float v) { return __float_as_uint(v) & 0x7FFFFFFFu; }

// An MFMA operand from a lane's 32 codes (16 bytes; the other half of the register octet is not read in
// the 4-bit format).
__device__ __forceinline__ v8i mx_operand(v4i c) { return (v8i){c.x, c.y, c.z, c.w, 0, 0, 0, 0}; }

// One block of 32 BF16 values (packed pairs, in order) -> codes and scale byte.  The converter divides by the
// scale itself and takes pairs; a subnormal scale (byte 0, amax below 2^-124) it would flush, so such a block
// takes the product with 2^127 instead.
__device__ __forceinline__ uint32_t mx_pack8_bf16(uint32_t a, uint32_t b, uint32_t c, uint32_t d, float scale) {
  uint32_t w = 0;
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(w, __builtin_bit_cast(bf16x2_t, a), scale, 0);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(w, __builtin_bit_cast(bf16x2_t, b), scale, 1);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(w, __builtin_bit_cast(bf16x2_t, c), scale, 2);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(w, __builtin_bit_cast(bf16x2_t, d), scale, 3);
  return w;
}
// The converter's scale of byte b >= 1 (1 for byte 0 and for the NaN byte).
__device__ __forceinline__ float mx_scale_of(uint32_t b) {
  return __uint_as_float(b == 0u || b == 255u ? 0x3F800000u : b << 23);
}
// A pair times 2^127, exact in BF16 for the magnitudes of a byte-0 block.
__device__ __forceinline__ uint32_t mx_lift_bf16(uint32_t w) {
  const float up = __uint_as_float(254u << 23);
  return pack_bf16x2(bf16lo(w) * up, bf16hi(w) * up);
}

}  // namespace fp8bq
