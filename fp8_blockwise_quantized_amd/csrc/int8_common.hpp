// 8-bit integer operands on the device: one FP32 scale s for each row of the operand (a token, an output channel),
// codes q in -127 .. 127 with value q s.
//
// Rule, per row: s = max(fp32(amax / 127), fp32(1e-12)), q = fp32(x / s) to the nearest integer, ties to even, both
// divisions IEEE.  The quotient is at most 127 (1 + 2^-24) / (1 - 2^-24), which rounds to 127: no clamp is needed.  A
// row that holds a NaN or an infinity has the scale NaN, so that every product over it is NaN.
#pragma once

#include "quant_common.hpp"

namespace fp8bq {

__device__ __forceinline__ uint32_t abs_bits(float v) { return __float_as_uint(v) & 0x7FFFFFFFu; }

// Scale of a row whose largest magnitude has the float bits amax (infinities and NaNs come last in their order).
__device__ __forceinline__ float int8_scale(uint32_t amax) {
  if (amax >= 0x7F800000u) return __uint_as_float(0x7FC00000u);
  const float s = __uint_as_float(amax) / 127.0f;
  return s < scale_floor() ? scale_floor() : s;
}

// Adding 1.5 2^23 to |y| < 2^22 rounds it to the nearest integer, ties to even, and leaves that integer in two's
// complement in the low bits: four sums and three byte permutations make four codes.
__device__ __forceinline__ uint32_t int8_pack4(float a, float b, float c, float d) {
  const float magic = 12582912.0f;
  const uint32_t x = __float_as_uint(a + magic), y = __float_as_uint(b + magic);
  const uint32_t z = __float_as_uint(c + magic), w = __float_as_uint(d + magic);
  const uint32_t lo = __builtin_amdgcn_perm(y, x, 0x0C0C0400u), hi = __builtin_amdgcn_perm(w, z, 0x04000C0Cu);
  return lo | hi;
}
__device__ __forceinline__ uint2 int8_quant8(const float (&v)[8], float s, float r) {
  float y[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) y[i] = div_by_scale(v[i], s, r);
  return make_uint2(int8_pack4(y[0], y[1], y[2], y[3]), int8_pack4(y[4], y[5], y[6], y[7]));
}

// Largest magnitude of eight values, as bits.
__device__ __forceinline__ uint32_t amax8(const float (&v)[8], uint32_t m) {
#pragma unroll
  for (int i = 0; i < 8; ++i) m = umax(m, abs_bits(v[i]));
  return m;
}
__device__ __forceinline__ uint32_t row16_umax(uint32_t u) {
  u = umax_partner<kDppXor8>(u, u);
  u = umax_partner<kDppMirror8>(u, u);
  u = umax_partner<kDppXor2>(u, u);
  return umax_partner<kDppXor1>(u, u);
}
__device__ __forceinline__ uint32_t wave_umax(uint32_t u) {
  u = row16_umax(u);
  const uint32_t a = umax((uint32_t)__builtin_amdgcn_readlane((int)u, 0), (uint32_t)__builtin_amdgcn_readlane((int)u, 16));
  const uint32_t b = umax((uint32_t)__builtin_amdgcn_readlane((int)u, 32), (uint32_t)__builtin_amdgcn_readlane((int)u, 48));
  return umax(a, b);
}

}  // namespace fp8bq
