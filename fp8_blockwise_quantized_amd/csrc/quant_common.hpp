// Loads, the quantize step and the LDS tile layouts that the quantize kernels share.
#pragma once

#include "device_common.hpp"

namespace fp8bq {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

// Plain (temporal) global accesses: inputs are often read again (an activation feeds both the 1x128
// and the 128x1 pass) and codes are read next by the GEMM, so letting them stay in the 256 MB
// Infinity Cache pays; non-temporal hints measured faster only on tensors larger than that cache.
__device__ __forceinline__ void store_codes8(uint8_t* p, uint2 w) {
  *reinterpret_cast<u32x2*>(p) = (u32x2){w.x, w.y};
}
__device__ __forceinline__ void store_codes16(uint8_t* p, uint4 w) {
  *reinterpret_cast<u32x4*>(p) = (u32x4){w.x, w.y, w.z, w.w};
}

// Load 8 consecutive input elements (16 bytes of BF16 or 32 bytes of FP32) as fp32.
template <typename TIn>
struct Load8;
template <>
struct Load8<uint16_t> {
  static __device__ __forceinline__ void run(const uint16_t* p, float (&v)[8]) {
    const u32x4 w = *reinterpret_cast<const u32x4*>(p);
    v[0] = bf16lo(w.x); v[1] = bf16hi(w.x);
    v[2] = bf16lo(w.y); v[3] = bf16hi(w.y);
    v[4] = bf16lo(w.z); v[5] = bf16hi(w.z);
    v[6] = bf16lo(w.w); v[7] = bf16hi(w.w);
  }
};
template <>
struct Load8<float> {
  static __device__ __forceinline__ void run(const float* p, float (&v)[8]) {
    const f32x4 a = *reinterpret_cast<const f32x4*>(p);
    const f32x4 b = *(reinterpret_cast<const f32x4*>(p) + 1);
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
  }
};

// Quantize 8 values with the group's (s, r) into two dwords of codes.  CLAMP: clamp the quotients to
// +-fmt_max before converting, which a per-tensor scale from a running amax needs (the tensor can
// exceed it); a blockwise scale comes from the group's own amax, so the quotients need no clamp
// (blockwise_quotient).
template <int FMT, bool CLAMP = false>
__device__ __forceinline__ uint2 quant8(const float (&v)[8], float s, float r) {
  float y[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) y[i] = CLAMP ? clamp_fmt<FMT>(div_by_scale(v[i], s, r)) : blockwise_quotient(v[i], s, r);
  return make_uint2(pack4<FMT>(y[0], y[1], y[2], y[3]), pack4<FMT>(y[4], y[5], y[6], y[7]));
}

constexpr int kQtCols = 128;

// LDS layouts of the 128-column tile kernels, chosen so that no access conflicts on LDS banks
// (64 banks of 4 bytes; a thread's 8 columns are 8*cc .. 8*cc+7, cc = t % 16, and the 4 row groups
// of a wave share them):
// - per-column arrays (partial maxima, scales) put column c at c + 4*(c/64): columns c and c+64,
//   which one instruction's lanes cc and cc+8 touch together, fall on different banks;
// - the transposed codes: column c's 128 codes (one byte per row) at byte 128*c + 128*(c/64), its
//   8-byte unit u (rows 8u .. 8u+7) at unit u ^ 2*((c ^ c/8) % 8).  The XOR value is even, so the
//   16-byte read of units 2h, 2h+1 stays one aligned access.
constexpr int kColPos = kQtCols + 4;   // entries per padded per-column array
constexpr int kRedStride = kColPos + 1;  // partial-maxima row stride (133: row groups 4 banks apart)
constexpr int kQtBytes = kQtCols * 128 + 128;
__device__ __forceinline__ int col_pos(int c) { return c + ((c >> 6) << 2); }
__device__ __forceinline__ int qt_off(int c, int u) {
  return (c << 7) + ((c >> 6) << 7) + ((u ^ (((c ^ (c >> 3)) & 7) << 1)) << 3);
}

}  // namespace fp8bq
