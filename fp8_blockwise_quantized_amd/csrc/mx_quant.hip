// MXFP4 quantizer: row blocks (32 consecutive elements of a row), column blocks (32 consecutive rows of a
// column, outputs transposed so that the contraction is contiguous), or both from one read.
//
// Bound by HBM: 2 (BF16) or 4 (FP32) bytes read and 0.53 written per element and layout.  16384 x 5632 BF16 takes
// 36 us in one layout and 56 us in both when it lies in the Infinity Cache (6.5 and 5.0 TB/s), 51-54 and 66 us from HBM
// (4.4-4.6 TB/s; a copy reaches 6.3 there).  Persistent workgroups that read a tile ahead were no faster from
// HBM (52-56 us), non-temporal reads and writes 10% faster there and 20-30% slower from the cache: not taken.
// A workgroup of four waves owns a tile of 128 rows by 128 columns; a wave holds 32 rows of it, a thread a patch of
// 8 rows by 8 columns (eight independent 16-byte loads of BF16).  A row block is then 4 neighbouring lanes (two DPP
// exchanges) and a column block the 4 lanes of the wave that are 16 apart, so neither maximum needs LDS or a
// barrier; only the transposed codes are staged in LDS, for stores of 64 contiguous bytes per column.
#include "launch.hpp"
#include "mx_common.hpp"
#include "quant_common.hpp"

namespace fp8bq {

// Both halves' value (or packed pair) with the lanes 16, 32 and 48 away, by f: the swaps give every lane its
// own and its partner's value in one of the two results each.
template <typename F>
__device__ __forceinline__ uint32_t over_row_groups(uint32_t v, F f) {
  const auto a = __builtin_amdgcn_permlane16_swap(v, v, false, false);
  v = f(a[0], a[1]);
  const auto b = __builtin_amdgcn_permlane32_swap(v, v, false, false);
  return f(b[0], b[1]);
}

// Staged codes of column c: 64 bytes (four 32-row blocks of 16), the 16-byte units XORed by the column so
// that the 16 columns one store instruction writes spread over the banks.
__device__ __forceinline__ int mx_stage(int c, int unit) { return 64 * c + 16 * (unit ^ ((c >> 3) & 3)); }

// A thread's 8 rows by 8 columns.  row(p) and column(i) give the scale byte and the codes of row p (its 8 columns) and
// of column i (its 8 rows); row blocks are the 4 lanes of a quad, column blocks the 4 row groups of the wave.
template <typename TIn>
struct MxPatch;
template <>
struct MxPatch<float> {
  float v[8][8];
  __device__ __forceinline__ void load(int p, const float* x) { Load8<float>::run(x, v[p]); }
  __device__ __forceinline__ void clear(int p) {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[p][i] = 0.0f;
  }
  __device__ __forceinline__ uint32_t row(int p, uint32_t& codes) const {
    uint32_t m = mx_abs_bits(v[p][0]);
#pragma unroll
    for (int i = 1; i < 8; ++i) m = umax(m, mx_abs_bits(v[p][i]));
    m = umax_partner<kDppXor1>(m, m);
    m = umax_partner<kDppXor2>(m, m);
    const uint32_t b = mx_scale_byte(m);
    const float inv = mx_inverse(b);
    float y[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) y[i] = v[p][i] * inv;
    codes = mx_pack8(y);
    return b;
  }
  // columns 2c and 2c + 1
  __device__ __forceinline__ void columns(int c, uint32_t (&b)[2], uint32_t (&codes)[2]) const {
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      uint32_t m = mx_abs_bits(v[0][2 * c + k]);
#pragma unroll
      for (int p = 1; p < 8; ++p) m = umax(m, mx_abs_bits(v[p][2 * c + k]));
      m = over_row_groups(m, [](uint32_t x, uint32_t y) { return umax(x, y); });
      b[k] = mx_scale_byte(m);
      const float inv = mx_inverse(b[k]);
      float y[8];
#pragma unroll
      for (int p = 0; p < 8; ++p) y[p] = v[p][2 * c + k] * inv;
      codes[k] = mx_pack8(y);
    }
  }
};
// BF16 stays packed: magnitudes compare as 16-bit integers, two at a time, and the converter takes pairs.  Half
// the registers of the unpacked form (and so about twice the waves to wait on memory with).
template <>
struct MxPatch<uint16_t> {
  u32x4 w[8];
  __device__ __forceinline__ void load(int p, const uint16_t* x) { w[p] = *reinterpret_cast<const u32x4*>(x); }
  __device__ __forceinline__ void clear(int p) { w[p] = (u32x4){0, 0, 0, 0}; }
  // codes of four pairs under scale byte b, of a block whose largest magnitude is m (BF16 bits)
  static __device__ __forceinline__ uint32_t pack(uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b,
                                                  uint32_t m) {
    if (b == 0u && m != 0u) {
      a0 = mx_lift_bf16(a0);
      a1 = mx_lift_bf16(a1);
      a2 = mx_lift_bf16(a2);
      a3 = mx_lift_bf16(a3);
    }
    return mx_pack8_bf16(a0, a1, a2, a3, mx_scale_of(b));
  }
  __device__ __forceinline__ uint32_t row(int p, uint32_t& codes) const {
    uint32_t m2 = w[p][0] & 0x7FFF7FFFu;
#pragma unroll
    for (int i = 1; i < 4; ++i) m2 = pk_umax16(m2, w[p][i] & 0x7FFF7FFFu);
    uint32_t m = umax(m2 & 0xFFFFu, m2 >> 16);
    m = umax_partner<kDppXor1>(m, m);
    m = umax_partner<kDppXor2>(m, m);
    const uint32_t b = mx_scale_byte(m << 16);
    codes = pack(w[p][0], w[p][1], w[p][2], w[p][3], b, m);
    return b;
  }
  __device__ __forceinline__ void columns(int c, uint32_t (&b)[2], uint32_t (&codes)[2]) const {
    uint32_t m2 = w[0][c] & 0x7FFF7FFFu;
#pragma unroll
    for (int p = 1; p < 8; ++p) m2 = pk_umax16(m2, w[p][c] & 0x7FFF7FFFu);
    m2 = over_row_groups(m2, [](uint32_t x, uint32_t y) { return pk_umax16(x, y); });
    uint32_t lo[4], hi[4];  // pairs of rows of the even and of the odd column
#pragma unroll
    for (int p = 0; p < 4; ++p) {
      lo[p] = __builtin_amdgcn_perm(w[2 * p + 1][c], w[2 * p][c], 0x05040100u);
      hi[p] = __builtin_amdgcn_perm(w[2 * p + 1][c], w[2 * p][c], 0x07060302u);
    }
    b[0] = mx_scale_byte(m2 << 16);
    b[1] = mx_scale_byte(m2 & 0xFFFF0000u);
    codes[0] = pack(lo[0], lo[1], lo[2], lo[3], b[0], m2 & 0xFFFFu);
    codes[1] = pack(hi[0], hi[1], hi[2], hi[3], b[1], m2 >> 16);
  }
};

template <typename TIn, bool ROWS, bool COLS>
__global__ __launch_bounds__(256) void mx_quant_kernel(const TIn* __restrict__ x, int64_t R, int64_t C, int64_t ldx,
                                                       uint8_t* __restrict__ q, int64_t ldq,
                                                       uint32_t* __restrict__ s, int64_t lds,
                                                       uint8_t* __restrict__ qt, int64_t ldqt,
                                                       uint32_t* __restrict__ st, int64_t ldst, uint32_t ncg) {
  __shared__ __attribute__((aligned(16))) uint8_t codes[COLS ? 128 * 64 : 16];
  __shared__ uint8_t scales[COLS ? 128 * 4 : 4];

  const int t = threadIdx.x;
  const int wid = t >> 6;
  const int cc = t & 15;        // 8-column chunk of the tile
  const int rg = (t >> 4) & 3;  // 8-row group of the wave's 32 rows
  const TileRC tile = tile_of_block(ncg);
  const int64_t r0 = tile.row * 128 + 32 * wid + 8 * rg;
  const int64_t col = tile.col * 128 + 8 * cc;
  const bool cvalid = col < C;  // C % 8 == 0: a chunk is all in or all out

  MxPatch<TIn> v;
#pragma unroll
  for (int p = 0; p < 8; ++p) {
    if (cvalid && r0 + p < R)
      v.load(p, x + (r0 + p) * ldx + col);
    else
      v.clear(p);
  }

  if constexpr (ROWS) {
#pragma unroll
    for (int p = 0; p < 8; ++p) {
      uint32_t c;
      const uint32_t b = v.row(p, c);
      if (cvalid && r0 + p < R) *reinterpret_cast<uint32_t*>(q + (r0 + p) * ldq + col / 2) = c;
      // the word of the row's four blocks, from lanes 0, 4, 8 and 12 of the 16
      const uint32_t w = dpp_read<0x150>(b) | dpp_read<0x154>(b) << 8 | dpp_read<0x158>(b) << 16 | dpp_read<0x15C>(b) << 24;
      if (cc == 0 && r0 + p < R) s[tile.col * lds + r0 + p] = w;
    }
  }

  if constexpr (COLS) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      uint32_t b[2], c[2];
      v.columns(i, b, c);
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const int n = 8 * cc + 2 * i + k;
        *reinterpret_cast<uint32_t*>(codes + mx_stage(n, wid) + 4 * rg) = c[k];
        if (rg == 0) scales[4 * n + wid] = (uint8_t)b[k];
      }
    }
    __syncthreads();
    const int64_t rows32 = (R + 31) / 32;  // 32-row blocks of a column that exist
#pragma unroll
    for (int pass = 0; pass < 2; ++pass) {
      const int c = (t >> 2) + 64 * pass, unit = t & 3;
      if (tile.col * 128 + c < C && tile.row * 4 + unit < rows32)
        store_codes16(qt + (tile.col * 128 + c) * ldqt + (tile.row * 4 + unit) * 16,
                      *reinterpret_cast<const uint4*>(codes + mx_stage(c, unit)));
    }
    if (t < 128 && tile.col * 128 + t < C)
      st[tile.row * ldst + tile.col * 128 + t] = *reinterpret_cast<const uint32_t*>(scales + 4 * t);
  }
}

template <typename TIn>
static hipError_t launch_in(const void* x, int64_t R, int64_t C, int64_t ldx, uint8_t* q, int64_t ldq, uint32_t* s,
                            int64_t lds, uint8_t* qt, int64_t ldqt, uint32_t* st_, int64_t ldst, hipStream_t st) {
  const uint32_t ncg = (uint32_t)((C + 127) / 128);
  const dim3 grid((unsigned)((R + 127) / 128) * ncg);
  if (q && qt)
    hipLaunchKernelGGL((mx_quant_kernel<TIn, true, true>), grid, dim3(256), 0, st, (const TIn*)x, R, C, ldx, q, ldq, s,
                       lds, qt, ldqt, st_, ldst, ncg);
  else if (q)
    hipLaunchKernelGGL((mx_quant_kernel<TIn, true, false>), grid, dim3(256), 0, st, (const TIn*)x, R, C, ldx, q, ldq,
                       s, lds, qt, ldqt, st_, ldst, ncg);
  else
    hipLaunchKernelGGL((mx_quant_kernel<TIn, false, true>), grid, dim3(256), 0, st, (const TIn*)x, R, C, ldx, q, ldq,
                       s, lds, qt, ldqt, st_, ldst, ncg);
  return hipGetLastError();
}

hipError_t launch_mx_quant(const void* x, int xt, int64_t R, int64_t C, int64_t ldx, uint8_t* q, int64_t ldq,
                           uint32_t* s, int64_t lds, uint8_t* qt, int64_t ldqt, uint32_t* st_, int64_t ldst,
                           hipStream_t st) {
  return xt == 0 ? launch_in<uint16_t>(x, R, C, ldx, q, ldq, s, lds, qt, ldqt, st_, ldst, st)
                 : launch_in<float>(x, R, C, ldx, q, ldq, s, lds, qt, ldqt, st_, ldst, st);
}

}  // namespace fp8bq
