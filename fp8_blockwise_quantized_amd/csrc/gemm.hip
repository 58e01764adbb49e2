// Host launchers of the scaled FP8 GEMM (the kernel: gemm_kernel.hpp), the reduction of its split
// partial sums, and the byte transpose and zero fill that the products use.
#include "gemm_kernel.hpp"

namespace fp8bq {

// Sum of the split partial sums in split order, converted to the output type:
// out[m, n] = sum_s partial[s][m][n]  (OUTF32 == 2: out[m, n] += that sum, in FP32).
template <int OUTF32>
__global__ __launch_bounds__(256) void splitk_reduce_kernel(const float* __restrict__ partial, int nsplit, int64_t M,
                                                            int64_t N, void* __restrict__ out, int64_t ldo) {
  const int64_t total = M * (N / 4);
  for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < total; i += (int64_t)gridDim.x * blockDim.x) {
    const int64_t m = i / (N / 4), n = 4 * (i - m * (N / 4));
    v4f s = *reinterpret_cast<const v4f*>(partial + m * N + n);
    for (int k = 1; k < nsplit; ++k) s += *reinterpret_cast<const v4f*>(partial + ((int64_t)k * M + m) * N + n);
    if constexpr (OUTF32 == 2) {
      v4f* o = reinterpret_cast<v4f*>(reinterpret_cast<float*>(out) + m * ldo + n);
      *o = *o + s;
    } else if constexpr (OUTF32) {
      *reinterpret_cast<v4f*>(reinterpret_cast<float*>(out) + m * ldo + n) = s;
    } else {
      *reinterpret_cast<uint2*>(reinterpret_cast<uint16_t*>(out) + m * ldo + n) =
          make_uint2(pack_bf16x2(s[0], s[1]), pack_bf16x2(s[2], s[3]));
    }
  }
}

template <int OP, int BM, int BN, int WGM, int WGN, int NSTAGE, int SBM, int FA, int FB, int OUTF32>
static hipError_t launch_variant(const GemmDesc& d, const GemmPlan& p, float* partial, hipStream_t st) {
  hipLaunchKernelGGL((gemm_tn_kernel<OP, BM, BN, WGM, WGN, NSTAGE, SBM, FA, FB, OUTF32>), dim3((unsigned)p.grid),
                     dim3(WGM * WGN * 64), 0, st, d, (uint32_t)p.tiles_m, (uint32_t)p.tiles_n, p.split_k, partial,
                     GroupArgs<kGroupNone>{});
  return hipGetLastError();
}

template <int OP, int SBM, int FA, int FB, int OUTF32>
static hipError_t launch_fmt(const GemmDesc& d, const GemmPlan& p, float* partial, hipStream_t st) {
  switch (p.shape) {
    case k128x256: return launch_variant<OP, 128, 256, 2, 4, 2, SBM, FA, FB, OUTF32>(d, p, partial, st);
    case k256x128: return launch_variant<OP, 256, 128, 4, 2, 2, SBM, FA, FB, OUTF32>(d, p, partial, st);
    case k256x256: return launch_variant<OP, 256, 256, 2, 4, 2, SBM, FA, FB, OUTF32>(d, p, partial, st);
    case k64x64: return launch_variant<OP, 64, 64, 4, 1, 2, SBM, FA, FB, OUTF32>(d, p, partial, st);
    default: return launch_variant<OP, 128, 128, 2, 2, 2, SBM, FA, FB, OUTF32>(d, p, partial, st);
  }
}

template <int OP, int SBM, int OUTF32>
static hipError_t launch_formats(const GemmDesc& d, const GemmPlan& p, float* partial, hipStream_t st) {
  if (d.fa == kE4M3 && d.fb == kE4M3) return launch_fmt<OP, SBM, kE4M3, kE4M3, OUTF32>(d, p, partial, st);
  if (d.fa == kE5M2 && d.fb == kE4M3) return launch_fmt<OP, SBM, kE5M2, kE4M3, OUTF32>(d, p, partial, st);
  if (d.fa == kE4M3 && d.fb == kE5M2) return launch_fmt<OP, SBM, kE4M3, kE5M2, OUTF32>(d, p, partial, st);
  return launch_fmt<OP, SBM, kE5M2, kE5M2, OUTF32>(d, p, partial, st);
}

template <int OP, int SBM>
static hipError_t launch_out(const GemmDesc& d, const GemmPlan& p, float* partial, hipStream_t st) {
  if constexpr (OP == kOpWgrad) {
    if (d.out_f32 == 2) return launch_formats<OP, SBM, 2>(d, p, partial, st);
  }
  return d.out_f32 ? launch_formats<OP, SBM, 1>(d, p, partial, st) : launch_formats<OP, SBM, 0>(d, p, partial, st);
}

hipError_t launch_gemm(int op, const GemmDesc& d, const GemmPlan& p, void* ws, hipStream_t st) {
  float* partial = p.split_k > 1 ? reinterpret_cast<float*>(ws) : nullptr;
  hipError_t e;
  if (op == kOpFprop)
    e = launch_out<kOpFprop, kSbBlock128>(d, p, partial, st);
  else if (op == kOpDgrad)
    e = launch_out<kOpDgrad, kSbBlock128>(d, p, partial, st);
  else
    e = launch_out<kOpWgrad, kSbColumn>(d, p, partial, st);
  if (e != hipSuccess || p.split_k <= 1) return e;
  const int64_t total = d.M * (d.N / 4);
  int64_t blocks = (total + 255) / 256;
  if (blocks > 8192) blocks = 8192;
  if (d.out_f32 == 2)
    hipLaunchKernelGGL(splitk_reduce_kernel<2>, dim3((unsigned)blocks), dim3(256), 0, st, partial, p.split_k, d.M,
                       d.N, d.c, d.ldc);
  else if (d.out_f32)
    hipLaunchKernelGGL(splitk_reduce_kernel<1>, dim3((unsigned)blocks), dim3(256), 0, st, partial, p.split_k, d.M,
                       d.N, d.c, d.ldc);
  else
    hipLaunchKernelGGL(splitk_reduce_kernel<0>, dim3((unsigned)blocks), dim3(256), 0, st, partial, p.split_k, d.M,
                       d.N, d.c, d.ldc);
  return hipGetLastError();
}

// ---------------------------------------------------------------------------------------------
// Byte transpose, 128x128 tiles: each thread loads a 4-row x 16-byte patch, transposes 4x4 byte
// blocks with v_perm_b32, stages dwords (4 source rows of one column) in LDS, and writes 16-byte
// runs of the destination rows.
// ---------------------------------------------------------------------------------------------
constexpr int kTrStride = 33;

__device__ __forceinline__ void transpose4x4(uint32_t d0, uint32_t d1, uint32_t d2, uint32_t d3, uint32_t (&o)[4]) {
  // v_perm_b32(hi, lo, sel): byte i of the result is byte sel_i of the 8-byte value {hi, lo}.
  const uint32_t p01l = __builtin_amdgcn_perm(d1, d0, 0x05010400u);  // d0.b0 d1.b0 d0.b1 d1.b1
  const uint32_t p01h = __builtin_amdgcn_perm(d1, d0, 0x07030602u);  // d0.b2 d1.b2 d0.b3 d1.b3
  const uint32_t p23l = __builtin_amdgcn_perm(d3, d2, 0x05010400u);
  const uint32_t p23h = __builtin_amdgcn_perm(d3, d2, 0x07030602u);
  o[0] = __builtin_amdgcn_perm(p23l, p01l, 0x05040100u);  // d0.b0 d1.b0 d2.b0 d3.b0
  o[1] = __builtin_amdgcn_perm(p23l, p01l, 0x07060302u);
  o[2] = __builtin_amdgcn_perm(p23h, p01h, 0x05040100u);
  o[3] = __builtin_amdgcn_perm(p23h, p01h, 0x07060302u);
}

__global__ __launch_bounds__(256) void transpose_u8_kernel(const uint8_t* __restrict__ src, int64_t lds,
                                                           uint8_t* __restrict__ dst, int64_t ldd, uint32_t ncb) {
  __shared__ uint32_t tileT[128 * kTrStride];
  const int t = threadIdx.x;
  const TileRC tile = tile_of_block(ncb);
  const int64_t r0 = tile.row * 128, c0 = tile.col * 128;
  const int rq = t >> 3, cq = t & 7;
  uint4 d[4];
#pragma unroll
  for (int p = 0; p < 4; ++p) d[p] = *reinterpret_cast<const uint4*>(src + (r0 + 4 * rq + p) * lds + c0 + 16 * cq);
  const uint32_t* w0 = reinterpret_cast<const uint32_t*>(&d[0]);
  const uint32_t* w1 = reinterpret_cast<const uint32_t*>(&d[1]);
  const uint32_t* w2 = reinterpret_cast<const uint32_t*>(&d[2]);
  const uint32_t* w3 = reinterpret_cast<const uint32_t*>(&d[3]);
#pragma unroll
  for (int w = 0; w < 4; ++w) {
    uint32_t o[4];
    transpose4x4(w0[w], w1[w], w2[w], w3[w], o);
#pragma unroll
    for (int b = 0; b < 4; ++b) tileT[(16 * cq + 4 * w + b) * kTrStride + rq] = o[b];
  }
  __syncthreads();
#pragma unroll
  for (int pass = 0; pass < 4; ++pass) {
    const int id = t + 256 * pass, k = id >> 3, ch = id & 7;
    const uint32_t* s4 = tileT + k * kTrStride + 4 * ch;
    *reinterpret_cast<uint4*>(dst + (c0 + k) * ldd + r0 + 16 * ch) = make_uint4(s4[0], s4[1], s4[2], s4[3]);
  }
}

hipError_t launch_transpose_u8(const uint8_t* src, int64_t lds, uint8_t* dst, int64_t ldd, int64_t R, int64_t C,
                               hipStream_t st) {
  const uint32_t ncb = (uint32_t)(C / 128);
  hipLaunchKernelGGL(transpose_u8_kernel, dim3((unsigned)(R / 128) * ncb), dim3(256), 0, st, src, lds, dst, ldd, ncb);
  return hipGetLastError();
}

__global__ void zero_fill_kernel(uint8_t* dst, int64_t rows, int64_t row_bytes, int64_t ld_bytes) {
  const int64_t total = rows * row_bytes;
  for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < total; i += (int64_t)gridDim.x * blockDim.x) {
    const int64_t r = i / row_bytes, c = i - r * row_bytes;
    dst[r * ld_bytes + c] = 0;
  }
}

hipError_t launch_zero_fill(void* dst, int64_t rows, int64_t row_bytes, int64_t ld_bytes, hipStream_t st) {
  const int64_t total = rows * row_bytes;
  int64_t blocks = (total + 255) / 256;
  if (blocks > 4096) blocks = 4096;
  if (blocks < 1) blocks = 1;
  hipLaunchKernelGGL(zero_fill_kernel, dim3((unsigned)blocks), dim3(256), 0, st, (uint8_t*)dst, rows, row_bytes,
                     ld_bytes);
  return hipGetLastError();
}

}  // namespace fp8bq
