// 8-bit integer product for many rows: C[m, n] = sa[m] sb[n] sum_k A[m, k] B[n, k], tiles staged in LDS.
//
// Mathematics: the sum of products of 8-bit codes is exact in 32-bit integers for contractions below 2^17, so neither
// the tile's shape nor a split of the contraction changes it; it is rounded once to FP32 and once by each scale.
//
// Measured: 8192 x 8192 x 8192 2.44 POP/s (the library's plain 8-bit product without scales 2.35), 16384 x 11264 x 2048 331 us
// (2.28), 4099 x 5632 x 2048 56 us (1.69), 64 experts of 2816 x 2048 with 768 rows 66 us (the weights' 369 MB at 5.6
// TB/s).  Bound by the matrix pipes at the clock that the power allows (busy 73% of the cycles for 8192 x 8192 x 8192,
// 58% for 16384 x 11264 x 2048; the bare instruction runs at 3.45 POP/s on such data), and with short contractions by the output: without its stores 2048 long ones take 23% less,
// 8192 long ones 11%; without the loads 13 to 15% less.
#include "int8_common.hpp"
#include "row_gemm.hpp"

namespace fp8bq {

struct Int8Out {
  const float* sa;
  const float* sb;
  void* c;
  int64_t ldc;
  int past, vec;
  int32_t* partial;  // [split][M][ldp] sums of a split contraction
  int64_t ldp;
};

// OUT: 0 BF16, 1 FP32, 2 FP32 added to the output, kPartial the sums of a split contraction.
constexpr int kPartial = 3;
template <int BM, int BN, int WGM, int WGN, int NST, int OUT, bool GROUPED>
__global__ __launch_bounds__(WGM* WGN * 64, (RowTile<BM, BN, WGM * WGN, NST>::kMinWaves)) void int8_gemm_kernel(
    RowDesc d, Int8Out o, uint32_t tiles_m, uint32_t tiles_n, int nsplit, GroupArgs<kGroupRowsMode> grp) {
  using Tile = RowTile<BM, BN, WGM * WGN, NST>;
  constexpr int MI = BM / WGM / 32, NI = BN / WGN / 32;
  __shared__ __attribute__((aligned(1024))) uint8_t smem[Tile::kRing + (GROUPED ? kGroupTableBytes : 0)];
  // (a row of patches at a time: the whole tile in FP32 beside its sums took more registers than there are)
  auto end = [&](const v16i (&acc)[MI][NI], const RowPlace& p) {
    const bool full = o.vec && p.whole;
    if constexpr (OUT == kPartial) {
      float* w = reinterpret_cast<float*>(o.partial) + ((int64_t)p.split * d.M + p.m) * o.ldp + p.n;
#pragma unroll
      for (int i = 0; i < MI; ++i) {
        v16f y[1][NI];
#pragma unroll
        for (int j = 0; j < NI; ++j) y[0][j] = __builtin_bit_cast(v16f, acc[i][j]);
        store_tile_f32<false>(y, w + 32 * i * o.ldp, o.ldp, TileEdge{p.m + 32 * i, p.n, p.mlim, p.nlim, p.whole, true}, false,
                              false, p.lane);
        __builtin_amdgcn_sched_barrier(0);
      }
      return;
    }
    float sb[NI][16];
    const bool wide = p.whole && (p.n & 3) == 0;
#pragma unroll
    for (int j = 0; j < NI; ++j)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int64_t n = p.n + 32 * j + 16 * (r >> 1) + 4 * (r & 1);
        if (wide) {
          const v4f w = *reinterpret_cast<const v4f*>(o.sb + n);
#pragma unroll
          for (int k = 0; k < 4; ++k) sb[j][4 * r + k] = w[k];
        } else {
#pragma unroll
          for (int k = 0; k < 4; ++k) sb[j][4 * r + k] = o.sb[n + k < p.nlim ? n + k : p.nlim - 1];
        }
      }
#pragma unroll
    for (int i = 0; i < MI; ++i) {
      const int64_t m = p.m + 32 * i;
      const float sa = o.sa[m < p.mlim ? m : p.mlim - 1];
      v16f y[1][NI];
#pragma unroll
      for (int j = 0; j < NI; ++j)
#pragma unroll
        for (int r = 0; r < 16; ++r) y[0][j][r] = (float)acc[i][j][r] * sa * sb[j][r];
      const TileEdge at{m, p.n, p.mlim, p.nlim, full, o.vec != 0};
      if constexpr (OUT == 0)
        store_tile_bf16(y, reinterpret_cast<uint16_t*>(o.c) + m * o.ldc + p.n + p.ccol, o.ldc, at, o.past != 0, p.lane);
      else
        store_tile_f32<OUT == 2>(y, reinterpret_cast<float*>(o.c) + m * o.ldc + p.n + p.ccol, o.ldc, at, OUT == 2,
                                 o.past != 0, p.lane);
      __builtin_amdgcn_sched_barrier(0);
    }
  };
  row_gemm_units<kRowsI8, BM, BN, WGM, WGN, NST, GROUPED ? kUnitsGrouped : kUnitsFull>(d, tiles_m, tiles_n, nsplit, 1, &grp,
                                                                                  smem, end);
}

// Sum of the split partial sums, scaled and converted to the output type (or added to it); four columns a thread.
template <int OUT>
__global__ __launch_bounds__(256) void int8_reduce_kernel(Int8Out o, int nsplit, int64_t M, int64_t N) {
  const int64_t quads = o.ldp / 4, total = M * quads;
  for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < total; i += (int64_t)gridDim.x * blockDim.x) {
    const int64_t m = i / quads, n = 4 * (i - m * quads);
    v4i s = *reinterpret_cast<const v4i*>(o.partial + m * o.ldp + n);
    for (int k = 1; k < nsplit; ++k) s += *reinterpret_cast<const v4i*>(o.partial + ((int64_t)k * M + m) * o.ldp + n);
    float y[4];
#pragma unroll
    for (int r = 0; r < 4; ++r) y[r] = (float)s[r] * o.sa[m] * o.sb[n + r < N ? n + r : N - 1];
    if constexpr (OUT == 0) {
      uint16_t* c = reinterpret_cast<uint16_t*>(o.c) + m * o.ldc + n;
      const uint32_t lo = pack_bf16x2(y[0], y[1]), hi = pack_bf16x2(y[2], y[3]);
      if (n + 4 <= N && ((uintptr_t)c & 7) == 0) {
        *reinterpret_cast<uint2*>(c) = make_uint2(lo, hi);
      } else {
        const uint16_t e[4] = {(uint16_t)lo, (uint16_t)(lo >> 16), (uint16_t)hi, (uint16_t)(hi >> 16)};
#pragma unroll
        for (int r = 0; r < 4; ++r)
          if (n + r < N) c[r] = e[r];
      }
    } else {
      float* c = reinterpret_cast<float*>(o.c) + m * o.ldc + n;
#pragma unroll
      for (int r = 0; r < 4; ++r)
        if (n + r < N) c[r] = OUT == 2 ? c[r] + y[r] : y[r];
    }
  }
}

template <int BM, int BN, int WGM, int WGN, int NST, int OUT>
static hipError_t launch_tile(const RowDesc& r, const Int8Out& o, const MxGroups& grp, const MxPlan& p, hipStream_t st) {
  const dim3 grid((unsigned)p.grid), block(WGM * WGN * 64);
  const GroupArgs<kGroupRowsMode> none{nullptr, 0, 0};
  if constexpr (OUT < 2) {  // (a grouped product is not added to the output, nor split)
    if (grp.offsets) {
      hipLaunchKernelGGL((int8_gemm_kernel<BM, BN, WGM, WGN, NST, OUT, true>), grid, block, 0, st, r, o, (uint32_t)p.tiles_m,
                         (uint32_t)p.tiles_n, 1, GroupArgs<kGroupRowsMode>{grp.offsets, grp.experts, r.M});
      return hipGetLastError();
    }
  }
  hipLaunchKernelGGL((int8_gemm_kernel<BM, BN, WGM, WGN, NST, OUT, false>), grid, block, 0, st, r, o, (uint32_t)p.tiles_m,
                     (uint32_t)p.tiles_n, p.split_k, none);
  return hipGetLastError();
}

template <int OUT>
static hipError_t launch_out(const Int8Desc& d, const MxGroups& grp, const MxPlan& p, void* ws, hipStream_t st) {
  RowDesc r{};
  r.a = (const uint8_t*)d.a;
  r.lda = d.lda;
  r.b = d.b;
  r.ldb = d.ldb;
  r.M = d.M;
  r.N = d.N;
  r.K = d.K;
  const Int8Out o{d.sa, d.sb, d.c, d.ldc, d.past, (d.ldc * (OUT == 0 ? 2 : 4)) % 16 == 0, (int32_t*)ws, (d.N + 3) / 4 * 4};
  switch (p.shape) {
    case k256x256: return launch_tile<256, 256, 2, 4, 2, OUT>(r, o, grp, p, st);
    case k256x192: return launch_tile<256, 192, 4, 2, 2, OUT>(r, o, grp, p, st);
    case k64x64:
      return p.deep ? launch_tile<64, 64, 2, 2, 3, OUT>(r, o, grp, p, st) : launch_tile<64, 64, 2, 2, 2, OUT>(r, o, grp, p, st);
    default: return launch_tile<128, 128, 2, 2, 2, OUT>(r, o, grp, p, st);
  }
}

template <int OUT>
static hipError_t launch_split(const Int8Desc& d, const MxPlan& p, void* ws, hipStream_t st) {
  const hipError_t e = launch_out<kPartial>(d, MxGroups{nullptr, 0}, p, ws, st);
  if (e != hipSuccess) return e;
  const Int8Out o{d.sa, d.sb, d.c, d.ldc, 0, 0, (int32_t*)ws, (d.N + 3) / 4 * 4};
  int64_t blocks = (d.M * (o.ldp / 4) + 255) / 256;
  blocks = blocks < 8192 ? blocks : 8192;
  hipLaunchKernelGGL((int8_reduce_kernel<OUT>), dim3((unsigned)blocks), dim3(256), 0, st, o, p.split_k, d.M, d.N);
  return hipGetLastError();
}

hipError_t launch_int8_gemm(const Int8Desc& d, const MxGroups& grp, const MxPlan& p, void* ws, hipStream_t st) {
  if (p.split_k > 1)
    return d.out_t == 0 ? launch_split<0>(d, p, ws, st) : d.out_t == 1 ? launch_split<1>(d, p, ws, st) : launch_split<2>(d, p, ws, st);
  if (d.out_t == 0) return launch_out<0>(d, grp, p, ws, st);
  return d.out_t == 1 ? launch_out<1>(d, grp, p, ws, st) : launch_out<2>(d, grp, p, ws, st);
}

}  // namespace fp8bq
