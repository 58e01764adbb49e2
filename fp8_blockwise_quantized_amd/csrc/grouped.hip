// Host launchers of the FP8 products grouped by expert.  The kernel is the dense product's
// (gemm_kernel.hpp) with work units that are tiles of one expert; see GroupMode there.
#include "gemm_kernel.hpp"

namespace fp8bq {

template <int GM>
static GroupArgs<GM> group_args(const GroupDesc& g, const GemmPlan& p) {
  if constexpr (GM == kGroupContract)
    return GroupArgs<GM>{g.offsets, g.experts, g.tokens, p.group_split, (uint32_t*)g.ws};
  else
    return GroupArgs<GM>{g.offsets, g.experts, g.tokens};
}

static float* partial_of(const GroupDesc& g) {
  return g.ws ? reinterpret_cast<float*>((uint8_t*)g.ws + kSplitListBytes) : nullptr;
}

template <int OP, int BM, int BN, int WGM, int WGN, int SBM, int FA, int FB, int OUTF32, int GM>
static hipError_t launch_tile(const GemmDesc& d, const GroupDesc& g, const GemmPlan& p, hipStream_t st) {
  hipLaunchKernelGGL((gemm_tn_kernel<OP, BM, BN, WGM, WGN, 2, SBM, FA, FB, OUTF32, GM>), dim3((unsigned)p.grid),
                     dim3(WGM * WGN * 64), 0, st, d, (uint32_t)p.tiles_m, (uint32_t)p.tiles_n, 1, partial_of(g),
                     group_args<GM>(g, p));
  return hipGetLastError();
}

template <int OP, int SBM, int FA, int FB, int OUTF32, int GM>
static hipError_t launch_shape(const GemmDesc& d, const GroupDesc& g, const GemmPlan& p, hipStream_t st) {
  switch (p.shape) {
    case k256x256:
      if constexpr (GM == kGroupContract) {
        return launch_tile<OP, 256, 256, 2, 4, SBM, FA, FB, OUTF32, GM>(d, g, p, st);
      } else {
        hipLaunchKernelGGL((gemm_tn_grouped_kernel<OP, SBM, FA, FB, OUTF32, GM>), dim3((unsigned)p.grid), dim3(512), 0,
                           st, d, (uint32_t)p.tiles_n, group_args<GM>(g, p));
        return hipGetLastError();
      }
    case k64x64: return launch_tile<OP, 64, 64, 4, 1, SBM, FA, FB, OUTF32, GM>(d, g, p, st);
    default: return launch_tile<OP, 128, 128, 2, 2, SBM, FA, FB, OUTF32, GM>(d, g, p, st);
  }
}

// The outputs of the experts whose contraction was split: the sum of their chunks' partial sums [M, N] in an order that
// the number of chunks fixes (OUTF32 == 2: added to the output).  A thread adds four values of one to three
// chunks; with more chunks the workgroup's four waves take every fourth chunk each and add up in LDS.  Bound by
// memory, and by its latency for small outputs: 4 bytes read for every chunk and value.
template <int OUTF32>
__global__ __launch_bounds__(256) void grouped_sum_kernel(const uint32_t* __restrict__ list, const float* __restrict__ partial,
                                                          int64_t M, int64_t N, void* __restrict__ out, int64_t ldo) {
  __shared__ v4f other[4][64];
  const int n = (int)list[0];
  const int64_t total = M * (N / 4);
  const int wave = (int)threadIdx.x >> 6, lane = (int)threadIdx.x & 63;
  int64_t before = 0;  // workgroups' shares of the experts so far: the next expert's begin where these end
  for (int i = 0; i < n; ++i) {
    const GroupEntry e = entry_of(list[1 + i]);
    const bool waves = e.chunks >= 4;
    const int64_t per = waves ? 64 : 256, shares = (total + per - 1) / per;
    const int64_t G = gridDim.x, first = (blockIdx.x + G - before % G) % G;
    before += shares;
    for (int64_t g = first; g < shares; g += G) {
      const int64_t v = g * per + (waves ? lane : (int)threadIdx.x);
      const bool in = v < total;
      v4f s = {0.0f, 0.0f, 0.0f, 0.0f};
      if (in) {
        const v4f* p = reinterpret_cast<const v4f*>(partial) + e.set * total + v;
        if (waves) {
          s = p[wave * total];
#pragma unroll 4
          for (int k = wave + 4; k < e.chunks; k += 4) s += p[k * total];
        } else {
          s = p[0] + p[total];
          if (e.chunks == 3) s += p[2 * total];
        }
      }
      if (waves) {
        __syncthreads();
        other[wave][lane] = s;
        __syncthreads();
        if (wave != 0) continue;
        s = (s + other[1][lane]) + (other[2][lane] + other[3][lane]);
      }
      if (!in) continue;
      const int64_t m = v / (N / 4), c = 4 * (v - m * (N / 4));
      const int64_t at = (e.expert * M + m) * ldo + c;
      if constexpr (OUTF32 == 2) {
        v4f* o = reinterpret_cast<v4f*>(reinterpret_cast<float*>(out) + at);
        *o = *o + s;
      } else if constexpr (OUTF32) {
        *reinterpret_cast<v4f*>(reinterpret_cast<float*>(out) + at) = s;
      } else {
        *reinterpret_cast<uint2*>(reinterpret_cast<uint16_t*>(out) + at) =
            make_uint2(pack_bf16x2(s[0], s[1]), pack_bf16x2(s[2], s[3]));
      }
    }
  }
}

template <int OP, int SBM, int OUTF32, int GM>
static hipError_t launch_formats(const GemmDesc& d, const GroupDesc& g, const GemmPlan& p, hipStream_t st) {
  if (d.fa == kE4M3 && d.fb == kE4M3) return launch_shape<OP, SBM, kE4M3, kE4M3, OUTF32, GM>(d, g, p, st);
  if (d.fa == kE5M2 && d.fb == kE4M3) return launch_shape<OP, SBM, kE5M2, kE4M3, OUTF32, GM>(d, g, p, st);
  if (d.fa == kE4M3 && d.fb == kE5M2) return launch_shape<OP, SBM, kE4M3, kE5M2, OUTF32, GM>(d, g, p, st);
  return launch_shape<OP, SBM, kE5M2, kE5M2, OUTF32, GM>(d, g, p, st);
}

template <int OP, int SBM, int GM>
static hipError_t launch_out(const GemmDesc& d, const GroupDesc& g, const GemmPlan& p, hipStream_t st) {
  if constexpr (OP == kOpWgrad) {
    if (d.out_f32 == 2) return launch_formats<OP, SBM, 2, GM>(d, g, p, st);
  }
  return d.out_f32 ? launch_formats<OP, SBM, 1, GM>(d, g, p, st) : launch_formats<OP, SBM, 0, GM>(d, g, p, st);
}

hipError_t launch_grouped_gemm(int op, const GemmDesc& d, const GroupDesc& g, const GemmPlan& p, hipStream_t st) {
  if (op == kOpFprop) return launch_out<kOpFprop, kSbBlock128, kGroupRowsMode>(d, g, p, st);
  if (op == kOpDgrad) return launch_out<kOpDgrad, kSbBlock128, kGroupWindow>(d, g, p, st);
  hipError_t e = launch_out<kOpWgrad, kSbColumn, kGroupContract>(d, g, p, st);
  if (e != hipSuccess || p.group_split.sets == 0) return e;
  const uint32_t* list = (const uint32_t*)g.ws;
  const float* partial = partial_of(g);
  int64_t blocks = (d.M * (d.N / 4) + 63) / 64;  // (one expert's shares)
  if (blocks > 1024) blocks = 1024;
  if (d.out_f32 == 2)
    hipLaunchKernelGGL(grouped_sum_kernel<2>, dim3((unsigned)blocks), dim3(256), 0, st, list, partial, d.M,
                       d.N, d.c, d.ldc);
  else if (d.out_f32)
    hipLaunchKernelGGL(grouped_sum_kernel<1>, dim3((unsigned)blocks), dim3(256), 0, st, list, partial, d.M,
                       d.N, d.c, d.ldc);
  else
    hipLaunchKernelGGL(grouped_sum_kernel<0>, dim3((unsigned)blocks), dim3(256), 0, st, list, partial, d.M,
                       d.N, d.c, d.ldc);
  return hipGetLastError();
}

}  // namespace fp8bq
