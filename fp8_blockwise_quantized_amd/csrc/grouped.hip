// Host launchers of the FP8 products grouped by expert.  The kernel is the dense product's
// (gemm_kernel.hpp) with work units that are tiles of one expert; see GroupMode there.
#include "gemm_kernel.hpp"

namespace fp8bq {

template <int OP, int BM, int BN, int WGM, int WGN, int SBM, int FA, int FB, int OUTF32, int GM>
static hipError_t launch_tile(const GemmDesc& d, const GroupDesc& g, const GemmPlan& p, hipStream_t st) {
  hipLaunchKernelGGL((gemm_tn_kernel<OP, BM, BN, WGM, WGN, 2, SBM, FA, FB, OUTF32, GM>), dim3((unsigned)p.grid),
                     dim3(WGM * WGN * 64), 0, st, d, (uint32_t)p.tiles_m, (uint32_t)p.tiles_n, 1, (float*)nullptr,
                     GroupArgs<GM>{g.offsets, g.experts, g.tokens});
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
                           st, d, (uint32_t)p.tiles_n, GroupArgs<GM>{g.offsets, g.experts, g.tokens});
        return hipGetLastError();
      }
    case k64x64: return launch_tile<OP, 64, 64, 4, 1, SBM, FA, FB, OUTF32, GM>(d, g, p, st);
    default: return launch_tile<OP, 128, 128, 2, 2, SBM, FA, FB, OUTF32, GM>(d, g, p, st);
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
  return launch_out<kOpWgrad, kSbColumn, kGroupContract>(d, g, p, st);
}

}  // namespace fp8bq
