// The experts' rows: tokens' choices sorted by expert, rows of x brought into that order, the experts' rows added up per
// token with their weights, and the gradients of both.
//
// All of it moves bytes; nothing here has arithmetic to speak of.  Every sum runs in a fixed order (a token's choices
// in theirs, a dot product over the threads in theirs), so results do not change from call to call.
//
// Measured, 16384 tokens of 2048 BF16 values with two choices each on 64 experts (us): sort 5 + 9, gather 41 (201 MB, 4.9 TB/s),
// combine 40 to 48 (as much), its backward 55 (328 MB, 6.0 TB/s; a streaming copy does 6.1).  Five tokens with six
// choices: 2.8, 2.7 and 4.0, a launch and its latency.  A workgroup takes a token (or a row of the output), so that its
// choices' rows are read and summed in registers and written once.
#include "group_table.hpp"
#include "launch.hpp"
#include "quant_common.hpp"

namespace fp8bq {

// Sort.  n choices in chunks of whole 64s, one workgroup a chunk, a wave a piece of it.  First kernel: a chunk's counts
// (left out when there is one chunk).  Second: each workgroup adds up the counts of all chunks and of those before
// its own, counts its waves' pieces, and each wave walks its piece once more, 64 choices at a time: the lanes with the
// same expert find each other with one ballot for each bit of the index, and a lane's row is the expert's next free
// one plus the lanes before it.  The order within an expert is that of the choices.
constexpr int kSortThreads = 1024, kSortWaves = kSortThreads / 64;

int expert_rows_chunks(int64_t n) {
  const int64_t c = (n + 2047) / 2048;
  return (int)(c < 1 ? 1 : c > 64 ? 64 : c);
}
static int64_t chunk_length(int64_t n) {
  const int64_t c = expert_rows_chunks(n);
  return ((n + c - 1) / c + 63) / 64 * 64;
}

__device__ __forceinline__ int choice_at(const int32_t* experts, int64_t i, int64_t end, int E) {
  const int e = i < end ? experts[i] : -1;
  return e >= 0 && e < E ? e : -1;
}

__global__ __launch_bounds__(kSortThreads) void expert_counts_kernel(const int32_t* __restrict__ experts, int64_t n, int E,
                                                                     int64_t len, uint32_t* __restrict__ counts) {
  __shared__ uint32_t have[kMaxExperts];
  for (int e = threadIdx.x; e < E; e += kSortThreads) have[e] = 0;
  __syncthreads();
  const int64_t begin = (int64_t)blockIdx.x * len, end = begin + len < n ? begin + len : n;
  for (int64_t i = begin + threadIdx.x; i < end; i += kSortThreads) {
    const int e = choice_at(experts, i, end, E);
    if (e >= 0) atomicAdd(&have[e], 1u);
  }
  __syncthreads();
  for (int e = threadIdx.x; e < E; e += kSortThreads) counts[(int64_t)blockIdx.x * E + e] = have[e];
}

__global__ __launch_bounds__(kSortThreads) void expert_rows_kernel(const int32_t* __restrict__ experts, int64_t n, int E,
                                                                   int64_t len, const uint32_t* __restrict__ counts,
                                                                   int64_t* __restrict__ offsets, int32_t* __restrict__ rows,
                                                                   int32_t* __restrict__ slots) {
  __shared__ uint32_t next[kSortWaves][kMaxExperts];  // counts of each wave's piece, then its next rows
  __shared__ uint32_t sums[kSortWaves], total;
  const int t = threadIdx.x, lane = t & 63, wid = t >> 6;
  const int64_t begin = (int64_t)blockIdx.x * len, end = begin + len < n ? begin + len : n;
  const int64_t piece = (len / 64 + kSortWaves - 1) / kSortWaves * 64;
  const int64_t p0 = begin + wid * piece < end ? begin + wid * piece : end;
  const int64_t p1 = p0 + piece < end ? p0 + piece : end;
  for (int i = t; i < kSortWaves * kMaxExperts; i += kSortThreads) next[i / kMaxExperts][i % kMaxExperts] = 0;
  __syncthreads();
  for (int64_t i = p0 + lane; i < p1; i += 64) {
    const int e = choice_at(experts, i, p1, E);
    if (e >= 0) atomicAdd(&next[wid][e], 1u);
  }
  __syncthreads();
  // thread e: all choices of expert e, and those of the chunks before this one
  uint32_t all = 0, before = 0;
  if (t < E) {
    if (counts) {
      for (int b = 0; b < (int)gridDim.x; ++b) {
        const uint32_t c = counts[(int64_t)b * E + t];
        all += c;
        before += b < (int)blockIdx.x ? c : 0;
      }
    } else {
      for (int w = 0; w < kSortWaves; ++w) all += next[w][t];
    }
  }
  const uint32_t upto = wave_scan_add(all);
  if (lane == 63) sums[wid] = upto;
  __syncthreads();
  uint32_t at = upto - all;
  for (int w = 0; w < wid; ++w) at += sums[w];
  if (t < E) {
    if (blockIdx.x == 0) {
      offsets[t] = at;
      if (t == E - 1) offsets[E] = at + all;
    }
    if (t == E - 1) total = at + all;
    uint32_t row = at + before;
    for (int w = 0; w < kSortWaves; ++w) {
      const uint32_t c = next[w][t];
      next[w][t] = row;
      row += c;
    }
  }
  __syncthreads();
  const int bits = 32 - __builtin_clz((unsigned)E);
  for (int64_t i0 = p0; i0 < p1; i0 += 64) {
    const int64_t i = i0 + lane;
    const int e = choice_at(experts, i, p1, E);
    uint64_t same = __ballot(e >= 0);
    for (int b = 0; b < bits; ++b) {
      const uint64_t set = __ballot((e >> b) & 1);
      same &= (e >> b) & 1 ? set : ~set;
    }
    if (e >= 0) {
      const uint32_t ahead = (uint32_t)__popcll(same & (((uint64_t)1 << lane) - 1));
      const uint32_t row = next[wid][e] + ahead;
      rows[i] = (int32_t)row;
      slots[row] = (int32_t)i;
      // (the wave's reads above are done before the last of the lanes writes: LDS serves a wave in order)
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
      if ((same >> lane) == 1) next[wid][e] = row + 1;
    } else if (i < p1) {
      rows[i] = -1;
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
  }
  // rows that no choice has
  for (int64_t r = (int64_t)total + (int64_t)blockIdx.x * kSortThreads + t; r < n; r += (int64_t)gridDim.x * kSortThreads)
    slots[r] = -1;
}

hipError_t launch_expert_rows(const int32_t* experts, int64_t n, int E, int64_t* offsets, int32_t* rows, int32_t* slots,
                              void* ws, hipStream_t st) {
  const int chunks = expert_rows_chunks(n);
  const int64_t len = chunk_length(n);
  uint32_t* counts = chunks > 1 ? (uint32_t*)ws : nullptr;
  if (counts) {
    hipLaunchKernelGGL(expert_counts_kernel, dim3((unsigned)chunks), dim3(kSortThreads), 0, st, experts, n, E, len, counts);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  hipLaunchKernelGGL(expert_rows_kernel, dim3((unsigned)chunks), dim3(kSortThreads), 0, st, experts, n, E, len, counts,
                     offsets, rows, slots);
  return hipGetLastError();
}

constexpr int kMoveThreads = 256;

// A row of the output: the token's row, or zeros where no choice has the row.  16 bytes a thread.
__global__ __launch_bounds__(kMoveThreads) void gather_rows_kernel(const uint8_t* __restrict__ x, int64_t T, int64_t chunks,
                                                                   int64_t ldx, const int32_t* __restrict__ slots, int k,
                                                                   int64_t n, uint8_t* __restrict__ out, int64_t ldo) {
  for (int64_t r = blockIdx.x; r < n; r += gridDim.x) {
    const int32_t s = slots[r];
    const int64_t token = s / k;
    const bool live = s >= 0 && token < T;
    const uint8_t* from = x + token * ldx;
    uint8_t* to = out + r * ldo;
    for (int64_t c = threadIdx.x; c < chunks; c += kMoveThreads) {
      u32x4 w = {0, 0, 0, 0};
      if (live) w = *reinterpret_cast<const u32x4*>(from + 16 * c);
      *reinterpret_cast<u32x4*>(to + 16 * c) = w;
    }
  }
}

template <typename TOut>
__device__ __forceinline__ void store8(TOut* p, const float (&v)[8]) {
  if constexpr (sizeof(TOut) == 2) {
    *reinterpret_cast<u32x4*>(p) = (u32x4){pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]),
                                           pack_bf16x2(v[6], v[7])};
  } else {
    *reinterpret_cast<f32x4*>(p) = (f32x4){v[0], v[1], v[2], v[3]};
    *(reinterpret_cast<f32x4*>(p) + 1) = (f32x4){v[4], v[5], v[6], v[7]};
  }
}

// out[t] = sum_j w[t, j] y[rows[t, j]], FP32, in the order of j; choices without a row add nothing.
template <typename TY, typename TOut>
__global__ __launch_bounds__(kMoveThreads) void combine_rows_kernel(const TY* __restrict__ y, int64_t T, int k, int64_t n,
                                                                    int64_t H, int64_t ldy, const int32_t* __restrict__ rows,
                                                                    const float* __restrict__ weights,
                                                                    TOut* __restrict__ out, int64_t ldo) {
  for (int64_t t = blockIdx.x; t < T; t += gridDim.x) {
    for (int64_t c = 8 * (int64_t)threadIdx.x; c < H; c += 8 * kMoveThreads) {
      float sum[8] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 4
      for (int j = 0; j < k; ++j) {
        const int32_t r = rows[t * k + j];
        if (r < 0 || r >= n) continue;
        const float w = weights ? weights[t * k + j] : 1.0f;
        float v[8];
        Load8<TY>::run(y + r * ldy + c, v);
#pragma unroll
        for (int i = 0; i < 8; ++i) sum[i] = __builtin_fmaf(w, v[i], sum[i]);
      }
      store8(out + t * ldo + c, sum);
    }
  }
}

// dy[rows[t, j]] = w[t, j] dout[t] and dw[t, j] = sum_h dout[t, h] y[rows[t, j], h]; zeros for choices without a row and
// rows without a choice (of the k rows t k .. t k + k - 1 each workgroup clears those).
template <typename TD, typename TY>
__global__ __launch_bounds__(kMoveThreads) void combine_rows_backward_kernel(
    const TD* __restrict__ dout, int64_t lddo, const TY* __restrict__ y, int64_t ldy, int64_t T, int k, int64_t n, int64_t H,
    const int32_t* __restrict__ rows, const float* __restrict__ weights, const int32_t* __restrict__ slots,
    TY* __restrict__ dy, int64_t lddy, float* __restrict__ dweights) {
  __shared__ float part[kMoveThreads / 64];
  const int tid = threadIdx.x, lane = tid & 63, wid = tid >> 6;
  for (int64_t t = blockIdx.x; t < T; t += gridDim.x) {
    for (int j = 0; j < k; ++j) {
      const int32_t r = rows[t * k + j];
      const bool live = r >= 0 && r < n;
      const float w = weights[t * k + j];
      float dot = 0.0f;
      if (live) {
        for (int64_t c = 8 * (int64_t)tid; c < H; c += 8 * kMoveThreads) {
          float d[8], v[8];
          Load8<TD>::run(dout + t * lddo + c, d);
          Load8<TY>::run(y + r * ldy + c, v);
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            dot = __builtin_fmaf(d[i], v[i], dot);
            v[i] = w * d[i];
          }
          store8(dy + r * lddy + c, v);
        }
      }
#pragma unroll
      for (int s = 1; s < 64; s <<= 1) dot += __shfl_xor(dot, s);
      if (lane == 0) part[wid] = dot;
      __syncthreads();
      if (tid == 0) {
        float sum = part[0];
        for (int i = 1; i < kMoveThreads / 64; ++i) sum += part[i];
        dweights[t * k + j] = sum;
      }
      __syncthreads();
      if (slots[t * k + j] < 0) {
        const float zero[8] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
        for (int64_t c = 8 * (int64_t)tid; c < H; c += 8 * kMoveThreads) store8(dy + (t * k + j) * lddy + c, zero);
      }
    }
  }
}

static dim3 row_grid(int64_t n) { return dim3((unsigned)(n < ((int64_t)1 << 20) ? n : (int64_t)1 << 20)); }

hipError_t launch_gather_rows(const void* x, int xt, int64_t T, int64_t H, int64_t ldx, const int32_t* slots, int64_t k,
                              void* out, int64_t ldo, hipStream_t st) {
  const int64_t es = xt == 0 ? 2 : 4;
  hipLaunchKernelGGL(gather_rows_kernel, row_grid(T * k), dim3(kMoveThreads), 0, st, (const uint8_t*)x, T, H * es / 16,
                     ldx * es, slots, (int)k, T * k, (uint8_t*)out, ldo * es);
  return hipGetLastError();
}

template <typename TY, typename TOut>
static hipError_t launch_combine(const void* y, int64_t T, int64_t k, int64_t H, int64_t ldy, const int32_t* rows,
                                 const float* weights, void* out, int64_t ldo, hipStream_t st) {
  hipLaunchKernelGGL((combine_rows_kernel<TY, TOut>), row_grid(T), dim3(kMoveThreads), 0, st, (const TY*)y, T, (int)k, T * k,
                     H, ldy, rows, weights, (TOut*)out, ldo);
  return hipGetLastError();
}

hipError_t launch_combine_rows(const void* y, int yt, int64_t T, int64_t k, int64_t H, int64_t ldy, const int32_t* rows,
                               const float* weights, void* out, int ot, int64_t ldo, hipStream_t st) {
  if (yt == 0)
    return ot == 0 ? launch_combine<uint16_t, uint16_t>(y, T, k, H, ldy, rows, weights, out, ldo, st)
                   : launch_combine<uint16_t, float>(y, T, k, H, ldy, rows, weights, out, ldo, st);
  return ot == 0 ? launch_combine<float, uint16_t>(y, T, k, H, ldy, rows, weights, out, ldo, st)
                 : launch_combine<float, float>(y, T, k, H, ldy, rows, weights, out, ldo, st);
}

template <typename TD, typename TY>
static hipError_t launch_backward(const void* dout, int64_t lddo, const void* y, int64_t ldy, int64_t T, int64_t k, int64_t H,
                                  const int32_t* rows, const float* weights, const int32_t* slots, void* dy, int64_t lddy,
                                  float* dweights, hipStream_t st) {
  hipLaunchKernelGGL((combine_rows_backward_kernel<TD, TY>), row_grid(T), dim3(kMoveThreads), 0, st, (const TD*)dout, lddo,
                     (const TY*)y, ldy, T, (int)k, T * k, H, rows, weights, slots, (TY*)dy, lddy, dweights);
  return hipGetLastError();
}

hipError_t launch_combine_rows_backward(const void* dout, int dt, int64_t lddo, const void* y, int yt, int64_t ldy, int64_t T,
                                        int64_t k, int64_t H, const int32_t* rows, const float* weights,
                                        const int32_t* slots, void* dy, int64_t lddy, float* dweights, hipStream_t st) {
  if (dt == 0)
    return yt == 0 ? launch_backward<uint16_t, uint16_t>(dout, lddo, y, ldy, T, k, H, rows, weights, slots, dy, lddy, dweights, st)
                   : launch_backward<uint16_t, float>(dout, lddo, y, ldy, T, k, H, rows, weights, slots, dy, lddy, dweights, st);
  return yt == 0 ? launch_backward<float, uint16_t>(dout, lddo, y, ldy, T, k, H, rows, weights, slots, dy, lddy, dweights, st)
                 : launch_backward<float, float>(dout, lddo, y, ldy, T, k, H, rows, weights, slots, dy, lddy, dweights, st);
}

}  // namespace fp8bq
