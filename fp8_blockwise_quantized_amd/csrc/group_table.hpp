// Per-expert tables of the products grouped by expert (device side).
//
// offsets[0..E] (int64, on the device) hold where each expert's tokens begin; the tokens of expert e
// are offsets[e] .. offsets[e+1]-1.  The values come from a router on the device, so a kernel makes them
// safe itself: each is clamped to [0, T] and to at least the one before it, whatever the buffer holds.
// One wave builds the tables in LDS: lane l owns experts 8l .. 8l+7 and two wave scans (a maximum for
// the clamped offsets, a sum for the counts) join the lanes; about a microsecond, most of it the load.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace fp8bq {

constexpr int kMaxExperts = 512;
constexpr int kExpertsPerLane = kMaxExperts / 64;
constexpr int kGroupTableBytes = (2 * (kMaxExperts + 1) * 4 + 15) / 16 * 16;  // unit counts and starts

// Inclusive wave scans by DPP: four shifts within the rows of 16 lanes, then each row's last lane into the
// next row and lane 31 into the upper half.  Lanes without a source take 0, the identity of both operations.
template <int CTRL, int ROWS>
__device__ __forceinline__ uint32_t scan_source(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, ROWS, 0xF, false);
}
__device__ __forceinline__ uint32_t wave_scan_add(uint32_t v) {
  v += scan_source<0x111, 0xF>(v);
  v += scan_source<0x112, 0xF>(v);
  v += scan_source<0x114, 0xF>(v);
  v += scan_source<0x118, 0xF>(v);
  v += scan_source<0x142, 0xA>(v);
  v += scan_source<0x143, 0xC>(v);
  return v;
}
__device__ __forceinline__ int wave_scan_max(int v) {  // v >= 0
  const auto up = [&](uint32_t o) { v = (int)o > v ? (int)o : v; };
  up(scan_source<0x111, 0xF>(v));
  up(scan_source<0x112, 0xF>(v));
  up(scan_source<0x114, 0xF>(v));
  up(scan_source<0x118, 0xF>(v));
  up(scan_source<0x142, 0xA>(v));
  up(scan_source<0x143, 0xC>(v));
  return v;
}

// The lane's safe offsets o[i] = offset of expert 8*lane + i, i = 0 .. 8 (T < 2^31); experts past E
// are empty.
__device__ __forceinline__ void group_offsets(const int64_t* offsets, int E, int64_t T, int lane,
                                              int (&o)[kExpertsPerLane + 1]) {
#pragma unroll
  for (int i = 0; i <= kExpertsPerLane; ++i) {
    const int j = kExpertsPerLane * lane + i;
    const int64_t v = offsets[j < E ? j : E];
    o[i] = (int)(v < 0 ? 0 : (v > T ? T : v));
  }
#pragma unroll
  for (int i = 1; i <= kExpertsPerLane; ++i) o[i] = o[i] > o[i - 1] ? o[i] : o[i - 1];
  const int upto = wave_scan_max(o[kExpertsPerLane]);
  int before = __shfl_up(upto, 1);
  before = lane == 0 ? 0 : before;
#pragma unroll
  for (int i = 0; i <= kExpertsPerLane; ++i) o[i] = o[i] > before ? o[i] : before;
}

// Exclusive sums of the lane's counts c[i] over all experts, written to pre[0 .. E] (pre[E] = total).
__device__ __forceinline__ void group_sums(const uint32_t (&c)[kExpertsPerLane], int E, int lane, uint32_t* pre) {
  uint32_t mine = 0;
#pragma unroll
  for (int i = 0; i < kExpertsPerLane; ++i) mine += c[i];
  uint32_t at = wave_scan_add(mine) - mine;
#pragma unroll
  for (int i = 0; i < kExpertsPerLane; ++i) {
    const int j = kExpertsPerLane * lane + i;
    if (j <= E) pre[j] = at;
    at += c[i];
  }
  if (lane == 63 && E == kMaxExperts) pre[E] = at;
}

// starts[e] = first token of expert e, units[e] = tiles of the experts before e, of tile_rows tokens by
// tiles_n columns of tiles.
__device__ __forceinline__ void group_table_rows(const int64_t* offsets, int E, int64_t T, int tile_rows,
                                                 uint32_t tiles_n, int* starts, uint32_t* units, int lane) {
  int o[kExpertsPerLane + 1];
  group_offsets(offsets, E, T, lane, o);
  uint32_t c[kExpertsPerLane];
#pragma unroll
  for (int i = 0; i < kExpertsPerLane; ++i) {
    const int j = kExpertsPerLane * lane + i;
    if (j <= E) starts[j] = o[i];
    c[i] = (uint32_t)((o[i + 1] - o[i] + tile_rows - 1) / tile_rows) * tiles_n;
  }
  if (lane == 63 && E == kMaxExperts) starts[E] = o[kExpertsPerLane];
  group_sums(c, E, lane, units);
}

// Row tiles of an expert's n tokens when its last tile may be short: tall tiles of 256 rows, and one of 128 where
// 1 to 128 rows are left after them.
constexpr int kTall = 256, kShort = 128;
__device__ __forceinline__ int tall_tiles(int n) { return n / kTall + (n % kTall > kShort ? 1 : 0); }
__device__ __forceinline__ int short_tiles(int n) { return n % kTall > 0 && n % kTall <= kShort ? 1 : 0; }

// As group_table_rows for both lists.
__device__ __forceinline__ void group_table_two(const int64_t* offsets, int E, int64_t T, uint32_t tiles_n,
                                                int* starts, uint32_t* tall, uint32_t* rest, int lane) {
  int o[kExpertsPerLane + 1];
  group_offsets(offsets, E, T, lane, o);
  uint32_t a[kExpertsPerLane], b[kExpertsPerLane];
#pragma unroll
  for (int i = 0; i < kExpertsPerLane; ++i) {
    const int j = kExpertsPerLane * lane + i;
    if (j <= E) starts[j] = o[i];
    a[i] = (uint32_t)tall_tiles(o[i + 1] - o[i]) * tiles_n;
    b[i] = (uint32_t)short_tiles(o[i + 1] - o[i]) * tiles_n;
  }
  if (lane == 63 && E == kMaxExperts) starts[E] = o[kExpertsPerLane];
  group_sums(a, E, lane, tall);
  group_sums(b, E, lane, rest);
}

// The lane's counts of 128-token blocks, for tokens padded to whole blocks per expert.
__device__ __forceinline__ void group_block_counts(const int (&o)[kExpertsPerLane + 1],
                                                   uint32_t (&c)[kExpertsPerLane]) {
#pragma unroll
  for (int i = 0; i < kExpertsPerLane; ++i) c[i] = (uint32_t)(o[i + 1] - o[i] + 127) / 128;
}

// starts[e] = first 128-token block of expert e in the padded layout, at most padded / 128; order[0 .. n) = the
// experts that have a block, by the bit length of their block count, most first (in expert order within one
// length); order[kMaxExperts] = n.  Products that contract over the blocks take the long experts first: a
// last round of long units on few workgroups is what costs most (64 experts with shares from 1/5 to 1/300:
// 614 us in expert order, contiguous per XCD).
__device__ __forceinline__ void group_table_blocks(const int64_t* offsets, int E, int64_t padded, int* starts,
                                                   uint32_t* order, int lane) {
  int o[kExpertsPerLane + 1];
  group_offsets(offsets, E, padded, lane, o);
  uint32_t c[kExpertsPerLane];
  group_block_counts(o, c);
  uint32_t mine = 0;
#pragma unroll
  for (int i = 0; i < kExpertsPerLane; ++i) mine += c[i];
  uint32_t at = wave_scan_add(mine) - mine;
  const uint32_t cap = (uint32_t)(padded / 128);
  uint32_t lengths = 0;  // bit l: an expert of mine has a count of l + 1 bits
#pragma unroll
  for (int i = 0; i < kExpertsPerLane; ++i) {
    const int j = kExpertsPerLane * lane + i;
    const uint32_t b0 = at < cap ? at : cap;
    at += c[i];
    const uint32_t b1 = at < cap ? at : cap;
    if (j <= E) starts[j] = (int)b0;
    c[i] = b1 - b0;
    if (c[i]) lengths |= 1u << (31 - __clz((int)c[i]));
  }
  if (lane == 63 && E == kMaxExperts) starts[E] = (int)(at < cap ? at : cap);
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) lengths |= (uint32_t)__shfl_xor((int)lengths, d);
  uint32_t n = 0;
  while (lengths) {  // (the same in every lane)
    const int l = 31 - __clz((int)lengths);
    lengths &= ~(1u << l);
    uint32_t have = 0;
#pragma unroll
    for (int i = 0; i < kExpertsPerLane; ++i) have += c[i] && 31 - __clz((int)c[i]) == l ? 1u : 0u;
    const uint32_t upto = wave_scan_add(have);
    uint32_t p = n + upto - have;
#pragma unroll
    for (int i = 0; i < kExpertsPerLane; ++i)
      if (c[i] && 31 - __clz((int)c[i]) == l) order[p++] = (uint32_t)(kExpertsPerLane * lane + i);
    n += (uint32_t)__builtin_amdgcn_readlane((int)upto, 63);
  }
  if (lane == 0) order[kMaxExperts] = n;
}

// The expert of unit u: pre[e] <= u < pre[e+1], by a count of the experts that end at or before u (all
// 64 lanes take part; the result is the same in each).
__device__ __forceinline__ int group_find(const uint32_t* pre, int E, uint32_t u, int lane) {
  int e = 0;
  for (int b = 0; b < E; b += 64) {
    const int j = b + lane;
    const bool le = j < E && pre[j + 1] <= u;
    e += __popcll(__ballot(le));
  }
  return __builtin_amdgcn_readfirstlane(e);
}

}  // namespace fp8bq
