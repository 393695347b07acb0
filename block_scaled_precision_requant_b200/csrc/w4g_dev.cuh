// Device helpers shared by the integer 4-bit projection kernels: unpacking and
// the tiles of rows grouped by expert.
#pragma once

#include <cuda_fp16.h>

#include <cstdint>

#include "w4g.h"

namespace bsr {

__device__ __forceinline__ float scale_f32(uint16_t s, int half) {
  return half ? __half2float(__ushort_as_half(s)) : __uint_as_float((uint32_t)s << 16);
}

__device__ __forceinline__ uint32_t fma_bf16x2(uint32_t a, uint32_t b, uint32_t c) {
  uint32_t d;
  asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
  return d;
}

// Both kernels unpack a code to the BF16 value (q - z) / 64, exactly, and
// multiply the sums by 64.  Bits below 256 read as BF16 are that integer times
// 2^-133 (subnormal below 128, the first normal binade above), so a nibble in
// bits 0-3 or 4-7 of a half needs neither shift nor exponent: one FMA scales
// it by 2^127 or 2^123 and subtracts z / 64.
constexpr uint32_t kLow2 = 0x7F007F00u;     // both nibbles in bits 0-3: 2^127, 2^127
constexpr uint32_t kHigh2 = 0x7D007D00u;    // both in bits 4-7: 2^123, 2^123
constexpr uint32_t kLowHigh = 0x7D007F00u;  // low half in 0-3, high half in 4-7
constexpr uint32_t kZero8 = 0xBE00BE00u;    // the pair -8 / 64

// The BF16 pair -z / 64.
__device__ __forceinline__ uint32_t zero_pair(uint32_t z) {
  const uint32_t h = __float_as_uint(-0.015625f * (float)z) & 0xFFFF0000u;
  return h | (h >> 16);
}

// One warp: off[e] = first row of expert e, each offset clamped to [the one
// before, rows_max]; pre[e] = tiles (of `rows` activation rows x `blocks`
// weight blocks) before expert e.  experts + 1 entries each.
__device__ __forceinline__ void count_tiles(const W4gArgs& g, int rows, int blocks, int lane, int* off, int* pre) {
  int edge = 0, sum = 0;
  const int rows_max = (int)g.rows_max;
  for (int e0 = 0; e0 < g.experts; e0 += 32) {
    const int e = e0 + lane;
    int hi = 0;
    if (e < g.experts) hi = g.offsets ? g.offsets[e + 1] : rows_max;
    hi = min(max(hi, edge), rows_max);
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xFFFFFFFFu, hi, o);
      if (lane >= o) hi = max(hi, v);
    }
    int lo = __shfl_up_sync(0xFFFFFFFFu, hi, 1);
    if (lane == 0) lo = edge;
    int s = e < g.experts ? (int)(((unsigned)(hi - lo) + (unsigned)rows - 1u) / (unsigned)rows) * blocks : 0;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xFFFFFFFFu, s, o);
      if (lane >= o) s += v;
    }
    if (e < g.experts) {
      off[e + 1] = hi;
      pre[e + 1] = sum + s;
    }
    edge = __shfl_sync(0xFFFFFFFFu, hi, 31);
    sum += __shfl_sync(0xFFFFFFFFu, s, 31);
  }
  if (lane == 0) off[0] = pre[0] = 0;
}

// Tile i < pre[experts]: its expert, weight block, first row and rows.  The
// row tiles of one weight block are neighbours, so that CTAs running together
// read the same weight.
struct GroupTile {
  int expert, n, row0, cnt;
};
__device__ __forceinline__ GroupTile find_tile(int i, int experts, int rows, const int* off, const int* pre) {
  int lo = 0, hi = experts;  // pre[lo] <= i < pre[hi]
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (pre[mid] <= i)
      lo = mid;
    else
      hi = mid;
  }
  const int count = off[lo + 1] - off[lo];
  const int local = i - pre[lo];
  GroupTile t = {lo, local, off[lo], min(rows, count)};
  if (count > rows) {
    const int tiles = (int)(((unsigned)count + (unsigned)rows - 1u) / (unsigned)rows);
    t.n = local / tiles;
    const int first = (local - t.n * tiles) * rows;
    t.row0 += first;
    t.cnt = min(rows, count - first);
  }
  return t;
}

}  // namespace bsr
