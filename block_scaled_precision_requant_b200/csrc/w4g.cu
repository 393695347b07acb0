// Projections with integer 4-bit weights and group scales, grouped by expert:
//   out[r, n] = bf16( sum_g s[n, g] * sum_{k in g} a[r, k] * (q[n, k] - z[n, g]) )
// One warp per weight row and up to 4 rows of one expert; lane l takes the
// 8-element words l, l + 32, ...; products and sums in float32.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "w4g.h"

namespace bsr {
namespace {

constexpr int kRows = 4;

__device__ __forceinline__ float scale_value(uint16_t s, int half) {
  return half ? __half2float(__ushort_as_half(s)) : __uint_as_float((uint32_t)s << 16);
}

__global__ void __launch_bounds__(256) w4g_simple_kernel(const W4gArgs g) {
  const int lane = threadIdx.x & 31;
  const int n = blockIdx.x * 8 + (threadIdx.x >> 5);
  if (n >= g.n) return;
  // the expert and first row of this block's row tile
  long long tile = blockIdx.y, r0 = 0;
  int e = 0;
  long long cnt = 0;
  bool found = false;
  long long lo = 0;
  for (; e < g.experts; ++e) {
    long long hi = g.offsets ? (long long)g.offsets[e + 1] : g.rows_max;
    hi = hi < lo ? lo : (hi > g.rows_max ? g.rows_max : hi);
    const long long tiles = (hi - lo + kRows - 1) / kRows;
    if (tile < tiles) {
      r0 = lo + tile * kRows;
      cnt = hi - r0 < kRows ? hi - r0 : kRows;
      found = true;
      break;
    }
    tile -= tiles;
    lo = hi;
  }
  if (!found) return;
  const size_t wrow = (size_t)e * g.n + n;
  const int groups = g.k / g.group;
  float acc[kRows] = {};
  for (int w = lane; w < g.k / 8; w += 32) {
    const uint32_t q = reinterpret_cast<const uint32_t*>(g.q + wrow * (size_t)(g.k / 2))[w];
    const int gi = w * 8 / g.group;
    const float s = scale_value(g.scale[wrow * groups + gi], g.half_scale);
    const float z = g.zero ? (float)g.zero[wrow * groups + gi] : 8.0f;
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      if (i >= cnt) break;
      const long long src = g.rows ? (long long)g.rows[r0 + i] : r0 + i;
      if (src < 0 || src >= g.a_rows) continue;
      const uint16_t* a = g.a + (size_t)src * g.k + (size_t)w * 8;
      float p = 0.0f;
#pragma unroll
      for (int j = 0; j < 8; ++j)
        p = fmaf(__uint_as_float((uint32_t)a[j] << 16), (float)((q >> (4 * j)) & 15u) - z, p);
      acc[i] = fmaf(p, s, acc[i]);
    }
  }
#pragma unroll
  for (int i = 0; i < kRows; ++i) {
    for (int off = 16; off; off >>= 1) acc[i] += __shfl_xor_sync(0xFFFFFFFFu, acc[i], off);
    if (lane == 0 && i < cnt)
      reinterpret_cast<__nv_bfloat16*>(g.out)[(size_t)(r0 + i) * g.n + n] = __float2bfloat16_rn(acc[i]);
  }
}

}  // namespace

cudaError_t launch_w4g_simple(const W4gArgs& g, cudaStream_t stream) {
  const long long tiles = (g.rows_max + kRows - 1) / kRows + (g.experts > 1 ? g.experts : 0);
  // grid.y is limited to 65535: row tiles beyond it are not reachable here
  if (tiles > 65535) return cudaErrorInvalidValue;
  w4g_simple_kernel<<<dim3((unsigned)((g.n + 7) / 8), (unsigned)tiles), 256, 0, stream>>>(g);
  return cudaGetLastError();
}

}  // namespace bsr
