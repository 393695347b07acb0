// Internal launch interface of the integer 4-bit (group-scale) projections and
// of the expert router and combine.
#pragma once

#include <cmath>
#include <cstddef>
#include <cstdint>
#include <cuda.h>
#include <cuda_runtime.h>

namespace bsr {

// One product over weight rows stacked by expert (dense: one expert, no
// offsets).  Row r of the output, off[e] <= r < off[e + 1], is row rows[r] of
// a (r itself when rows is null) times expert e's weight; off[0] = 0 and off[e]
// = min(max(off[e - 1], offsets[e]), rows_max).
struct W4gArgs {
  const uint16_t* a;       // [a_rows, K] BF16
  const int32_t* offsets;  // [experts + 1], or null: one expert with `rows_max` rows
  const int32_t* rows;     // [rows_max], or null
  const uint8_t* q;        // [experts * N, K/2], element 2i in the low nibble of byte i
  const uint16_t* scale;   // [experts * N, K/G] BF16 or FP16
  const uint8_t* zero;     // [experts * N, K/G], or null: 8
  uint16_t* out;           // [rows_max, N] BF16
  long long a_rows, rows_max;
  int experts, n, k, group;
  int half_scale;          // scales are FP16
};

// What the host knows of the groups: the experts that have rows and their mean
// number of rows, for choices without preference.
struct W4gSpread {
  double active, mean;
  bool one;  // a single expert: all rows are its
  // Tiles of `rows` activation rows over all experts; a group's last tile is
  // half empty on average.
  double tiles(int rows) const {
    if (one) return std::ceil(mean / rows);
    return active * (mean <= 0.5 * rows ? 1.0 : 0.5 + mean / rows);
  }
};
inline W4gSpread w4g_spread(const W4gArgs& g) {
  W4gSpread s;
  const double experts = (double)g.experts, pairs = (double)g.rows_max;
  s.one = g.experts == 1;
  s.active = s.one ? 1.0 : experts * (1.0 - std::pow(1.0 - 1.0 / experts, pairs));
  s.mean = pairs / s.active;
  return s;
}

// Few rows per expert: warp-level tensor instructions fed by a streamed weight.
// Items of rt (1, 2 or 4) tiles of 16 weight rows x 8 nt activation rows, ks
// warps along K; the codes' tensor map has boxes of a tile x 128 bytes with the
// 128-byte swizzle.
constexpr int kW4gGemvRows = 16;
struct W4gGemvPlan {
  int rt, nt, ks, slots, nblk, chunks, grid;
  size_t smem;
  double us;  // estimated time
};
W4gGemvPlan w4g_gemv_plan(const W4gArgs& g, int num_sms);
cudaError_t launch_w4g_gemv(const CUtensorMap& tm_q, const W4gArgs& g, const W4gGemvPlan& p, int* status,
                            cudaStream_t stream);

// Many rows per expert: the tcgen05 tensor cores, tiles of 128 weight rows x
// bm activation rows.  Tensor maps: codes [experts * N, K/2] bytes, box 128
// rows x 64 bytes, 64-byte swizzle; activations [a_rows, K] BF16, box bm rows
// x 64, 128-byte swizzle.  Takes no row index.
struct W4gGemmPlan {
  int bm, grid;
  int split;  // CTAs (a cluster) that share the K of a tile; more than one only without offsets
  double us;  // estimated time
};
W4gGemmPlan w4g_gemm_plan(const W4gArgs& g, int num_sms);
// out[r] = a[rows[r]] for the rows of all groups (offsets as in W4gArgs, clamped
// alike); zeros where the index is outside a.  16-byte aligned rows.
cudaError_t launch_w4g_gather(const uint16_t* a, long long a_rows, const int32_t* rows, const int32_t* offsets,
                              int experts, uint16_t* out, long long rows_max, int k, cudaStream_t stream,
                              int num_sms);
cudaError_t launch_w4g_gemm(const CUtensorMap& tm_q, const CUtensorMap& tm_a, const W4gArgs& g, const W4gGemmPlan& p,
                            int* status, cudaStream_t stream);

// Which of the two takes a product.  `gemv` is filled where it may, `gemm`
// always.  At most kW4gFewRows rows per expert always take the first, so that
// they need no scratch.  The host does not know the groups: where they are even
// that is the faster one, where all rows fall on one expert the slower (us,
// decode / tensor-core: 512 rows on one of 128 experts of 1536 x 2048 35.9 /
// 20.3, 256 on one of 64 of 2048 x 2048 22.6 / 10.5, 32 on one of 8 of 14336 x
// 4096 41.7 / 16.8; at 5 rows each of the 128 64.4 / 87.0).
constexpr int kW4gFewRows = 4;
struct W4gPlan {
  bool few = false;
  W4gGemvPlan gemv = {};
  W4gGemmPlan gemm = {};
};
W4gPlan w4g_plan(const W4gArgs& g, int num_sms);

// Router.  Blocks of route_block_tokens(tokens) tokens; scratch holds one
// row of `experts` counts per block (none when there is one block).
constexpr int kRouteMaxExperts = 1024;
constexpr int kRouteMaxTopK = 32;
long long route_block_tokens(long long tokens);
size_t route_scratch_bytes(long long tokens, int experts);
cudaError_t launch_route(const void* logits, bool bf16, long long tokens, int experts, int top_k, bool renorm,
                         int32_t* ids, float* weights, int32_t* offsets, int32_t* rows, int32_t* pos, void* scratch,
                         size_t smem_optin, cudaStream_t stream);

cudaError_t launch_combine(const uint16_t* y, long long y_rows, const int32_t* pos, const float* weights,
                           const uint16_t* residual, uint16_t* out, long long tokens, int top_k, int n,
                           cudaStream_t stream, int num_sms);

}  // namespace bsr
