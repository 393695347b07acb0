// Expert router and combine.
//
// Router: per token the top_k experts by logit (ties to the lowest index),
// their softmax weights, and the grouping of the (token, slot) pairs by
// expert.  An expert whose logit is -inf or NaN is masked: it is never
// chosen and has probability 0; slots left without an expert get id -1,
// weight 0 and position -1 and join no group.  The pairs of one expert keep
// their order (token, then slot), so the groups never depend on scheduling:
// positions come from counts, not from atomically drawn tickets (the only
// atomics are integer histogram counts).
//
// One warp per token (up to four in turn, for their latencies); lane l holds
// experts l, l + 32, ...: a logit as an unsigned key of the same order (0 =
// masked).  Each slot takes one hardware warp maximum over keys and one warp
// minimum over the indices that hold it.
// A block of tokens counts its pairs by expert.  With one block the same
// launch groups them; otherwise a second launch (programmatic dependent, same
// blocks) sums the counts of the blocks before it and the totals, then places
// its pairs: each warp counts its contiguous part of the block's pairs by
// expert, the warps' counts are scanned, and ranks within 32 pairs come from
// match_any.  Blocks of at least 32 tokens (one per warp) and at most 128 of
// them, so that the second launch reads at most 128 x E counts per block; up
// to 64 tokens take one block and one launch.
//
// Bound by latency: the chain of top_k warp reductions and the second launch,
// with one block of 32 warps per SM.  Measured: 33 tokens of 64 experts, top
// 8, 7.2 us; 16384 tokens of 128 experts, top 8, 23 us (4 tokens per warp;
// their 4 MB of logits take 0.7 us to read).
//
// Combine: out[t, :] = bf16(residual[t, :] + sum_j w[t, j] * y[pos[t, j], :]),
// summed in float32 in slot order; one read of each row, 16 bytes of up to four
// rows in flight per thread.  Bound by HBM: 8192 tokens, 8 rows of 2048 and a
// residual 56 us = 5.5 TB/s; 16 tokens 2.2 us (launch).
#include <cuda_bf16.h>

#include <climits>

#include "w4g.h"

namespace bsr {
namespace {

constexpr int kThreads = 1024;
constexpr int kWarps = kThreads / 32;
constexpr int kHeld = 4;  // rounds of 32 pairs whose ids a warp keeps in registers
constexpr int kMaxBlocks = 128;
constexpr int kMinBlockTokens = 32;   // a token per warp
constexpr int kOneBlockTokens = 64;   // at most this many in a single block: one launch, 7 us where two take 9

// Order-preserving key of a logit; 0 marks a masked expert.  +0 and -0 share
// a key.
__device__ __forceinline__ uint32_t logit_key(float x) {
  if (!(x > -INFINITY)) return 0u;  // -inf or NaN
  const uint32_t b = __float_as_uint(x + 0.0f);
  return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}
__device__ __forceinline__ float key_logit(uint32_t key) {
  return __uint_as_float((key & 0x80000000u) ? (key & 0x7FFFFFFFu) : ~key);
}
// exp(x - top) with +inf logits sharing the whole probability
__device__ __forceinline__ float shifted_exp(float x, float top) {
  if (x == top) return 1.0f;
  return expf(x - top);
}

struct RouteArgs {
  const void* logits;
  long long tokens, block_tokens;
  int experts, top_k, bf16, renorm, blocks;
  int32_t* ids;
  float* weights;
  int32_t* offsets;
  int32_t* rows;
  int32_t* pos;
  int32_t* counts;  // [blocks, experts]
};

// The chosen experts of TP tokens t, t + step, ..., one step of each in turn so
// that the warp reductions' latencies overlap: slot j's id and weight end in
// lane j.  Each lane keeps its largest key and that key's expert.  Up to four
// keys are sorted once, so that the lane whose expert was chosen moves on to
// its next; with more it looks through its keys again.
template <int V, int TP>
__device__ __forceinline__ void route_tokens(const RouteArgs& r, long long t, long long step, long long t1, int lane,
                                             int* hist) {
  uint32_t key[TP][V], best[TP], my_key[TP];
  unsigned best_at[TP];
  int my_id[TP];
  float top[TP], all[TP];
  bool left[TP];
#pragma unroll
  for (int p = 0; p < TP; ++p) {
    const long long tp = t + p * step;
    left[p] = tp < t1;
    const size_t row = (size_t)(left[p] ? tp : t) * (size_t)r.experts;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int e = v * 32 + lane;
      float x = -INFINITY;
      if (left[p] && e < r.experts)
        x = r.bf16 ? __uint_as_float((uint32_t)__ldg(static_cast<const uint16_t*>(r.logits) + row + e) << 16)
                   : __ldg(static_cast<const float*>(r.logits) + row + e);
      key[p][v] = logit_key(x);
    }
  }
  // keys in falling order and, in bytes from the lowest, their v
  constexpr bool kSorted = V <= 4;
  uint32_t order[TP];
  auto sort_keys = [&](int p) {
    uint32_t at[V];
#pragma unroll
    for (int v = 0; v < V; ++v) at[v] = (uint32_t)v;
#pragma unroll
    for (int end = V - 1; end > 0; --end)
#pragma unroll
      for (int v = 0; v < end; ++v) {  // neighbours, strictly: equal keys stay in order
        const uint32_t a = key[p][v], b = key[p][v + 1], i = at[v], j = at[v + 1];
        const bool swap = b > a;
        key[p][v] = swap ? b : a;
        key[p][v + 1] = swap ? a : b;
        at[v] = swap ? j : i;
        at[v + 1] = swap ? i : j;
      }
    order[p] = 0u;
#pragma unroll
    for (int v = 0; v < V && v < 4; ++v) order[p] |= at[v] << (8 * v);
  };
  auto head = [&](int p) {
    best[p] = key[p][0];
    best_at[p] = (order[p] & 0xFFu) * 32u + (unsigned)lane;
  };
  auto rescan = [&](int p) {
    best[p] = key[p][V - 1];
    best_at[p] = (unsigned)((V - 1) * 32 + lane);
#pragma unroll
    for (int v = V - 2; v >= 0; --v)
      if (key[p][v] >= best[p]) {
        best[p] = key[p][v];
        best_at[p] = (unsigned)(v * 32 + lane);
      }
  };
#pragma unroll
  for (int p = 0; p < TP; ++p) {
    if constexpr (kSorted) {
      sort_keys(p);
      head(p);
    } else {
      rescan(p);
    }
    my_id[p] = -1;
    my_key[p] = 0u;
    top[p] = all[p] = 0.0f;
    const uint32_t m = __reduce_max_sync(0xFFFFFFFFu, best[p]);
    if (m) top[p] = key_logit(m);
    if (!r.renorm && m) {
#pragma unroll
      for (int v = 0; v < V; ++v)
        if (key[p][v]) all[p] += shifted_exp(key_logit(key[p][v]), top[p]);
    }
  }
  for (int j = 0; j < r.top_k; ++j) {
    uint32_t m[TP];
    unsigned at[TP];
#pragma unroll
    for (int p = 0; p < TP; ++p) m[p] = __reduce_max_sync(0xFFFFFFFFu, best[p]);
#pragma unroll
    for (int p = 0; p < TP; ++p) at[p] = __reduce_min_sync(0xFFFFFFFFu, best[p] == m[p] ? best_at[p] : UINT_MAX);
#pragma unroll
    for (int p = 0; p < TP; ++p) {
      if (m[p] == 0u) continue;  // every expert left is masked
      if (lane == j) {
        my_id[p] = (int)at[p];
        my_key[p] = m[p];
      }
      if ((at[p] & 31u) == (unsigned)lane) {
        if constexpr (kSorted) {
#pragma unroll
          for (int v = 0; v + 1 < V; ++v) key[p][v] = key[p][v + 1];
          key[p][V - 1] = 0u;
          order[p] >>= 8;
          head(p);
        } else {
#pragma unroll
          for (int v = 0; v < V; ++v)
            if ((unsigned)(v * 32 + lane) == at[p]) key[p][v] = 0u;
          rescan(p);
        }
      }
    }
  }
#pragma unroll
  for (int p = 0; p < TP; ++p) {
    const float e = my_id[p] >= 0 ? shifted_exp(key_logit(my_key[p]), top[p]) : 0.0f;
    float total = r.renorm ? e : all[p];
#pragma unroll
    for (int off = 16; off; off >>= 1) total += __shfl_xor_sync(0xFFFFFFFFu, total, off);
    if (lane < r.top_k && left[p]) {
      const size_t at = (size_t)(t + p * step) * r.top_k + lane;
      r.ids[at] = my_id[p];
      r.weights[at] = my_id[p] >= 0 ? e / total : 0.0f;
      if (my_id[p] >= 0) atomicAdd(&hist[my_id[p]], 1);
    }
  }
}

template <int V>
__device__ void route_block(const RouteArgs& r, int* hist) {
  constexpr int TP = V <= 4 ? 4 : V <= 8 ? 2 : 1;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  for (int e = threadIdx.x; e < r.experts; e += kThreads) hist[e] = 0;
  __syncthreads();
  const long long t0 = blockIdx.x * r.block_tokens;
  const long long t1 = min(r.tokens, t0 + r.block_tokens);
  if (TP == 1 || t1 - t0 <= kWarps) {
    for (long long t = t0 + warp; t < t1; t += kWarps) route_tokens<V, 1>(r, t, kWarps, t1, lane, hist);
  } else if (TP == 2 || t1 - t0 <= 2 * kWarps) {
    for (long long t = t0 + warp; t < t1; t += 2 * kWarps) route_tokens<V, 2>(r, t, kWarps, t1, lane, hist);
  } else {
    for (long long t = t0 + warp; t < t1; t += TP * kWarps) route_tokens<V, TP>(r, t, kWarps, t1, lane, hist);
  }
  __syncthreads();
}

// Exclusive scan over experts of total[], in place into first[] (first[E] =
// sum); every thread of the block takes part.
__device__ void scan_experts(const int* total, int* first, int experts) {
  if (threadIdx.x < 32) {
    const int lane = threadIdx.x;
    int carry = 0;
    for (int e0 = 0; e0 < experts; e0 += 32) {
      const int v = e0 + lane < experts ? total[e0 + lane] : 0;
      int s = v;
#pragma unroll
      for (int off = 1; off < 32; off <<= 1) {
        const int o = __shfl_up_sync(0xFFFFFFFFu, s, off);
        if (lane >= off) s += o;
      }
      if (e0 + lane < experts) first[e0 + lane] = carry + s - v;
      carry += __shfl_sync(0xFFFFFFFFu, s, 31);
    }
    if (lane == 0) first[experts] = carry;
  }
  __syncthreads();
}

// A warp's contiguous part of the block's pairs, the ids of its first rounds
// in registers.
struct Part {
  long long a, b;
  int id[kHeld];
};
__device__ __forceinline__ Part load_part(const RouteArgs& r) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const long long p0 = blockIdx.x * r.block_tokens * r.top_k;
  const long long p1 = min(r.tokens * r.top_k, p0 + r.block_tokens * r.top_k);
  long long part = (p1 - p0 + kWarps - 1) / kWarps;
  part = (part + 31) / 32 * 32;
  Part w;
  w.a = min(p1, p0 + warp * part);
  w.b = min(p1, w.a + part);
#pragma unroll
  for (int i = 0; i < kHeld; ++i) {
    const long long p = w.a + i * 32 + lane;
    w.id[i] = p < w.b ? r.ids[p] : -1;
  }
  return w;
}

// Places the block's pairs.  start[e]: position of the block's first pair of
// expert e.  warp_counts [kWarps][experts].
__device__ void place_pairs(const RouteArgs& r, const Part& w, const int* start, int* warp_counts) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int* mine = warp_counts + warp * r.experts;
  for (int e = lane; e < r.experts; e += 32) mine[e] = 0;
  __syncwarp();
#pragma unroll
  for (int i = 0; i < kHeld; ++i)
    if (w.id[i] >= 0) atomicAdd(&mine[w.id[i]], 1);
  for (long long p = w.a + kHeld * 32 + lane; p < w.b; p += 32) {
    const int id = r.ids[p];
    if (id >= 0) atomicAdd(&mine[id], 1);
  }
  __syncthreads();
  for (int e = threadIdx.x; e < r.experts; e += kThreads) {
    int at = start[e];
#pragma unroll 8
    for (int i = 0; i < kWarps; ++i) {
      const int c = warp_counts[i * r.experts + e];
      warp_counts[i * r.experts + e] = at;
      at += c;
    }
  }
  __syncthreads();
  auto round = [&](long long p, int id) {  // p: this lane's pair
    const unsigned same = __match_any_sync(0xFFFFFFFFu, id);
    int at = -1;
    if (id >= 0) {
      at = mine[id] + __popc(same & ((1u << lane) - 1u));
      r.rows[at] = (int)(p / r.top_k);
    }
    if (p < w.b) r.pos[p] = at;
    __syncwarp();
    if (id >= 0 && (same >> lane) == 1u) mine[id] = at + 1;  // the last lane of each set
    __syncwarp();
  };
#pragma unroll
  for (int i = 0; i < kHeld; ++i)
    if (w.a + i * 32 < w.b) round(w.a + i * 32 + lane, w.id[i]);
  for (long long p = w.a + kHeld * 32; p < w.b; p += 32) round(p + lane, p + lane < w.b ? r.ids[p + lane] : -1);
}

// rows[] past the last group, the block's share of them
__device__ void fill_tail(const RouteArgs& r, int used) {
  const long long pairs = r.tokens * r.top_k;
  for (long long p = used + blockIdx.x * (long long)kThreads + threadIdx.x; p < pairs;
       p += (long long)gridDim.x * kThreads)
    r.rows[p] = -1;
}

// Shared memory: hist/total [E], first [E + 1], then kWarps x E counts.
template <int V, bool ONE>
__global__ void __launch_bounds__(kThreads) route_kernel(const RouteArgs r) {
  extern __shared__ int smem[];
  int* hist = smem;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  route_block<V>(r, hist);
  if constexpr (ONE) {
    int* first = hist + r.experts;
    scan_experts(hist, first, r.experts);
    for (int e = threadIdx.x; e <= r.experts; e += kThreads) r.offsets[e] = first[e];
    place_pairs(r, load_part(r), first, first + r.experts + 1);
    fill_tail(r, first[r.experts]);
  } else {
    for (int e = threadIdx.x; e < r.experts; e += kThreads)
      r.counts[(size_t)blockIdx.x * r.experts + e] = hist[e];
  }
}

__global__ void __launch_bounds__(kThreads) route_group_kernel(const RouteArgs r) {
  extern __shared__ int smem[];
  int* total = smem;
  int* first = total + r.experts;
  int* warp_counts = first + r.experts + 1;
  int* before = warp_counts;  // [E], consumed before the warp counts are made
  for (int e = threadIdx.x; e < 2 * r.experts + 1; e += kThreads) total[e] = 0;
  for (int e = threadIdx.x; e < r.experts; e += kThreads) before[e] = 0;
  __syncthreads();
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const Part w = load_part(r);  // on its way while the counts are summed
  // counts of all blocks, and of the blocks before this one
  const int lanes_e = r.experts < kThreads ? r.experts : kThreads;
  const int parts = kThreads / lanes_e;
  const int part = threadIdx.x / lanes_e;
  if (part < parts) {
    for (int e = threadIdx.x - part * lanes_e; e < r.experts; e += lanes_e) {
      int sum = 0, pre = 0;
#pragma unroll 8
      for (int b = part; b < r.blocks; b += parts) {
        const int c = r.counts[(size_t)b * r.experts + e];
        sum += c;
        pre += b < (int)blockIdx.x ? c : 0;
      }
      atomicAdd(&total[e], sum);
      atomicAdd(&before[e], pre);
    }
  }
  __syncthreads();
  scan_experts(total, first, r.experts);
  if (blockIdx.x == 0)
    for (int e = threadIdx.x; e <= r.experts; e += kThreads) r.offsets[e] = first[e];
  const int used = first[r.experts];
  __syncthreads();
  for (int e = threadIdx.x; e < r.experts; e += kThreads) total[e] = first[e] + before[e];
  __syncthreads();
  place_pairs(r, w, total, warp_counts);
  fill_tail(r, used);
}

size_t route_smem(int experts) { return ((size_t)(2 + kWarps) * experts + 1) * sizeof(int); }

template <int V>
cudaError_t launch_route_v(const RouteArgs& r, size_t smem_optin, cudaStream_t stream) {
  const size_t smem = route_smem(r.experts);
  if (smem > smem_optin) return cudaErrorInvalidValue;
  cudaError_t e = cudaSuccess;
  if (r.blocks == 1) {
    if (smem > 48 * 1024)
      e = cudaFuncSetAttribute(route_kernel<V, true>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    route_kernel<V, true><<<1, kThreads, smem, stream>>>(r);
    return cudaGetLastError();
  }
  if (smem > 48 * 1024) {
    e = cudaFuncSetAttribute(route_group_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
  }
  route_kernel<V, false><<<r.blocks, kThreads, (size_t)r.experts * sizeof(int), stream>>>(r);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)r.blocks);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, route_group_kernel, r);
}

// VE elements (16, 8, 4 or 2 bytes) per thread and step.
template <int VE>
struct Vec;
template <>
struct Vec<8> {
  using T = uint4;
};
template <>
struct Vec<4> {
  using T = uint2;
};
template <>
struct Vec<2> {
  using T = uint32_t;
};
template <>
struct Vec<1> {
  using T = uint16_t;
};

template <int VE>
union Pack {
  typename Vec<VE>::T v;
  uint16_t h[VE];
};

template <int VE>
__global__ void __launch_bounds__(256)
    combine_kernel(const uint16_t* __restrict__ y, long long y_rows, const int32_t* __restrict__ pos,
                   const float* __restrict__ weights, const uint16_t* residual, uint16_t* out, long long tokens,
                   int top_k, int n) {
  const int cols = n / VE;
  const long long items = tokens * cols;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  for (long long i = (long long)blockIdx.x * 256 + threadIdx.x; i < items; i += (long long)gridDim.x * 256) {
    const long long t = i / cols;
    const int c = (int)(i - t * cols);
    float acc[VE];
#pragma unroll
    for (int v = 0; v < VE; ++v) acc[v] = 0.0f;
    if (residual) {
      Pack<VE> x;
      x.v = *reinterpret_cast<const typename Vec<VE>::T*>(residual + (size_t)t * n + (size_t)c * VE);
#pragma unroll
      for (int v = 0; v < VE; ++v) acc[v] = __uint_as_float((uint32_t)x.h[v] << 16);
    }
    for (int j0 = 0; j0 < top_k; j0 += 4) {
      Pack<VE> x[4];
      float w[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        long long p = -1;
        w[j] = 0.0f;
        if (j0 + j < top_k) {
          p = pos[t * top_k + j0 + j];
          w[j] = weights[t * top_k + j0 + j];
        }
        if (p >= 0 && p < y_rows)
          x[j].v = *reinterpret_cast<const typename Vec<VE>::T*>(y + (size_t)p * n + (size_t)c * VE);
        else {
          w[j] = 0.0f;
#pragma unroll
          for (int v = 0; v < VE; ++v) x[j].h[v] = 0;
        }
      }
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int v = 0; v < VE; ++v) acc[v] = fmaf(w[j], __uint_as_float((uint32_t)x[j].h[v] << 16), acc[v]);
    }
    Pack<VE> o;
#pragma unroll
    for (int v = 0; v < VE; ++v) o.h[v] = __bfloat16_as_ushort(__float2bfloat16_rn(acc[v]));
    *reinterpret_cast<typename Vec<VE>::T*>(out + (size_t)t * n + (size_t)c * VE) = o.v;
  }
}

template <int VE>
cudaError_t launch_combine_v(const uint16_t* y, long long y_rows, const int32_t* pos, const float* weights,
                             const uint16_t* residual, uint16_t* out, long long tokens, int top_k, int n,
                             cudaStream_t stream, int num_sms) {
  const long long blocks = (tokens * (n / VE) + 255) / 256;
  const long long cap = (long long)num_sms * 8 * 64;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(blocks < cap ? blocks : cap));
  cfg.blockDim = dim3(256);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, combine_kernel<VE>, y, y_rows, pos, weights, residual, out, tokens, top_k, n);
}

}  // namespace

long long route_block_tokens(long long tokens) {
  if (tokens <= kOneBlockTokens) return kOneBlockTokens;
  const long long b = (tokens + kMaxBlocks - 1) / kMaxBlocks;
  return b < kMinBlockTokens ? kMinBlockTokens : b;
}

size_t route_scratch_bytes(long long tokens, int experts) {
  const long long b = route_block_tokens(tokens);
  const long long blocks = (tokens + b - 1) / b;
  return blocks <= 1 ? 0 : (size_t)blocks * (size_t)experts * sizeof(int32_t);
}

cudaError_t launch_route(const void* logits, bool bf16, long long tokens, int experts, int top_k, bool renorm,
                         int32_t* ids, float* weights, int32_t* offsets, int32_t* rows, int32_t* pos, void* scratch,
                         size_t smem_optin, cudaStream_t stream) {
  RouteArgs r = {};
  r.logits = logits;
  r.tokens = tokens;
  r.block_tokens = route_block_tokens(tokens);
  r.experts = experts;
  r.top_k = top_k;
  r.bf16 = bf16 ? 1 : 0;
  r.renorm = renorm ? 1 : 0;
  r.blocks = (int)((tokens + r.block_tokens - 1) / r.block_tokens);
  if (r.blocks < 1) r.blocks = 1;  // no tokens: the offsets are still written
  r.ids = ids;
  r.weights = weights;
  r.offsets = offsets;
  r.rows = rows;
  r.pos = pos;
  r.counts = static_cast<int32_t*>(scratch);
  const int v = (experts + 31) / 32;
  if (v <= 1) return launch_route_v<1>(r, smem_optin, stream);
  if (v <= 2) return launch_route_v<2>(r, smem_optin, stream);
  if (v <= 4) return launch_route_v<4>(r, smem_optin, stream);
  if (v <= 8) return launch_route_v<8>(r, smem_optin, stream);
  if (v <= 16) return launch_route_v<16>(r, smem_optin, stream);
  return launch_route_v<32>(r, smem_optin, stream);
}

cudaError_t launch_combine(const uint16_t* y, long long y_rows, const int32_t* pos, const float* weights,
                           const uint16_t* residual, uint16_t* out, long long tokens, int top_k, int n,
                           cudaStream_t stream, int num_sms) {
  const uintptr_t bits = reinterpret_cast<uintptr_t>(y) | reinterpret_cast<uintptr_t>(out) |
                         reinterpret_cast<uintptr_t>(residual) | (uintptr_t)((size_t)n * 2);
  auto launch = [&](auto kernel) {
    return kernel(y, y_rows, pos, weights, residual, out, tokens, top_k, n, stream, num_sms);
  };
  if (bits % 16 == 0) return launch(launch_combine_v<8>);
  if (bits % 8 == 0) return launch(launch_combine_v<4>);
  if (bits % 4 == 0) return launch(launch_combine_v<2>);
  return launch(launch_combine_v<1>);
}

}  // namespace bsr
