// Integer 4-bit projections for few rows per expert (decode):
//   out[r, n] = bf16( sum_g s[n, g] * sum_{k in g} a[r, k] * (q[n, k] - z[n, g]) )
// on the weight as stored, rows grouped by expert (dense: one expert).
//
// Bound: the weight stream from HBM, half a byte per element, 46 elements per
// SM and clock at the copy rate.  A CUDA-core FMA per element (after a
// conversion) would need most of an SM's issue slots for one activation row
// and more than all of them for several, so the products go through the
// warp-level tensor instruction (mma.sync m16n8k16, BF16 -> F32): 16 weight
// rows times up to 8 activation rows per instruction at the same cost for 1
// row as for 8.  What is left on the CUDA cores is the unpacking, 11
// instructions per 8 elements: shift and mask a pair of nibbles into the
// mantissas of two BF16 values 128 + q, subtract 128 + z (both exact).  An
// mma sums over K in any order, so nibble pairs (j, j + 4) of a 32-bit word
// are taken as they come and the activations are permuted to match.  A
// group's products are summed from zero by the mma, then scaled in float32.
//
// Work split: an item is `rb` weight rows (at most 16 RT) of one expert times
// up to 8 NT of its activation rows; ks warps of a CTA split its K in chunks of
// 256 (128 bytes) dealt cyclically, and add their sums in a fixed order
// through shared memory.  The split depends on K only: a row's bits depend
// neither on the other rows nor on the grid.  rb is chosen so that the items
// fill whole waves of the resident CTAs.
//
// Memory: each warp streams its chunks (rb rows x 128 bytes, 128-byte
// swizzle) by TMA into its own ring of slots, issued ahead across items; no
// CTA barrier in the stream.  Row g of an mma is slot row bitreverse3(g): with
// the swizzle, the lanes of one shared-memory phase then hit distinct banks
// for groups of 32, 64 and 128 (4, 8 and 16 bytes per lane).
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <mutex>

#include "common.cuh"
#include "w4g.h"

namespace bsr {
namespace {

constexpr int kWarps = 8;
constexpr int kChunk = 256;       // elements of K per chunk
constexpr int kChunkBytes = 128;  // of codes

struct GemvCfg {
  int rb, ks, slots, nblk, chunks;
};

struct GemvSmem {
  uint32_t slot_bytes, red, bars, off, pre, abort_flag, total;
};

__host__ __device__ inline GemvSmem gemv_smem(int rt, int nt, int slots, int experts) {
  GemvSmem L;
  L.slot_bytes = (uint32_t)rt * 16u * kChunkBytes;
  L.red = kWarps * (uint32_t)slots * L.slot_bytes;
  L.bars = L.red + kWarps * (uint32_t)(rt * 16 + 1) * (uint32_t)(nt * 8) * 4u;
  L.off = L.bars + kWarps * (uint32_t)slots * 8u;
  L.pre = L.off + (uint32_t)(experts + 1) * 4u;
  L.abort_flag = L.pre + (uint32_t)(experts + 1) * 4u;
  L.total = L.abort_flag + 16u + 1024u;  // 1 KB to align the slots
  return L;
}

__device__ __forceinline__ float scale_f32(uint16_t s, int half) {
  return half ? __half2float(__ushort_as_half(s)) : __uint_as_float((uint32_t)s << 16);
}

__device__ __forceinline__ uint32_t sub_bf16x2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}

// 8 codes of a word -> four BF16 pairs (q_j - z, q_{j+4} - z); zc = the pair
// 128 + z.
__device__ __forceinline__ void unpack8(uint32_t w, uint32_t zc, uint32_t (&p)[4]) {
#pragma unroll
  for (int j = 0; j < 4; ++j) p[j] = sub_bf16x2(((w >> (4 * j)) & 0x000F000Fu) | 0x43004300u, zc);
}

__device__ __forceinline__ void mma_bf16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

template <int W>
__device__ __forceinline__ void lds_words(uint32_t addr, uint32_t (&w)[W]) {
  if constexpr (W == 4)
    asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]) : "r"(addr));
  else if constexpr (W == 2)
    asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(w[0]), "=r"(w[1]) : "r"(addr));
  else
    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(w[0]) : "r"(addr));
}

struct Item {
  int e, blk;
  int row0, cnt;  // first grouped row, rows (at most 8 NT)
};

template <int G, int RT, int NT>
__global__ void __launch_bounds__(kWarps * 32, 2)
    w4g_gemv_kernel(const __grid_constant__ CUtensorMap tm_q, const W4gArgs g, const GemvCfg c,
                    int* __restrict__ status) {
  constexpr int W = G / 32;           // words per lane, row and group
  constexpr int GC = kChunk / G;      // groups per chunk
  constexpr int SPL = (GC + 3) / 4;   // scales per lane, row and chunk
  constexpr int TOK = 8 * NT;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  const GemvSmem L = gemv_smem(RT, NT, c.slots, g.experts);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int grp = warp / c.ks, wk = warp - grp * c.ks;
  const int ngrp = kWarps / c.ks;
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + L.bars) + (size_t)warp * c.slots;
  int* s_off = reinterpret_cast<int*>(smem + L.off);
  int* s_pre = reinterpret_cast<int*>(smem + L.pre);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + L.abort_flag);
  const uint32_t ring = smem_u32(smem) + (uint32_t)warp * (uint32_t)c.slots * L.slot_bytes;

  if (threadIdx.x == 0) *abort_flag = 0;
  if (lane == 0) {
    for (int s = 0; s < c.slots; ++s) mbar_init(&bars[s], 1);
    fence_mbar_init();
  }
  if (threadIdx.x == 0) tma_prefetch_desc(&tm_q);
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  // items before each expert; the offsets clamped to [the one before, R]
  if (warp == 0) {
    int edge = 0, sum = 0;
    for (int e0 = 0; e0 < g.experts; e0 += 32) {
      const int e = e0 + lane;
      int hi = 0;
      if (e < g.experts) hi = g.offsets ? g.offsets[e + 1] : (int)g.rows_max;
      hi = min(max(hi, edge), (int)g.rows_max);
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xFFFFFFFFu, hi, o);
        if (lane >= o) hi = max(hi, v);
      }
      int lo = __shfl_up_sync(0xFFFFFFFFu, hi, 1);
      if (lane == 0) lo = edge;
      const int items = e < g.experts ? (hi - lo + TOK - 1) / TOK * c.nblk : 0;
      int s = items;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xFFFFFFFFu, s, o);
        if (lane >= o) s += v;
      }
      if (e < g.experts) {
        s_off[e + 1] = hi;
        s_pre[e + 1] = sum + s;
      }
      edge = __shfl_sync(0xFFFFFFFFu, hi, 31);
      sum += __shfl_sync(0xFFFFFFFFu, s, 31);
    }
    if (lane == 0) s_off[0] = s_pre[0] = 0;
  }
  __syncthreads();
  const int items = s_pre[g.experts];
  const int step = (int)gridDim.x * ngrp;
  const int first = (int)blockIdx.x * ngrp + grp;

  auto find = [&](int i) {
    Item t;
    int lo = 0, hi = g.experts;  // s_pre[lo] <= i < s_pre[hi]
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (s_pre[mid] <= i)
        lo = mid;
      else
        hi = mid;
    }
    t.e = lo;
    const int rows = s_off[lo + 1] - s_off[lo];
    const int tiles = (rows + TOK - 1) / TOK;
    const int local = i - s_pre[lo];
    t.blk = local / tiles;
    const int tile = local - t.blk * tiles;
    t.row0 = s_off[lo] + tile * TOK;
    t.cnt = min(TOK, rows - tile * TOK);
    return t;
  };

  // the warp's issue position: next (item, chunk) to request
  int iss_item = first, iss_c = wk, iss_y = 0;
  uint32_t issued = 0, used = 0;
  if (iss_item < items) {
    const Item t = find(iss_item);
    iss_y = t.e * g.n + t.blk * c.rb;
  }
  auto issue = [&]() {
    if (iss_item >= items) return;
    const uint32_t s = issued % (uint32_t)c.slots;
    if (lane == 0) {
      mbar_arrive_expect_tx(&bars[s], (uint32_t)c.rb * kChunkBytes);
      tma_load_2d(smem + (ring - smem_u32(smem)) + s * L.slot_bytes, &tm_q, &bars[s], iss_c * kChunkBytes, iss_y);
    }
    ++issued;
    iss_c += c.ks;
    if (iss_c >= c.chunks) {
      iss_c = wk;
      iss_item += step;
      if (iss_item < items) {
        const Item t = find(iss_item);
        iss_y = t.e * g.n + t.blk * c.rb;
      }
    }
  };
  if (wk < c.chunks)
    for (int s = 0; s < c.slots; ++s) issue();

  const int t4 = lane & 3, g8 = lane >> 2;
  const int r8 = ((g8 & 1) << 2) | (g8 & 2) | (g8 >> 2);  // bit reversal
  const int groups = g.k / G;
  bool dead = false;
  for (int it = first; it < items; it += step) {
    const Item t = find(it);
    const int n0 = t.blk * c.rb;
    const uint16_t* ap[NT];
#pragma unroll
    for (int tt = 0; tt < NT; ++tt) {
      const int r = tt * 8 + g8;
      ap[tt] = nullptr;
      if (r < t.cnt) {
        const long long src = g.rows ? (long long)g.rows[t.row0 + r] : (long long)t.row0 + r;
        if (src >= 0 && src < g.a_rows) ap[tt] = g.a + (size_t)src * (size_t)g.k;
      }
    }
    float tot[RT][NT][4];
#pragma unroll
    for (int i = 0; i < RT; ++i)
#pragma unroll
      for (int tt = 0; tt < NT; ++tt)
#pragma unroll
        for (int j = 0; j < 4; ++j) tot[i][tt][j] = 0.0f;

    for (int ch = wk; ch < c.chunks; ch += c.ks) {
      const int gbase = ch * GC;
      // scales and zero points: lane t4 holds groups t4 (and t4 + 4) of its rows
      uint16_t sc[RT][2][SPL];
      uint8_t zp[RT][2][SPL];
#pragma unroll
      for (int i = 0; i < RT; ++i)
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int v = 0; v < SPL; ++v) {
            const int gi = gbase + v * 4 + t4;
            const int n = n0 + i * 16 + h * 8 + r8;
            sc[i][h][v] = 0;
            zp[i][h][v] = 8;
            if (v * 4 + t4 < GC && gi < groups && n < g.n) {
              const size_t at = ((size_t)t.e * g.n + n) * (size_t)groups + gi;
              sc[i][h][v] = g.scale[at];
              if (g.zero) zp[i][h][v] = g.zero[at];
            }
          }
      // activations of the chunk: lane t4 of each group's G/4 elements
      uint4 x[NT][GC][W];
#pragma unroll
      for (int tt = 0; tt < NT; ++tt)
#pragma unroll
        for (int gi = 0; gi < GC; ++gi)
#pragma unroll
          for (int w = 0; w < W; ++w) {
            x[tt][gi][w] = make_uint4(0, 0, 0, 0);
            if (ap[tt] && gbase + gi < groups)
              x[tt][gi][w] =
                  __ldg(reinterpret_cast<const uint4*>(ap[tt] + (size_t)(gbase + gi) * G + t4 * (G / 4) + w * 8));
          }
      const uint32_t s = used % (uint32_t)c.slots;
      bool landed = !dead;
      if (!dead)
        landed = mbar_wait(&bars[s], (used / (uint32_t)c.slots) & 1u, abort_flag, status, DEV_ERR_TIMEOUT_DECODE);
      if (__any_sync(0xFFFFFFFFu, !landed)) dead = true;
      const uint32_t slot = ring + s * L.slot_bytes;
#pragma unroll
      for (int gi = 0; gi < GC; ++gi) {
        if (gbase + gi >= groups) break;
        uint32_t b[NT][W][4];
#pragma unroll
        for (int tt = 0; tt < NT; ++tt)
#pragma unroll
          for (int w = 0; w < W; ++w) {
            const uint4 v = x[tt][gi][w];
            b[tt][w][0] = __byte_perm(v.x, v.z, 0x5410);
            b[tt][w][1] = __byte_perm(v.x, v.z, 0x7632);
            b[tt][w][2] = __byte_perm(v.y, v.w, 0x5410);
            b[tt][w][3] = __byte_perm(v.y, v.w, 0x7632);
          }
        const int src = (lane & ~3) | (gi & 3);
        const uint32_t boff = (uint32_t)(gi * (G / 2) + t4 * (G / 8));
#pragma unroll
        for (int i = 0; i < RT; ++i) {
          uint32_t zc[2];
          float sv[2];
          uint32_t w0[W], w1[W];
          const uint32_t ra = (uint32_t)(i * 16 + r8);
          const uint32_t at = slot + ra * kChunkBytes + ((((boff >> 4) ^ (uint32_t)r8) << 4) | (boff & 15u));
          lds_words<W>(at, w0);
          lds_words<W>(at + 8u * kChunkBytes, w1);
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            sv[h] = scale_f32((uint16_t)__shfl_sync(0xFFFFFFFFu, (int)sc[i][h][gi / 4], src), g.half_scale);
            zc[h] = (g.zero ? (uint32_t)__shfl_sync(0xFFFFFFFFu, (int)zp[i][h][gi / 4], src) : 8u) * 0x00010001u |
                    0x43004300u;
          }
          float d[NT][4];
#pragma unroll
          for (int tt = 0; tt < NT; ++tt)
#pragma unroll
            for (int j = 0; j < 4; ++j) d[tt][j] = 0.0f;
#pragma unroll
          for (int w = 0; w < W; ++w) {
            uint32_t p0[4], p1[4];
            unpack8(w0[w], zc[0], p0);
            unpack8(w1[w], zc[1], p1);
#pragma unroll
            for (int tt = 0; tt < NT; ++tt) {
              mma_bf16(d[tt], p0[0], p1[0], p0[1], p1[1], b[tt][w][0], b[tt][w][1]);
              mma_bf16(d[tt], p0[2], p1[2], p0[3], p1[3], b[tt][w][2], b[tt][w][3]);
            }
          }
#pragma unroll
          for (int tt = 0; tt < NT; ++tt) {
            tot[i][tt][0] = fmaf(d[tt][0], sv[0], tot[i][tt][0]);
            tot[i][tt][1] = fmaf(d[tt][1], sv[0], tot[i][tt][1]);
            tot[i][tt][2] = fmaf(d[tt][2], sv[1], tot[i][tt][2]);
            tot[i][tt][3] = fmaf(d[tt][3], sv[1], tot[i][tt][3]);
          }
        }
      }
      ++used;
      // every lane has read the slot: it may be refilled (async proxy)
      __syncwarp();
      if (!dead) {
        fence_proxy_async_smem();
        issue();
      }
    }

    // sum of the item's ks warps, in warp order
    constexpr int PITCH = RT * 16 + 1;
    float* red = reinterpret_cast<float*>(smem + L.red);
    float* mine = red + (size_t)warp * PITCH * TOK;
#pragma unroll
    for (int i = 0; i < RT; ++i)
#pragma unroll
      for (int tt = 0; tt < NT; ++tt)
#pragma unroll
        for (int j = 0; j < 4; ++j)
          mine[(tt * 8 + t4 * 2 + (j & 1)) * PITCH + i * 16 + (j >> 1) * 8 + r8] = tot[i][tt][j];
    const int bar_threads = c.ks * 32;
    asm volatile("bar.sync %0, %1;" ::"r"(grp + 1), "r"(bar_threads) : "memory");
    const int nrows = min(c.rb, g.n - n0);
    const float* part = red + (size_t)grp * c.ks * PITCH * TOK;
    for (int i = wk * 32 + lane; i < nrows * t.cnt; i += bar_threads) {
      const int tok = i / nrows, r = i - tok * nrows;
      float v = 0.0f;
      for (int w = 0; w < c.ks; ++w) v += part[((size_t)w * TOK + tok) * PITCH + r];
      reinterpret_cast<__nv_bfloat16*>(g.out)[(size_t)(t.row0 + tok) * (size_t)g.n + n0 + r] = __float2bfloat16_rn(v);
    }
    asm volatile("bar.sync %0, %1;" ::"r"(grp + 1), "r"(bar_threads) : "memory");
  }
  // a warp that gave up waiting may still have copies in flight: wait for
  // them once more, again bounded, so the CTA does not exit under them
  if (dead && lane == 0) {
    const unsigned long long t0 = globaltimer_ns();
    for (uint32_t j = issued > (uint32_t)c.slots ? issued - c.slots : 0u; j < issued; ++j)
      while (!mbar_try_wait(&bars[j % c.slots], (j / c.slots) & 1u) && globaltimer_ns() - t0 < kWaitLimitNs) {
      }
  }
}

std::mutex g_mu;

template <int G, int RT, int NT>
cudaError_t launch(const CUtensorMap& tm, const W4gArgs& g, const GemvCfg& c, int grid, size_t smem, int* status,
                   cudaStream_t stream) {
  auto kern = w4g_gemv_kernel<G, RT, NT>;
  static size_t granted[64] = {};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  {
    std::lock_guard<std::mutex> lk(g_mu);
    if (smem > granted[dev]) {
      if ((e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem)) != cudaSuccess)
        return e;
      granted[dev] = smem;
    }
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3(kWarps * 32);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, tm, g, c, status);
}

template <int G>
cudaError_t launch_g(const CUtensorMap& tm, const W4gArgs& g, const W4gGemvPlan& p, int* status,
                     cudaStream_t stream) {
  const GemvCfg c = {p.rb, p.ks, p.slots, p.nblk, p.chunks};
  if (p.rt == 1)
    return p.nt == 1 ? launch<G, 1, 1>(tm, g, c, p.grid, p.smem, status, stream)
                     : launch<G, 1, 2>(tm, g, c, p.grid, p.smem, status, stream);
  return p.nt == 1 ? launch<G, 2, 1>(tm, g, c, p.grid, p.smem, status, stream)
                   : launch<G, 2, 2>(tm, g, c, p.grid, p.smem, status, stream);
}

}  // namespace

W4gGemvPlan w4g_gemv_plan(const W4gArgs& g, int num_sms) {
  W4gGemvPlan p = {};
  p.chunks = (g.k + kChunk - 1) / kChunk;
  p.ks = 1;
  while (p.ks < kWarps && p.ks * 2 <= p.chunks) p.ks *= 2;
  const int ngrp = kWarps / p.ks;
  // activation rows per item by the rows that an expert gets on average
  const long long active = g.rows_max < g.experts ? g.rows_max : g.experts;
  p.nt = (g.rows_max + active - 1) / active <= 8 ? 1 : 2;
  const long long tok = 8 * p.nt;
  const long long tiles = active + (g.rows_max - active) / tok;
  // rows per item: the fewest row steps over whole waves of two CTAs per SM
  const long long slots_all = 2LL * num_sms * ngrp;
  double best = 0.0;
  for (int rb = 32; rb >= 8; rb -= 2) {
    const long long items = ((g.n + rb - 1) / rb) * tiles;
    const long long waves = (items + slots_all - 1) / slots_all;
    const double cost = (double)waves * (rb + 4);
    if (best == 0.0 || cost < best - 1e-9) {
      best = cost;
      p.rb = rb;
    }
  }
  p.rt = p.rb <= 16 ? 1 : 2;
  p.nblk = (g.n + p.rb - 1) / p.rb;
  // slots: as many as leave room for two CTAs per SM (228 KB less 1 KB per CTA)
  p.slots = 6;
  while (p.slots > 2 && gemv_smem(p.rt, p.nt, p.slots, g.experts).total > 115712u) --p.slots;
  p.smem = gemv_smem(p.rt, p.nt, p.slots, g.experts).total;
  const long long items = (long long)p.nblk * (tiles + active);  // ragged tails add at most one tile per expert
  const long long ctas = (items + ngrp - 1) / ngrp;
  p.grid = (int)(ctas < 2LL * num_sms ? ctas : 2LL * num_sms);
  return p;
}

cudaError_t launch_w4g_gemv(const CUtensorMap& tm_q, const W4gArgs& g, const W4gGemvPlan& p, int* status,
                            cudaStream_t stream) {
  switch (g.group) {
    case 32: return launch_g<32>(tm_q, g, p, status, stream);
    case 64: return launch_g<64>(tm_q, g, p, status, stream);
    case 128: return launch_g<128>(tm_q, g, p, status, stream);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace bsr
