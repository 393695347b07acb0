// Integer 4-bit projections for few rows per expert (decode):
//   out[r, n] = bf16( sum_g s[n, g] * sum_{k in g} a[r, k] * (q[n, k] - z[n, g]) )
// on the weight as stored, rows grouped by expert (dense: one expert).
//
// Bound: the weight stream from HBM, half a byte per element, is 46 elements
// per SM and clock at the copy rate.  A CUDA-core FMA per element (after a
// conversion) would need most of an SM's issue slots for one activation row
// and more than all of them for several, so the products go through the
// warp-level tensor instruction (mma.sync m16n8k16, BF16 -> F32): 16 weight
// rows times up to 8 activation rows per instruction, at the same cost for 1
// row as for 8.  (tcgen05.mma wants 128 weight rows per tile and its operands
// staged for one issuing thread; at 8 rows the staging is the work.)  What is
// left on the CUDA cores is the unpacking: per word of 8 codes a shift, four
// masks and four BF16-pair FMAs (w4g_dev.cuh).  An mma sums over K in any
// order, so nibble pairs (j, j + 4) of a word are taken as they come and the
// activations are permuted to match.  A group's products are summed from zero
// by the mma, then scaled in float32.
//
// Work split: an item is rt = 1, 2 or 4 tiles of 16 weight rows of one expert
// times up to 8 NT of its activation rows; ks warps of a CTA split its K in
// chunks of 256 (128 bytes) dealt cyclically, and add their sums in a fixed
// order through shared memory.  The split depends on K only: a row's bits
// depend neither on the other rows nor on the grid.  Larger items use an
// activation load for more weight rows, smaller ones fill the last wave of
// CTAs: the plan weighs the two by measured costs.
// Consecutive items go to different SMs, so that a partial last wave is
// shared by all of them (64 tokens, top 8 of 128 experts of 1536 x 2048: 62.7
// us; with a CTA's warps taking consecutive items 68.7).
//
// One CTA per SM: 16 multiplying warps, and a producer warp whose lane w keeps
// warp w's ring full of tiles (16 rows x 128 bytes, 128-byte swizzle, by TMA)
// across chunks and items; no CTA barrier in the stream.  With the copies
// issued by the multiplying warps themselves the same work took 17% longer (dense
// 14336 x 4096, 1 row: 15.6 us against 13.3), and three or four smaller CTAs
// per SM, which leave 56 to 72 registers per thread, spilled and took longer
// still.  Row g of an mma is slot row bitreverse3(g): with the swizzle, the
// lanes of one shared-memory phase then hit distinct banks for groups of 32,
// 64 and 128 (4, 8 and 16 bytes per lane).  A chunk's scales and zero points
// are read a chunk ahead and kept as stored until they are staged in shared
// memory: converting them at the load would wait for it.
//
// Measured (inputs larger than L2): 14336 x 4096, groups of 128: 1 row 12.5
// us = 2.4 TB/s, 8 rows 14.1 us; five or six experts of that size (4 tokens,
// top 2 of 8) 43.4 us = 3.8 TB/s; 122 experts of 1536 x 2048 (48 tokens, top 8
// of 128, groups of 64, zero points) 67.4 us = 3.1 TB/s.  With the
// multiplication taken out the stream alone reaches 5.25 TB/s: the kernel is
// bound by issue and instruction latency (about 20 instructions per word and
// warp, 54% of the issue slots with 4 warps per scheduler; without the
// unpacking's FMAs, 22% of all instructions, it is 9% faster), at one or two
// waves also by the launch and the first bytes.
#include <cuda_bf16.h>

#include <cmath>
#include <mutex>

#include "common.cuh"
#include "w4g.h"
#include "w4g_dev.cuh"
#include "w4g_ring.h"

namespace bsr {
namespace {

constexpr int kWarps = 16;        // that multiply
constexpr int kWarp0 = 4;         // the warps before them: one requests the codes
constexpr int kThreads = 32 * (kWarp0 + kWarps);
constexpr int kMaxSplit = 8;      // warps along K
constexpr int kDoneBar = 15;      // named barrier; those of the groups along K are 1 to 8
// register split: launched with 96 per thread
constexpr int kLaunchRegs = 96, kCodesRegs = 24, kMulRegs = 112;
static_assert(128 * kCodesRegs + 32 * kWarps * kMulRegs <= kThreads * kLaunchRegs, "register split");
constexpr int kChunk = 256;       // elements of K per chunk
constexpr int kChunkBytes = 128;  // of codes

constexpr int kRows = kW4gGemvRows;  // weight rows per tile: the mma's
static_assert(kRows == 16, "mma.m16n8k16");
constexpr int kSlotBytes = kRows * kChunkBytes;

struct GemvCfg {
  int rt, ks, slots, nblk, chunks;
  int vec;  // scales (and zero points) of a lane may be read as one vector
};

struct GemvSmem {
  uint32_t meta, red, bars, off, pre, abort_flag, total;
};

// Per-warp ring of tile slots, per-warp scales of a chunk, the warps' sums of
// an item, barriers, offsets and items before each expert.
__host__ __device__ inline GemvSmem gemv_smem(int rt, int nt, int group, int slots, int experts) {
  GemvSmem L;
  L.meta = kWarps * (uint32_t)slots * kSlotBytes;
  L.red = L.meta + kWarps * (uint32_t)(kChunk / group) * (uint32_t)rt * 8u * 16u;
  L.bars = L.red + kWarps * (uint32_t)(rt * 16) * (uint32_t)(nt * 8) * 4u;
  L.off = L.bars + kWarps * (uint32_t)slots * 16u;  // full and empty
  L.pre = L.off + (uint32_t)(experts + 1) * 4u;
  L.abort_flag = L.pre + (uint32_t)(experts + 1) * 4u;
  L.total = L.abort_flag + 16u + 1024u;  // 1 KB to align the slots
  return L;
}

// 8 codes of a word -> four BF16 pairs ((q_j - z) / 64, (q_{j+4} - z) / 64);
// zc = the pair -z / 64.
__device__ __forceinline__ void unpack8(uint32_t w, uint32_t zc, uint32_t (&p)[4]) {
  const uint32_t v = w >> 8;
  p[0] = fma_bf16x2(w & 0x000F000Fu, kLow2, zc);
  p[1] = fma_bf16x2(w & 0x00F000F0u, kHigh2, zc);
  p[2] = fma_bf16x2(v & 0x000F000Fu, kLow2, zc);
  p[3] = fma_bf16x2(v & 0x00F000F0u, kHigh2, zc);
}

__device__ __forceinline__ void mma_bf16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// the same from a zero accumulator
__device__ __forceinline__ void mma_bf16_first(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                               uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.0f));
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

// G: group.  RT: most 16-row tiles of an item (2: one or two; 4: four).  NT:
// 8-row activation tiles.
template <int G, int RT, int NT>
__global__ void __launch_bounds__(kThreads, 1)
    w4g_gemv_kernel(const __grid_constant__ CUtensorMap tm_q, const W4gArgs g, const GemvCfg c,
                    int* __restrict__ status) {
  constexpr int W = G / 32;                     // words per lane, row and group
  constexpr int GS = kChunk / G / NT;           // groups per segment
  constexpr int SEG = kChunk / NT;              // elements of K per segment
  constexpr int GC = kChunk / G;                // groups per chunk
  constexpr int ML = (RT * 16 + 31) / 32;       // rows whose scales one lane loads
  constexpr int TOK = 8 * NT;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  const GemvSmem L = gemv_smem(RT, NT, G, c.slots, g.experts);
  const int warp = (int)(threadIdx.x >> 5) - kWarp0, lane = threadIdx.x & 31;
  const int ngrp = kWarps / c.ks;
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + L.bars);  // [warp][slot]
  uint64_t* empty = full + (size_t)kWarps * c.slots;
  int* s_off = reinterpret_cast<int*>(smem + L.off);
  int* s_pre = reinterpret_cast<int*>(smem + L.pre);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + L.abort_flag);

  if (threadIdx.x == 0) *abort_flag = 0;
  if (threadIdx.x < kWarps * c.slots) {
    mbar_init(&full[threadIdx.x], 1);
    mbar_init(&empty[threadIdx.x], 1);
    fence_mbar_init();
  }
  if (threadIdx.x == 0) tma_prefetch_desc(&tm_q);
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  if (warp == -kWarp0) count_tiles(g, TOK, c.nblk, lane, s_off, s_pre);
  __syncthreads();
  const int items = s_pre[g.experts];
  const int step = (int)gridDim.x * ngrp;
  const int rt = RT == 4 ? 4 : c.rt;
  const int rb = kRows * rt;  // weight rows of an item
  auto find = [&](int i) {
    const GroupTile f = find_tile(i, g.experts, TOK, s_off, s_pre);
    return Item{f.expert, f.n, f.row0, f.cnt};
  };

  // the multiplying warps and the one that requests the codes, once each
  auto warps_done = [] { asm volatile("bar.sync %0, %1;" ::"n"(kDoneBar), "n"(32 * (kWarps + 1)) : "memory"); };

  if (warp < 0) {
    setmaxnreg_dec<kCodesRegs>();
    if (warp != -kWarp0) return;
    // ---------------------------------------------------------- codes
    // lane w keeps warp w's ring full, across its chunks, tiles and items
    const int grp = lane / c.ks, wk = lane - grp * c.ks;
    uint64_t* f = full + lane * c.slots;
    uint64_t* e = empty + lane * c.slots;
    uint8_t* ring = smem + (size_t)lane * (size_t)c.slots * kSlotBytes;
    int slot = 0;
    uint32_t phase = 1, issued = 0;
    bool ok = true;
    if (lane < kWarps) {
      for (int it = grp * (int)gridDim.x + (int)blockIdx.x; ok && it < items; it += step) {
        const Item t = find(it);
        const int y = t.e * g.n + t.blk * rb;
        for (int ch = wk; ok && ch < c.chunks; ch += c.ks)
          for (int i = 0; i < rt; ++i) {
            ok = mbar_wait(&e[slot], phase, abort_flag, status, DEV_ERR_TIMEOUT_DECODE);
            if (!ok) break;
            mbar_arrive_expect_tx(&f[slot], (uint32_t)kSlotBytes);
            tma_load_2d(ring + (size_t)slot * kSlotBytes, &tm_q, &f[slot], ch * kChunkBytes, y + i * kRows);
            ++issued;
            if (++slot == c.slots) {
              slot = 0;
              phase ^= 1u;
            }
          }
      }
    }
    // Once every warp is done: if any wait ran out, this lane's or its warp's,
    // copies may be in flight that no warp waits for, and the CTA must not exit
    // under them.  (Waiting for them here in every case, without the meeting,
    // took 1-1.5% longer at one row.)
    __syncwarp();
    warps_done();
    if (lane < kWarps && *abort_flag) {
      const unsigned long long t0 = globaltimer_ns();
      drain_ring(issued, (uint32_t)c.slots, [&](uint32_t s, uint32_t parity) {
        while (!mbar_try_wait(&f[s], parity))
          if (globaltimer_ns() - t0 > kWaitLimitNs) return false;
        return true;
      });
    }
    return;
  }
  setmaxnreg_inc<kMulRegs>();

  const int grp = warp / c.ks, wk = warp - grp * c.ks;
  const int first = grp * (int)gridDim.x + (int)blockIdx.x;
  uint64_t* bars = full + warp * c.slots;
  uint64_t* released = empty + warp * c.slots;
  const uint32_t ring_s = smem_u32(smem) + (uint32_t)(warp * c.slots * kSlotBytes);
  const uint32_t meta_s = smem_u32(smem) + L.meta + (uint32_t)(warp * RT * GC) * 128u;
  const int t4 = lane & 3, g8 = lane >> 2;
  const int r8 = ((g8 & 1) << 2) | (g8 & 2) | (g8 >> 2);  // bit reversal
  const int groups = g.k / G;

  // The activation rows of an item: row tt * 8 + g8 in this lane; -1 for none.
  // The index is read an item ahead, and looked at only when its item begins.
  struct Index {
    int r[NT];
  };
  auto index_of = [&](const Item& t) {
    Index x;
#pragma unroll
    for (int tt = 0; tt < NT; ++tt) {
      const int r = tt * 8 + g8;
      x.r[tt] = -1;
      if (r < t.cnt) x.r[tt] = g.rows ? __ldg(g.rows + t.row0 + r) : t.row0 + r;
    }
    return x;
  };
  struct Rows {
    const uint16_t* p[NT];
  };
  auto rows_of = [&](const Index& x) {
    Rows q;
#pragma unroll
    for (int tt = 0; tt < NT; ++tt)
      q.p[tt] = x.r[tt] >= 0 && x.r[tt] < g.a_rows ? g.a + (size_t)x.r[tt] * (size_t)g.k + t4 * (G / 4) : nullptr;
    return q;
  };
  // One segment's activations: of each group, this lane's G/4 elements.
  struct Acts {
    uint4 v[NT][GS][W];
  };
  auto load_acts = [&](const Rows& r, int gi0) {
    Acts x;
#pragma unroll
    for (int tt = 0; tt < NT; ++tt)
#pragma unroll
      for (int gi = 0; gi < GS; ++gi)
#pragma unroll
        for (int w = 0; w < W; ++w) {
          x.v[tt][gi][w] = make_uint4(0, 0, 0, 0);
          if (r.p[tt] && gi0 + gi < groups)
            x.v[tt][gi][w] = __ldg(reinterpret_cast<const uint4*>(r.p[tt] + (size_t)(gi0 + gi) * G + w * 8));
        }
    return x;
  };
  // Scales and zero points of one chunk, as stored: lane l has rows l, l + 32 of
  // the item's 16-row tiles.
  struct alignas(16) Meta {
    alignas(16) uint16_t s[ML][GC];
    alignas(8) uint8_t z[ML][GC];
  };
  // this lane's rows within an item; groups are taken from the item's base
  int mrow[ML];
#pragma unroll
  for (int l = 0; l < ML; ++l) {
    const int r = l * 32 + lane;
    mrow[l] = r < rb ? r : 1 << 30;
  }
  auto load_meta = [&](const Item& t, int ch) {
    Meta m;
    const int gi = ch * GC;
    const int left = g.n - t.blk * rb;  // rows of the item that exist
    const size_t base = ((size_t)t.e * g.n + (size_t)t.blk * rb) * (size_t)groups + gi;
    const uint16_t* sp = g.scale + base;
    const uint8_t* zp = g.zero + base;
#pragma unroll
    for (int l = 0; l < ML; ++l) {
      const bool ok = mrow[l] < left;
      const uint32_t at = (uint32_t)mrow[l] * (uint32_t)groups;  // below 64 x 2^26
#pragma unroll
      for (int v = 0; v < GC; ++v) {
        m.s[l][v] = 0;
        m.z[l][v] = 8;
      }
      if (c.vec) {
        if (ok) {
          if constexpr (GC == 2) {
            *reinterpret_cast<uint32_t*>(m.s[l]) = __ldg(reinterpret_cast<const uint32_t*>(sp + at));
            if (g.zero) *reinterpret_cast<uint16_t*>(m.z[l]) = __ldg(reinterpret_cast<const uint16_t*>(zp + at));
          } else if constexpr (GC == 4) {
            *reinterpret_cast<uint2*>(m.s[l]) = __ldg(reinterpret_cast<const uint2*>(sp + at));
            if (g.zero) *reinterpret_cast<uint32_t*>(m.z[l]) = __ldg(reinterpret_cast<const uint32_t*>(zp + at));
          } else {
            *reinterpret_cast<uint4*>(m.s[l]) = __ldg(reinterpret_cast<const uint4*>(sp + at));
            if (g.zero) *reinterpret_cast<uint2*>(m.z[l]) = __ldg(reinterpret_cast<const uint2*>(zp + at));
          }
        }
      } else {
#pragma unroll
        for (int v = 0; v < GC; ++v)
          if (ok && gi + v < groups) {
            m.s[l][v] = __ldg(sp + at + v);
            if (g.zero) m.z[l][v] = __ldg(zp + at + v);
          }
      }
    }
    return m;
  };
  // ... to shared memory, per tile, group and mma row pair: {s(r), s(r + 8),
  // -z/64 of r, of r + 8}
  const uint32_t meta_w =
      meta_s + (uint32_t)(lane >> 4) * (GC * 128u) + (uint32_t)(lane & 7) * 16u + (uint32_t)((lane >> 3) & 1) * 4u;
  auto put_scale = [&](uint32_t at, float v) {
    asm volatile("st.shared.f32 [%0], %1;" ::"r"(meta_w + at), "f"(v) : "memory");
  };
  auto put_zero = [&](uint32_t at, uint32_t v) {
    asm volatile("st.shared.u32 [%0], %1;" ::"r"(meta_w + at + 8u), "r"(v) : "memory");
  };
  auto put_meta = [&](const Meta& m) {
    if (g.half_scale) {
#pragma unroll
      for (int l = 0; l < ML; ++l)
#pragma unroll
        for (int v = 0; v < GC; ++v) put_scale((uint32_t)((l * 2 * GC + v) * 128), scale_f32(m.s[l][v], 1));
    } else {
#pragma unroll
      for (int l = 0; l < ML; ++l)
#pragma unroll
        for (int v = 0; v < GC; ++v) put_scale((uint32_t)((l * 2 * GC + v) * 128), scale_f32(m.s[l][v], 0));
    }
    if (g.zero) {
#pragma unroll
      for (int l = 0; l < ML; ++l)
#pragma unroll
        for (int v = 0; v < GC; ++v) put_zero((uint32_t)((l * 2 * GC + v) * 128), zero_pair(m.z[l][v]));
    }
  };
  if (!g.zero) {  // the same for every chunk
#pragma unroll
    for (int l = 0; l < ML; ++l)
#pragma unroll
      for (int v = 0; v < GC; ++v) put_zero((uint32_t)((l * 2 * GC + v) * 128), kZero8);
  }

  // A warp whose wait ran out goes on without waiting (its outputs are not to be
  // used) and releases no slot: its copy may still be on its way.
  bool dead = false;
  Item next = {};
  Index next_index = {};
  Meta meta = {};
  if (first < items) {
    next = find(first);
    next_index = index_of(next);
    meta = load_meta(next, wk);
  }
  int slot = 0;
  uint32_t phase = 0;
  for (int it = first; it < items; it += step) {
    const Item t = next;
    const Rows rows = rows_of(next_index);
    const int n0 = t.blk * rb;
    if (it + step < items) {
      next = find(it + step);
      next_index = index_of(next);
    }
    float tot[RT][NT][4];
#pragma unroll
    for (int i = 0; i < RT; ++i)
#pragma unroll
      for (int tt = 0; tt < NT; ++tt)
#pragma unroll
        for (int j = 0; j < 4; ++j) tot[i][tt][j] = 0.0f;

    for (int ch = wk; ch < c.chunks; ch += c.ks) {
      const bool last = ch + c.ks >= c.chunks;
      __syncwarp();
      put_meta(meta);
      __syncwarp();
      meta = load_meta(last ? next : t, last ? wk : ch + c.ks);
      const int slot0 = slot;  // the chunk's first tile
      const uint32_t phase0 = phase;
#pragma unroll
      for (int seg = 0; seg < NT; ++seg) {
        const int gbase = (ch * NT + seg) * GS;
        const Acts acts = load_acts(rows, gbase);
        uint32_t b[NT][GS][W][4];
#pragma unroll
        for (int tt = 0; tt < NT; ++tt)
#pragma unroll
          for (int gi = 0; gi < GS; ++gi)
#pragma unroll
            for (int w = 0; w < W; ++w) {
              const uint4 v = acts.v[tt][gi][w];
              b[tt][gi][w][0] = __byte_perm(v.x, v.z, 0x5410);
              b[tt][gi][w][1] = __byte_perm(v.x, v.z, 0x7632);
              b[tt][gi][w][2] = __byte_perm(v.y, v.w, 0x5410);
              b[tt][gi][w][3] = __byte_perm(v.y, v.w, 0x7632);
            }
        slot = slot0;
        phase = phase0;
#pragma unroll
        for (int i = 0; i < RT; ++i) {
          if (i < rt) {
            if (seg == 0 && !dead) {
              const bool landed = mbar_wait(&bars[slot], phase, abort_flag, status, DEV_ERR_TIMEOUT_DECODE);
              if (__any_sync(0xFFFFFFFFu, !landed)) dead = true;
            }
            const uint32_t sl = ring_s + (uint32_t)slot * kSlotBytes + (uint32_t)r8 * kChunkBytes;
#pragma unroll
            for (int gi = 0; gi < GS; ++gi) {
              uint32_t w0[W], w1[W];
              const uint32_t boff = (uint32_t)(seg * (SEG / 2) + gi * (G / 2) + t4 * (G / 8));
              const uint32_t at = sl + ((((boff >> 4) ^ (uint32_t)r8) << 4) | (boff & 15u));
              lds_words<W>(at, w0);
              lds_words<W>(at + 8u * kChunkBytes, w1);
              float s0, s1;
              uint32_t z0, z1;
              const uint32_t ma = meta_s + (uint32_t)((i * GC + seg * GS + gi) * 128) + (uint32_t)r8 * 16u;
              asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];" : "=f"(s0), "=f"(s1), "=r"(z0), "=r"(z1) : "r"(ma));
              // two chains of products, so that one's latency passes during the other
              float d[NT][2][4];
#pragma unroll
              for (int w = 0; w < W; ++w) {
                uint32_t p0[4], p1[4];
                unpack8(w0[w], z0, p0);
                unpack8(w1[w], z1, p1);
#pragma unroll
                for (int tt = 0; tt < NT; ++tt) {
                  if (w == 0) {
                    mma_bf16_first(d[tt][0], p0[0], p1[0], p0[1], p1[1], b[tt][gi][w][0], b[tt][gi][w][1]);
                    mma_bf16_first(d[tt][1], p0[2], p1[2], p0[3], p1[3], b[tt][gi][w][2], b[tt][gi][w][3]);
                  } else {
                    mma_bf16(d[tt][0], p0[0], p1[0], p0[1], p1[1], b[tt][gi][w][0], b[tt][gi][w][1]);
                    mma_bf16(d[tt][1], p0[2], p1[2], p0[3], p1[3], b[tt][gi][w][2], b[tt][gi][w][3]);
                  }
                }
              }
#pragma unroll
              for (int tt = 0; tt < NT; ++tt) {
                tot[i][tt][0] = fmaf(d[tt][0][0] + d[tt][1][0], s0, tot[i][tt][0]);
                tot[i][tt][1] = fmaf(d[tt][0][1] + d[tt][1][1], s0, tot[i][tt][1]);
                tot[i][tt][2] = fmaf(d[tt][0][2] + d[tt][1][2], s1, tot[i][tt][2]);
                tot[i][tt][3] = fmaf(d[tt][0][3] + d[tt][1][3], s1, tot[i][tt][3]);
              }
            }
            if (seg + 1 == NT) {  // every lane has read the slot: it may be refilled
              __syncwarp();
              if (lane == 0 && !dead) mbar_arrive(&released[slot]);
            }
            if (++slot == c.slots) {
              slot = 0;
              phase ^= 1u;
            }
          }
        }
      }
    }

    // sum of the item's ks warps, in warp order; the codes were taken / 64
    constexpr int PITCH = RT * 16;
    float* red = reinterpret_cast<float*>(smem + L.red);
    float* mine = red + (size_t)warp * PITCH * TOK;
#pragma unroll
    for (int i = 0; i < RT; ++i)
      if (i < rt) {
#pragma unroll
        for (int tt = 0; tt < NT; ++tt)
#pragma unroll
          for (int j = 0; j < 4; ++j)
            mine[(tt * 8 + t4 * 2 + (j & 1)) * PITCH + i * 16 + (j >> 1) * 8 + r8] = tot[i][tt][j];
      }
    const int bar_threads = c.ks * 32;
    if (c.ks > 1)
      asm volatile("bar.sync %0, %1;" ::"r"(grp + 1), "r"(bar_threads) : "memory");
    else
      __syncwarp();
    const float* part = red + (size_t)grp * c.ks * PITCH * TOK;
    for (int i = wk * 32 + lane; i < PITCH * t.cnt; i += bar_threads) {
      const int tok = i / PITCH, r = i & (PITCH - 1);
      const int row = n0 + r;
      if (r >= rb || row >= g.n) continue;
      float v = 0.0f;
      for (int w = 0; w < c.ks; ++w) v += part[((size_t)w * TOK + tok) * PITCH + r];
      reinterpret_cast<__nv_bfloat16*>(g.out)[(size_t)(t.row0 + tok) * (size_t)g.n + row] =
          __float2bfloat16_rn(64.0f * v);
    }
    if (c.ks > 1)
      asm volatile("bar.sync %0, %1;" ::"r"(grp + 1), "r"(bar_threads) : "memory");
    else
      __syncwarp();
  }
  warps_done();
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
      cudaFuncAttributes fa;
      if ((e = cudaFuncGetAttributes(&fa, kern)) != cudaSuccess) return e;
      // the register split assumes every thread starts with kLaunchRegs registers
      if (fa.numRegs < kLaunchRegs) return cudaErrorInvalidConfiguration;
      if ((e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem)) != cudaSuccess)
        return e;
      granted[dev] = smem;
    }
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3(kThreads);
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
  GemvCfg c = {p.rt, p.ks, p.slots, p.nblk, p.chunks, 0};
  constexpr int gc = kChunk / G;  // a chunk's scales start at a multiple of gc groups of the row
  c.vec = (g.k / G) % gc == 0 && reinterpret_cast<uintptr_t>(g.scale) % (2u * gc) == 0 &&
          reinterpret_cast<uintptr_t>(g.zero) % (unsigned)gc == 0;
  if constexpr (G != 32) {  // at most two tiles there (see the plan)
    if (p.rt > 2) return launch<G, 4, 1>(tm, g, c, p.grid, p.smem, status, stream);
  }
  return p.nt == 1 ? launch<G, 2, 1>(tm, g, c, p.grid, p.smem, status, stream)
                   : launch<G, 2, 2>(tm, g, c, p.grid, p.smem, status, stream);
}

}  // namespace

W4gGemvPlan w4g_gemv_plan(const W4gArgs& g, int num_sms) {
  W4gGemvPlan p = {};
  p.chunks = (g.k + kChunk - 1) / kChunk;
  // at least two chunks per warp: an item's fixed cost (its lookup, the first
  // activations, the sum over warps) is that of two tiles' chunks.  By K only,
  // so that the order of a row's sum is.
  p.ks = 1;
  while (p.ks < kMaxSplit && p.ks * 4 <= p.chunks) p.ks *= 2;
  const int ngrp = kWarps / p.ks;
  const int per_warp = (p.chunks + p.ks - 1) / p.ks;
  const W4gSpread sp = w4g_spread(g);
  p.nt = sp.mean <= 8.0 ? 1 : 2;
  const int tok = 8 * p.nt;
  const double tiles = sp.tiles(tok);
  // rt tiles of 16 rows per item: the least estimated time over whole waves.
  // Measured per wave, us: 2.3, and per chunk of a warp 0.7 (its activations and
  // scales) + 0.9 per tile (16 / 32 / 64 rows at K = 2048: 5.2 / 7.5 / 13.3, at
  // K = 14336: 13.4 / 19 / 33).  (Three tiles took as long as four, tiles of
  // fewer rows as long as full ones.)
  const double slots_all = (double)num_sms * ngrp;
  double best = 0.0;
  // (At G = 32 four tiles' scales, with two activation tiles their sums, leave
  // too little room for the ring.)
  for (int rt = g.group == 32 || p.nt == 2 ? 2 : 4; rt >= 1; rt /= 2) {
    const double items = (double)((g.n + rt * kRows - 1) / (rt * kRows)) * tiles;
    const double cost = ceil(items / slots_all) * (2.3 + per_warp * (0.7 + 0.9 * rt));
    if (best == 0.0 || cost < best - 1e-9) {
      best = cost;
      p.rt = rt;
    }
  }
  // The call: a launch, and by group and activation tiles (measured, us, 14336 x
  // 4096, estimate before factors 10.9, at groups of 32 and two activation tiles
  // 14.6: groups of 128 13.6, two tiles 21.0; 64 15.3 and 21.6; 32 17.5 and 27).
  const double f = p.nt == 1 ? (g.group == 64 ? 1.15 : 1.0) : (g.group == 32 ? 1.65 : 1.25);
  p.us = 2.7 + best * f;
  const int rb = p.rt * kRows;
  p.nblk = (g.n + rb - 1) / rb;
  // slots: as many as the shared memory of an SM (227 KB) has room for.  A
  // chunk's tiles stay until its last segment.
  const int rt_max = p.rt <= 2 ? 2 : 4;
  const int least = p.nt == 1 ? 3 : p.rt + 1;
  p.slots = 6;
  while (p.slots > least && gemv_smem(rt_max, p.nt, g.group, p.slots, g.experts).total > 232448u) --p.slots;
  p.smem = gemv_smem(rt_max, p.nt, g.group, p.slots, g.experts).total;
  // of any grouping: each expert's last tile may be ragged
  const long long items = (long long)p.nblk * ((g.rows_max < g.experts ? g.rows_max : g.experts) + g.rows_max / tok);
  p.grid = (int)(items < num_sms ? items : num_sms);
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
