// Integer 4-bit projections on the 5th-generation tensor cores, rows grouped
// by expert with ragged sizes (dense: one expert):
//   out[r, n] = bf16( sum_g s[n, g] * P[r, n, g] ),
//   P = sum_{k in g} a[r, k] * (q[n, k] - z[n, g])
// BF16 activations x BF16 integers (exact), float32 accumulation in tensor
// memory per group, one float32 FMA per element and group outside it.
//
// Tile: 128 weight rows (tensor-memory lanes, MMA M) x BM activation rows of
// one expert (columns, MMA N; a ragged tile multiplies its rows only).  The
// codes are the A operand and go through tensor memory: a stage's codes (128
// rows x 128 elements, 8 KB) come by TMA, eight warps unpack them to BF16
// pairs (w4g_dev.cuh) and store them with tcgen05.st as the A operand of
// `tcgen05.mma kind::f16`.  Through shared memory the unpacked tile (32 KB per
// stage, written once and read once) would compete with the activation tile
// for its bandwidth.  Activations (B operand) come by TMA into
// 128-byte-swizzled tiles, so a row index is resolved by a copy of the rows
// beforehand (w4g_gather_kernel): the tile's rows gathered here measured 454
// (TMA four-row gathers) and 284 TFLOP/s (16-byte asynchronous copies of two
// warps) against 1040 for tile loads, while the copy of 8192 rows of 4096 (23
// us) is 3% of their product with 14336 weight rows.
//
// The scale changes every G elements of K, so each group accumulates into its
// own tensor-memory buffer (two to six, what the unpacked stages leave of 512
// columns) and the epilogue adds s * P to float32 registers: a thread owns one
// weight row, so the scale is one register, and BM / 2 columns.  Per SM and
// group that is 128 x BM FMAs (two per instruction) against BM x G x 128
// tensor FMAs.
//
// Tiles are dealt to persistent CTAs in order of expert, weight tile,
// activation tile (activation fastest, so that CTAs running together read the
// same weight tile), from offsets read on the device.
//
// A dense product of few tiles leaves most SMs without one; clusters of 2, 4 or
// 8 CTAs then share a tile's K, and the first adds the others' float32 sums, in
// their order, from its own shared memory (17 rows of 4096 x 4096: 16.2 us with
// 32 CTAs, 9.0 with clusters of 4; 64 rows of 4096 x 14336: 49.5 and 19.6).
//
// Warps (20): 0 TMA loads, 1 MMAs (one elected lane; owns the tensor memory),
// 2-3 idle, 4-11 unpack (warp w: lanes 32 (w % 4).., half of each stage's K),
// 12-19 epilogue (lanes 32 (w % 4).., half of the columns).  Every wait is
// bounded: a wait that runs out sets a status bit and every role leaves its
// loop; copies and MMAs in flight are drained (bounded) before the tensor
// memory is freed.
//
// Measured, 2048 x 14336 x 4096, in short runs: G = 128 192-196 us = 1230-1250
// TFLOP/s, G = 64 225-235 us = 1020-1070, G = 32 366-377 us = 640-657; for
// seconds on end, under the power limit of 1000 W: 219 us at 1575 MHz, 260 at
// 1700, 366 at 1965.  G = 128 is bound by the MMAs and that limit (without the
// MMAs the rest takes 137 us), G = 32 by the epilogue's chain of wait, load and
// FMAs per group, about 520 cycles (no pipe is above 42%).  Narrow tiles are bound by the unpacking and the MMA warp's fixed work
// per group: 50 rows 18 us.  Tried and slower: 16 epilogue warps (G = 32 457 ->
// 620 us), two warps that issue MMAs (190 -> 206); no faster: a third buffer at
// BM = 128, the epilogue's loads a chunk ahead within a group (more than 16
// columns of them spill) or across groups.
#include <cuda_bf16.h>

#include <cmath>
#include <mutex>

#include "common.cuh"
#include "w4g.h"
#include "w4g_dev.cuh"
#include "w4g_ring.h"

namespace bsr {
namespace {

constexpr int kBn = 128;       // weight rows per tile
constexpr int kKs = 128;       // elements of K per stage
constexpr int kRaw = kBn * kKs / 2;
constexpr int kThreads = 640;
constexpr int kDeqWarp0 = 4, kEpiWarp0 = 12;
constexpr int kDeqWarps = 8, kEpiWarps = 8;
constexpr uint32_t kTmemCols = 512;
constexpr int kMaxStages = 12;
constexpr size_t kSmemMax = 232448;
constexpr int kLaunchRegs = 96, kCtrlRegs = 48;
constexpr int kSumBytes = 160 * 1024;  // of any width's stages, for the sums of a cluster's other CTAs

template <int BM>
struct Cfg {
  // tensor memory: the groups' accumulators, then the unpacked stages of 64
  // columns (128 elements of K, two per column)
  static constexpr int ASTAGES = BM == 192 ? 2 : 4;
  static constexpr uint32_t COL_A = kTmemCols - 64u * ASTAGES;
  static constexpr int TBUF = (int)COL_A / BM < 6 ? (int)COL_A / BM : 6;
  static constexpr int COLS = BM / 2;                     // columns per epilogue warp
  static constexpr int CH = BM == 192 ? 2 : 1;            // chunks that go through registers at once
  static constexpr int CW = COLS / CH;                    // columns of a chunk: 48, 64, 32, 16
  static constexpr int ACT = BM * 256;                    // two 128-byte-swizzled tiles of 64 elements of K
  static constexpr int STAGE = kRaw + ACT;
  // register split: launched with kLaunchRegs per thread
  static constexpr int EPI_REGS = BM == 192 ? 168 : 136;
  static constexpr int DEQ_REGS = BM == 192 ? 48 : 80;
  static_assert(128 * kCtrlRegs + 256 * (DEQ_REGS + EPI_REGS) <= kThreads * kLaunchRegs, "register split");
};

struct Ctrl {
  uint64_t full[kMaxStages], empty[kMaxStages];
  uint64_t aready[4];
  uint64_t tfull[6], tempty[6];
  uint64_t drain;
  uint32_t tmem_base;
  int abort_flag;
};

// kind::f16, D = F32, A = B = BF16, both K-major.
constexpr uint32_t idesc_bf16(int m, int n) {
  return (1u << 4) | (1u << 7) | (1u << 10) | ((uint32_t)(n >> 3) << 17) | ((uint32_t)(m >> 4) << 24);
}

// D[tmem] (+)= A[tmem] x B[smem]^T
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b_desc, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}

__device__ __forceinline__ void tmem_st_x16(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(
          taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}

__device__ __forceinline__ void tmem_ld(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}
__device__ __forceinline__ void tmem_ld(uint32_t taddr, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,"
      "%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
        "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
        "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr));
}

// CW columns as loads of 32 and 16.
template <int CW>
__device__ __forceinline__ void tmem_ld_chunk(uint32_t taddr, uint32_t (&r)[CW]) {
#pragma unroll
  for (int i = 0; i + 32 <= CW; i += 32) tmem_ld(taddr + (uint32_t)i, reinterpret_cast<uint32_t(&)[32]>(r[i]));
  if constexpr (CW % 32 == 16)
    tmem_ld(taddr + (uint32_t)(CW - 16), reinterpret_cast<uint32_t(&)[16]>(r[CW - 16]));
}

// Ties registers written by a tensor-memory load to this point of the
// program (after tcgen05.wait::ld).
template <int R>
__device__ __forceinline__ void regs_after_wait(uint32_t (&r)[R]) {
#pragma unroll
  for (int i = 0; i < R; i += 8)
    asm volatile("" : "+r"(r[i]), "+r"(r[i + 1]), "+r"(r[i + 2]), "+r"(r[i + 3]), "+r"(r[i + 4]), "+r"(r[i + 5]),
                      "+r"(r[i + 6]), "+r"(r[i + 7]));
}

// prmt, whose selectors with bit 3 set give a byte of copies of the sign bit.
__device__ __forceinline__ uint32_t prmt(uint32_t a, uint32_t b, uint32_t sel) {
  uint32_t d;
  asm("prmt.b32 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(sel));
  return d;
}

// Bounded wait that ignores the abort flag (used while draining).
__device__ __forceinline__ bool wait_drain(uint64_t* bar, uint32_t parity) {
  const unsigned long long t0 = globaltimer_ns();
  while (!mbar_try_wait(bar, parity))
    if (globaltimer_ns() - t0 > kWaitLimitNs) return false;
  return true;
}

// One lane of the converged warp.
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred P;\n\telect.sync _|P, 0xFFFFFFFF;\n\tselp.b32 %0, 1, 0, P;\n\t}" : "=r"(p));
  return p != 0;
}

struct TileAt {
  int e, n0, row0, cnt;
};

// All threads of the cluster, from any place of the program.
__device__ __forceinline__ void cluster_meet() {
  asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
}

// Ring position.
struct Pos {
  int i = 0;
  uint32_t phase = 0;
  __device__ __forceinline__ void next(int n) {
    if (++i == n) {
      i = 0;
      phase ^= 1u;
    }
  }
};

template <int BM, int G>
__global__ void __launch_bounds__(kThreads, 1)
    w4g_gemm_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_a,
                    const W4gArgs g, const int stages, const int split, int* __restrict__ status) {
  using C = Cfg<BM>;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  Ctrl* ctrl = reinterpret_cast<Ctrl*>(smem + (size_t)stages * C::STAGE);
  int* s_off = reinterpret_cast<int*>(ctrl + 1);
  int* s_pre = s_off + g.experts + 1;
  volatile int* abort_flag = &ctrl->abort_flag;
  // through a shuffle, so that the compiler knows it uniform: the roles' loops
  // then keep their descriptors and addresses in uniform registers
  const int warp = __shfl_sync(0xFFFFFFFFu, (int)(threadIdx.x >> 5), 0);
  const int lane = threadIdx.x & 31;
  const int n_tiles = (g.n + kBn - 1) / kBn;
  // K of this CTA: its share of the stages
  const int kstages = (g.k + kKs - 1) / kKs;
  const int rank = (int)blockIdx.x % split;
  const int ks0 = rank * kstages / split, ks1 = (rank + 1) * kstages / split;
  const int first_tile = (int)blockIdx.x / split, tile_step = (int)gridDim.x / split;
  const int groups = g.k / G;
  // a stage: the activation tile, then the codes
  auto stage_ptr = [&](int s) { return smem + (size_t)s * C::STAGE; };

  if (threadIdx.x == 0) {
    for (int s = 0; s < stages; ++s) {
      mbar_init(&ctrl->full[s], 1);
      mbar_init(&ctrl->empty[s], 1 + kDeqWarps);  // the MMA commit + the unpacking warps
    }
    for (int s = 0; s < C::ASTAGES; ++s) mbar_init(&ctrl->aready[s], kDeqWarps);
    for (int b = 0; b < C::TBUF; ++b) {
      mbar_init(&ctrl->tfull[b], 1);
      mbar_init(&ctrl->tempty[b], kEpiWarps);
    }
    mbar_init(&ctrl->drain, 1);
    ctrl->abort_flag = 0;
    fence_mbar_init();
    tma_prefetch_desc(&tm_q);
    tma_prefetch_desc(&tm_a);
  }
  if (warp == 1) {
    tmem_alloc(&ctrl->tmem_base, kTmemCols);
    tmem_relinquish();
  }
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (warp == 0) count_tiles(g, BM, n_tiles, lane, s_off, s_pre);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = ctrl->tmem_base;
  const int tiles = s_pre[g.experts];
  auto find = [&](int i) {
    const GroupTile f = find_tile(i, g.experts, BM, s_off, s_pre);
    return TileAt{f.expert, f.n * kBn, f.row0, f.cnt};
  };

  if (warp < kDeqWarp0) {
    setmaxnreg_dec<kCtrlRegs>();
    if (warp == 0) {
      // ---------------------------------------------------------------- loads
      Pos p;
      uint32_t it = 0;
      bool ok = true;
      for (int tile = first_tile; ok && tile < tiles; tile += tile_step) {
        const TileAt t = find(tile);
        for (int ks = ks0; ks < ks1; ++ks) {
          ok = mbar_wait(&ctrl->empty[p.i], p.phase ^ 1u, abort_flag, status, DEV_ERR_TIMEOUT_TMA);
          if (__any_sync(0xFFFFFFFFu, !ok)) {
            ok = false;
            break;
          }
          if (elect_one()) {
            uint8_t* st = stage_ptr(p.i);
            mbar_arrive_expect_tx(&ctrl->full[p.i], C::STAGE);
            tma_load_2d(st + C::ACT, &tm_q, &ctrl->full[p.i], ks * (kKs / 2), t.e * g.n + t.n0);
            tma_load_2d(st, &tm_a, &ctrl->full[p.i], ks * kKs, t.row0);
            tma_load_2d(st + BM * 128, &tm_a, &ctrl->full[p.i], ks * kKs + 64, t.row0);  // zeros past K
          }
          __syncwarp();
          ++it;
          p.next(stages);
        }
      }
      // the last stages' copies must have landed before the CTA may exit or, with
      // a shared K, its stages take the other CTAs' sums, also when an unpacking
      // warp gave up after the last issue here
      if (lane == 0)
        drain_ring(it, (uint32_t)stages,
                   [&](uint32_t s, uint32_t parity) { return wait_drain(&ctrl->full[s], parity); });
      __syncwarp();
    } else if (warp == 1) {
      // ---------------------------------------------------------------- MMA
      // A stage's unpacked codes are ready only after its activations landed
      // (the unpacking warps waited for both), so that is the one wait.
      Pos p, ap, tp;
      bool ok = true;
      // a ragged tile multiplies its rows only, in whole steps of 16 (what the
      // epilogue then reads past them it does not store)
      uint32_t idesc = idesc_bf16(kBn, BM);
      const uint64_t b_desc0 = smem_desc_k_sw128(smem_u32(smem));
      // The MMAs of the stage's group `gi` (16 elements of K each) into the
      // current buffer and its commit; after the last group the stage's
      auto group = [&](int gi, bool last) {
        const uint64_t b = b_desc0 + (uint64_t)(p.i * (C::STAGE >> 4));
        const uint32_t a = tmem + C::COL_A + (uint32_t)ap.i * 64u;
        const uint32_t d = tmem + (uint32_t)(tp.i * BM);
        if (elect_one()) {
#pragma unroll
          for (int j = 0; j < G / 16; ++j) {
            const int k16 = gi * (G / 16) + j;  // of the stage's 8: tile k16 / 4, 32 bytes each
            mma_ts(d, a + (uint32_t)k16 * 8u, b + (uint64_t)((k16 >> 2) * (BM * 128 >> 4) + (k16 & 3) * 2), idesc,
                   j > 0 ? 1u : 0u);
          }
          tc_commit(&ctrl->tfull[tp.i]);
          if (last) tc_commit(&ctrl->empty[p.i]);
        }
        __syncwarp();
        tp.next(C::TBUF);
      };
      auto buffer_wait = [&]() {
        const bool in = mbar_wait(&ctrl->tempty[tp.i], tp.phase ^ 1u, abort_flag, status, DEV_ERR_TIMEOUT_MMA);
        return !__any_sync(0xFFFFFFFFu, !in);
      };
      for (int tile = first_tile; ok && tile < tiles; tile += tile_step) {
        idesc = idesc_bf16(kBn, (find(tile).cnt + 15) & ~15);
        for (int ks = ks0; ks < ks1; ++ks) {
          const int count = min(kKs, g.k - ks * kKs) / G;  // groups of the stage
          if (!(ok = buffer_wait())) break;
          ok = mbar_wait(&ctrl->aready[ap.i], ap.phase, abort_flag, status, DEV_ERR_TIMEOUT_MMA);
          ok = !__any_sync(0xFFFFFFFFu, !ok);
          if (!ok) break;
          tc_fence_after();
#pragma unroll
          for (int gi = 0; gi < kKs / G; ++gi) {
            if (gi >= count) break;
            if (gi > 0) {
              if (!(ok = buffer_wait())) break;
              tc_fence_after();
            }
            group(gi, gi + 1 == count);
          }
          if (!ok) break;
          p.next(stages);
          ap.next(C::ASTAGES);
        }
      }
      // every MMA issued so far has completed once this commit arrives
      if (elect_one()) tc_commit(&ctrl->drain);
      wait_drain(&ctrl->drain, 0u);
      __syncwarp();
    }
  } else if (warp < kEpiWarp0) {
    setmaxnreg_dec<C::DEQ_REGS>();
    // ------------------------------------------------------------------ unpack
    // warp w: lanes 32 (w % 4).., K half (w - 4) / 4 of each stage
    const int q = warp & 3, half = (warp - kDeqWarp0) >> 2;
    const int row = q * 32 + lane;
    // the row's 64 bytes, this half's 32: 16-byte quarters under the 64-byte
    // swizzle
    const uint32_t roff = (uint32_t)(C::ACT + row * 64), rsw = (uint32_t)((row >> 1) & 3) * 16u;
    const uint32_t t_addr = tmem + ((uint32_t)(q * 32) << 16) + C::COL_A + (uint32_t)half * 32u;
    Pos p, ap, fp;  // stage, operand buffer, the stage whose MMAs free that buffer
    // The last stage whose stores are in flight: they are waited for, and
    // the stage handed on, once the next stage's codes have been read, so that
    // the stores' latency passes during the reads.
    int last_stage = -1, last_buf = 0;
    auto finish = [&]() {
      if (last_stage < 0) return;
      asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(&ctrl->aready[last_buf]);
        mbar_arrive(&ctrl->empty[last_stage]);
      }
      last_stage = -1;
    };
    uint32_t it = 0;
    bool ok = true;
    for (int tile = first_tile; ok && tile < tiles; tile += tile_step) {
      const uint8_t* zrow = nullptr;
      if (g.zero) {
        const TileAt t = find(tile);
        if (t.n0 + row < g.n) zrow = g.zero + ((size_t)t.e * g.n + t.n0 + row) * (size_t)groups;
      }
      // zero points of the half's two 32-element parts, as stored
      struct Zeros {
        uint8_t a, b;
      };
      auto zero_at = [&](int ks) {
        const int k0 = ks * kKs + half * 64;
        const int g0 = k0 / G, g1 = (k0 + 32) / G;
        Zeros z = {8, 8};
        if (zrow && g0 < groups) z.a = __ldg(zrow + g0);
        if (G == 32 && zrow && g1 < groups) z.b = __ldg(zrow + g1);
        return z;
      };
      // of this and the next two stages
      Zeros z0 = {8, 8}, z1 = {8, 8}, z2 = {8, 8};
      if (g.zero) {
        z0 = zero_at(ks0);
        z1 = zero_at(ks0 + 1);
        z2 = zero_at(ks0 + 2);
      }
      for (int ks = ks0; ks < ks1; ++ks, ++it) {
        uint32_t zc[2] = {kZero8, kZero8};
        if (g.zero) {
          zc[0] = zero_pair(z0.a);
          zc[1] = G == 32 ? zero_pair(z0.b) : zc[0];
          z0 = z1;
          z1 = z2;
          z2 = zero_at(ks + 3);
        }
        ok = mbar_wait(&ctrl->full[p.i], p.phase, abort_flag, status, DEV_ERR_TIMEOUT_PREP);
        if (__any_sync(0xFFFFFFFFu, !ok)) {
          ok = false;
          break;
        }
        const uint32_t raw = smem_u32(stage_ptr(p.i)) + roff;
        uint32_t w[2][4];
#pragma unroll
        for (int hk = 0; hk < 2; ++hk)
          asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];"
                       : "=r"(w[hk][0]), "=r"(w[hk][1]), "=r"(w[hk][2]), "=r"(w[hk][3])
                       : "r"(raw + ((uint32_t)(half * 32 + hk * 16) ^ rsw))
                       : "memory");
        finish();
        // the operand buffer is free once the MMAs of ASTAGES stages ago have
        // completed, which their stage's release says (this warp's own arrival
        // for that stage is long past, and the stage cannot be released again
        // before this warp reaches it)
        if (it >= (uint32_t)C::ASTAGES) {
          ok = mbar_wait(&ctrl->empty[fp.i], fp.phase, abort_flag, status, DEV_ERR_TIMEOUT_PREP);
          if (__any_sync(0xFFFFFFFFu, !ok)) {
            ok = false;
            break;
          }
          fp.next(stages);
        }
        tc_fence_after();
#pragma unroll
        for (int hk = 0; hk < 2; ++hk) {
          uint32_t v[16];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            // low and high nibbles of the four bytes; byte j of each makes a
            // pair of halves (a sign byte of `lo` is zero): the low nibble in
            // bits 0-3, the high one in bits 4-7.  Bits below 256 read as BF16
            // are that integer times 2^-133.
            const uint32_t lo = w[hk][i] & 0x0F0F0F0Fu, hi = w[hk][i] & 0xF0F0F0F0u;
#pragma unroll
            for (int j = 0; j < 4; ++j)
              v[i * 4 + j] =
                  fma_bf16x2(prmt(lo, hi, 0x8080u | (uint32_t)(j | (4 + j) << 8)), kLowHigh, zc[hk]);
          }
          tmem_st_x16(t_addr + (uint32_t)(ap.i * 64 + hk * 16), v);
        }
        last_stage = p.i;
        last_buf = ap.i;
        p.next(stages);
        ap.next(C::ASTAGES);
      }
    }
    finish();
  } else {
    setmaxnreg_inc<C::EPI_REGS>();
    // ---------------------------------------------------------------- epilogue
    const int q = warp & 3, h = (warp - kEpiWarp0) >> 2;
    const uint32_t tl = tmem + ((uint32_t)(q * 32) << 16) + (uint32_t)(h * C::COLS);
    constexpr int CH = C::CH, CW = C::CW;
    static_assert(C::COLS == CH * CW && CW % 16 == 0, "whole chunks");
    float2 acc[CH][CW / 2];
    Pos tp;
    bool ok = true;
    // scales of the next four groups of this thread's weight row, as stored (a
    // conversion here would wait for the load)
    uint16_t sq[4];
    const uint16_t* srow = nullptr;
    const int gi0 = ks0 * (kKs / G), gi1 = min(groups, ks1 * (kKs / G));
    bool met = false;
    auto scale_at = [&](int gi) -> uint16_t { return srow && gi < groups ? __ldg(srow + gi) : (uint16_t)0; };
    auto open_tile = [&](const TileAt& t) {
      const int n = t.n0 + q * 32 + lane;
      srow = n < g.n ? g.scale + ((size_t)t.e * g.n + n) * (size_t)groups : nullptr;
#pragma unroll
      for (int i = 0; i < 4; ++i) sq[i] = scale_at(gi0 + i);
    };
    TileAt t = {};
    if (first_tile < tiles) {
      t = find(first_tile);
      open_tile(t);
    }
    for (int tile = first_tile; ok && tile < tiles; tile += tile_step) {
#pragma unroll
      for (int c = 0; c < CH; ++c)
#pragma unroll
        for (int j = 0; j < CW / 2; ++j) acc[c][j] = make_float2(0.0f, 0.0f);
      for (int gi = gi0; gi < gi1; ++gi) {
        const float sc = scale_f32(sq[0], g.half_scale);
        const float2 s2 = make_float2(sc, sc);
        sq[0] = sq[1];
        sq[1] = sq[2];
        sq[2] = sq[3];
        sq[3] = scale_at(gi + 4);
        if (!mbar_wait(&ctrl->tfull[tp.i], tp.phase, abort_flag, status, DEV_ERR_TIMEOUT_EPI)) ok = false;
        if (__any_sync(0xFFFFFFFFu, !ok)) {
          ok = false;
          break;
        }
        tc_fence_after();
        const uint32_t tb = tl + (uint32_t)(tp.i * BM);
#pragma unroll
        for (int c = 0; c < CH; ++c) {
          uint32_t r[CW];
          tmem_ld_chunk(tb + (uint32_t)(CW * c), r);
          tc_wait_ld();
          regs_after_wait(r);
          if (c + 1 == CH) {  // the buffer is in registers: hand it back to the MMA
            tc_fence_before();
            mbar_arrive_lane0(&ctrl->tempty[tp.i], lane);
          }
#pragma unroll
          for (int j = 0; j < CW / 2; ++j)
            acc[c][j] =
                __ffma2_rn(make_float2(__uint_as_float(r[2 * j]), __uint_as_float(r[2 * j + 1])), s2, acc[c][j]);
        }
        tp.next(C::TBUF);
      }
      if (split > 1) {
        // The first CTA adds the others' sums, in their order, from its own
        // stages' memory, which nothing uses once all are here.  (A cluster has
        // one tile; after an abort too its CTAs meet.)
        met = true;
        constexpr uint32_t kPart = (uint32_t)BM * 128u * 4u;
        const uint32_t mine = (uint32_t)((h * C::COLS) * 128 + q * 32 + lane) * 4u;
        cluster_meet();
        if (rank > 0) {
          uint32_t at;
          asm volatile("mapa.shared::cluster.u32 %0, %1, 0;"
                       : "=r"(at)
                       : "r"(smem_u32(smem) + (uint32_t)(rank - 1) * kPart + mine));
#pragma unroll
          for (int c = 0; c < CH; ++c)
#pragma unroll
            for (int j = 0; j < CW; ++j)
              asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(at + (uint32_t)(c * CW + j) * 512u),
                           "f"((j & 1) ? acc[c][j >> 1].y : acc[c][j >> 1].x)
                           : "memory");
        }
        cluster_meet();
        if (rank > 0) break;
        for (int r = 0; r + 1 < split; ++r) {
          const float* part = reinterpret_cast<const float*>(smem + (size_t)r * kPart + mine);
#pragma unroll
          for (int c = 0; c < CH; ++c)
#pragma unroll
            for (int j = 0; j < CW / 2; ++j) {
              acc[c][j].x += part[(c * CW + 2 * j) * 128];
              acc[c][j].y += part[(c * CW + 2 * j + 1) * 128];
            }
        }
      }
      if (!ok) break;
      const TileAt now = t;
      if (tile + tile_step < tiles) {  // the next tile's scales are on their way during the stores
        t = find(tile + tile_step);
        open_tile(t);
      }
      const int n = now.n0 + q * 32 + lane;
      const int c0 = h * C::COLS;
      __nv_bfloat16* o = reinterpret_cast<__nv_bfloat16*>(g.out) + ((size_t)now.row0 + c0) * (size_t)g.n + n;
      if (n < g.n) {
#pragma unroll
        for (int c = 0; c < CH; ++c)
#pragma unroll
          for (int j = 0; j < CW; ++j) {
            const float v = (j & 1) ? acc[c][j >> 1].y : acc[c][j >> 1].x;
            if (c0 + c * CW + j < now.cnt) *o = __float2bfloat16_rn(64.0f * v);  // the codes were taken / 64
            asm volatile("add.s64 %0, %0, %1;" : "+l"(o) : "l"((long long)g.n * 2));
          }
      }
      __syncwarp();
      if (split > 1) break;
    }
    if (split > 1 && !met) {
      cluster_meet();
      cluster_meet();
    }
  }
  if (split > 1 && warp < kEpiWarp0) {  // with the epilogue's two meetings
    __syncwarp();
    cluster_meet();
    cluster_meet();
  }

  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tmem, kTmemCols);
}

// Rows of a, by index, in the order of the groups: 16 bytes per thread.  An
// index outside a gives a row of zeros; rows past the last group are left.  The
// last group ends where count_tiles lets it end, at the largest offset: one that
// falls stands for the one before it.  (Each warp reads all offsets, which costs
// nothing that shows: a call of 8192 rows of 4096 of 128 experts, 128 weight rows
// each, 46.4 us with and without, of 8192 rows of 256 of 1024 experts 29.3.)
__global__ void __launch_bounds__(256) w4g_gather_kernel(const uint4* __restrict__ a, const int32_t* __restrict__ rows,
                                                         const int32_t* __restrict__ offsets, uint4* __restrict__ out,
                                                         int rows_max, int a_rows, int experts, int cols) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  int last = 0;
#pragma unroll 4
  for (int e = 1 + (threadIdx.x & 31); e <= experts; e += 32) last = max(last, __ldg(offsets + e));
  last = __reduce_max_sync(0xFFFFFFFFu, last);
  const long long items = (long long)min(last, rows_max) * cols;
  const long long stride = (long long)gridDim.x * 256;
  for (long long i = (long long)blockIdx.x * 256 + threadIdx.x; i < items; i += 4 * stride) {
    uint4 v[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const long long at = i + u * stride;
      v[u] = make_uint4(0, 0, 0, 0);
      if (at < items) {
        const int r = (int)(at / cols);
        const int src = __ldg(rows + r);
        if (src >= 0 && src < a_rows) v[u] = __ldg(a + (size_t)src * cols + (size_t)(at - (long long)r * cols));
      }
    }
#pragma unroll
    for (int u = 0; u < 4; ++u)
      if (i + u * stride < items) out[i + u * stride] = v[u];
  }
}

template <int BM>
size_t smem_bytes(int stages, int experts) {
  return 1024 + (size_t)stages * Cfg<BM>::STAGE + sizeof(Ctrl) + 2 * sizeof(int) * ((size_t)experts + 1);
}

template <int BM>
int stage_count(int experts) {
  int s = kMaxStages;
  while (s > Cfg<BM>::ASTAGES + 1 && smem_bytes<BM>(s, experts) > kSmemMax) --s;
  return s;
}

std::mutex g_mu;

template <int BM, int G>
cudaError_t launch(const CUtensorMap& tm_q, const CUtensorMap& tm_a, const W4gArgs& g, const W4gGemmPlan& p,
                   int* status, cudaStream_t stream) {
  auto kern = w4g_gemm_kernel<BM, G>;
  static bool granted[64] = {};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  {
    std::lock_guard<std::mutex> lk(g_mu);
    if (!granted[dev]) {
      cudaFuncAttributes fa;
      if ((e = cudaFuncGetAttributes(&fa, kern)) != cudaSuccess) return e;
      // the register split assumes every thread starts with kLaunchRegs registers
      if (fa.numRegs < kLaunchRegs) return cudaErrorInvalidConfiguration;
      if ((e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmemMax)) != cudaSuccess)
        return e;
      granted[dev] = true;
    }
  }
  const int stages = stage_count<BM>(g.experts);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)p.grid);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem_bytes<BM>(stages, g.experts);
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = (unsigned)p.split;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = p.split > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kern, tm_q, tm_a, g, stages, p.split, status);
}

template <int BM>
cudaError_t launch_bm(const CUtensorMap& tm_q, const CUtensorMap& tm_a, const W4gArgs& g, const W4gGemmPlan& p,
                      int* status, cudaStream_t stream) {
  switch (g.group) {
    case 32: return launch<BM, 32>(tm_q, tm_a, g, p, status, stream);
    case 64: return launch<BM, 64>(tm_q, tm_a, g, p, status, stream);
    case 128: return launch<BM, 128>(tm_q, tm_a, g, p, status, stream);
    default: return cudaErrorInvalidValue;
  }
}

// Clusters of `split` CTAs that the current device runs at once: a cluster lies
// within one group of SMs, so that of 148 SMs 33 clusters of 4 and 15 of 8 were
// found to fit (one more takes a second wave: 4736 weight rows in 37 clusters of
// 4 16.0 us, 4224 in 33 9.2).
int cluster_room(int split) {
  static int room[64][9] = {};  // + 1
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 0;
  std::lock_guard<std::mutex> lk(g_mu);
  int& r = room[dev][split];
  if (r == 0) {
    auto kern = w4g_gemm_kernel<32, 128>;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)split);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = kSmemMax;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)split;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    int n = 0;
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmemMax) != cudaSuccess ||
        cudaOccupancyMaxActiveClusters(&n, kern, &cfg) != cudaSuccess) {
      cudaGetLastError();  // answered by not splitting
      n = 0;
    }
    r = n + 1;
  }
  return r - 1;
}

}  // namespace

W4gGemmPlan w4g_gemm_plan(const W4gArgs& g, int num_sms) {
  W4gGemmPlan p = {};
  const long long n_tiles = (g.n + kBn - 1) / kBn;
  // Time of a tile at K = 4096 by width and group (128, 64, 32), us: a 2048 x
  // 14336 x 4096 product divided by its waves of tiles.
  const int widths[4] = {192, 128, 64, 32};
  const double tile_us[3][4] = {{21.5, 16.7, 14.0, 13.5}, {25.5, 21.5, 17.1, 15.9}, {42.4, 35.2, 25.9, 24.1}};
  const double* us = tile_us[g.group == 128 ? 0 : g.group == 64 ? 1 : 2];
  const W4gSpread sp = w4g_spread(g);
  const int kstages = (g.k + kKs - 1) / kKs;
  p.split = 1;
  for (int i = 0; i < 4; ++i) {
    const double tiles = (double)n_tiles * sp.tiles(widths[i]);
    const auto cost = [&](int split) {
      return ceil(tiles * split / num_sms) * (0.6 + (us[i] - 0.6) * ((double)g.k / split / 4096.0));
    };
    if (i == 0 || cost(1) < p.us) {
      p.us = cost(1);
      p.bm = widths[i];
      p.split = 1;
    }
    // Few tiles of a dense product: clusters share their K, where it has work
    // for all, the first CTA's stages hold the others' sums and all clusters run
    // at once.  1.5: the two meetings and the sums.
    for (int split = 2; split <= 8 && !g.offsets; split *= 2) {
      if (tiles * split > num_sms || kstages < 4 * split || (split - 1) * widths[i] * 512 > kSumBytes ||
          tiles > cluster_room(split))
        break;
      const double us_split = cost(split) + 1.5;
      if (us_split < p.us) {
        p.us = us_split;
        p.bm = widths[i];
        p.split = split;
      }
    }
  }
  // the launch and the set-up (50 rows of 14336 x 4096, one wave of 13.5: 17.3),
  // and the copy of the rows
  p.us += g.rows ? 5.5 : 3.0;
  // of any grouping: each expert's last tile may be ragged
  const long long most =
      n_tiles * ((g.rows_max < g.experts ? g.rows_max : (long long)g.experts) + g.rows_max / p.bm);
  p.grid = (int)(most < num_sms ? most : num_sms);
  if (p.split > 1) p.grid = p.split * (int)(n_tiles * ((g.rows_max + p.bm - 1) / p.bm));
  return p;
}

cudaError_t launch_w4g_gather(const uint16_t* a, long long a_rows, const int32_t* rows, const int32_t* offsets,
                              int experts, uint16_t* out, long long rows_max, int k, cudaStream_t stream,
                              int num_sms) {
  const int cols = k / 8;
  const long long blocks = (rows_max * cols + 1023) / 1024;
  const long long cap = (long long)num_sms * 8;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(blocks < cap ? blocks : cap));
  cfg.blockDim = dim3(256);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, w4g_gather_kernel, reinterpret_cast<const uint4*>(a), rows, offsets,
                            reinterpret_cast<uint4*>(out), (int)rows_max, (int)a_rows, experts, cols);
}

cudaError_t launch_w4g_gemm(const CUtensorMap& tm_q, const CUtensorMap& tm_a, const W4gArgs& g, const W4gGemmPlan& p,
                            int* status, cudaStream_t stream) {
  switch (p.bm) {
    case 32: return launch_bm<32>(tm_q, tm_a, g, p, status, stream);
    case 64: return launch_bm<64>(tm_q, tm_a, g, p, status, stream);
    case 128: return launch_bm<128>(tm_q, tm_a, g, p, status, stream);
    case 192: return launch_bm<192>(tm_q, tm_a, g, p, status, stream);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace bsr
