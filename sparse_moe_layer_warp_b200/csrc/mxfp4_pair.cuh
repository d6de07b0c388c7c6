// mxfp4_pair.cuh -- the experts over MXFP4 weights on CTA pairs (tcgen05 cta_group::2), for groups of
// many tokens.  Arithmetic, units and waits are mxfp4_layer.cuh's.
//
// What would bound one-CTA tiles there is shared memory: a stage of two 128-row weight tiles and 56
// tokens takes 448 clocks of tensor time, but its operands cross the 128 bytes a clock of shared
// memory for 830 (codes are one byte there; they are written by the copy, and read once for every
// 112 columns of N).  A pair runs M = 256, N = 224: a CTA's codes are read once for 112 tokens, and
// each CTA holds and reads only half of the token rows -- the hi rows in the leader, the lo rows in
// its peer.  A stage of 896 clocks then moves 106 KB, and the tensor cores bind (8192 tokens: 1.84
// to 1.88 ms alone, the tensor pipe 71 % active).  256 tokens stream 2.4 GB of weights in 0.39 to 0.40
// ms, 0.92 to 0.94 of the copy rate.
//
// CTA r of a pair holds weight rows [128 r, 128 r + 128) of each 256-row tile; a unit has two tiles
// (gate and up; two neighbours of W_d).  N follows the unit's tokens (2 x the next multiple of 8).
// TMEM: 2 x 224 accumulator columns (of 112-token tiles), so one unit at a time, and two sets of
// scales.  The scales of all N columns are needed by both CTAs, those of the weight rows by the CTA
// that holds them.
// The combine is a launch of its own: at these sizes y is larger than L2 and wants every warp.
#pragma once
#include <limits.h>

#include "mxfp4_layer.cuh"

namespace moe {

constexpr int kMxPairEpiWarps = 16;  // warps 0-15: four for each TMEM lane quadrant
// then MMA (two warps in the leader: one for each weight tile, as in mxfp4_layer.cuh; the first is the
// peer's scheduler), weights, token rows.  20 warps leave 96 registers a thread: the epilogue of
// 112-token tiles spills 40 bytes (none with 32).  A 21st warp would leave 80 and spill 116.
constexpr int kMxPairThreads = 32 * (kMxPairEpiWarps + 4);

struct MxPairParams {
  StreamBase b;
  CUtensorMap tm_g, tm_u, tm_d;      // codes, box {128, 128}, padded 4-bit
  CUtensorMap tm_sg, tm_su, tm_sd;   // their scale blocks as words, box {128, 1}
  CUtensorMap tm_x[3], tm_h[3];      // token rows, hi then lo [2 P, cols]: boxes of pair_box rows
  CUtensorMap tm_xs, tm_hs;          // scale blocks as words, box {128, blocks of a tile}
  SplitRows h;
  uint8_t *hs;
};

// Rows of the three token boxes: a tile of few tokens loads few rows.
template <int BN>
__host__ __device__ constexpr int pair_box(int i) {
  return i == 2 ? BN : (i == 1 ? BN / 2 : (BN > 32 ? 16 : 8));
}

// BN: token rows of a tile.  112 where the tensor cores bind.  32 where weights are streamed for a few
// rows of each expert: what counts is then the ring, five stages against four.
template <int kBN>
struct MxPairCfg {
  static constexpr int BN = kBN;
  static constexpr int A_BYTES = 2 * kMxTile * 128;
  static constexpr int B_BYTES = BN * 128;  // hi rows (leader) or lo rows (peer)
  static constexpr int SA_BYTES = 2 * kMxScaleBlock, SB_BYTES = scale_block_bytes(BN);
  static constexpr int STAGE_BYTES = A_BYTES + B_BYTES + SA_BYTES + SB_BYTES;
  static constexpr int TILE_COLS = 2 * BN, ACC_COLS = 2 * TILE_COLS;
  static constexpr int SF_COLS = 24;  // for each of the two MMA warps: weights 4, tokens 8
  static constexpr int TMEM_USED = ACC_COLS + 2 * SF_COLS;
  static constexpr int TMEM_COLS = TMEM_USED <= 128 ? 128 : 512;
  static_assert(TMEM_USED <= TMEM_COLS && BN % 16 == 0 && 2 * BN <= 256, "tile");
  static constexpr int FIXED = StreamTables::BYTES + 1024 /*barriers*/ + 1024 /*alignment*/;
  static constexpr int STAGES = (226 * 1024 - FIXED) / STAGE_BYTES;
  static_assert(STAGES >= 4 && B_BYTES % 1024 == 0, "pipeline");
  static constexpr size_t SMEM = FIXED + (size_t)STAGES * STAGE_BYTES;
};

__device__ __forceinline__ void tc_mma_mx_pair(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                               uint32_t sf_a, uint32_t sf_b, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::mxf8f6f4.block_scale [%0], %1, %2, %3, [%5], [%6], p;\n\t}" ::"r"(
          d),
      "l"(a), "l"(b), "r"(idesc), "r"(accumulate), "r"(sf_a), "r"(sf_b)
      : "memory");
}
// one scale block in each CTA of the pair, to the same TMEM columns of each
__device__ __forceinline__ void tc_cp_scales_pair(uint32_t taddr, uint32_t smem_addr) {
  asm volatile("tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;" ::"r"(taddr),
               "l"(scale_block_desc(smem_addr))
               : "memory");
}

template <int BN>
__global__ void __launch_bounds__(kMxPairThreads, 1)
    mxfp4_pair_kernel(const __grid_constant__ MxPairParams p) {
  using C = MxPairCfg<BN>;
  constexpr int S = C::STAGES;
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint8_t *sA = smem;                       // [S][2 tiles][128 rows][128 B]
  uint8_t *sB = sA + S * C::A_BYTES;        // [S][BN rows][128 B]
  uint8_t *sSA = sB + S * C::B_BYTES;       // [S][2][512]
  uint8_t *sSB = sSA + S * C::SA_BYTES;     // [S][1024] (32 rows: 512)
  uint64_t *full = reinterpret_cast<uint64_t *>(sSB + S * C::SB_BYTES);  // the leader's: both CTAs'
  uint64_t *empty = full + S;
  uint64_t *tfull = empty + S;
  uint64_t *tempty = tfull + 1;             // the leader's: both CTAs' epilogue warps
  uint64_t *uq_full = tempty + 1;
  uint64_t *uq_empty = uq_full + kUnitQ;    // the peer's: both CTAs' readers
  uint64_t *mma_end = uq_empty + kUnitQ;
  Unit *uq = reinterpret_cast<Unit *>(mma_end + 1);
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(uq + kUnitQ);
  volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);
  const StreamTables tb(reinterpret_cast<uint8_t *>(full) + 1024, p.b.E, p.b.n_shared);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();
  const bool leader = rank == 0;
  const int Tk = p.b.T * p.b.k, d = p.b.d, f = p.b.f;
  const int up_tiles = (f + 255) / 256, down_tiles = (d + 511) / 512;
  const int n_rows = Tk + p.b.n_shared * p.b.T;

  if (threadIdx.x == 0) {
    for (int s = 0; s < S; ++s) {
      mbar_init(&full[s], 2);  // the leader's two producer warps
      mbar_init(&empty[s], 2);  // MMA warps
    }
    mbar_init(tfull, 2);
    mbar_init(tempty, 2 * kMxPairEpiWarps);
    for (int q = 0; q < kUnitQ; ++q) {
      mbar_init(&uq_full[q], 1);
      mbar_init(&uq_empty[q], 2 * (kMxPairEpiWarps + 2) + 2);
    }
    mbar_init(mma_end, 2);
    *abort_flag = 0;
    fence_mbar_init();
    tma_prefetch_desc(&p.tm_g);
    tma_prefetch_desc(&p.tm_u);
    tma_prefetch_desc(&p.tm_d);
  }
  if (warp == kMxPairEpiWarps) tmem_alloc_pair(tmem_slot, C::TMEM_COLS);
  griddep_wait();
  griddep_launch_dependents();
  // The scheduler's first ticket, asked for here: its round trip passes behind the tables.  Pairs of
  // one grid need not run at once (another kernel may hold SMs), so none has units by position.
  auto claim = [&] { return atomicAdd(p.b.sched, 1); };
  int first_ticket = 0;
  if (warp == kMxPairEpiWarps && !leader && lane == 0) first_ticket = claim();
  for (int e = threadIdx.x; e <= p.b.E; e += blockDim.x) tb.offsets[e] = p.b.offsets[e];
  __syncthreads();
  if (warp == 0) build_tile_prefix(p.b, tb, BN);
  tc_fence_before();
  __syncthreads();
  cluster_sync();  // both CTAs' barriers are initialised, their TMEM allocated
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;

  auto warp_wait = [&](uint64_t *bar, uint32_t parity, int where) -> bool {
    return __all_sync(0xffffffffu, mbar_wait_suspend(bar, parity, abort_flag, p.b.status, where));
  };
  int qi = 0;
  uint32_t qph = 0;
  const uint32_t full_leader = mapa_shared(smem_u32(full), 0);
  const uint32_t uq_empty_peer = mapa_shared(smem_u32(uq_empty), 1);
  auto next_unit = [&](Unit &w, int where) -> bool {
    if (!__all_sync(0xffffffffu, mbar_wait_suspend<true>(&uq_full[qi], qph, abort_flag,
                                                         p.b.status, where)))
      return false;
    w = load_unit(&uq[qi]);
    // The arrival has no release (it would wait for the epilogue's stores in flight, 2500 clocks a
    // unit); its address depends on every word read, so it cannot pass the reads.
    const int all = w.kind | w.g | w.mt | w.tok0 | w.n | w.row0 | w.uses | w.rows | w.tile;
    const bool read = all != INT_MIN;
    if (lane == 0) mbar_arrive_remote_relaxed(uq_empty_peer + (read ? qi : 0) * 8);
    if (++qi == kUnitQ) {
      qi = 0;
      qph ^= 1;
    }
    return true;
  };
  // first row (of the group's weights) of tile j of a unit in CTA r
  auto tile_row = [&](const Unit &w, int j, int r) {
    return w.kind == 0 ? w.mt * 256 + r * kMxTile : w.mt * 512 + j * 256 + r * kMxTile;
  };
  bool alive = true;

  if (warp == kMxPairEpiWarps && !leader) {
    // ---------------------------------------------------------------- scheduler (peer)
    if (lane == 0)
      schedule_units(p.b, tb, BN, up_tiles, down_tiles,
                     tickets_claimed(first_ticket, claim), claim,
                     [&](const Unit &r) {
                       if (!mbar_wait_suspend<true>(&uq_empty[qi], qph ^ 1, abort_flag, p.b.status,
                                                    31))
                         return false;
                       uq[qi] = r;
                       const uint32_t to = mapa_shared(smem_u32(&uq[qi]), 0);
                       const int *v = reinterpret_cast<const int *>(&r);
#pragma unroll
                       for (int i = 0; i < (int)(sizeof(Unit) / 4); ++i)
                         st_shared_remote(to + 4 * i, v[i]);
                       mbar_arrive(&uq_full[qi]);
                       mbar_arrive_remote(mapa_shared(smem_u32(&uq_full[qi]), 0));
                       if (++qi == kUnitQ) {
                         qi = 0;
                         qph ^= 1;
                       }
                       return true;
                     });
    __syncwarp();
  } else if (warp == kMxPairEpiWarps + 2) {
    // ---------------------------------------------------------------- weights
    const uint64_t pol_once = policy_evict_first(), pol_reuse = policy_evict_last();
    int st = 0, filled = 0;
    uint32_t ph = 0;
    Unit w;
    bool ok = true;
    while ((ok = next_unit(w, 45)) && w.kind >= 0) {
      const bool up = w.kind == 0;
      const int nk = (up ? d : f) / 128, m_rows = up ? f : d, row = w.g * m_rows;
      const int row_a = tile_row(w, 0, rank), row_b = tile_row(w, 1, rank);
      int tiles = 0;  // of both CTAs
#pragma unroll
      for (int i = 0; i < 4; ++i) tiles += tile_row(w, i >> 1, i & 1) < m_rows;
      const CUtensorMap *ma = up ? &p.tm_g : &p.tm_d, *mb = up ? &p.tm_u : &p.tm_d;
      const CUtensorMap *sa = up ? &p.tm_sg : &p.tm_sd, *sb = up ? &p.tm_su : &p.tm_sd;
      const uint64_t pol = w.uses == 1 ? pol_once : pol_reuse;
      for (int kc = 0; kc < nk; ++kc) {
        ok = warp_wait(&empty[st], ph ^ 1, 32);
        if (!ok) break;
        if (elect_one()) {
          const uint32_t bar = full_leader + st * 8;
          uint8_t *a = sA + st * C::A_BYTES, *s = sSA + st * C::SA_BYTES;
          if (leader) mbar_arrive_expect_tx(&full[st], tiles * (kMxTile * 64 + kMxScaleBlock));
          if (row_a < m_rows) {
            tma_load_2d_pair(a, ma, bar, kc * 128, row + row_a, pol);
            tma_load_2d_pair(s, sa, bar, 0, (row + row_a) / kMxTile * nk + kc, pol);
          }
          if (row_b < m_rows) {
            tma_load_2d_pair(a + C::A_BYTES / 2, mb, bar, kc * 128, row + row_b, pol);
            tma_load_2d_pair(s + kMxScaleBlock, sb, bar, 0, (row + row_b) / kMxTile * nk + kc, pol);
          }
        }
        __syncwarp();
        ++filled;
        if (++st == S) {
          st = 0;
          ph ^= 1;
        }
      }
      if (!ok) break;
    }
    if (!ok && lane == 0 && leader) drain_stages(full, filled, S);
    __syncwarp();
  } else if (warp == kMxPairEpiWarps + 3) {
    // ---------------------------------------------------------------- token rows
    const int h_target = n_rows * up_tiles * 8;
    const uint64_t pol = policy_evict_last();
    bool all_ready = false;
    int st = 0, filled = 0;
    uint32_t ph = 0;
    Unit w;
    bool ok = true;
    while ((ok = next_unit(w, 33)) && w.kind >= 0) {
      const bool up = w.kind == 0;
      if (!up && !all_ready) {
        int got = 1;
        if (lane == 0)
          got = counter_wait_bounded(p.b.done + w.g, w.rows * up_tiles * 8, abort_flag, p.b.status,
                                     34);
        if (lane == 1) got = counter_load(p.b.done_all) == h_target ? 2 : 1;
        ok = __shfl_sync(0xffffffffu, got, 0) != 0;
        if (!ok) break;
        all_ready = __shfl_sync(0xffffffffu, got, 1) == 2;
        __syncwarp();  // the elected lane's copies follow those two loads
        fence_proxy_async_global();  // other CTAs' stores, read by TMA
      }
      const int nk = (up ? d : f) / 128, box = w.n <= pair_box<BN>(0) ? 0 : (w.n <= pair_box<BN>(1) ? 1 : 2);
      const CUtensorMap *m = up ? &p.tm_x[box] : &p.tm_h[box], *sc = up ? &p.tm_xs : &p.tm_hs;
      for (int kc = 0; kc < nk; ++kc) {
        ok = warp_wait(&empty[st], ph ^ 1, 35);
        if (!ok) break;
        if (elect_one()) {
          const uint32_t bar = full_leader + st * 8;
          if (leader)
            mbar_arrive_expect_tx(&full[st], 2 * (pair_box<BN>(box) * 128 + C::SB_BYTES));
          tma_load_2d_pair(sB + st * C::B_BYTES, m, bar, kc * 128, (int)rank * n_rows + w.row0,
                           pol);
          tma_load_2d_pair(sSB + st * C::SB_BYTES, sc, bar, 0,
                           (w.tile * nk + kc) * (C::SB_BYTES / kMxScaleBlock), pol);
        }
        __syncwarp();
        ++filled;
        if (++st == S) {
          st = 0;
          ph ^= 1;
        }
      }
      if (!ok) break;
    }
    if (!ok && lane == 0 && leader) drain_stages(full, filled, S);
    __syncwarp();
  } else if (warp == kMxPairEpiWarps || warp == kMxPairEpiWarps + 1) {
    // ---------------------------------------------------------------- MMA (leader)
    if (leader) {
      const int j = __reduce_max_sync(0xffffffffu, warp) - kMxPairEpiWarps;
      int st = 0, it = 0;
      uint32_t ph = 0;
      Unit w;
      const uint32_t tm = __reduce_max_sync(0xffffffffu, tmem_base), d0 = tm + j * C::TILE_COLS;
      const uint32_t a_base = smem_u32(sA) + j * (C::A_BYTES / 2), b_base = smem_u32(sB),
                     sa_base = smem_u32(sSA) + j * kMxScaleBlock, sb_base = smem_u32(sSB);
      while (next_unit(w, 36) && w.kind >= 0) {
        const int nk = (w.kind == 0 ? d : f) / 128, half = pair_lo_row(w.n);
        const bool there = tile_row(w, j, 0) < (w.kind == 0 ? f : d);
        const uint32_t id0 = idesc_mx(256, 2 * half);
        bool ok = warp_wait(tempty, (it & 1) ^ 1, 46), ready = false;
        ++it;
        for (int kc = 0; ok && kc < nk; ++kc) {
          if (!__all_sync(0xffffffffu, ready)) ok = warp_wait(&full[st], ph, 37);
          if (!ok) break;
          tc_fence_after();
          const int st1 = st + 1 == S ? 0 : st + 1;
          const uint32_t ph1 = st + 1 == S ? ph ^ 1 : ph;
          ready = kc + 1 < nk && mbar_test_wait(&full[st1], ph1);
          const uint32_t sf = tm + C::ACC_COLS + (kc & 1) * C::SF_COLS + j * (C::SF_COLS / 2);
          if (elect_one()) {
            if (there) {
              const uint32_t sb = sb_base + st * C::SB_BYTES;
              tc_cp_scales_pair(sf, sa_base + st * C::SA_BYTES);
              tc_cp_scales_pair(sf + 4, sb);
              if (BN > 64 && half > 64) tc_cp_scales_pair(sf + 8, sb + kMxScaleBlock);
              const uint64_t a = sdesc_k_sw128(a_base + st * C::A_BYTES),
                             b = sdesc_k_sw128(b_base + st * C::B_BYTES);
#pragma unroll
              for (int kk = 0; kk < 4; ++kk)
                tc_mma_mx_pair(d0, a + 2 * kk, b + 2 * kk,
                               id0 | ((uint32_t)kk << 4) | ((uint32_t)kk << 29), sf, sf + 4,
                               (kc | kk) ? 1u : 0u);
            }
            tc_commit_pair_both(&empty[st]);
            if (kc == nk - 1) tc_commit_pair_both(tfull);
          }
          __syncwarp();
          st = st1;
          ph = ph1;
        }
        if (!ok) break;
      }
      if (lane == 0) {
        tc_commit_pair_local(mma_end);
        volatile int no_abort = 0;
        mbar_wait_bounded(mma_end, 0, &no_abort, nullptr, 0);
      }
    }
    __syncwarp();
  } else if (warp < kMxPairEpiWarps) {
    // ---------------------------------------------------------------- epilogue
    // Chunks of 8 tokens, dealt to the four warps of a quadrant.  All of a unit's values are read
    // before the first is stored, and the accumulator goes back at once.  y is left without the
    // gates, which the combine applies: looking them up cost two dependent loads a unit here.
    constexpr int CH = (BN / 8 + 3) / 4;
    const int q = warp & 3, c0 = warp >> 2 << 3;
    const uint32_t tempty_leader = mapa_shared(smem_u32(tempty), 0);
    int it = 0;
    Unit w;
    while ((alive = next_unit(w, 42)) && w.kind >= 0) {
      const bool up = w.kind == 0;
      const int m_rows = up ? f : d, half = pair_lo_row(w.n);
      const int row_a = tile_row(w, 0, rank), row_b = tile_row(w, 1, rank);
      const bool one = row_a < m_rows, two = row_b < m_rows;
      alive = warp_wait(tfull, it & 1, 39);
      if (!alive) break;
      ++it;
      tc_fence_after();
      const uint32_t ta = tmem_base + ((uint32_t)(q * 32) << 16);
      float v0[CH][8], v1[CH][8];
#pragma unroll
      for (int i = 0; i < CH; ++i) {
        const int c = 32 * i + c0;
        if (c >= w.n || !one) continue;
        uint32_t r0[8], r1[8];
        tmem_ld8(ta + c, r0);
        tmem_ld8(ta + half + c, r1);
        tmem_ld_wait();
#pragma unroll
        for (int j = 0; j < 8; ++j) v0[i][j] = __uint_as_float(r0[j]) + __uint_as_float(r1[j]);
        if (!two) continue;
        tmem_ld8(ta + C::TILE_COLS + c, r0);
        tmem_ld8(ta + C::TILE_COLS + half + c, r1);
        tmem_ld_wait();
#pragma unroll
        for (int j = 0; j < 8; ++j) v1[i][j] = __uint_as_float(r0[j]) + __uint_as_float(r1[j]);
      }
      // the loads have completed (tcgen05.wait::ld); nothing else is handed over
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_remote_relaxed(tempty_leader);
      int count = 0;
#pragma unroll
      for (int i = 0; i < CH; ++i) {
        const int c = 32 * i + c0;
        if (c >= w.n) continue;
        count += min(8, w.n - c);
        if (!one) continue;
        if (up) {
#pragma unroll
          for (int j = 0; j < 8; ++j) v0[i][j] = swiglu(v0[i][j], v1[i][j]);
          store_h_chunk(p.h, p.hs + ((size_t)w.tile * (f / 128) + row_a / 128) * C::SB_BYTES, f,
                        w.row0, row_a + q * 32, c, w.n, half, q, lane, v0[i]);
        } else {
          float *y = p.b.y + (size_t)(w.row0 + c) * d + row_a + q * 32 + lane;
#pragma unroll
          for (int j = 0; j < 8; ++j)
            if (c + j < w.n) {
              y[(size_t)j * d] = v0[i][j];
              if (two) y[(size_t)j * d + 256] = v1[i][j];
            }
        }
      }
      __syncwarp();
      if (up && lane == 0) {
        __threadfence();
        atomicAdd(p.b.done + w.g, count);
        atomicAdd(p.b.done_all, count);
      }
    }
  }
  // the pair leaves together: the leader's MMAs read the peer's shared memory, and the peer's
  // copies signal the leader's barriers
  tc_fence_before();
  __syncthreads();
  cluster_sync();
  if (warp == kMxPairEpiWarps) {
    tc_fence_after();
    tmem_dealloc_pair(tmem_base, C::TMEM_COLS);
  }
}

// out[t] = sum_j routed_scale * gate[t, j] * y[slot_row[t, j]] + y[shared row t], in this order in
// fp32, one rounding.  Four columns a thread; bound by HBM (y is read once).
__global__ void __launch_bounds__(256)
    mxfp4_combine_kernel(const float *__restrict__ y, const int *__restrict__ slot_row,
                         const float *__restrict__ gate, float routed_scale, int T, int k,
                         int n_shared, int d, __nv_bfloat16 *__restrict__ out) {
  griddep_wait();
  griddep_launch_dependents();
  const int vpr = d / 4;
  const size_t n = (size_t)T * vpr, step = (size_t)gridDim.x * blockDim.x;
  for (size_t i = (size_t)blockIdx.x * blockDim.x + threadIdx.x; i < n; i += step) {
    const size_t t = i / vpr, c = i % vpr * 4;
    float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int j0 = 0; j0 < k; j0 += 8) {  // eight rows in flight, added in slot order
      float g[8];
      float4 v[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const bool in = j0 + j < k;
        g[j] = in ? routed_scale * __ldg(gate + t * k + j0 + j) : 0.f;
        v[j] = in ? __ldg(reinterpret_cast<const float4 *>(
                        y + (size_t)__ldg(slot_row + t * k + j0 + j) * d + c))
                  : make_float4(0.f, 0.f, 0.f, 0.f);
      }
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (j0 + j < k) {
          s.x = fmaf(g[j], v[j].x, s.x);
          s.y = fmaf(g[j], v[j].y, s.y);
          s.z = fmaf(g[j], v[j].z, s.z);
          s.w = fmaf(g[j], v[j].w, s.w);
        }
    }
    if (n_shared) {
      const float4 v = __ldg(reinterpret_cast<const float4 *>(y + ((size_t)T * k + t) * d + c));
      s.x += v.x;
      s.y += v.y;
      s.z += v.z;
      s.w += v.w;
    }
    store4(out + t * d + c, s);
  }
}

}  // namespace moe
