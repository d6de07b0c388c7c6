// weight_stream.cuh -- the experts of a few tokens in one persistent kernel: every SM streams
// expert weights (bf16 or MXFP4) from HBM without a pause across the up projection, the down
// projection and the combine; the one-launch layer (kRoute) also routes the tokens.
//
//   up    h[r, c]  = silu(x_r . W_g[e, c]) * (x_r . W_u[e, c])      row r of the sorted space
//   down  y[r, c]  = scale_r * (h_r . W_d[e, c])       scale_r = routed_scale * gate, shared 1
//   out[t]         = sum_j y[slot_row[t, j]] + y[shared row t]      fixed order, fp32, one rounding
//
// With one to sixteen tokens for each expert the layer is bound by the bytes of its weights, so
// the kernel is built around their stream: a ring of shared-memory stages is filled by two
// producer warps -- one for the weights, which depend on nothing but the routing and so run ahead
// through the up projection's end into the down projection, one for the token rows, which wait
// for h where they must -- and emptied by 16 consumer warps.  Work units (expert, weight rows,
// token tile) are claimed from a counter, all up units before the down units.
//
// The products run on mma.sync with the weights as the 16-row operand and 8 tokens as the other:
// at 8 tokens a tile the tensor work is a few percent of what the SM can do, and a weight that
// is a 4-bit code has to pass through registers anyway.  (tcgen05 takes bf16 operands from shared
// memory: every code would be converted, stored and read back.)
//
// MXFP4: a stage holds 64 weight rows x 256 codes (TMA boxes of 32 rows x 128 bytes, 128-byte
// swizzle) and their scales.  The order of K inside a block of 32 is free as long as both operands
// agree on it, so lane t of a row's four lanes takes codes 8t .. 8t + 7 of the block: one 32-bit
// word of shared memory, four hardware conversions to half pairs, two mma steps.  The products
// of a block are summed apart (fp32) and enter the accumulator times 2^(weight scale) * 2^(token
// scale).  The token rows are halves with a power-of-two scale for each 32 values
// (kActChunkBytes): the largest of a block lies in [2^14, 2^15), so a bf16 value loses nothing
// unless it is 2^-28 of its block's largest, and h keeps 11 bits.
// bf16: a stage holds 32 weight rows x 256 columns; lane t takes 16-byte chunk 2t or 2t + 1 of
// each 64 columns, which the swizzle spreads over all banks.
//
// Waiting: a down unit's token rows wait for counts of finished h rows, the combine for counts of
// finished y rows.  A unit is only ever claimed by a CTA that runs, and finishing it waits for
// up units alone (claimed before), so the waits end whatever the residency of the grid.  kRoute
// adds one barrier of the grid after the router's logits, so that kernel is a cooperative launch.
// All waits are bounded.
#pragma once
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <stdint.h>

#include "expert_simt.cuh"
#include "grouped_gemm.cuh"
#include "mxfp4.cuh"
#include "ptx_sm100.cuh"
#include "routing.cuh"

namespace moe {

constexpr int kStreamK = 256;       // K of a stage
constexpr int kStreamWarps = 16;    // consumer warps: two groups of 8 take stages in turn
constexpr int kStreamThreads = 32 * (kStreamWarps + 2);
constexpr int kStreamMaxT = 64;     // kRoute: tokens, (token, slot) pairs
constexpr int kStreamMaxPairs = 512;
constexpr int kStreamMinTile = 32;  // smallest d tile of a down unit (StreamCfg::DOWN_ROWS)
// block-scaled fp16 activations: chunks of 256 values, 512 bytes of halves then 8 fp32 scales
constexpr int kActChunkBytes = 512 + 32;
__host__ __device__ constexpr int act_chunks(int cols) { return (cols + 255) / 256; }

struct StreamParams {
  CUtensorMap tm_g, tm_u, tm_d;            // weights (MX: code bytes)
  const uint8_t *sc_g, *sc_u, *sc_d;       // MX: scales
  const __nv_bfloat16 *x;                  // [T, d]
  __nv_bfloat16 *out;                      // [T, d]
  uint8_t *xq, *hq;                        // MX: block-scaled x [T], h [P] (act_chunks a row)
  __nv_bfloat16 *h;                        // bf16: h [P, f]
  float *y;                                // [P, d]
  const int *offsets, *perm, *slot_row;    // routing (kRoute: made by the kernel itself)
  const float *gate;
  const __nv_bfloat16 *w_router;           // kRoute
  const float *bias;
  float *logits;                           // [T, E]
  int *done, *tile_done;                   // h rows x up tiles of a group; y rows of a d tile
  int *sched;                              // units claimed beyond the first of each CTA
  int *grid_bar;                           // kRoute: arrivals, departures
  DevStatus *status;
  int T, d, f, E, k, n_shared;
  float routed_scale;
};

template <bool kMx, int NT>
struct StreamCfg {
  static constexpr int BT = 8 * NT;                      // tokens of a unit
  static constexpr int UP_ROWS = kMx ? 32 : 16;          // h columns of an up unit
  static constexpr int DOWN_ROWS = 2 * UP_ROWS;          // y columns of a down unit
  static constexpr int A_BYTES = kMx ? 64 * 128 : 32 * 512;
  static constexpr int PITCH = kMx ? 576 : 528;          // bytes of a token row in a stage
  static constexpr int B_BYTES = BT * PITCH;
  static constexpr int S_BYTES = kMx ? 64 * 8 : 0;
  static constexpr int PARTS = kMx ? 8 : 16;             // partial sums of an output
  static constexpr int RP = kMx ? 68 : 36;               // pitch of a partial tile's token row
  static constexpr int RED_BYTES = NT * PARTS * 8 * RP * 4;
  static constexpr int FIXED = RED_BYTES + 12 * 1024 /*tables*/ + 1024 /*barriers*/ + 1024;
  static constexpr int STAGES_RAW = (226 * 1024 - FIXED) / (A_BYTES + B_BYTES + S_BYTES);
  static constexpr int STAGES = STAGES_RAW & ~1;  // even: a slot's group never changes
  static_assert(STAGES >= 4, "pipeline too shallow");
  static constexpr size_t SMEM = FIXED + (size_t)STAGES * (A_BYTES + B_BYTES + S_BYTES);
};

// Untiled copy of `bytes` (a multiple of 16) from global into shared memory.
__device__ __forceinline__ void bulk_load(void *dst, const void *src, uint32_t bytes,
                                          uint64_t *bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
          smem_u32(dst)),
      "l"(src), "r"(bytes), "r"(smem_u32(bar))
      : "memory");
}
__device__ __forceinline__ void cp_async4(void *dst, const void *src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(smem_u32(dst)), "l"(src)
               : "memory");
}
// one arrival on `bar` when this thread's cp.async copies so far have landed
__device__ __forceinline__ void cp_async_arrive(uint64_t *bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(bar))
               : "memory");
}

__device__ __forceinline__ void mma_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                        uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_bf16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Power-of-two scale of a block of activations from its largest magnitude (fp32 bits): 2^(e - 14)
// for a largest value in [2^e, 2^(e+1)), at least 2^-126; an infinity or NaN counts as the largest
// finite exponent (it stays itself).  Returns the exponent field of the scale.
__device__ __forceinline__ uint32_t act_scale_field(uint32_t amax_bits) {
  const uint32_t e = min(amax_bits >> 23, 254u);
  return e > 15u ? e - 14u : 1u;
}

// x [T, d] bf16 -> block-scaled halves (kActChunkBytes layout); thread i of n_threads.
__device__ __forceinline__ void convert_rows_block_scaled(const __nv_bfloat16 *x, int T, int d,
                                                          uint8_t *xq, size_t i0,
                                                          size_t n_threads) {
  const int lanes = d / kMxPerLane, nch = act_chunks(d);
  const size_t n = (size_t)T * lanes;  // a multiple of 16; whole blocks of four lanes
  for (size_t i = i0; i < ((n + 31) & ~(size_t)31); i += n_threads) {
    float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    if (i < n) load8(x + i * kMxPerLane, v);
    const uint32_t field = act_scale_field(block_amax_bits(v));
    if (i < n) {
      const float inv = __uint_as_float((254u - field) << 23);
      uint4 u;
      uint32_t *w = reinterpret_cast<uint32_t *>(&u);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const __half2 h = __floats2half2_rn(v[2 * j] * inv, v[2 * j + 1] * inv);
        w[j] = *reinterpret_cast<const uint32_t *>(&h);
      }
      const size_t t = i / lanes;
      const int c = (int)(i % lanes) * kMxPerLane;
      uint8_t *chunk = xq + (t * nch + (c >> 8)) * kActChunkBytes;
      *reinterpret_cast<uint4 *>(chunk + (c & 255) * 2) = u;
      if ((c & 31) == 0)
        *reinterpret_cast<float *>(chunk + 512 + ((c & 255) >> 5) * 4) =
            __uint_as_float(field << 23);
    }
  }
}

__global__ void __launch_bounds__(256) act_block_scale_kernel(const __nv_bfloat16 *x, int T,
                                                              int d, uint8_t *xq) {
  griddep_wait();
  griddep_launch_dependents();
  convert_rows_block_scaled(x, T, d, xq, (size_t)blockIdx.x * blockDim.x + threadIdx.x,
                            (size_t)gridDim.x * blockDim.x);
}

template <bool kMx, int NT, bool kRoute>
__global__ void __launch_bounds__(kStreamThreads, 1)
    weight_stream_kernel(const __grid_constant__ StreamParams p) {
  using C = StreamCfg<kMx, NT>;
  constexpr int S = C::STAGES, BT = C::BT;
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint8_t *sA = smem;
  uint8_t *sB = sA + S * C::A_BYTES;
  uint8_t *sS = sB + S * C::B_BYTES;
  float *red = reinterpret_cast<float *>(sS + S * C::S_BYTES);
  uint64_t *full = reinterpret_cast<uint64_t *>(reinterpret_cast<uint8_t *>(red) + C::RED_BYTES);
  uint64_t *full_b = full + S;
  uint64_t *empty = full_b + S;
  uint64_t *uq_full = empty + S;
  uint64_t *uq_empty = uq_full + kUnitQ;
  uint64_t *red_full = uq_empty + kUnitQ;
  uint64_t *red_empty = red_full + 1;
  volatile int *uq = reinterpret_cast<volatile int *>(red_empty + 1);  // [kUnitQ]
  volatile int *abort_flag = uq + kUnitQ;
  int *tables = reinterpret_cast<int *>(reinterpret_cast<uint8_t *>(full) + 1024);
  // group order: the shared expert first (known before the routing is), then the experts
  int *tile_prefix = tables;                                   // [G + 1] token tiles
  int *s_offsets = tile_prefix + (p.E + p.n_shared + 1);       // [E + 1]
  int *s_perm = s_offsets + (p.E + 1);                         // kRoute: [Tk]
  int *s_slot = s_perm + kStreamMaxPairs;                      // kRoute: [Tk]
  float *s_gate = reinterpret_cast<float *>(s_slot + kStreamMaxPairs);  // kRoute: [Tk]

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int G = p.E + p.n_shared, Tk = p.T * p.k;
  const int nch_up = (p.d + kStreamK - 1) / kStreamK, nch_down = (p.f + kStreamK - 1) / kStreamK;
  const int up_tiles = p.f / C::UP_ROWS, down_tiles = p.d / C::DOWN_ROWS;

  if (threadIdx.x == 0) {
    for (int s = 0; s < S; ++s) {
      mbar_init(&full[s], kMx ? 33 : 1);  // weights; MX: and each lane's scale copies
      mbar_init(&full_b[s], 1);           // token rows
      mbar_init(&empty[s], kStreamWarps / 2);
    }
    for (int q = 0; q < kUnitQ; ++q) {
      mbar_init(&uq_full[q], 1);
      mbar_init(&uq_empty[q], kStreamWarps + 1);  // the consumers and the token producer
    }
    mbar_init(red_full, kStreamWarps);
    mbar_init(red_empty, kStreamWarps);
    *abort_flag = 0;
    fence_mbar_init();
    tma_prefetch_desc(&p.tm_g);
    tma_prefetch_desc(&p.tm_u);
    tma_prefetch_desc(&p.tm_d);
  }
  const int *perm = kRoute ? s_perm : p.perm;
  const int *slot_row = kRoute ? s_slot : p.slot_row;
  const float *gate = kRoute ? s_gate : p.gate;
  bool alive = true;

  if (kRoute) {
    const int n_thr = gridDim.x * blockDim.x, thr = blockIdx.x * blockDim.x + threadIdx.x;
    for (int i = thr; i < G + down_tiles; i += n_thr) {  // done and tile_done
      if (i < G) p.done[i] = 0;
      else p.tile_done[i - G] = 0;
    }
    if (thr == 0) *p.sched = 0;
    if (kMx) convert_rows_block_scaled(p.x, p.T, p.d, p.xq, thr, n_thr);
    // router logits of two experts a CTA (16 warps), as the decode routing kernel's
    for (int e0 = blockIdx.x * kDecodeEPC; e0 < p.E; e0 += gridDim.x * kDecodeEPC) {
      uint4 wr[kDecodeMaxC][kDecodeEPC];
      decode_load_router_rows(p.w_router, e0, p.d, p.E, wr);
      decode_router_rows(p.x, e0, p.T, p.d, p.E, wr, p.logits, red);
    }
    __syncthreads();
    if (threadIdx.x == 0) {
      __threadfence();
      atomicAdd(p.grid_bar, 1);
      counter_wait_bounded(p.grid_bar, gridDim.x, abort_flag, p.status, 30);
      __threadfence();
    }
    __syncthreads();
    alive = *abort_flag == 0;
    // every CTA selects for all tokens itself: no second barrier
    int *s_idx = reinterpret_cast<int *>(red), *hist = s_idx + kStreamMaxPairs;
    uint32_t *bits = reinterpret_cast<uint32_t *>(hist + kDecodeMaxExperts);  // [E][2]
    int *warp_sum = reinterpret_cast<int *>(bits + 2 * kDecodeMaxExperts);
    for (int e = threadIdx.x; e < p.E; e += blockDim.x) {
      hist[e] = 0;
      bits[2 * e] = bits[2 * e + 1] = 0u;
    }
    __syncthreads();
    for (int t = warp; t < p.T; t += kStreamWarps + 2) {
      int my_e;
      float my_gate;
      topk_token<9>(p.logits + (size_t)t * p.E, p.bias, p.E, p.k, nullptr, lane, my_e, my_gate);
      if (lane < p.k) {
        s_idx[t * p.k + lane] = my_e;
        s_gate[t * p.k + lane] = my_gate;
        atomicAdd(&hist[my_e], 1);
        atomicOr(&bits[2 * my_e + (t >> 5)], 1u << (t & 31));
      }
    }
    __syncthreads();
    block_exclusive_scan(hist, s_offsets, p.E, warp_sum);
    if (threadIdx.x == 0) s_offsets[p.E] = Tk;
    for (int q = threadIdx.x; q < Tk; q += blockDim.x) {
      const int t = q / p.k, e = s_idx[q];
      int rank = __popc(bits[2 * e + (t >> 5)] & ((1u << (t & 31)) - 1u));
      if (t >= 32) rank += __popc(bits[2 * e]);
      const int row = s_offsets[e] + rank;
      s_perm[row] = q;
      s_slot[q] = row;
    }
  } else {
    griddep_wait();
    griddep_launch_dependents();
    for (int e = threadIdx.x; e <= p.E; e += blockDim.x) s_offsets[e] = p.offsets[e];
  }
  __syncthreads();
  auto group_at = [&](int o) { return p.n_shared ? (o == 0 ? p.E : o - 1) : o; };
  auto group_rows = [&](int g) { return g < p.E ? s_offsets[g + 1] - s_offsets[g] : p.T; };
  auto group_row0 = [&](int g) { return g < p.E ? s_offsets[g] : Tk; };
  if (warp == 0) {  // token tiles before each group
    const int per = (G + 31) / 32, lo = min(G, lane * per), hi = min(G, lo + per);
    int run = 0;
    for (int o = lo; o < hi; ++o) run += (group_rows(group_at(o)) + BT - 1) / BT;
    int incl = run;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += v;
    }
    int excl = incl - run;
    for (int o = lo; o < hi; ++o) {
      tile_prefix[o] = excl;
      excl += (group_rows(group_at(o)) + BT - 1) / BT;
    }
    if (lane == 31) tile_prefix[G] = incl;
  }
  __syncthreads();
  const int n_up = tile_prefix[G] * up_tiles, n_units = n_up + tile_prefix[G] * down_tiles;

  struct Unit {
    bool up;
    int g, mt, tok0, n, row0, uses;  // group, weight tile, first token, tokens, first sorted row
  };
  auto decode = [&](int u) {
    Unit r;
    r.up = u < n_up;
    const int tiles = r.up ? up_tiles : down_tiles;
    if (!r.up) u -= n_up;
    int lo = 0, hi = G - 1;
    while (lo < hi) {  // last group whose units start at or before u
      const int mid = (lo + hi + 1) >> 1;
      if (tile_prefix[mid] * tiles <= u) lo = mid;
      else hi = mid - 1;
    }
    r.g = group_at(lo);
    r.uses = tile_prefix[lo + 1] - tile_prefix[lo];
    const int loc = u - tile_prefix[lo] * tiles;
    r.mt = loc / r.uses;  // token tile innermost: its weights are read by neighbours in time
    r.tok0 = (loc - r.mt * r.uses) * BT;
    r.n = min(BT, group_rows(r.g) - r.tok0);
    r.row0 = group_row0(r.g) + r.tok0;
    return r;
  };
  // lane 0 polls, the warp follows
  auto warp_wait = [&](uint64_t *bar, uint32_t parity, int where) -> bool {
    if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
    int ok = 1;
    if (lane == 0) ok = mbar_wait_bounded(bar, parity, abort_flag, p.status, where) ? 1 : 0;
    ok = __shfl_sync(0xffffffffu, ok, 0);
    // the other lanes see the completed phase themselves
    return ok != 0 && __all_sync(0xffffffffu, mbar_try_wait(bar, parity));
  };

  if (!alive) {
    // the grid barrier gave up: no unit is claimed
  } else if (warp == kStreamWarps) {
    // ---------------------------------------------------------------- weight producer
    const uint64_t pol_once = policy_evict_first(), pol_reuse = policy_evict_last();
    int c = 0;  // stages filled so far
    int u = blockIdx.x, qi = 0;
    uint32_t qph = 0;
    bool ok = true;
    while (ok) {
      ok = warp_wait(&uq_empty[qi], qph ^ 1, 31);
      if (!ok) break;
      const int uid = u < n_units ? u : -1;
      if (lane == 0) {
        uq[qi] = uid;
        mbar_arrive(&uq_full[qi]);
      }
      if (++qi == kUnitQ) {
        qi = 0;
        qph ^= 1;
      }
      if (uid < 0) break;
      int next = 0;  // claimed while this unit's loads are issued
      if (lane == 0) next = atomicAdd(p.sched, 1) + gridDim.x;
      const Unit w = decode(uid);
      const int K = w.up ? p.d : p.f, nch = w.up ? nch_up : nch_down;
      const size_t m_rows = w.up ? p.f : p.d;
      const size_t row = (size_t)w.g * m_rows + (size_t)w.mt * (w.up ? C::UP_ROWS : C::DOWN_ROWS);
      const uint64_t pol = w.uses == 1 ? pol_once : pol_reuse;
      const CUtensorMap *m0 = w.up ? &p.tm_g : &p.tm_d, *m1 = w.up ? &p.tm_u : &p.tm_d;
      const int row1 = (int)row + (w.up ? 0 : C::UP_ROWS);  // rows of the second half
      for (int kc = 0; kc < nch; ++kc, ++c) {
        const int st = c % S;
        ok = warp_wait(&empty[st], ((c / S) & 1) ^ 1, 32);
        if (!ok) break;
        uint8_t *a = sA + st * C::A_BYTES;
        if (kMx) {
          if (lane == 0) {
            mbar_arrive_expect_tx(&full[st], C::A_BYTES);
            tma_load_2d_hint(a, m0, &full[st], kc * 128, (int)row, pol);
            tma_load_2d_hint(a + 4096, m1, &full[st], kc * 128, row1, pol);
          }
          // 64 rows x 8 scale bytes, in words (K / 32 is a multiple of 4)
          const uint8_t *s0 = w.up ? p.sc_g : p.sc_d, *s1 = w.up ? p.sc_u : p.sc_d;
          const size_t ld = K / kMxBlock;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int r = i * 16 + (lane >> 1), col = kc * 8 + (lane & 1) * 4;
            const uint8_t *src =
                r < 32 ? s0 + (row + r) * ld : s1 + ((size_t)row1 + (r - 32)) * ld;
            if (col < (int)ld) cp_async4(sS + st * C::S_BYTES + r * 8 + (lane & 1) * 4, src + col);
          }
          cp_async_arrive(&full[st]);
        } else if (lane == 0) {
          const int nb = min(4, (K - kc * kStreamK) / 64);  // boxes of 16 rows x 64 columns
          mbar_arrive_expect_tx(&full[st], nb * 4096);
          for (int j = 0; j < nb; ++j) {
            tma_load_2d_hint(a + j * 2048, m0, &full[st], kc * kStreamK + 64 * j, (int)row, pol);
            tma_load_2d_hint(a + 8192 + j * 2048, m1, &full[st], kc * kStreamK + 64 * j, row1,
                             pol);
          }
        }
      }
      u = __shfl_sync(0xffffffffu, next, 0);
    }
    if (!ok) {  // leave no copy in flight
      for (int i = max(0, c - S); i < c; ++i) {
        volatile int no_abort = 0;
        if (lane == 0) mbar_wait_bounded(&full[i % S], (i / S) & 1, &no_abort, nullptr, 0);
      }
      asm volatile("cp.async.wait_all;" ::: "memory");
    }
  } else if (warp == kStreamWarps + 1) {
    // ---------------------------------------------------------------- token-row producer
    int c = 0, qi = 0, ready = -1;
    uint32_t qph = 0;
    bool ok = true;
    while (ok) {
      ok = warp_wait(&uq_full[qi], qph, 33);
      if (!ok) break;
      const int uid = uq[qi];
      __syncwarp();
      if (lane == 0) mbar_arrive(&uq_empty[qi]);
      if (++qi == kUnitQ) {
        qi = 0;
        qph ^= 1;
      }
      if (uid < 0) break;
      const Unit w = decode(uid);
      if (!w.up && w.g != ready) {
        int got = 1;
        if (lane == 0)
          got = counter_wait_bounded(p.done + w.g, group_rows(w.g) * up_tiles, abort_flag,
                                     p.status, 34)
                    ? 1
                    : 0;
        ok = __shfl_sync(0xffffffffu, got, 0) != 0;
        if (!ok) break;
        ready = w.g;
      }
      __syncwarp();
      fence_proxy_async_global();  // the rows may be other CTAs' stores, read by bulk copies
      const int K = w.up ? p.d : p.f, nch = w.up ? nch_up : nch_down;
      const uint8_t *src = nullptr;  // lane i: token row i of the unit
      if (lane < w.n) {
        if (w.up) {
          const size_t t = w.g < p.E ? perm[w.row0 + lane] / p.k : w.tok0 + lane;
          src = kMx ? p.xq + t * nch * kActChunkBytes
                    : reinterpret_cast<const uint8_t *>(p.x + t * p.d);
        } else {
          const size_t r = w.row0 + lane;
          src = kMx ? p.hq + r * nch * kActChunkBytes
                    : reinterpret_cast<const uint8_t *>(p.h + r * p.f);
        }
      }
      for (int kc = 0; kc < nch; ++kc, ++c) {
        const int st = c % S;
        ok = warp_wait(&empty[st], ((c / S) & 1) ^ 1, 35);
        if (!ok) break;
        const uint32_t bytes = kMx ? kActChunkBytes : min(kStreamK, K - kc * kStreamK) * 2;
        if (lane == 0) mbar_arrive_expect_tx(&full_b[st], bytes * w.n);
        __syncwarp();
        if (lane < w.n)
          bulk_load(sB + st * C::B_BYTES + lane * C::PITCH,
                    src + (size_t)kc * (kMx ? kActChunkBytes : kStreamK * 2), bytes, &full_b[st]);
      }
    }
    if (!ok) {
      for (int i = max(0, c - S); i < c; ++i) {
        volatile int no_abort = 0;
        if (lane == 0) mbar_wait_bounded(&full_b[i % S], (i / S) & 1, &no_abort, nullptr, 0);
      }
    }
  } else {
    // ---------------------------------------------------------------- consumers
    const int grp = warp >> 3, w8 = warp & 7, gr = lane >> 2, t4 = lane & 3;
    // MX: m half (16 of each 32 rows) and K quarter of a stage; bf16: K eighth
    const int mh = kMx ? w8 >> 2 : 0, kq = kMx ? (w8 & 3) : w8;
    const int part = kMx ? grp * 4 + kq : grp * 8 + kq;
    int c = 0, qi = 0;
    uint32_t qph = 0, rph = 0;
    while (true) {
      if (!warp_wait(&uq_full[qi], qph, 36)) {
        alive = false;
        break;
      }
      const int uid = uq[qi];
      __syncwarp();
      if (lane == 0) mbar_arrive(&uq_empty[qi]);
      if (++qi == kUnitQ) {
        qi = 0;
        qph ^= 1;
      }
      if (uid < 0) break;
      const Unit w = decode(uid);
      const int K = w.up ? p.d : p.f, nch = w.up ? nch_up : nch_down;
      float acc[NT][2][4];
#pragma unroll
      for (int i = 0; i < NT * 8; ++i) (&acc[0][0][0])[i] = 0.f;
      for (int kc = 0; kc < nch; ++kc, ++c) {
        if ((c & 1) != grp) continue;
        const int st = c % S;
        if (!warp_wait(&full[st], (c / S) & 1, 37) || !warp_wait(&full_b[st], (c / S) & 1, 41)) {
          alive = false;
          break;
        }
        const uint8_t *a = sA + st * C::A_BYTES, *b = sB + st * C::B_BYTES;
        if (kMx) {
          if (kc * 8 + 2 * kq < K / kMxBlock) {
            float sw[2][2][2];  // [m][row, row + 8][block]
#pragma unroll
            for (int m = 0; m < 2; ++m)
#pragma unroll
              for (int r = 0; r < 2; ++r) {
                const uint32_t two = *reinterpret_cast<const uint16_t *>(
                    sS + st * C::S_BYTES + (m * 32 + mh * 16 + r * 8 + gr) * 8 + 2 * kq);
                const __nv_bfloat162_raw f =
                    __nv_cvt_e8m0x2_to_bf162raw(static_cast<__nv_fp8x2_storage_t>(two));
                sw[m][r][0] = __uint_as_float((uint32_t)f.x << 16);
                sw[m][r][1] = __uint_as_float((uint32_t)f.y << 16);
              }
            float2 sx[NT][2];  // tokens 2t, 2t + 1: both blocks
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
              for (int j = 0; j < 2; ++j)
                sx[n][j] = *reinterpret_cast<const float2 *>(
                    b + (n * 8 + 2 * t4 + j) * C::PITCH + 512 + 8 * kq);
#pragma unroll
            for (int bl = 0; bl < 2; ++bl) {
              const int blk = 2 * kq + bl;
              uint32_t av[2][2][4];  // [m][row, row + 8]: codes 8t .. 8t + 7 as half pairs
#pragma unroll
              for (int m = 0; m < 2; ++m)
#pragma unroll
                for (int r = 0; r < 2; ++r)
                  e2m1x8_to_half(*reinterpret_cast<const uint32_t *>(
                                     a + m * 4096 + (mh * 16 + r * 8 + gr) * 128 +
                                     ((blk ^ gr) << 4) + t4 * 4),
                                 av[m][r]);
#pragma unroll
              for (int n = 0; n < NT; ++n) {
                if (n * 8 >= w.n) break;
                const uint4 bv = *reinterpret_cast<const uint4 *>(b + (n * 8 + gr) * C::PITCH +
                                                                  blk * 64 + t4 * 16);
                const float s0 = bl ? sx[n][0].y : sx[n][0].x, s1 = bl ? sx[n][1].y : sx[n][1].x;
#pragma unroll
                for (int m = 0; m < 2; ++m) {
                  float t[4] = {0.f, 0.f, 0.f, 0.f};
                  mma_f16(t, av[m][0][0], av[m][1][0], av[m][0][1], av[m][1][1], bv.x, bv.y);
                  mma_f16(t, av[m][0][2], av[m][1][2], av[m][0][3], av[m][1][3], bv.z, bv.w);
                  acc[n][m][0] = fmaf(t[0], sw[m][0][bl] * s0, acc[n][m][0]);
                  acc[n][m][1] = fmaf(t[1], sw[m][0][bl] * s1, acc[n][m][1]);
                  acc[n][m][2] = fmaf(t[2], sw[m][1][bl] * s0, acc[n][m][2]);
                  acc[n][m][3] = fmaf(t[3], sw[m][1][bl] * s1, acc[n][m][3]);
                }
              }
            }
          }
        } else if (kc * 8 + kq < K / 32) {
          // the half of 64-column box kq / 2 whose 16-byte chunks are 2t + (kq & 1)
          const int box = kq >> 1, ch = 2 * t4 + (kq & 1);
          uint4 av[2][2];
#pragma unroll
          for (int m = 0; m < 2; ++m)
#pragma unroll
            for (int r = 0; r < 2; ++r)
              av[m][r] = *reinterpret_cast<const uint4 *>(a + m * 8192 + box * 2048 +
                                                          (r * 8 + gr) * 128 + ((ch ^ gr) << 4));
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            if (n * 8 >= w.n) break;
            const uint4 bv = *reinterpret_cast<const uint4 *>(b + (n * 8 + gr) * C::PITCH +
                                                              box * 128 + ch * 16);
#pragma unroll
            for (int m = 0; m < 2; ++m) {
              mma_bf16(acc[n][m], av[m][0].x, av[m][1].x, av[m][0].y, av[m][1].y, bv.x, bv.y);
              mma_bf16(acc[n][m], av[m][0].z, av[m][1].z, av[m][0].w, av[m][1].w, bv.z, bv.w);
            }
          }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&empty[st]);
      }
      if (!alive) break;
      // the warps' partial sums meet in shared memory; warp i then finishes token i of the unit
      if (!warp_wait(red_empty, rph ^ 1, 38)) {
        alive = false;
        break;
      }
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        if (n * 8 >= w.n) break;
#pragma unroll
        for (int m = 0; m < 2; ++m)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int tok = 2 * t4 + (i & 1);
            const int row = m * (kMx ? 32 : 16) + mh * 16 + (i >> 1) * 8 + gr;
            red[((n * C::PARTS + part) * 8 + tok) * C::RP + row] = acc[n][m][i];
          }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(red_full);
      if (!warp_wait(red_full, rph, 39)) {
        alive = false;
        break;
      }
      rph ^= 1;
      if (warp < w.n) {
        const float *src = red + ((size_t)(warp >> 3) * C::PARTS * 8 + (warp & 7)) * C::RP + lane;
        float v0 = 0.f, v1 = 0.f;
#pragma unroll
        for (int i = 0; i < C::PARTS; ++i) {
          v0 += src[i * 8 * C::RP];
          if (kMx) v1 += src[i * 8 * C::RP + 32];
        }
        const size_t row = w.row0 + warp;
        if (w.up) {
          if (kMx) {  // a block of 32 columns of h
            const float h = swiglu(v0, v1);
            uint32_t amax = __float_as_uint(h) & 0x7fffffffu;
            amax = __reduce_max_sync(0xffffffffu, amax);
            const uint32_t field = act_scale_field(amax);
            uint8_t *chunk = p.hq + (row * nch_down + (w.mt >> 3)) * kActChunkBytes;
            reinterpret_cast<__half *>(chunk)[(w.mt & 7) * 32 + lane] =
                __float2half_rn(h * __uint_as_float((254u - field) << 23));
            if (lane == 0)
              reinterpret_cast<float *>(chunk + 512)[w.mt & 7] = __uint_as_float(field << 23);
          } else {  // lanes 0..15 gate, 16..31 up
            const float u = __shfl_down_sync(0xffffffffu, v0, 16);
            if (lane < 16) p.h[row * p.f + w.mt * 16 + lane] = __float2bfloat16_rn(swiglu(v0, u));
          }
        } else {
          const float sc = w.g < p.E ? p.routed_scale * gate[perm[row]] : 1.f;
          float *y = p.y + row * p.d + w.mt * C::DOWN_ROWS + lane;
          y[0] = v0 * sc;
          if (kMx) y[32] = v1 * sc;
        }
        // publish: stores, then the count
        __threadfence();
        __syncwarp();
        if (lane == 0) {
          __threadfence();
          atomicAdd(w.up ? p.done + w.g : p.tile_done + w.mt, 1);
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(red_empty);
    }
    // ---------------------------------------------------------------- combine
    // Pieces of 128 output columns of a token, dealt to the warps of the grid.
    if (alive) {
      constexpr int TPP = 128 / C::DOWN_ROWS;  // d tiles of a piece
      const int n_rows = Tk + p.n_shared * p.T, per_tok = p.d / 128;
      for (int i = blockIdx.x + gridDim.x * warp; i < p.T * per_tok;
           i += gridDim.x * kStreamWarps) {
        const int t = i / per_tok, piece = i % per_tok;
        int ok = 1;
        if (lane < TPP)
          ok = counter_wait_bounded(p.tile_done + piece * TPP + lane, n_rows, abort_flag,
                                    p.status, 40)
                   ? 1
                   : 0;
        if (!__all_sync(0xffffffffu, ok)) break;
        const float *y = p.y + piece * 128 + lane * 4;
        float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int j0 = 0; j0 < p.k; j0 += 8) {  // eight rows in flight, added in slot order
          float4 v[8];
#pragma unroll
          for (int j = 0; j < 8; ++j)
            v[j] = j0 + j < p.k ? __ldcg(reinterpret_cast<const float4 *>(
                                      y + (size_t)slot_row[(size_t)t * p.k + j0 + j] * p.d))
                                : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
          for (int j = 0; j < 8; ++j)
            if (j0 + j < p.k) {
              s.x += v[j].x;
              s.y += v[j].y;
              s.z += v[j].z;
              s.w += v[j].w;
            }
        }
        if (p.n_shared) {
          const float4 v = __ldcg(reinterpret_cast<const float4 *>(y + (size_t)(Tk + t) * p.d));
          s.x += v.x;
          s.y += v.y;
          s.z += v.z;
          s.w += v.w;
        }
        store4(p.out + (size_t)t * p.d + piece * 128 + lane * 4, s);
      }
    }
  }
  if (kRoute) {
    // the last CTA to leave clears the barrier for the next launch
    __syncthreads();
    if (threadIdx.x == 0) {
      __threadfence();
      if (atomicAdd(p.grid_bar + 1, 1) == (int)gridDim.x - 1) {
        p.grid_bar[0] = 0;
        p.grid_bar[1] = 0;
        __threadfence();
      }
    }
  }
}

}  // namespace moe
