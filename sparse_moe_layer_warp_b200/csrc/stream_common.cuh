// stream_common.cuh -- what the persistent whole-layer kernels share (weight_stream.cuh: one launch,
// bf16 weights; mxfp4_layer.cuh: one launch, MXFP4 weights; mxfp4_pair.cuh: the experts of many
// tokens, MXFP4 weights): routing inside the kernel, the work units and their scheduler, the
// combine, suspended waits.
//
//   up    h[r, c]  = silu(x_r . W_g[e, c]) * (x_r . W_u[e, c])      row r of the sorted space
//   down  y[r, c]  = scale_r * (h_r . W_d[e, c])       scale_r = routed_scale * gate, shared 1
//   out[t]         = sum_j y[slot_row[t, j]] + y[shared row t]      fixed order, fp32, one rounding
//
// With a few tokens for each expert the layer is bound by the bytes of its weights, so these
// kernels are built around their stream: a ring of shared-memory stages is filled by producer
// warps -- weights, which depend on nothing but the routing and so run ahead through the up
// projection's end into the down projection, and token rows, which wait for h where they must.
// Work units (group, weight rows, token tile) are claimed from a counter, all up units before the
// down units.
//
// Waiting: a down unit's token rows wait for counts of finished h rows, the combine for counts of
// finished y rows.  Finishing a unit waits for up units alone, whose tickets are lower, and a CTA
// takes its own in order: these waits end if whoever owns an up unit runs.  The CTA pairs draw every
// ticket from the counter, so only a pair that runs owns any, whatever the residency of the grid.
// The one-launch layer has a barrier of the grid after the router's logits and is a cooperative launch
// for that: all its CTAs run at once, and each owns its first tickets by position.  All waits are
// bounded.
#pragma once
#include <cuda.h>
#include <cuda_bf16.h>
#include <stdint.h>

#include "expert_simt.cuh"
#include "grouped_gemm.cuh"
#include "ptx_sm100.cuh"
#include "routing.cuh"

namespace moe {

constexpr int kStreamMaxT = 64;       // one-launch layer: tokens, (token, slot) pairs
constexpr int kStreamMaxPairs = 512;
constexpr int kStreamMinTile = 32;    // smallest d tile of a down unit
// Units a CTA claims ahead of the one it hands out: a claim takes an L2 round trip under load
// (1.5 us measured, as long as a whole down unit takes)
constexpr int kClaimAhead = 3;
constexpr unsigned long long kDrainLimitNs = 10000000ull;  // copies in flight land in microseconds

struct StreamBase {
  const __nv_bfloat16 *x;                  // [T, d]
  __nv_bfloat16 *out;                      // [T, d]
  float *y;                                // [P, d]
  const int *offsets;                      // CTA pairs: [E + 1], from the routing kernels
  const __nv_bfloat16 *w_router;           // one-launch layer
  const float *bias;
  float *logits;                           // [T, E]
  int *done, *done_all, *tile_done;        // finished pieces of h of a group, of all groups; of y
                                           // of a d tile (zero at launch, or zeroed by the kernel)
  int *sched;                              // tickets drawn from the counter (Tickets)
  int *grid_bar;                           // one-launch layer: arrivals, departures
  DevStatus *status;
  int T, d, f, E, k, n_shared;
  float routed_scale;
};

// A unit of work: token rows [row0, row0 + n) of group g against weight tile mt.
struct Unit {
  int kind;  // 0 up, 1 down, -1 no more
  int g, mt, tok0, n, row0;
  int uses;  // token tiles of the group: how often its weights are read
  int rows;  // rows of the group
  int tile;  // number of the token tile (token_tile_number)
};

// A unit as the queue holds it, in uniform registers: every lane reads the same words, and the
// compiler knows it.  Producers and the MMA warp stay converged and let one elected lane issue: a
// copy or a tcgen05 operation whose operands are uniform issues in about 25 clocks, under
// `if (lane == 0)` in 70 to 130 -- two copies and a wait a stage then bound the whole kernel (760
// clocks a stage whatever its work).
__device__ __forceinline__ Unit load_unit(const Unit *q) {
  Unit w;
  const int *src = reinterpret_cast<const int *>(q);
  int *dst = reinterpret_cast<int *>(&w);
#pragma unroll
  for (int i = 0; i < (int)(sizeof(Unit) / sizeof(int)); ++i)
    dst[i] = __reduce_max_sync(0xffffffffu, src[i]);
  return w;
}

// Token tile i (of bt rows) of group g, whose first sorted row is off, has number off / bt + g + i:
// distinct for all tiles (a group of n rows moves the quotient by n / bt at least, rounded down,
// and g by one), below rows / bt + groups.
__host__ __device__ __forceinline__ int token_tile_number(int off, int g, int i, int bt) {
  return off / bt + g + i;
}

// mbar_wait_bounded with long suspended tries: a dozen warps that poll would take the issue
// slots of those that work.
template <bool kCluster = false>
__device__ __forceinline__ bool mbar_wait_suspend(uint64_t *bar, uint32_t parity,
                                                  volatile int *abort_flag, DevStatus *status,
                                                  int where,
                                                  unsigned long long limit_ns = kWaitLimitNs) {
  auto try_wait = [&]() {
    uint32_t ok;
    if (kCluster)  // arrivals and data from the other CTA of a pair
      asm volatile(
          "{\n\t.reg .pred p;\n\t"
          "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2, %3;\n\t"
          "selp.u32 %0, 1, 0, p;\n\t}"
          : "=r"(ok)
          : "r"(smem_u32(bar)), "r"(parity), "r"(20000u)  // ns
          : "memory");
    else
      asm volatile(
          "{\n\t.reg .pred p;\n\t"
          "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\t"
          "selp.u32 %0, 1, 0, p;\n\t}"
          : "=r"(ok)
          : "r"(smem_u32(bar)), "r"(parity), "r"(20000u)  // ns
          : "memory");
    return ok != 0;
  };
  if (try_wait()) return true;
  const unsigned long long t0 = globaltimer_ns();
  while (!try_wait()) {
    if (*abort_flag) return false;
    if (globaltimer_ns() - t0 > limit_ns) {
      *abort_flag = 1;
      if (status) {
        atomicExch(&status->error, 1);
        atomicExch(&status->where, where);
      }
      return false;
    }
  }
  return true;
}

// After a wait gave up: none of the last `filled` stages' copies is left in flight (bounded).
__device__ __forceinline__ void drain_stages(uint64_t *full, int filled, int stages) {
  for (int i = max(0, filled - stages); i < filled; ++i) {
    volatile int no_abort = 0;
    mbar_wait_bounded(&full[i % stages], (i / stages) & 1, &no_abort, nullptr, 0, kDrainLimitNs);
  }
}

__device__ __forceinline__ int counter_load(const int *ctr) {
  int v;
  asm volatile("ld.acquire.gpu.global.b32 %0, [%1];" : "=r"(v) : "l"(ctr) : "memory");
  return v;
}

__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src) {  // not through L1
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async4(uint32_t dst, const void *src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}
// This thread's arrival on `bar` once its cp.async so far have landed (one of the expected arrivals).
__device__ __forceinline__ void cp_async_arrive(uint64_t *bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(bar))
               : "memory");
}
__device__ __forceinline__ void mbar_arrive_n(uint64_t *bar, uint32_t n) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0], %1;" ::"r"(smem_u32(bar)), "r"(n)
               : "memory");
}
__device__ __forceinline__ void cp_async_commit() {
  asm volatile("cp.async.commit_group;" ::: "memory");
}
__device__ __forceinline__ void cp_async_wait_all() {
  asm volatile("cp.async.wait_all;" ::: "memory");
}
template <int N>
__device__ __forceinline__ void cp_async_wait() {  // all but the last N groups have landed
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// Shared-memory tables of the units, built by the whole CTA.  Group order: the shared expert
// first, then the experts.
struct StreamTables {
  int *tile_prefix;  // [G + 1] token tiles before each group
  int *offsets;      // [E + 1]
  int *perm, *slot;  // one-launch layer: [Tk]
  float *gate;
  __host__ __device__ __forceinline__ StreamTables(void *mem, int E, int n_shared) {
    tile_prefix = static_cast<int *>(mem);
    offsets = tile_prefix + (E + n_shared + 1);
    perm = offsets + (E + 1);
    slot = perm + kStreamMaxPairs;
    gate = reinterpret_cast<float *>(slot + kStreamMaxPairs);
  }
  // largest size: 1025 groups without, or 289 groups with the routing of 512 pairs (no more: at
  // 9 KB the smallest stages would not fit six times)
  static constexpr int BYTES = 17 * 512;
};
static_assert((2 * (kMaxExperts + 1) + 1) * 4 <= StreamTables::BYTES, "tables");
static_assert((2 * (kDecodeMaxExperts + 1) + 1 + 3 * kStreamMaxPairs) * 4 <= StreamTables::BYTES,
              "tables");

// Bytes of scratch that route_tokens needs.
constexpr int kRouteScratch =
    (kStreamMaxPairs + 3 * kDecodeMaxExperts + 32) * 4 > kDecodeWarps * 32 * 4
        ? (kStreamMaxPairs + 3 * kDecodeMaxExperts + 32) * 4
        : kDecodeWarps * 32 * 4;

// Routing of the one-launch layer, by the whole CTA (16 warps or more).  Zeroes the counters,
// computes the router's logits of two experts a CTA (the decode routing kernel's sums, so the
// selection is moe_route's), meets the other CTAs, then selects for all tokens itself: no second
// barrier.  Fills the tables, tile_prefix for token tiles of bt rows among them.  False when the
// barrier gave up.
__device__ __forceinline__ bool route_tokens(const StreamBase &p, const StreamTables &tb, int bt,
                                             int n_done, void *scratch,
                                             volatile int *abort_flag) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, n_warps = blockDim.x >> 5;
  const int n_thr = gridDim.x * blockDim.x, thr = blockIdx.x * blockDim.x + threadIdx.x;
  for (int i = thr; i < n_done; i += n_thr) p.done[i] = 0;  // done, done_all, tile_done
  if (thr == 0) *p.sched = 0;
  for (int e0 = blockIdx.x * kDecodeEPC; e0 < p.E; e0 += gridDim.x * kDecodeEPC) {
    uint4 wr[kDecodeMaxC][kDecodeEPC];
    decode_load_router_rows(p.w_router, e0, p.d, p.E, wr);
    decode_router_rows(p.x, e0, p.T, p.d, p.E, wr, p.logits, static_cast<float *>(scratch));
  }
  __syncthreads();
  if (threadIdx.x == 0) {
    __threadfence();
    atomicAdd(p.grid_bar, 1);
    counter_wait_bounded(p.grid_bar, gridDim.x, abort_flag, p.status, 30);
    __threadfence();
  }
  int *s_idx = static_cast<int *>(scratch), *hist = s_idx + kStreamMaxPairs;
  uint32_t *bits = reinterpret_cast<uint32_t *>(hist + kDecodeMaxExperts);  // [E][2] by token
  int *warp_sum = reinterpret_cast<int *>(bits + 2 * kDecodeMaxExperts);
  for (int e = threadIdx.x; e < p.E; e += blockDim.x) {
    hist[e] = 0;
    bits[2 * e] = bits[2 * e + 1] = 0u;
  }
  __syncthreads();
  if (*abort_flag) return false;
  for (int t = warp; t < p.T; t += n_warps) {
    int my_e;
    float my_gate;
    topk_token<9>(p.logits + (size_t)t * p.E, p.bias, p.E, p.k, nullptr, lane, my_e, my_gate);
    if (lane < p.k) {
      s_idx[t * p.k + lane] = my_e;
      tb.gate[t * p.k + lane] = my_gate;
      atomicAdd(&hist[my_e], 1);
      atomicOr(&bits[2 * my_e + (t >> 5)], 1u << (t & 31));
    }
  }
  __syncthreads();
  // one scan of rows (low half) and token tiles (high half): both sums stay below 2^10
  static_assert(kStreamMaxPairs < 65536, "halves of a word");
  for (int e = threadIdx.x; e < p.E; e += blockDim.x)
    hist[e] |= (hist[e] + bt - 1) / bt << 16;
  __syncthreads();
  block_exclusive_scan(hist, tb.offsets, p.E, warp_sum);
  const int s_tiles = p.n_shared ? (p.T + bt - 1) / bt : 0;  // the shared expert's come first
  for (int e = threadIdx.x; e < p.E; e += blockDim.x) {
    const int both = tb.offsets[e];
    tb.offsets[e] = both & 0xffff;
    tb.tile_prefix[e + p.n_shared] = (both >> 16) + s_tiles;
    if (e == p.E - 1) {
      tb.offsets[p.E] = p.T * p.k;
      tb.tile_prefix[p.E + p.n_shared] = ((both + hist[e]) >> 16) + s_tiles;
      if (p.n_shared) tb.tile_prefix[0] = 0;
    }
  }
  __syncthreads();
  for (int q = threadIdx.x; q < p.T * p.k; q += blockDim.x) {
    const int t = q / p.k, e = s_idx[q];
    int rank = __popc(bits[2 * e + (t >> 5)] & ((1u << (t & 31)) - 1u));
    if (t >= 32) rank += __popc(bits[2 * e]);
    const int row = tb.offsets[e] + rank;
    tb.perm[row] = q;
    tb.slot[q] = row;
  }
  return true;
}

__host__ __device__ __forceinline__ int group_at(const StreamBase &p, int o) {
  return p.n_shared ? (o == 0 ? p.E : o - 1) : o;
}
__host__ __device__ __forceinline__ int group_rows(const StreamBase &p, const StreamTables &tb, int g) {
  return g < p.E ? tb.offsets[g + 1] - tb.offsets[g] : p.T;
}

// tile_prefix for token tiles of bt rows from the offsets, by one warp.
__device__ __forceinline__ void build_tile_prefix(const StreamBase &p, const StreamTables &tb,
                                                  int bt) {
  const int lane = threadIdx.x & 31, G = p.E + p.n_shared;
  const int per = (G + 31) / 32, lo = min(G, lane * per), hi = min(G, lo + per);
  int run = 0;
  for (int o = lo; o < hi; ++o) run += (group_rows(p, tb, group_at(p, o)) + bt - 1) / bt;
  int incl = run;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += v;
  }
  int excl = incl - run;
  for (int o = lo; o < hi; ++o) {
    tb.tile_prefix[o] = excl;
    excl += (group_rows(p, tb, group_at(p, o)) + bt - 1) / bt;
  }
  if (lane == 31) tb.tile_prefix[G] = incl;
}

// The kClaimAhead tickets that a scheduler has in hand, as the counter gave them (nothing is computed
// from a claim before its turn: the thread would wait for the answer): ticket t is unit t + base.
struct Tickets {
  int t0, t1, t2, base;
};
static_assert(kClaimAhead == 3, "t0, t1, t2");
// All drawn from the counter, t0 by the caller before: a scheduler that does not run yet owns no unit.
// t2 is drawn once t1 has come, and t1 some time after t0, so that those who start together get units a
// round apart: with three draws in a row a third of the pairs took all the units of a small batch
// (200 tokens, 16 experts: 75 us, so drawn 60; 77 tokens of a small model 50, so drawn 46).
template <typename Claim>
__host__ __device__ __forceinline__ Tickets tickets_claimed(int t0, Claim claim) {
  Tickets k;
  k.t0 = t0;
  k.t1 = claim();
  k.t2 = k.t1 >= 0 ? claim() : 0;  // (no ticket is negative: this waits for t1)
  k.base = 0;
  return k;
}
// The first of scheduler `me` of n by position, which saves a round trip at the start.  Only where
// all n schedulers are sure to run at once: another's first units are not done by anyone else.
__host__ __device__ __forceinline__ Tickets tickets_by_position(int me, int n) {
  Tickets k;
  k.base = kClaimAhead * n;
  k.t0 = me - k.base;
  k.t1 = k.t0 + n;
  k.t2 = k.t1 + n;
  return k;
}

// The scheduler: one thread claims units until none is left and hands each, the end (kind -1) last,
// to publish(unit), which returns false when a wait gave up.  claim() draws the counter's next ticket.
template <typename Claim, typename Publish>
__host__ __device__ __forceinline__ void schedule_units(const StreamBase &p,
                                                        const StreamTables &tb, int bt,
                                                        int up_tiles, int down_tiles, Tickets k,
                                                        Claim claim, Publish publish) {
  const int G = p.E + p.n_shared, n_tiles = tb.tile_prefix[G];
  const int n_up = n_tiles * up_tiles, n_units = n_up + n_tiles * down_tiles;
  int pos = 0;  // group (in group order) of the last unit
  bool down = false;
  while (true) {
    int u = k.t0 + k.base;
    k.t0 = k.t1;
    k.t1 = k.t2;
    k.t2 = claim();
    Unit r;
    r.kind = u < n_up ? 0 : (u < n_units ? 1 : -1);
    if (r.kind >= 0) {
      // a scheduler's tickets only grow, so the group is found from the last one's on
      if (r.kind == 1) {
        u -= n_up;
        if (!down) pos = 0;
        down = true;
      }
      const int tiles = down ? down_tiles : up_tiles;
      // bisection: with few tokens most groups are empty, and stepping over 288 of them took 8 us
      if (tb.tile_prefix[pos + 1] * tiles <= u) {
        int last = G - 1;
        while (pos < last) {
          const int mid = (pos + last) >> 1;
          if (tb.tile_prefix[mid + 1] * tiles <= u) pos = mid + 1;
          else last = mid;
        }
      }
      r.g = group_at(p, pos);
      r.uses = tb.tile_prefix[pos + 1] - tb.tile_prefix[pos];
      const int loc = u - tb.tile_prefix[pos] * tiles;
      r.mt = loc / r.uses;  // token tile innermost: its weights are read by neighbours in time
      r.tok0 = (loc - r.mt * r.uses) * bt;
      r.rows = group_rows(p, tb, r.g);
      r.n = min(bt, r.rows - r.tok0);
      const int off = r.g < p.E ? tb.offsets[r.g] : p.T * p.k;
      r.row0 = off + r.tok0;
      r.tile = token_tile_number(off, r.g, r.tok0 / bt, bt);
    }
    if (!publish(r) || r.kind < 0) break;
  }
}

// Combine: pieces of 128 output columns of a token, dealt to the grid's combine warps (this one is
// `worker` of n_workers in its CTA).  A piece waits until every row of its d tile(s), tile_cols
// columns wide, is there: `target` pieces a tile.
__device__ __forceinline__ void combine_pieces(const StreamBase &p, const int *slot_row,
                                               int tile_cols, int target, int worker,
                                               int n_workers, volatile int *abort_flag) {
  const int lane = threadIdx.x & 31, Tk = p.T * p.k, per_tok = p.d / 128;
  const int tpp = tile_cols >= 128 ? 1 : 128 / tile_cols;  // d tiles of a piece
  for (long long i = blockIdx.x + (long long)gridDim.x * worker; i < (long long)p.T * per_tok;
       i += (long long)gridDim.x * n_workers) {
    const int t = (int)(i / per_tok), piece = (int)(i % per_tok);
    int ok = 1;
    if (lane < tpp)
      ok = counter_wait_bounded(p.tile_done + piece * 128 / tile_cols + lane, target, abort_flag,
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

// One-launch layer: the last CTA to leave clears the grid barrier for the next launch.  Called by
// one thread after its CTA's last use of it.
__device__ __forceinline__ void leave_grid(const StreamBase &p) {
  __threadfence();
  if (atomicAdd(p.grid_bar + 1, 1) == (int)gridDim.x - 1) {
    p.grid_bar[0] = 0;
    p.grid_bar[1] = 0;
    __threadfence();
  }
}

}  // namespace moe
