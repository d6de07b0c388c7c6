// weight_stream.cuh -- the whole layer for a few tokens over bf16 weights in one persistent kernel:
// every SM streams expert weights from HBM without a pause across the up projection, the down
// projection and the combine (stream_common.cuh: units, waits, routing).
//
// The ring is filled by producer warps -- two for the weights, one for the token rows -- and emptied
// by 8 consumer warps that split K.
//
// The products run on mma.sync with the weights as the 16-row operand and 8 tokens as the other:
// at 8 tokens a tile the tensor work is a few percent of what the SM can do, and a warp that
// reads its fragments straight from the ring gives the slot back without an accumulator hand-over.
//
// A stage holds 32 weight rows x 256 columns; lane t of a row's four lanes takes 16-byte chunk 2t or
// 2t + 1 of each 64 columns, which the swizzle spreads over all banks (the order of K inside a
// block of 32 is free as long as both operands agree on it).
//
// Bound by HBM: 16 tokens stream 3.3 GB in 0.50 to 0.55 ms (0.92 to 1.0 of the copy rate), 1 token
// 285 MB in 63 us, of which routing is 10 and the combine 3.
#pragma once
#include <cuda.h>
#include <cuda_bf16.h>
#include <stdint.h>

#include <type_traits>

#include "stream_common.cuh"

namespace moe {

constexpr int kStreamWarps = 8;     // consumer warps: each an eighth of a stage's K
constexpr int kStreamEpiWarps = 4;  // sum the partials of a unit, store, publish
// weights (one warp for each half of a stage's rows), token rows, scheduler
constexpr int kStreamProdWarps = 4;
constexpr int kStreamAllWarps = kStreamWarps + kStreamProdWarps + kStreamEpiWarps;
constexpr int kStreamThreads = 32 * kStreamAllWarps;
constexpr int kRedSlots = 2;        // 8-token tiles of partial sums in flight

struct StreamParams {
  StreamBase b;
  CUtensorMap tm_g, tm_u, tm_d;  // weights
  __nv_bfloat16 *h;              // [P, f]
};

template <int NT>
struct StreamCfg {
  static constexpr int BT = 8 * NT;                      // tokens of a unit
  static constexpr int UP_ROWS = 16;                     // h columns of an up unit
  static constexpr int DOWN_ROWS = 2 * UP_ROWS;          // y columns of a down unit
  static constexpr int KS = 256;                         // K of a stage
  static constexpr int A_BYTES = 32 * 512;
  static constexpr int PITCH = 528;                      // bytes of a token row in a stage
  static constexpr int B_BYTES = BT * PITCH;
  static constexpr int STAGE_BYTES = A_BYTES + B_BYTES;
  static constexpr int MT = 2;                           // m tiles (16 rows) of a stage
  static constexpr int PARTS = kStreamWarps;             // partial sums of an output
  static constexpr int RP = 36;                          // pitch of a partial tile's token row
  static constexpr int RED_BYTES = kRedSlots * PARTS * 8 * RP * 4;
  static constexpr int FIXED = RED_BYTES + StreamTables::BYTES + 1024 /*barriers*/ + 1024;
  static constexpr int STAGES_RAW = (226 * 1024 - FIXED) / STAGE_BYTES;
  static constexpr int STAGES = STAGES_RAW > 16 ? 16 : STAGES_RAW;
  static_assert(STAGES >= 4, "pipeline too shallow");
  static_assert(DOWN_ROWS >= kStreamMinTile, "workspace holds the tile counts");
  static_assert(STAGES * STAGE_BYTES >= kRouteScratch, "the ring holds the routing's scratch");
  static constexpr size_t SMEM = FIXED + (size_t)STAGES * STAGE_BYTES;
};

// shared-memory loads by 32-bit address
__device__ __forceinline__ uint32_t lds32(uint32_t a) {
  uint32_t v;
  asm volatile("ld.shared.b32 %0, [%1];" : "=r"(v) : "r"(a));
  return v;
}
__device__ __forceinline__ float lds_f32(uint32_t a) { return __uint_as_float(lds32(a)); }
__device__ __forceinline__ uint4 lds128(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(a));
  return v;
}
__device__ __forceinline__ void sts_f32(uint32_t a, float v) {
  asm volatile("st.shared.f32 [%0], %1;" ::"r"(a), "f"(v) : "memory");
}

__device__ __forceinline__ void mma_bf16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

template <int NT>
__global__ void __launch_bounds__(kStreamThreads, 1)
    weight_stream_kernel(const __grid_constant__ StreamParams p) {
  using C = StreamCfg<NT>;
  constexpr int S = C::STAGES, BT = C::BT;
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint8_t *sA = smem;
  uint8_t *sB = sA + S * C::A_BYTES;
  float *red = reinterpret_cast<float *>(sB + S * C::B_BYTES);
  uint64_t *full = reinterpret_cast<uint64_t *>(reinterpret_cast<uint8_t *>(red) + C::RED_BYTES);
  uint64_t *empty = full + S;
  uint64_t *uq_full = empty + S;
  uint64_t *uq_empty = uq_full + kUnitQ;
  uint64_t *red_full = uq_empty + kUnitQ;
  uint64_t *red_empty = red_full + kRedSlots;
  Unit *uq = reinterpret_cast<Unit *>(red_empty + kRedSlots);  // [kUnitQ]
  volatile int *abort_flag = reinterpret_cast<volatile int *>(uq + kUnitQ);
  const StreamTables tb(reinterpret_cast<uint8_t *>(full) + 1024, p.b.E, p.b.n_shared);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int G = p.b.E + p.b.n_shared, Tk = p.b.T * p.b.k, d = p.b.d, f = p.b.f;
  const int nch_up = (d + C::KS - 1) / C::KS, nch_down = (f + C::KS - 1) / C::KS;
  const int up_tiles = f / C::UP_ROWS, down_tiles = d / C::DOWN_ROWS;
  const int n_rows = Tk + p.b.n_shared * p.b.T;

  if (threadIdx.x == 0) {
    for (int s = 0; s < S; ++s) {
      mbar_init(&full[s], 3);  // weights (two warps), token rows
      mbar_init(&empty[s], kStreamWarps);
    }
    for (int q = 0; q < kUnitQ; ++q) {
      mbar_init(&uq_full[q], 1);
      mbar_init(&uq_empty[q], kStreamAllWarps - 1);  // all but the scheduler
    }
    for (int i = 0; i < kRedSlots; ++i) {
      mbar_init(&red_full[i], kStreamWarps);
      mbar_init(&red_empty[i], kStreamEpiWarps / kRedSlots);
    }
    *abort_flag = 0;
    fence_mbar_init();
    tma_prefetch_desc(&p.tm_g);
    tma_prefetch_desc(&p.tm_u);
    tma_prefetch_desc(&p.tm_d);
  }
  __syncthreads();  // the abort flag is clear
  bool alive = route_tokens(p.b, tb, BT, G + 1 + down_tiles, smem, abort_flag);
  // the ring was the routing's scratch: its generic accesses precede the asynchronous copies
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  __syncthreads();

  // every lane polls; all of them see the phase, or the warp gives up
  auto warp_wait = [&](uint64_t *bar, uint32_t parity, int where) -> bool {
    return __all_sync(0xffffffffu, mbar_wait_suspend(bar, parity, abort_flag, p.b.status, where));
  };

  // the next unit of the queue (qi, qph: this role's cursor); false when a wait gave up
  int qi = 0;
  uint32_t qph = 0;
  auto next_unit = [&](Unit &w, int where) -> bool {
    if (!warp_wait(&uq_full[qi], qph, where)) return false;
    w = load_unit(&uq[qi]);
    __syncwarp();
    if (lane == 0) mbar_arrive(&uq_empty[qi]);
    if (++qi == kUnitQ) {
      qi = 0;
      qph ^= 1;
    }
    return true;
  };

  if (!alive) {
    // the grid barrier gave up: no unit is claimed
  } else if (warp == kStreamWarps || warp == kStreamWarps + 1) {
    // ---------------------------------------------------------------- weight producers
    // Warp 0 loads the first half of a stage's rows (gate, or the first rows of W_d), warp 1 the
    // other (up, or the next rows).
    const int half = __reduce_max_sync(0xffffffffu, warp) - kStreamWarps;
    const uint64_t pol_once = policy_evict_first(), pol_reuse = policy_evict_last();
    int st = 0, filled = 0;
    uint32_t ph = 0;
    bool ok = true;
    Unit w;
    while ((ok = next_unit(w, 45)) && w.kind >= 0) {
      const bool up = w.kind == 0;
      const int nch = up ? nch_up : nch_down;
      const int row = w.g * (up ? f : d) + w.mt * (up ? C::UP_ROWS : C::DOWN_ROWS) +
                      (up ? 0 : half * C::UP_ROWS);
      const uint64_t pol = w.uses == 1 ? pol_once : pol_reuse;
      const CUtensorMap *m = up ? (half ? &p.tm_u : &p.tm_g) : &p.tm_d;
      for (int kc = 0; kc < nch; ++kc) {
        ok = warp_wait(&empty[st], ph ^ 1, 32);
        if (!ok) break;
        if (elect_one()) {
          mbar_arrive_expect_tx(&full[st], C::A_BYTES / 2);
          // a half's four tiles of 64 columns in one load; those past K are zero
          tma_load_3d_hint(sA + st * C::A_BYTES + half * (C::A_BYTES / 2), m, &full[st], 0, row,
                           kc * 4, pol);
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
    if (!ok && lane == 0) drain_stages(full, filled, S);
    __syncwarp();
  } else if (warp == kStreamWarps + 2) {
    // ---------------------------------------------------------------- token-row producer
    // A lane copies 16 bytes of a row: a row of a stage is one or two copies by the warp.  The
    // copies of up to kRowsAhead stages are in flight; one lane announces a stage when they have
    // landed (32 arrivals, one a lane, cost more than the copies).  Nothing is held back while the
    // warp waits: it announces everything first.
    constexpr int kRowsAhead = 3;
    const int h_target = n_rows * up_tiles;
    bool all_ready = false;
    int st = 0, pending = 0;
    uint32_t ph = 0;
    Unit w;
    bool ok = true;
    auto announce = [&](int n) {  // the n oldest pending stages, whose copies have landed
      __syncwarp();
      if (lane == 0)
        for (int i = 0; i < n; ++i) {
          const int s = st - pending + i;
          mbar_arrive(&full[s < 0 ? s + S : s]);
        }
      pending -= n;
    };
    auto flush = [&]() {
      if (pending == 0) return;
      cp_async_wait<0>();
      announce(pending);
    };
    while (true) {
      if (!__all_sync(0xffffffffu, mbar_try_wait(&uq_full[qi], qph))) flush();
      ok = next_unit(w, 33);
      if (!ok || w.kind < 0) break;
      const bool up = w.kind == 0;
      if (!up && !all_ready) {
        flush();
        // lane 0 waits for the group's h; lane 1 looks whether all of h is there, after which
        // no unit asks again (each look costs an L2 round trip)
        int got = 1;
        if (lane == 0)
          got = counter_wait_bounded(p.b.done + w.g, w.rows * up_tiles, abort_flag,
                                     p.b.status, 34);
        if (lane == 1) got = counter_load(p.b.done_all) == h_target ? 2 : 1;
        ok = __shfl_sync(0xffffffffu, got, 0) != 0;
        if (!ok) break;
        all_ready = __shfl_sync(0xffffffffu, got, 1) == 2;
        __syncwarp();  // the other lanes' copies follow those two loads
      }
      const int K = up ? d : f, nch = up ? nch_up : nch_down;
      // row of x or h that lane i names for token i of the unit
      int my_row = w.row0 + lane;
      if (up && lane < w.n)
        my_row = w.g < p.b.E ? tb.perm[w.row0 + lane] / p.b.k : w.tok0 + lane;
      const uint8_t *base = reinterpret_cast<const uint8_t *>(up ? p.b.x : p.h) + lane * 16;
      for (int kc = 0; kc < nch; ++kc) {
        if (!__all_sync(0xffffffffu, mbar_try_wait(&empty[st], ph ^ 1))) {
          flush();
          ok = warp_wait(&empty[st], ph ^ 1, 35);
          if (!ok) break;
        }
        const int bytes = min(C::KS, K - kc * C::KS) * 2 - lane * 16;  // of a row, from this lane on
        const uint32_t dst = smem_u32(sB) + st * C::B_BYTES + lane * 16;
        for (int i = 0; i < w.n; ++i) {
          const uint8_t *src = base + ((size_t)__shfl_sync(0xffffffffu, my_row, i) * K +
                                       kc * C::KS) * 2;
          if (bytes > 0) cp_async16(dst + i * C::PITCH, src);
        }
        cp_async_commit();
        ++pending;
        if (++st == S) {
          st = 0;
          ph ^= 1;
        }
        if (pending == kRowsAhead) {
          cp_async_wait<kRowsAhead - 1>();
          announce(1);
        }
      }
    }
    flush();
  } else if (warp == kStreamWarps + 3) {
    // ---------------------------------------------------------------- scheduler
    if (lane == 0)
      schedule_units(p.b, tb, BT, up_tiles, down_tiles,
                     tickets_by_position(blockIdx.x, gridDim.x),
                     [&] { return atomicAdd(p.b.sched, 1); },
                     [&](const Unit &r) {
                       if (!mbar_wait_suspend(&uq_empty[qi], qph ^ 1, abort_flag, p.b.status, 31))
                         return false;
                       uq[qi] = r;
                       mbar_arrive(&uq_full[qi]);
                       if (++qi == kUnitQ) {
                         qi = 0;
                         qph ^= 1;
                       }
                       return true;
                     });
    __syncwarp();
  } else if (warp >= kStreamWarps + kStreamProdWarps) {
    // ---------------------------------------------------------------- epilogue
    // The warps of a slot share its tiles of partial sums (alternate tokens): add them in a fixed
    // order, free the slot, finish and publish the rows.  Every warp of a slot follows all the
    // slot's phases: one that skipped some could take an older phase for its own.
    const int my_slot = (warp - (kStreamWarps + kStreamProdWarps)) % kRedSlots;
    const int j0 = (warp - (kStreamWarps + kStreamProdWarps)) / kRedSlots;
    constexpr int JN = 8 * kRedSlots / kStreamEpiWarps;  // tokens of a tile for each warp
    constexpr int JS = kStreamEpiWarps / kRedSlots;
    int tile = 0;
    Unit w;
    bool ok = true;
    while (ok && next_unit(w, 42) && w.kind >= 0) {
      const bool up = w.kind == 0;
      for (int n0 = 0; n0 < w.n; n0 += 8, ++tile) {
        const int slot = tile % kRedSlots, n = min(8, w.n - n0);
        if (slot != my_slot) continue;
        // factor of each row, asked for before the wait: routed_scale * gate
        float sc[JN];
#pragma unroll
        for (int j = 0; j < JN; ++j)
          sc[j] = !up && w.g < p.b.E && j0 + j * JS < n
                      ? p.b.routed_scale * tb.gate[tb.perm[w.row0 + n0 + j0 + j * JS]]
                      : 1.f;
        ok = warp_wait(&red_full[slot], (tile / kRedSlots) & 1, 39);
        if (!ok) break;
        const uint32_t src = smem_u32(red) + (slot * C::PARTS * 8 * C::RP + lane) * 4;
        float v0[JN];
#pragma unroll
        for (int j = 0; j < JN; ++j) {
          v0[j] = 0.f;
          if (j0 + j * JS < n) {
#pragma unroll
            for (int i = 0; i < C::PARTS; ++i)
              v0[j] += lds_f32(src + (i * 8 + j0 + j * JS) * C::RP * 4);
          }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&red_empty[slot]);
#pragma unroll
        for (int j = 0; j < JN; ++j) {
          if (j0 + j * JS >= n) break;
          const size_t row = w.row0 + n0 + j0 + j * JS;
          if (up) {
            // lanes 0..15 gate, 16..31 up
            const float u = __shfl_down_sync(0xffffffffu, v0[j], 16);
            if (lane < 16)
              p.h[row * f + w.mt * 16 + lane] = __float2bfloat16_rn(swiglu(v0[j], u));
          } else {
            p.b.y[row * d + w.mt * C::DOWN_ROWS + lane] = v0[j] * sc[j];
          }
        }
        // publish: the warp's stores (made visible by lane 0's fence, after the warp's barrier),
        // then the count of its rows
        const int rows = (n - j0 + JS - 1) / JS;
        if (rows <= 0) continue;
        __syncwarp();
        if (lane == 0) {
          __threadfence();
          atomicAdd(up ? p.b.done + w.g : p.b.tile_done + w.mt, rows);
          if (up) atomicAdd(p.b.done_all, rows);
        }
      }
    }
  } else {
    // ---------------------------------------------------------------- consumers
    // Warp i takes block i of each 8 blocks of 32 along K, for all rows of the stage.
    const int gr = lane >> 2, t4 = lane & 3;
    // this lane's addresses within a stage
    const uint32_t a_lane = smem_u32(sA) + gr * 128 + (warp >> 1) * 2048 +
                            (((2 * t4 + (warp & 1)) ^ gr) << 4);
    const uint32_t b_lane =
        smem_u32(sB) + gr * C::PITCH + (warp >> 1) * 128 + (2 * t4 + (warp & 1)) * 16;
    const uint32_t red_lane = smem_u32(red) + ((warp * 8 + 2 * t4) * C::RP + gr) * 4;
    int st = 0, tile = 0;  // tile: tiles of partial sums so far
    uint32_t ph = 0;
    Unit w;
    while ((alive = next_unit(w, 36)) && w.kind >= 0) {
      const int K = w.kind == 0 ? d : f, nch = w.kind == 0 ? nch_up : nch_down, n_tok = w.n;
      float acc[NT][C::MT][4];  // m tiles of 16 rows
#pragma unroll
      for (int i = 0; i < NT * C::MT * 4; ++i) (&acc[0][0][0])[i] = 0.f;
      // the unit's stages; NA tiles of 8 tokens are in use
      auto stages = [&](auto tiles) {
        constexpr int NA = decltype(tiles)::value;
        for (int kc = 0; kc < nch; ++kc) {
          if (!warp_wait(&full[st], ph, 37)) return false;
          const uint32_t a = a_lane + st * C::A_BYTES, b = b_lane + st * C::B_BYTES;
          if (kc * 8 + warp < K / 32) {
            uint4 av[2][2];
#pragma unroll
            for (int m = 0; m < 2; ++m)
#pragma unroll
              for (int r = 0; r < 2; ++r) av[m][r] = lds128(a + m * 8192 + r * 1024);
#pragma unroll
            for (int n = 0; n < NA; ++n) {
              const uint4 bv = lds128(b + n * 8 * C::PITCH);
#pragma unroll
              for (int m = 0; m < 2; ++m)
                mma_bf16(acc[n][m], av[m][0].x, av[m][1].x, av[m][0].y, av[m][1].y, bv.x, bv.y);
#pragma unroll
              for (int m = 0; m < 2; ++m)
                mma_bf16(acc[n][m], av[m][0].z, av[m][1].z, av[m][0].w, av[m][1].w, bv.z, bv.w);
            }
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(&empty[st]);
          if (++st == S) {
            st = 0;
            ph ^= 1;
          }
        }
        return true;
      };
      using One = std::integral_constant<int, 1>;
      using All = std::integral_constant<int, NT>;
      const bool one = NT == 1 || n_tok <= 8;
      alive = one ? stages(One{}) : stages(All{});
      if (!alive) break;
      // the warps' partial sums meet in shared memory, a tile of 8 tokens at a time
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        if (n * 8 >= n_tok || !alive) break;
        const int slot = tile % kRedSlots;
        if (!warp_wait(&red_empty[slot], ((tile / kRedSlots) & 1) ^ 1, 38)) {
          alive = false;
          break;
        }
        ++tile;
        const uint32_t dst = red_lane + slot * (C::PARTS * 8 * C::RP * 4);
#pragma unroll
        for (int m = 0; m < C::MT; ++m)
#pragma unroll
          for (int i = 0; i < 4; ++i)
            sts_f32(dst + ((i & 1) * C::RP + m * 16 + (i >> 1) * 8) * 4, acc[n][m][i]);
        __syncwarp();
        if (lane == 0) mbar_arrive(&red_full[slot]);
      }
      if (!alive) break;
    }
    if (alive)
      combine_pieces(p.b, tb.slot, C::DOWN_ROWS, n_rows, warp, kStreamWarps, abort_flag);
  }
  __syncthreads();
  if (threadIdx.x == 0) leave_grid(p.b);
}

}  // namespace moe
