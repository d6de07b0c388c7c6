// mxfp4_layer.cuh -- the whole layer for a few tokens over MXFP4 weights in one persistent kernel on
// the block-scaled tensor cores (stream_common.cuh: units, waits, routing), and what it shares with
// the CTA-pair kernel for more tokens (mxfp4_pair.cuh).
//
// Arithmetic.  The weights' e2m1 codes and e8m0 scales go to tcgen05.mma (.kind::mxf8f6f4,
// .block_scale) as they are: no unpacking by the CUDA cores.  The other operand of that
// instruction has at most 8 bits, so an activation is the sum of two e4m3 values, hi = round(v) and
// lo = round(v - hi), each with one power-of-two scale for 32 neighbours (the largest of a block
// lies in [2^7, 2^8) of hi's scale; lo's scale is 2^-4 of hi's).  e4m3 keeps four bits, so hi + lo
// is a bf16 value exactly down to 2^-13 of its block's largest, and within 2^-21 of that largest
// below; h (fp32 from the SwiGLU) is held to 2^-9 of itself, as by a rounding to bf16.  hi and lo
// are separate columns of the N side; the epilogue adds the two fp32 accumulators.  N = 2 x tokens
// at twice the bf16 rate: the tensor time of bf16, at 17/64 of its weight bytes.
//
// A stage: 128 K of two tiles of 128 weight rows (gate and up; two neighbouring tiles of W_d), in
// shared memory one byte a code (the padded 4-bit TMA format: 8 bytes of codes, 8 of padding,
// whose transaction count is the bytes read), their scales, and the 2 x BN token rows with theirs.
// Scales are copied to TMEM by tcgen05.cp in the order of the instruction's scale layout: blocks of
// 512 bytes for 128 rows x 128 K, byte (r % 32) * 16 + r / 32 * 4 + k / 32.
//
// Bound at 16 tokens by the weight stream: 884 MB in 168 to 172 us, 0.79 of the copy rate (a stage of 17 KB
// of codes fills 33 KB of shared memory, so a ring of 5 or 6 stages holds 90 to 100 KB in flight;
// asking tiles into L2 ahead of their load made it 14 % slower).  At 1 token (37 us) by latency: 10 us
// of routing, 14 for up units of 32 stages, 6 for down units of 10, 3 for the combine.
#pragma once
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp8.h>
#include <stdint.h>

#include "mxfp4.cuh"
#include "stream_common.cuh"

namespace moe {

// 0-3 epilogue, 4-5 MMA, 6-7 weights, 8 token rows, 9 scheduler; all route, the others combine
constexpr int kMxWarps = 16;
constexpr int kMxThreads = 32 * kMxWarps;
constexpr int kMxTile = 128;  // weight rows of a tile: h columns of an up unit
constexpr int kMxDown = 2 * kMxTile;  // y columns of a down unit
constexpr int kMxScaleBlock = 512;

// Activations as hi and lo e4m3 values: hi [rows, cols], lo behind it.
struct SplitRows {
  uint8_t *hi, *lo;
};
__host__ __forceinline__ SplitRows split_rows(uint8_t *values, size_t rows, int cols) {
  return {values, values + rows * cols};
}

// Their scales come in blocks as the weights' do, one (or two, one behind the other, past 128 rows)
// for each token tile and 128 columns (token_tile_number): of a tile with n tokens, rows 0 .. n - 1
// are hi's; lo's begin at row BN, or on CTA pairs, whose N follows n, at the next multiple of 8.
__host__ __device__ constexpr int scale_block_bytes(int BN) {
  return (2 * BN + 127) / 128 * kMxScaleBlock;
}
__device__ __forceinline__ int pair_lo_row(int n) { return (n + 7) & ~7; }
__device__ __forceinline__ int scale_row_at(int r) {
  return (r >> 7) * kMxScaleBlock + (r & 31) * 16 + ((r >> 5) & 3) * 4;
}

struct MxParams {
  StreamBase b;
  CUtensorMap tm_g, tm_u, tm_d;              // codes, box {128, 128}, padded 4-bit
  CUtensorMap tm_h;                          // rows of h: box {128, BN, hi and lo}
  const uint8_t *sc_g, *sc_u, *sc_d;         // scale blocks (mxfp4_tile_scales_kernel)
  SplitRows x, h;                            // x: rows by token
  uint8_t *xs;                               // scale words of x by token and 128 columns
  uint8_t *hs;                               // scale blocks of h by token tile and 128 columns
};

template <int BN>
struct MxCfg {
  static constexpr int N = 2 * BN;                 // MMA N: hi rows, lo rows
  static constexpr int A_BYTES = 2 * kMxTile * 128;
  static constexpr int B_BYTES = N * 128;
  static constexpr int SA_BYTES = 2 * kMxScaleBlock, SB_BYTES = scale_block_bytes(BN);
  static constexpr int STAGE_BYTES = A_BYTES + B_BYTES + SA_BYTES + SB_BYTES;
  static constexpr int ACC_COLS = 2 * N;           // both weight tiles
  static constexpr int SF_COLS = 16;  // scale columns of a stage, 8 a weight tile; two sets in turn
  static constexpr int TMEM_USED = 2 * ACC_COLS + 2 * SF_COLS;
  static constexpr int TMEM_COLS = TMEM_USED <= 128 ? 128 : (TMEM_USED <= 256 ? 256 : 512);
  static_assert(TMEM_USED <= 512 && N % 16 == 0 && N <= 128 && B_BYTES % 1024 == 0, "tile");
  static constexpr int FIXED = StreamTables::BYTES + 1024 /*barriers*/ + 1024 /*alignment*/;
  static constexpr int STAGES_RAW = (226 * 1024 - FIXED) / STAGE_BYTES;
  static constexpr int STAGES = STAGES_RAW > 8 ? 8 : STAGES_RAW;
  static_assert(STAGES >= 3, "pipeline too shallow");
  static_assert(STAGES * STAGE_BYTES >= kRouteScratch, "the ring holds the routing's scratch");
  static constexpr size_t SMEM = FIXED + (size_t)STAGES * STAGE_BYTES;
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

// Instruction descriptor, .kind::mxf8f6f4: A e2m1 (5 at bits 7-9), B e4m3 (0 at 10-12), both
// K-major, N >> 3 at bits 17-22, e8m0 scales (bit 23), M >> 4 at bits 24-28; the byte of the scale
// words that a step uses (K block 0..3) at bits 4-5 (B) and 29-30 (A).
__device__ __forceinline__ constexpr uint32_t idesc_mx(int M, int N) {
  return (5u << 7) | ((uint32_t)(N >> 3) << 17) | (1u << 23) | ((uint32_t)(M >> 4) << 24);
}
__device__ __forceinline__ void tc_mma_mx(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                          uint32_t sf_a, uint32_t sf_b, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::mxf8f6f4.block_scale [%0], %1, %2, %3, [%5], [%6], p;\n\t}" ::"r"(
          d),
      "l"(a), "l"(b), "r"(idesc), "r"(accumulate), "r"(sf_a), "r"(sf_b)
      : "memory");
}
// One 512-byte scale block -> 4 TMEM columns of all four lane quadrants (rows of 16 bytes, groups
// of 8 rows 128 bytes apart, no swizzle).  Runs in order with the thread's MMAs.
__device__ __forceinline__ uint64_t scale_block_desc(uint32_t smem_addr) {
  return (uint64_t)((smem_addr >> 4) & 0x3FFFu) | (uint64_t)(128u >> 4) << 32 | (uint64_t)1u << 46;
}
__device__ __forceinline__ void tc_cp_scales(uint32_t taddr, uint32_t smem_addr) {
  asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(taddr),
               "l"(scale_block_desc(smem_addr))
               : "memory");
}
__device__ __forceinline__ void tmem_ld8(uint32_t taddr, uint32_t (&r)[8]) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]),
                 "=r"(r[6]), "=r"(r[7])
               : "r"(taddr)
               : "memory");
}

// Scale byte of hi for a block whose largest magnitude has these fp32 bits: the largest lies in
// [2^7, 2^8) of 2^(byte - 127).  lo's byte is 4 less (not below 0).
__device__ __forceinline__ uint32_t act_scale_byte(uint32_t amax_bits) {
  const uint32_t e = min(amax_bits >> 23, 254u);
  return e > 7u ? e - 7u : 0u;
}
// Two values of (up to) two blocks -> hi and lo byte pairs; s: the blocks' scale bytes.
__device__ __forceinline__ void split_pair(float a, float b, uint32_t sa, uint32_t sb, uint32_t &hi,
                                           uint32_t &lo) {
  // an infinity becomes NaN: e4m3 has none, and a finite stand-in would be a wrong answer
  a = fmaf(a, 0.f, a);
  b = fmaf(b, 0.f, b);
  a *= __uint_as_float((254u - sa) << 23);
  b *= __uint_as_float((254u - sb) << 23);
  uint16_t h, l;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(h) : "f"(b), "f"(a));
  uint32_t back;  // the pair as halves, exact
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(back) : "h"(h));
  const float2 r = __half22float2(*reinterpret_cast<const __half2 *>(&back));
  // lo's unit: 2^-4 of hi's, or the smallest scale there is
  const float ua = sa >= 4u ? 16.f : __uint_as_float((127u + sa) << 23);
  const float ub = sb >= 4u ? 16.f : __uint_as_float((127u + sb) << 23);
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(l) : "f"((b - r.y) * ub), "f"((a - r.x) * ua));
  hi = h;
  lo = l;
}
__device__ __forceinline__ uint32_t lo_scale_byte(uint32_t s) { return s > 4u ? s - 4u : 0u; }

// 16 neighbours a lane, two lanes a block, eight lanes a scale word: this lane's values as hi and lo
// bytes, and the four scale bytes of the eight lanes (valid in every lane).
__device__ __forceinline__ void split_lane(const float (&v)[16], uint4 &hi, uint4 &lo,
                                           uint32_t &s_hi, uint32_t &s_lo) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 16; ++i) m = max(m, __float_as_uint(v[i]) & 0x7fffffffu);
  const uint32_t s = act_scale_byte(max(m, __shfl_xor_sync(0xffffffffu, m, 1)));
  uint32_t h[8], l[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) split_pair(v[2 * j], v[2 * j + 1], s, s, h[j], l[j]);
  hi = make_uint4(h[0] | h[1] << 16, h[2] | h[3] << 16, h[4] | h[5] << 16, h[6] | h[7] << 16);
  lo = make_uint4(l[0] | l[1] << 16, l[2] | l[3] << 16, l[4] | l[5] << 16, l[6] | l[7] << 16);
  const int shift = (threadIdx.x & 6) * 4;  // block of this lane among the eight lanes' four
  s_hi = s << shift;
  s_lo = lo_scale_byte(s) << shift;
#pragma unroll
  for (int o = 2; o < 8; o <<= 1) {
    s_hi |= __shfl_xor_sync(0xffffffffu, s_hi, o);
    s_lo |= __shfl_xor_sync(0xffffffffu, s_lo, o);
  }
}
__device__ __forceinline__ void load16(const __nv_bfloat16 *p, float (&v)[16]) {
  float a[8], b[8];
  load8(p, a);
  load8(p + 8, b);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    v[i] = a[i];
    v[8 + i] = b[i];
  }
}

// 8 x 8 bytes across 8 neighbouring lanes: byte j of lane i (a: bytes 0-3, b: 4-7) becomes byte i of
// lane j.  Three exchanges of 32 bits.
__device__ __forceinline__ void transpose_bytes(uint32_t &a, uint32_t &b, int lane) {
  const bool u4 = lane & 4, u2 = lane & 2, u1 = lane & 1;
  uint32_t t = __shfl_xor_sync(0xffffffffu, u4 ? a : b, 4);
  if (u4) a = t;
  else b = t;
  // halves: lanes with bit 1 clear keep the low ones
  t = __shfl_xor_sync(0xffffffffu, __byte_perm(a, b, u2 ? 0x5410 : 0x7632), 2);
  a = __byte_perm(a, t, u2 ? 0x3254 : 0x5410);
  b = __byte_perm(b, t, u2 ? 0x3276 : 0x7610);
  // bytes: lanes with bit 0 clear keep bytes 0 and 2
  t = __shfl_xor_sync(0xffffffffu, __byte_perm(a, b, u1 ? 0x6420 : 0x7531), 1);
  a = __byte_perm(a, t, u1 ? 0x3514 : 0x5240);
  b = __byte_perm(b, t, u1 ? 0x3716 : 0x7260);
}

// Eight tokens (c .. c + 7 of a tile of n) x a warp's 32 columns of h (lane: column) as split values
// with the scale byte k of their rows: col the first column, hs the tile's scale block of these 128
// columns, lo0 the block's first lo row.  The bytes are transposed so that a lane stores 8
// neighbours of one token: as 16 one-byte stores a lane they took half of the up epilogue.
__device__ __forceinline__ void store_h_chunk(const SplitRows &h, uint8_t *hs, int f, int row0,
                                              int col, int c, int n, int lo0, int k, int lane,
                                              const float (&v)[8]) {
  uint32_t s[8], hi[4], lo[4];
#pragma unroll
  for (int j = 0; j < 8; ++j)
    s[j] = act_scale_byte(__reduce_max_sync(0xffffffffu, __float_as_uint(v[j]) & 0x7fffffffu));
#pragma unroll
  for (int j = 0; j < 4; ++j)
    split_pair(v[2 * j], v[2 * j + 1], s[2 * j], s[2 * j + 1], hi[j], lo[j]);
  uint32_t hi_a = hi[0] | hi[1] << 16, hi_b = hi[2] | hi[3] << 16;
  uint32_t lo_a = lo[0] | lo[1] << 16, lo_b = lo[2] | lo[3] << 16;
  transpose_bytes(hi_a, hi_b, lane);
  transpose_bytes(lo_a, lo_b, lane);
  // lanes t, 8 + t, 16 + t, 24 + t: token t.  Lane t also writes its hi scale, lane 8 + t its lo
  const int t = lane & 7, r = c + t;
  uint32_t mine = 0;
#pragma unroll
  for (int j = 0; j < 8; ++j)
    if (t == j) mine = s[j];
  if (r < n) {
    const size_t at = (size_t)(row0 + r) * f + col + (lane & 24);
    *reinterpret_cast<uint2 *>(h.hi + at) = make_uint2(hi_a, hi_b);
    *reinterpret_cast<uint2 *>(h.lo + at) = make_uint2(lo_a, lo_b);
    if (lane < 16)
      hs[scale_row_at(lane < 8 ? r : lo0 + r) + k] =
          (uint8_t)(lane < 8 ? mine : lo_scale_byte(mine));
  }
}

// x [T, d] -> the split rows of the sorted space with the scale blocks of CTA pairs' tiles of BN rows:
// token t to its k routed rows and its shared row.  One warp converts 512 columns of a token and
// stores them k + n_shared times; bound by HBM (2 d bytes read, 2 d (k + n_shared) written a token).
template <int BN>
__global__ void __launch_bounds__(256)
    split_rows_kernel(const __nv_bfloat16 *__restrict__ x, const int *__restrict__ slot_row,
                      const int *__restrict__ idx, const int *__restrict__ offsets, int T, int d,
                      int E, int k, int n_shared, SplitRows out, uint8_t *xs) {
  const int lane = threadIdx.x & 31, nk = d / 128, n_warps = gridDim.x * 8;
  const int chunks = (d + 511) / 512;
  griddep_wait();
  griddep_launch_dependents();
  for (long long item = blockIdx.x * 8 + (threadIdx.x >> 5); item < (long long)T * chunks;
       item += n_warps) {
    const int t = (int)(item / chunks), c = (int)(item % chunks) * 512 + lane * 16;
    float v[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) v[i] = 0.f;
    if (c < d) load16(x + (size_t)t * d + c, v);
    // lane j: row of slot j, its tile's number, its hi and lo rows in a block; the shared row (all 32
    // lanes may have slots) beside them
    auto place = [&](int g, int off, int rows, int row, int &tile, int &r, int &r_lo) {
      tile = token_tile_number(off, g, (row - off) / BN, BN);
      r = (row - off) % BN;
      r_lo = pair_lo_row(min(BN, rows - (row - off - r))) + r;
    };
    int row = 0, tile = 0, r = 0, r_lo = 0, s_tile, s_r, s_lo;
    if (lane < k) {
      const int g = idx[(size_t)t * k + lane], off = offsets[g];
      row = slot_row[(size_t)t * k + lane];
      place(g, off, offsets[g + 1] - off, row, tile, r, r_lo);
    }
    place(E, T * k, T, T * k + t, s_tile, s_r, s_lo);
    uint4 hi, lo;
    uint32_t w_hi, w_lo;  // scale words
    split_lane(v, hi, lo, w_hi, w_lo);
    for (int j = 0; j < k + n_shared; ++j) {
      const bool slot = j < k;
      const size_t rw = slot ? __shfl_sync(0xffffffffu, row, j) : T * k + t;
      const size_t tl = slot ? __shfl_sync(0xffffffffu, tile, j) : s_tile;
      const int rj = slot ? __shfl_sync(0xffffffffu, r, j) : s_r;
      const int lj = slot ? __shfl_sync(0xffffffffu, r_lo, j) : s_lo;
      if (c >= d) continue;
      *reinterpret_cast<uint4 *>(out.hi + rw * d + c) = hi;
      *reinterpret_cast<uint4 *>(out.lo + rw * d + c) = lo;
      if ((lane & 7) < 2)
        *reinterpret_cast<uint32_t *>(xs + (tl * nk + (c >> 7)) * scale_block_bytes(BN) +
                                      scale_row_at((lane & 1) ? lj : rj)) =
            (lane & 1) ? w_lo : w_hi;
    }
  }
}

template <int BN>
__global__ void __launch_bounds__(kMxThreads, 1)
    mxfp4_layer_kernel(const __grid_constant__ MxParams p) {
  using C = MxCfg<BN>;
  constexpr int S = C::STAGES, N = C::N;
  constexpr int kRowArrivals = 32;  // of the token rows' warp at a stage: one a lane
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint8_t *sA = smem;                       // [S][2 tiles][128 rows][128 B]
  uint8_t *sB = sA + S * C::A_BYTES;        // [S][hi rows, lo rows][128 B]
  uint8_t *sSA = sB + S * C::B_BYTES;       // [S][2][512]
  uint8_t *sSB = sSA + S * C::SA_BYTES;     // [S][512]
  uint64_t *full = reinterpret_cast<uint64_t *>(sSB + S * C::SB_BYTES);
  uint64_t *empty = full + S;
  uint64_t *tfull = empty + S;              // [2]
  uint64_t *tempty = tfull + 2;             // [2]
  uint64_t *uq_full = tempty + 2;
  uint64_t *uq_empty = uq_full + kUnitQ;
  uint64_t *mma_end = uq_empty + kUnitQ;    // all MMAs have completed
  Unit *uq = reinterpret_cast<Unit *>(mma_end + 1);
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(uq + kUnitQ);
  volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);
  StreamTables tb(reinterpret_cast<uint8_t *>(full) + 1024, p.b.E, p.b.n_shared);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int G = p.b.E + p.b.n_shared, Tk = p.b.T * p.b.k, d = p.b.d, f = p.b.f;
  const int up_tiles = f / kMxTile, down_tiles = (d + kMxDown - 1) / kMxDown;
  const int n_rows = Tk + p.b.n_shared * p.b.T;

  if (threadIdx.x == 0) {
    for (int s = 0; s < S; ++s) {
      mbar_init(&full[s], 2 + kRowArrivals);  // weights (two warps), token rows
      mbar_init(&empty[s], 2);  // MMA warps
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&tfull[i], 2);
      mbar_init(&tempty[i], 4);
    }
    for (int q = 0; q < kUnitQ; ++q) {
      mbar_init(&uq_full[q], 1);
      mbar_init(&uq_empty[q], 9);  // epilogue 4, MMA 2, weights 2, token rows
    }
    mbar_init(mma_end, 2);
    *abort_flag = 0;
    fence_mbar_init();
    tma_prefetch_desc(&p.tm_g);
    tma_prefetch_desc(&p.tm_u);
    tma_prefetch_desc(&p.tm_d);
  }
  if (warp == 4) tmem_alloc(tmem_slot, C::TMEM_COLS);
  __syncthreads();  // the abort flag is clear
  // split x by token, then route; the ring's memory is the scratch
  {
    const int nk = d / 128, chunks = (d + 511) / 512, n_warps = gridDim.x * kMxWarps;
    for (int i = blockIdx.x * kMxWarps + warp; i < p.b.T * chunks; i += n_warps) {
      const int t = i / chunks, c = (i % chunks) * 512 + lane * 16;
      float v[16];
#pragma unroll
      for (int j = 0; j < 16; ++j) v[j] = 0.f;
      if (c < d) load16(p.b.x + (size_t)t * d + c, v);
      uint4 hi, lo;
      uint32_t s_hi, s_lo;
      split_lane(v, hi, lo, s_hi, s_lo);
      if (c >= d) continue;
      *reinterpret_cast<uint4 *>(p.x.hi + (size_t)t * d + c) = hi;
      *reinterpret_cast<uint4 *>(p.x.lo + (size_t)t * d + c) = lo;
      if ((lane & 7) == 0)
        *reinterpret_cast<uint2 *>(p.xs + ((size_t)t * nk + (c >> 7)) * 8) =
            make_uint2(s_hi, s_lo);
    }
  }
  bool alive = route_tokens(p.b, tb, BN, G + 1 + down_tiles, smem, abort_flag);
  // the ring was the routing's scratch: its generic accesses precede the asynchronous copies
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;

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
  } else if (warp == 9) {
    if (lane == 0)
      schedule_units(p.b, tb, BN, up_tiles, down_tiles,
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
  } else if (warp == 6 || warp == 7) {
    // ---------------------------------------------------------------- weights
    // One warp for each of a stage's two tiles.
    const int half = __reduce_max_sync(0xffffffffu, warp) - 6;
    const uint64_t pol_once = policy_evict_first(), pol_reuse = policy_evict_last();
    int st = 0, filled = 0;
    uint32_t ph = 0;
    Unit w;
    bool ok = true;
    while ((ok = next_unit(w, 45)) && w.kind >= 0) {
      const bool up = w.kind == 0;
      const int nk = (up ? d : f) / 128, m_rows = up ? f : d;
      const int tile = up ? w.mt : 2 * w.mt + half;
      const bool there = tile * kMxTile < m_rows;  // d may be an odd number of tiles
      const int row = w.g * m_rows + tile * kMxTile;
      const CUtensorMap *m = up ? (half ? &p.tm_u : &p.tm_g) : &p.tm_d;
      const uint8_t *sc = (up ? (half ? p.sc_u : p.sc_g) : p.sc_d) +
                          (size_t)(row / kMxTile) * nk * kMxScaleBlock;
      const uint64_t pol = w.uses == 1 ? pol_once : pol_reuse;
      for (int kc = 0; kc < nk; ++kc) {
        ok = warp_wait(&empty[st], ph ^ 1, 32);
        if (!ok) break;
        if (elect_one()) {
          if (there) {
            mbar_arrive_expect_tx(&full[st], kMxTile * 64 + kMxScaleBlock);
            tma_load_2d_hint(sA + st * C::A_BYTES + half * (C::A_BYTES / 2), m, &full[st],
                             kc * 128, row, pol);
            bulk_load(sSA + st * C::SA_BYTES + half * kMxScaleBlock, sc + kc * kMxScaleBlock,
                      kMxScaleBlock, &full[st]);
          } else {
            mbar_arrive(&full[st]);
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
    if (!ok && lane == 0) drain_stages(full, filled, S);
    __syncwarp();
  } else if (warp == 8) {
    // ---------------------------------------------------------------- token rows
    // Rows of h are neighbours: a stage's come in one box, its scales in one block.  x is by token:
    // its rows are gathered by 16-byte asynchronous copies, 8 lanes a row, into the swizzled tile,
    // the scale words by 4-byte copies.  Every lane's copies arrive on the stage's barrier by
    // themselves: a warp that waited for them to land before it announced a stage filled one slot
    // in a copy's latency.
    const int h_target = n_rows * up_tiles * 4;
    bool all_ready = false;
    int st = 0, filled = 0;
    uint32_t ph = 0;
    Unit w;
    bool ok = true;
    while (true) {
      ok = next_unit(w, 33);
      if (!ok || w.kind < 0) break;
      const bool up = w.kind == 0;
      if (!up && !all_ready) {
        // lane 0 waits for the group's h; lane 1 looks whether all of h is there, after which
        // no unit asks again (each look costs an L2 round trip)
        int got = 1;
        if (lane == 0)
          got = counter_wait_bounded(p.b.done + w.g, w.rows * up_tiles * 4, abort_flag,
                                     p.b.status, 34);
        if (lane == 1) got = counter_load(p.b.done_all) == h_target ? 2 : 1;
        ok = __shfl_sync(0xffffffffu, got, 0) != 0;
        if (!ok) break;
        all_ready = __shfl_sync(0xffffffffu, got, 1) == 2;
        __syncwarp();  // the other lanes' copies follow those two loads
        fence_proxy_async_global();  // other CTAs' stores, read by TMA
      }
      const int K = up ? d : f, nk = K / 128;
      if (!up) {
        const uint8_t *sc = p.hs + (size_t)w.tile * nk * C::SB_BYTES;
        for (int kc = 0; kc < nk; ++kc) {
          ok = warp_wait(&empty[st], ph ^ 1, 35);
          if (!ok) break;
          if (elect_one()) {
            mbar_arrive_n(&full[st], kRowArrivals - 1);
            mbar_arrive_expect_tx(&full[st], C::B_BYTES + C::SB_BYTES);
            tma_load_3d(sB + st * C::B_BYTES, &p.tm_h, &full[st], kc * 128, w.row0, 0);
            bulk_load(sSB + st * C::SB_BYTES, sc + kc * C::SB_BYTES, C::SB_BYTES, &full[st]);
          }
          __syncwarp();
          ++filled;
          if (++st == S) {
            st = 0;
            ph ^= 1;
          }
        }
        if (!ok) break;
        continue;
      }
      // This lane's piece of the first 4 rows (hi, then lo) and its scale word: addresses once a
      // unit, so that a unit of one or two tokens -- most are -- takes two copies a stage.
      int my_row = w.row0 + lane;
      if (lane < w.n) my_row = w.g < p.b.E ? tb.perm[w.row0 + lane] / p.b.k : w.tok0 + lane;
      const int c = lane & 7;  // 16-byte chunk of a 128-byte row
      auto piece = [&](int r, uint32_t &to, const uint8_t *&src) {
        const int i = r < w.n ? r : r - w.n, t = r < w.n ? r : BN + i;  // row of the tile
        const size_t row = __shfl_sync(0xffffffffu, my_row, i & 31);
        to = t * 128 + ((c ^ (t & 7)) << 4);
        src = (r < w.n ? p.x.hi : p.x.lo) + row * K + c * 16;
      };
      auto word = [&](int r, uint32_t &to, const uint8_t *&src) {
        const int i = r < w.n ? r : r - w.n;
        const size_t row = __shfl_sync(0xffffffffu, my_row, i & 31);
        to = scale_row_at(r < w.n ? r : BN + i);
        src = p.xs + row * nk * 8 + (r < w.n ? 0 : 4);
      };
      uint32_t to0, to1;
      const uint8_t *src0, *src1;
      piece(lane >> 3, to0, src0);
      word(lane, to1, src1);
      for (int kc = 0; kc < nk; ++kc) {
        ok = warp_wait(&empty[st], ph ^ 1, 35);
        if (!ok) break;
        const uint32_t b = smem_u32(sB) + st * C::B_BYTES, sb = smem_u32(sSB) + st * C::SB_BYTES;
        if ((lane >> 3) < 2 * w.n) cp_async16(b + to0, src0 + kc * 128);
        if (lane < 2 * w.n) cp_async4(sb + to1, src1 + kc * 8);
        for (int r = 4 + (lane >> 3); r - (lane >> 3) < 2 * w.n; r += 4) {
          uint32_t to;
          const uint8_t *src;
          piece(r, to, src);
          if (r < 2 * w.n) cp_async16(b + to, src + kc * 128);
        }
        for (int r = 32 + lane; r - lane < 2 * w.n; r += 32) {
          uint32_t to;
          const uint8_t *src;
          word(r, to, src);
          if (r < 2 * w.n) cp_async4(sb + to, src + kc * 8);
        }
        cp_async_arrive(&full[st]);
        ++filled;
        if (++st == S) {
          st = 0;
          ph ^= 1;
        }
      }
      if (!ok) break;
    }
    cp_async_wait_all();
    if (!ok && lane == 0) drain_stages(full, filled, S);
    __syncwarp();
  } else if (warp == 4 || warp == 5) {
    // ---------------------------------------------------------------- MMA
    // One warp for each weight tile: a stage's loop turn (the wait, 11 tcgen05 operations, the
    // commit) takes one issuing thread 750 clocks, the products 330 at 16 columns.  The next stage's
    // barrier is looked at before this one's products are issued.
    const int j = __reduce_max_sync(0xffffffffu, warp) - 4;
    int st = 0, it = 0;
    uint32_t ph = 0;
    Unit w;
    const uint32_t tm = __reduce_max_sync(0xffffffffu, tmem_base);
    const uint32_t a_base = smem_u32(sA) + j * (C::A_BYTES / 2), b_base = smem_u32(sB),
                   sa_base = smem_u32(sSA) + j * kMxScaleBlock, sb_base = smem_u32(sSB);
    while (next_unit(w, 36) && w.kind >= 0) {
      const int acc = it & 1, nk = (w.kind == 0 ? d : f) / 128;
      const bool there = j == 0 || w.kind == 0 || (2 * w.mt + 1) * kMxTile < d;
      bool ok = warp_wait(&tempty[acc], ((it >> 1) & 1) ^ 1, 46);
      const uint32_t d0 = tm + acc * C::ACC_COLS + j * N;
      bool ready = false;
      for (int kc = 0; ok && kc < nk; ++kc) {
        if (!__all_sync(0xffffffffu, ready)) ok = warp_wait(&full[st], ph, 37);
        if (!ok) break;
        tc_fence_after();
        const int st1 = st + 1 == S ? 0 : st + 1;
        const uint32_t ph1 = st + 1 == S ? ph ^ 1 : ph;
        ready = kc + 1 < nk && mbar_test_wait(&full[st1], ph1);
        const uint32_t sf = tm + 2 * C::ACC_COLS + (kc & 1) * C::SF_COLS + j * 8;
        if (elect_one()) {
          if (there) {
            // gathered token rows: written by the copies' generic proxy, read by the tensor cores
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            tc_cp_scales(sf, sa_base + st * C::SA_BYTES);
            tc_cp_scales(sf + 4, sb_base + st * C::SB_BYTES);
            const uint64_t a = sdesc_k_sw128(a_base + st * C::A_BYTES),
                           b = sdesc_k_sw128(b_base + st * C::B_BYTES);
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)  // 32 bytes of a row: 2 units of the descriptors
              tc_mma_mx(d0, a + 2 * kk, b + 2 * kk,
                        idesc_mx(kMxTile, N) | ((uint32_t)kk << 4) | ((uint32_t)kk << 29), sf,
                        sf + 4, (kc | kk) ? 1u : 0u);
          }
          tc_commit(&empty[st]);
          if (kc == nk - 1) tc_commit(&tfull[acc]);
        }
        __syncwarp();
        st = st1;
        ph = ph1;
      }
      ++it;
      if (!ok) break;
    }
    if (lane == 0) {
      tc_commit(mma_end);
      volatile int no_abort = 0;
      mbar_wait_bounded(mma_end, 0, &no_abort, nullptr, 0);
    }
    __syncwarp();
  } else if (warp < 4) {
    // ---------------------------------------------------------------- epilogue
    int it = 0;
    Unit w;
    while ((alive = next_unit(w, 42)) && w.kind >= 0) {
      const int acc = it & 1;
      const bool up = w.kind == 0;
      const bool two = up || (2 * w.mt + 1) * kMxTile < d;
      // down: routed_scale * gate of tokens lane and 32 + lane, asked for before the wait
      float sc0 = 1.f, sc1 = 1.f;
      if (!up && w.g < p.b.E) {
        if (lane < w.n) sc0 = p.b.routed_scale * tb.gate[tb.perm[w.row0 + lane]];
        if (BN > 32 && 32 + lane < w.n) sc1 = p.b.routed_scale * tb.gate[tb.perm[w.row0 + 32 + lane]];
      }
      alive = warp_wait(&tfull[acc], (it >> 1) & 1, 39);
      if (!alive) break;
      ++it;
      tc_fence_after();
      const uint32_t ta = tmem_base + ((uint32_t)(warp * 32) << 16) + acc * C::ACC_COLS;
      for (int c = 0; c < w.n; c += 8) {
        uint32_t r0[8], r1[8], r2[8], r3[8];
        tmem_ld8(ta + c, r0);
        tmem_ld8(ta + BN + c, r1);
        if (two) {
          tmem_ld8(ta + N + c, r2);
          tmem_ld8(ta + N + BN + c, r3);
        }
        tmem_ld_wait();
        float v0[8], v1[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          v0[j] = __uint_as_float(r0[j]) + __uint_as_float(r1[j]);
          v1[j] = two ? __uint_as_float(r2[j]) + __uint_as_float(r3[j]) : 0.f;
        }
        if (up) {
#pragma unroll
          for (int j = 0; j < 8; ++j) v0[j] = swiglu(v0[j], v1[j]);
          store_h_chunk(p.h, p.hs + ((size_t)w.tile * (f / 128) + w.mt) * C::SB_BYTES, f, w.row0,
                        w.mt * kMxTile + warp * 32, c, w.n, BN, warp, lane, v0);
        } else {
          float *y = p.b.y + (size_t)(w.row0 + c) * d + w.mt * kMxDown + warp * 32 + lane;
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const float s = __shfl_sync(0xffffffffu, BN > 32 && c >= 32 ? sc1 : sc0, (c + j) & 31);
            if (c + j < w.n) {
              y[(size_t)j * d] = v0[j] * s;
              if (two) y[(size_t)j * d + kMxTile] = v1[j] * s;
            }
          }
        }
      }
      // every TMEM load has completed: the accumulator goes back before the stores drain
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(&tempty[acc]);
        // publish: the warp's stores (made visible by this fence, after the warp's barrier), then
        // the count of its pieces of rows
        __threadfence();
        atomicAdd(up ? p.b.done + w.g : p.b.tile_done + w.mt, w.n);
        if (up) atomicAdd(p.b.done_all, w.n);
      }
      __syncwarp();
    }
  } else {
    // ---------------------------------------------------------------- idle until the combine
    alive = warp_wait(mma_end, 0, 47);
  }
  if (alive && (warp < 4 || warp > 9))
    combine_pieces(p.b, tb.slot, kMxDown, n_rows * 4, warp < 4 ? warp : warp - 6, kMxWarps - 6,
                   abort_flag);
  tc_fence_before();
  __syncthreads();
  if (warp == 4) {
    tc_fence_after();
    tmem_dealloc(tmem_base, C::TMEM_COLS);
  }
  if (threadIdx.x == 0) leave_grid(p.b);
}

}  // namespace moe
