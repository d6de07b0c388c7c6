// mxfp4.cuh -- MXFP4 matrices (microscaled 4-bit floating point): quantisation, its inverse, and the
// order of the scales that the layer's kernels load.
//
// A matrix [rows, cols] (cols a multiple of 32) is held as codes [rows, cols / 2] (two e2m1
// values a byte, the lower column in the low nibble) and scales [rows, cols / 32] (one e8m0 byte
// for each 32 neighbours of a row: 2^(byte - 127), 255 = NaN).  e2m1 holds 0, 0.5, 1, 1.5, 2, 3,
// 4, 6 and their negatives.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp4.h>
#include <cuda_fp8.h>
#include <stdint.h>

#include "ptx_sm100.cuh"

namespace moe {

constexpr int kMxBlock = 32;   // values that share a scale
constexpr int kMxUnroll = 4;   // pieces of 8 values a thread takes at a time, 256 apart
constexpr int kMxPerLane = 8;  // values a lane converts: four lanes hold a block

// 2^(byte - 127): byte 0 is fp32's subnormal 2^-127, byte 255 NaN
__device__ __forceinline__ float e8m0_to_f32(uint32_t byte) {
  return __uint_as_float(byte == 0 ? 0x00400000u : (byte == 255u ? 0x7fffffffu : byte << 23));
}

// Eight e2m1 codes (low nibble first) -> eight halves, exact: one conversion for each byte.  The
// byte registers matter: through the header's 8-bit function, which packs and unpacks each result,
// the same conversions ran at 28 codes a clock and SM instead of 124.
__device__ __forceinline__ void e2m1x8_to_half(uint32_t codes, uint32_t (&h)[4]) {
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
      "mov.b32 {b0, b1, b2, b3}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, b0;\n\t"
      "cvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, b2;\n\t"
      "cvt.rn.f16x2.e2m1x2 %3, b3;\n\t}"
      : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
      : "r"(codes));
}

__device__ __forceinline__ void load8(const __nv_bfloat16 *p, float (&v)[8]) {
  const uint4 u = *reinterpret_cast<const uint4 *>(p);
  const __nv_bfloat162 *h = reinterpret_cast<const __nv_bfloat162 *>(&u);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = __bfloat1622float2(h[i]);
    v[2 * i] = f.x;
    v[2 * i + 1] = f.y;
  }
}
__device__ __forceinline__ void load8(const float *p, float (&v)[8]) {
  const float4 a = *reinterpret_cast<const float4 *>(p);
  const float4 b = *reinterpret_cast<const float4 *>(p + 4);
  v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
  v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
}
// (streaming stores: what is written is larger than L2 where the rate matters)
__device__ __forceinline__ void store8(__nv_bfloat16 *p, const float (&v)[8]) {
  uint4 u;
  uint32_t *w = reinterpret_cast<uint32_t *>(&u);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t *>(&h);
  }
  __stcs(reinterpret_cast<uint4 *>(p), u);
}
__device__ __forceinline__ void store8(float *p, const float (&v)[8]) {
  __stcs(reinterpret_cast<float4 *>(p), make_float4(v[0], v[1], v[2], v[3]));
  __stcs(reinterpret_cast<float4 *>(p + 4), make_float4(v[4], v[5], v[6], v[7]));
}

// largest magnitude of the four lanes' 32 values, as fp32 bits without the sign (the order of
// magnitudes is that of these integers; NaN above infinity)
__device__ __forceinline__ uint32_t block_amax_bits(const float (&v)[8]) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(v[i]) & 0x7fffffffu);
  m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
  return max(m, __shfl_xor_sync(0xffffffffu, m, 2));
}

// Quantisation.  scale = 2^s with s = floor(log2 max|v|) - 2, at least -127 (the exponent field
// of the largest magnitude less 2 is the e8m0 byte itself); each value becomes the nearest e2m1
// value of v / 2^s, ties to the even code, magnitudes past 6 saturate to 6.  v / 2^s is exact: a
// product with a power of two (only results far below the smallest code lose bits).  A block that
// holds an infinity or a NaN becomes NaN: byte 255, codes 0.
// One pass, 16 or 32 bytes read a lane, four lanes a block, kMxUnroll loads in flight a thread; bound
// by HBM: 185,000 x 4096 bf16 in 328 us, 5.85 TB/s, and back in 291 us, 6.6 TB/s (the copy rate).
template <typename Tin>
__global__ void __launch_bounds__(256)
    mxfp4_quantize_kernel(const Tin *__restrict__ src, size_t n_lanes, uint8_t *__restrict__ codes,
                          uint8_t *__restrict__ scales) {
  griddep_wait();
  griddep_launch_dependents();
  const size_t step = (size_t)gridDim.x * 256 * kMxUnroll;
  // whole warps take part in the shuffles
  for (size_t i0 = (size_t)blockIdx.x * 256 * kMxUnroll; i0 < n_lanes; i0 += step) {
    float v[kMxUnroll][8];
#pragma unroll
    for (int u = 0; u < kMxUnroll; ++u) {
      const size_t i = i0 + u * 256 + threadIdx.x;
#pragma unroll
      for (int j = 0; j < 8; ++j) v[u][j] = 0.f;
      if (i < n_lanes) load8(src + i * kMxPerLane, v[u]);
    }
#pragma unroll
    for (int u = 0; u < kMxUnroll; ++u) {
      const size_t i = i0 + u * 256 + threadIdx.x;
      const uint32_t field = block_amax_bits(v[u]) >> 23;
      const uint32_t byte = field == 255u ? 255u : (field > 2u ? field - 2u : 0u);
      const float inv = byte == 255u ? 0.f : __uint_as_float((254u - byte) << 23);
      uint32_t c = 0;
      if (byte != 255u) {
#pragma unroll
        for (int j = 0; j < 4; ++j)
          c |= (uint32_t)__nv_cvt_float2_to_fp4x2(
                   make_float2(v[u][2 * j] * inv, v[u][2 * j + 1] * inv), __NV_E2M1,
                   cudaRoundNearest)
               << (8 * j);
      }
      if (i < n_lanes) {
        __stcs(reinterpret_cast<uint32_t *>(codes + i * 4), c);
        if ((i & 3) == 0) scales[i >> 2] = (uint8_t)byte;
      }
    }
  }
}

// The values that codes and scales stand for: e2m1 times 2^(byte - 127).  Exact in fp32 and bf16
// for every byte up to 252 (what quantisation writes); past it the largest codes are infinite.
template <typename Tout>
__global__ void __launch_bounds__(256)
    mxfp4_dequantize_kernel(const uint8_t *__restrict__ codes, const uint8_t *__restrict__ scales,
                            size_t n_lanes, Tout *__restrict__ dst) {
  griddep_wait();
  griddep_launch_dependents();
  const size_t step = (size_t)gridDim.x * 256 * kMxUnroll;
  for (size_t i0 = (size_t)blockIdx.x * 256 * kMxUnroll; i0 < n_lanes; i0 += step) {
    uint32_t c[kMxUnroll], b[kMxUnroll];
#pragma unroll
    for (int u = 0; u < kMxUnroll; ++u) {
      const size_t i = i0 + u * 256 + threadIdx.x;
      c[u] = i < n_lanes ? *reinterpret_cast<const uint32_t *>(codes + i * 4) : 0u;
      b[u] = i < n_lanes ? scales[i >> 2] : 0u;
    }
#pragma unroll
    for (int u = 0; u < kMxUnroll; ++u) {
      const size_t i = i0 + u * 256 + threadIdx.x;
      uint32_t h[4];
      e2m1x8_to_half(c[u], h);
      const float s = e8m0_to_f32(b[u]);
      float v[8];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&h[j]));
        v[2 * j] = f.x * s;
        v[2 * j + 1] = f.y * s;
      }
      if (i < n_lanes) store8(dst + i * kMxPerLane, v);
    }
  }
}

// Scales in the order of the block-scaled tensor core instruction: blocks of 512 bytes for 128 rows
// x 128 K (a row of blocks after the other), in a block byte r % 32 * 16 + r / 32 * 4 + k / 32.
// One thread moves the four scales of a row of a block (one word); n words, nk blocks along K.
__global__ void __launch_bounds__(256)
    mxfp4_tile_scales_kernel(const uint32_t *__restrict__ scales, size_t n, int nk,
                             uint32_t *__restrict__ tiled) {
  griddep_wait();
  griddep_launch_dependents();
  const size_t step = (size_t)gridDim.x * blockDim.x;
  for (size_t i = (size_t)blockIdx.x * blockDim.x + threadIdx.x; i < n; i += step) {
    const size_t block = i >> 7, row = block / nk * 128 + (i & 3) * 32 + ((i >> 2) & 31);
    tiled[i] = scales[row * nk + block % nk];
  }
}

}  // namespace moe
