// mx4.cuh -- microscaled 4-bit blocks: 32 consecutive elements of the
// contraction share a power-of-two scale 2^(s - 127) (one byte, 255: NaN) and
// are held as e2m1 codes (0, .5, 1, 1.5, 2, 3, 4, 6 and their negatives).
//
// Scale of a block: s - 127 = floor(log2(max |v|)) - 2, so that the largest
// element lands in [4, 8); elements round to nearest even and saturate at 6.
// A block with an infinity or a NaN gets the scale NaN.
//
// Scale storage of an operand [rows, cols]: tiles of 128 rows x 4 blocks (128
// columns), 512 bytes each, tile (row / 128, block / 4) in row-major order;
// inside a tile byte (row % 32) * 16 + (row / 32 % 4) * 4 + block % 4.  That
// is the order in which the tensor cores' scale copy (32 lanes x 16 bytes)
// wants it: lane row % 32, column row / 32, byte block % 4.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <stdint.h>

#include "hmm_internal.h"

namespace hmm {

constexpr int MX_BLOCK = 32;
constexpr int MX_TILE_BYTES = 512;

// Scale byte of a block from the bits of its largest magnitude (an unsigned
// maximum of |v| bits, so that infinities and NaN come out on top).
__device__ __forceinline__ uint32_t mx_scale_byte(uint32_t amax_bits) {
  if (amax_bits >= 0x7F800000u) return 255u;
  const uint32_t e = amax_bits >> 23;  // 0 for zero and subnormal blocks: scale 2^-127
  return e > 2u ? e - 2u : 0u;
}
// 2^(127 - s), exact for every s of a finite block (0 .. 252); a NaN block
// (255) gets 0, its codes do not matter.
__device__ __forceinline__ float mx_inverse_scale(uint32_t s) {
  return s == 255u ? 0.0f : __uint_as_float((254u - s) << 23);
}
__device__ __forceinline__ float mx_scale(uint32_t s) {
  if (s == 255u) return __uint_as_float(0x7FC00000u);
  return __uint_as_float(s == 0u ? 0x00400000u : s << 23);
}

// Eight scaled values to eight codes, element 0 in the low half of byte 0.
__device__ __forceinline__ uint32_t mx_codes8(const float (&v)[8]) {
  uint32_t r;
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n\t"
      "mov.b32 %0, {b0, b1, b2, b3};\n\t}"
      : "=r"(r)
      : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]));
  return r;
}

// Eight codes to the values they stand for.
__device__ __forceinline__ void mx_values8(uint32_t codes, float scale, float (&v)[8]) {
  uint32_t h[4];
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
      "mov.b32 {b0, b1, b2, b3}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, b0;\n\t"
      "cvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, b2;\n\t"
      "cvt.rn.f16x2.e2m1x2 %3, b3;\n\t}"
      : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
      : "r"(codes));
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h[j]));
    v[2 * j] = f.x * scale;
    v[2 * j + 1] = f.y * scale;
  }
}

// Pairs of bf16 in 32-bit words (the low half first).
__device__ __forceinline__ float pair_lo(uint32_t v) { return __uint_as_float(v << 16); }
__device__ __forceinline__ float pair_hi(uint32_t v) { return __uint_as_float(v & 0xFFFF0000u); }
// Larger magnitude of each half, NaN if either is (m: a result of this).
__device__ __forceinline__ uint32_t pair_amax(uint32_t m, uint32_t v) {
  uint32_t r;
  asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(m), "r"(v & 0x7FFF7FFFu));
  return r;
}
// Each half times a power of two given as a pair (exact where the block's scale
// makes the product matter: results below 2^-126 round to 0 either way).
__device__ __forceinline__ uint32_t pair_mul(uint32_t v, uint32_t s) {
  uint32_t r;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(v), "r"(s));
  return r;
}

// The scale byte of a block whose 32 bf16 values are held by four neighbouring
// lanes, eight each (u: four pairs).
__device__ __forceinline__ uint32_t quad_scale_bf16(const uint32_t (&u)[4]) {
  uint32_t m = pair_amax(pair_amax(u[0] & 0x7FFF7FFFu, u[1]), pair_amax(u[2] & 0x7FFF7FFFu, u[3]));
  m = pair_amax(m, __shfl_xor_sync(0xffffffffu, m, 1));
  m = pair_amax(m, __shfl_xor_sync(0xffffffffu, m, 2));
  return mx_scale_byte(max(m << 16, m & 0xFFFF0000u));
}
// Eight bf16 values to codes (s: their block's scale byte).
__device__ __forceinline__ uint32_t codes8_bf16(const uint32_t (&u)[4], uint32_t s) {
  // (a power of two up to 2^127: its upper half is the bf16 value)
  const uint32_t i = __float_as_uint(mx_inverse_scale(s));
  const uint32_t inv = (i >> 16) | i;
  float w[8];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const uint32_t v = pair_mul(u[j], inv);
    w[2 * j] = pair_lo(v);
    w[2 * j + 1] = pair_hi(v);
  }
  return mx_codes8(w);
}

// Byte offset of the scale of (row, block) in an operand's scale array with
// kt = ceil(cols / 128) tiles per 128 rows.
__host__ __device__ __forceinline__ int64_t mx_scale_offset(int64_t row, int64_t block, int64_t kt) {
  return ((row >> 7) * kt + (block >> 2)) * MX_TILE_BYTES + (row & 31) * 16 +
         ((row >> 5) & 3) * 4 + (block & 3);
}

}  // namespace hmm
