// mx4.cuh -- the microscaled 4-bit format (dmoe_mx4 of dmoe.h) on the device: where a block's
// scale byte lies, the scale of a block, and the conversions of its elements.
#pragma once

#include <stdint.h>

#include "common.cuh"

namespace dmoe {

// Scales lie in tiles of 128 rows x 128 columns (4 blocks of 32): [row tile][column tile][32][4][4],
// byte [l][q][b] = row 32 q + l, block b of the tile.  It is the order in which the block-scaled
// tensor-core instructions take the scales of 128 rows from shared memory (one 512-byte tile
// is four tensor-memory columns), so the grouped GEMM copies whole tiles.
constexpr int kMx4TileBytes = 512;

// Offset of the four scale bytes of row r, column tile ct (a 4-byte word).
__device__ __forceinline__ size_t mx4_scale_word(long long r, int ct, int col_tiles) {
  const int rr = (int)(r & 127);
  return ((size_t)(r >> 7) * col_tiles + ct) * kMx4TileBytes + (rr & 31) * 16 + (rr >> 5) * 4;
}

// Scale byte of a block from the bits of its largest magnitude as fp32 (|x|, so no sign bit):
// floor(log2 amax) - 2, the power of two that puts amax into [4, 8) (6 is the largest element),
// kept within [2^-127, 2^127]; 255 (NaN) for an inf or NaN in the block.  Subnormal and zero
// maxima have exponent field 0 and get 2^-127.
__device__ __forceinline__ uint32_t mx4_scale_byte(uint32_t amax_bits) {
  const uint32_t e = amax_bits >> 23;
  return (e == 255u) ? 255u : (e > 2u ? e - 2u : 0u);
}

// 2^(127 - s): the factor that takes values into a block of scale byte s <= 252 (254 at most
// for s = 0: 2^127, a normal number).
__device__ __forceinline__ float mx4_inverse(uint32_t s) { return __uint_as_float((254u - s) << 23); }

// 2^(s - 127) in fp32: s = 0 is the subnormal 2^-127; s = 255 is NaN.
__device__ __forceinline__ float mx4_scale_value(uint32_t s) {
  const uint32_t b = (s == 0u) ? 0x00400000u : (s << 23);
  return __uint_as_float(s == 255u ? 0x7FC00000u : b);
}

// Eight values, scaled into their block, to eight elements (round to nearest even, saturated at
// +-6), element i in bits 4i .. 4i+3.
__device__ __forceinline__ uint32_t mx4_pack8(const float (&v)[8]) {
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

// Eight elements to fp16 pairs (exact): o[i] holds elements 2i (low half) and 2i + 1.
__device__ __forceinline__ void mx4_unpack8(uint32_t w, uint32_t (&o)[4]) {
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
      "mov.b32 {b0, b1, b2, b3}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, b0;\n\t"
      "cvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, b2;\n\t"
      "cvt.rn.f16x2.e2m1x2 %3, b3;\n\t}"
      : "=r"(o[0]), "=r"(o[1]), "=r"(o[2]), "=r"(o[3])
      : "r"(w));
}

// ---- block floating point rows (DMOE_SCALE_COLS of dmoe.h) -------------------------------------

// The power-of-two factor for 128 columns of largest magnitude m (into [2^13, 2^14), with the
// exceptions that DMOE_SCALE_COLS states); `stored` is what goes into the scale array.
__device__ __forceinline__ float bfp_scale(float m, float &stored) {
  int es = 13 - ((int)((__float_as_uint(m) >> 23) & 0xFFu) - 127);
  const bool finite = m <= 3.402823466e38f;
  if (m == 0.0f || !finite) es = 0;
  if (es > 24 && es <= 51) es = 24;
  es = min(max(es, -126), 126);
  const bool fits = finite && es >= -15 && es <= 24;
  stored = __uint_as_float(((uint32_t)(127 - es) << 23) | (fits ? 0u : 0x80000000u));
  return __uint_as_float((uint32_t)(127 + es) << 23);
}

}  // namespace dmoe
