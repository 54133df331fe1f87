// Microscaled 4-bit elements: e2m1 values (sign, two exponent bits, one
// fraction bit: 0, 0.5, 1, 1.5, 2, 3, 4, 6), two a byte with the even element
// in the low half, and one power-of-two scale (e8m0: 2^(byte - 127), 255 is
// NaN) of each 32 elements of a row.
#pragma once

#include <stdint.h>

namespace dsmh {

// The scale byte of 32 elements of which the largest magnitude has these bits:
// 2^(floor(log2 max) - 2), so that the largest lies in [4, 8) scaled, at least
// 2^-127; NaN where one element is infinite or NaN.
__device__ __forceinline__ uint32_t mx_scale_byte(uint32_t largest) {
  const uint32_t exponent = largest >> 23;
  return exponent == 255u ? 255u : (exponent > 2u ? exponent - 2u : 0u);
}
// The factor 2^(127 - byte) that brings elements to that scale: a normal float,
// since a finite block's byte is 252 at most.  0 for NaN blocks.
__device__ __forceinline__ float mx_inverse(uint32_t byte) {
  return byte == 255u ? 0.0f : __uint_as_float((254u - byte) << 23);
}

// Eight floats to e2m1, to the nearest, ties to the even code, saturating at 6: two a
// byte, the first in the low half of the lowest.
__device__ __forceinline__ uint32_t e2m1_word(const float2 (&v)[4]) {
  uint32_t r;
  asm("{\n\t.reg .b8 a, b, c, d;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\tcvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\tcvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
      "mov.b32 %0, {a, b, c, d};\n\t}"
      : "=r"(r)
      : "f"(v[0].x), "f"(v[0].y), "f"(v[1].x), "f"(v[1].y), "f"(v[2].x), "f"(v[2].y), "f"(v[3].x), "f"(v[3].y));
  return r;
}

// Eight 4-bit elements as bf16 pairs (0,4), (1,5), (2,6), (3,7), scaled.  An
// element's sign, exponent and fraction bits at those of a bf16 make its value
// times 2^-126; `factor` (twice, in a pair) makes up for it with the scale, an
// exact product.  A warp that has a scale for which no bf16 does both multiplies
// twice (again_of).
__device__ __forceinline__ uint32_t times_bf16(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ void decode8(uint32_t w, uint32_t factor, uint32_t (&r)[4]) {
  // One product moves an element's four bits twice, which the logic pipe, half as
  // wide as the others, need not do.
  constexpr uint32_t kBits = 0x81c081c0u, kLow = 0x000f000fu, kHigh = 0x00f000f0u;
  const uint32_t rest = w >> 8;
  r[0] = ((w & kLow) * 0x1040u) & kBits;
  r[1] = ((w & kHigh) * 0x0104u) & kBits;
  r[2] = ((rest & kLow) * 0x1040u) & kBits;
  r[3] = ((rest & kHigh) * 0x0104u) & kBits;
#pragma unroll
  for (int i = 0; i < 4; ++i) r[i] = times_bf16(r[i], factor);
}
// 2^(byte - 1) = 2^126 2^(byte - 127) as a bf16 pair where it is one, else
// 2^126, with 2^(byte - 127) (or NaN) for `again`.
__device__ __forceinline__ uint32_t factor_of(uint32_t byte, bool twice) {
  return (twice ? 253u : byte + 126u) * 0x00800080u;
}
__device__ __forceinline__ uint32_t again_of(uint32_t byte) {
  const uint32_t bits = byte == 0u ? 0x0040u : (byte == 255u ? 0x7fc0u : byte << 7);
  return bits | bits << 16;
}

}  // namespace dsmh
