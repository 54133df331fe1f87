// Microscaled 4-bit elements: e2m1 values (sign, two exponent bits, one
// fraction bit: 0, 0.5, 1, 1.5, 2, 3, 4, 6), two a byte with the even element
// in the low half, and one power-of-two scale (e8m0: 2^(byte - 127), 255 is
// NaN) of each 32 elements of a row.
#pragma once

#include <stdint.h>

namespace dsmh {

// 2^(byte - 127).  2^-127 lies below the normal 32-bit floats.
__device__ __forceinline__ float mx_scale(uint32_t byte) {
  if (byte == 0u) return __uint_as_float(0x00400000u);
  return byte == 255u ? __uint_as_float(0x7fc00000u) : __uint_as_float(byte << 23);
}

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

// Two floats to e2m1, to the nearest, ties to the even code, saturating at 6:
// `low` in the low half of the byte.
__device__ __forceinline__ uint32_t e2m1_pair(float low, float high) {
  uint32_t r;
  asm("{\n\t.reg .b8 p, z;\n\tcvt.rn.satfinite.e2m1x2.f32 p, %1, %2;\n\tmov.b32 %0, {p, z, z, z};\n\t}"
      : "=r"(r)
      : "f"(high), "f"(low));
  return r & 0xffu;
}
// Element i (0..7) of a word of eight, as a float.  Its bits at a float's
// exponent and fraction make the value times 2^-126, an exact product.
__device__ __forceinline__ float e2m1_value(uint32_t word, int i) {
  const uint32_t sign = (i < 7 ? word << (28 - 4 * i) : word) & 0x80000000u;
  const int up = 22 - 4 * i;
  const uint32_t rest = (up >= 0 ? word << up : word >> -up) & 0x01c00000u;
  return __uint_as_float(sign | rest) * 0x1p126f;
}

}  // namespace dsmh
