// Element types of the expert-layer kernels: conversion to 32-bit floats and
// one rounding back.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <stdint.h>

namespace dsmh {

__device__ __forceinline__ float to_float(float v) { return v; }
__device__ __forceinline__ float to_float(__half v) { return __half2float(v); }
__device__ __forceinline__ float to_float(__nv_bfloat16 v) { return __bfloat162float(v); }

template <typename T>
__device__ __forceinline__ T from_float(float v);
template <>
__device__ __forceinline__ float from_float<float>(float v) { return v; }
template <>
__device__ __forceinline__ __half from_float<__half>(float v) { return __float2half_rn(v); }
template <>
__device__ __forceinline__ __nv_bfloat16 from_float<__nv_bfloat16>(float v) {
  return __float2bfloat16_rn(v);
}

// Two elements of a type as floats, and back with one rounding each.  16-bit
// pairs are one 32-bit word, so a conversion back takes one instruction.
__device__ __forceinline__ float2 pair_to_floats(uint32_t w, __nv_bfloat16) {
  return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}
__device__ __forceinline__ float2 pair_to_floats(uint32_t w, __half) {
  return __half22float2(*reinterpret_cast<const __half2*>(&w));
}
__device__ __forceinline__ uint32_t floats_to_pair(float2 v, __nv_bfloat16) {
  const __nv_bfloat162 p = __float22bfloat162_rn(v);
  return *reinterpret_cast<const uint32_t*>(&p);
}
__device__ __forceinline__ uint32_t floats_to_pair(float2 v, __half) {
  const __half2 p = __float22half2_rn(v);
  return *reinterpret_cast<const uint32_t*>(&p);
}
// Number of float pairs in 16 bytes, the i-th of them, and replacing it.
template <typename T>
struct Vector16 {
  static constexpr int kPairs = sizeof(T) == 2 ? 4 : 2;
  uint32_t w[4];
  __device__ __forceinline__ float2 get(int i) const {
    if constexpr (sizeof(T) == 2) return pair_to_floats(w[i], T());
    else return make_float2(__uint_as_float(w[2 * i]), __uint_as_float(w[2 * i + 1]));
  }
  __device__ __forceinline__ void set(int i, float2 v) {
    if constexpr (sizeof(T) == 2) {
      w[i] = floats_to_pair(v, T());
    } else {
      w[2 * i] = __float_as_uint(v.x);
      w[2 * i + 1] = __float_as_uint(v.y);
    }
  }
  __device__ __forceinline__ uint4 words() const { return make_uint4(w[0], w[1], w[2], w[3]); }
  __device__ __forceinline__ void words(const uint4& v) { w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w; }
};

// a * b + c on both floats of a pair, one instruction.
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;"
      : "=l"(r)
      : "l"(*reinterpret_cast<const uint64_t*>(&a)), "l"(*reinterpret_cast<const uint64_t*>(&b)),
        "l"(*reinterpret_cast<const uint64_t*>(&c)));
  return *reinterpret_cast<const float2*>(&r);
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;"
      : "=l"(r)
      : "l"(*reinterpret_cast<const uint64_t*>(&a)), "l"(*reinterpret_cast<const uint64_t*>(&b)));
  return *reinterpret_cast<const float2*>(&r);
}

// V elements that move as one access of V * sizeof(T) bytes (up to 16).
template <typename T, int V>
struct alignas(sizeof(T) * V) Pack {
  T v[V];
};

}  // namespace dsmh
