// What routing's kernels share: the order of logits, softmax terms.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace dsmh {

constexpr uint32_t kFullWarp = 0xffffffffu;

// Floats as unsigned integers of the same order; 0 for what is masked (-inf
// and NaN).  Adding zero makes -0 equal to +0.
__device__ __forceinline__ uint32_t rank_key(float v) {
  if (!(v > -INFINITY)) return 0u;
  const uint32_t b = __float_as_uint(v + 0.0f);
  return b ^ ((b >> 31) ? 0xffffffffu : 0x80000000u);
}
__device__ __forceinline__ float rank_value(uint32_t key) {
  return __uint_as_float(key ^ ((key >> 31) ? 0x80000000u : 0xffffffffu));
}

// exp(v - top), the unnormalised softmax of an unmasked logit.  With top at
// +inf it is the limit: 1 for the entries at +inf, 0 for the others.
__device__ __forceinline__ float raised(float v, float top) {
  return top < INFINITY ? expf(v - top) : (v == top ? 1.0f : 0.0f);
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) v += __shfl_xor_sync(kFullWarp, v, d);
  return v;
}

}  // namespace dsmh
