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

// A lane's two largest rank keys that have not been picked, and their places.
// Equal keys come by rising place.
struct Best {
  uint32_t key = 0, next = 0;
  int at = 0, next_at = 0;
};
template <int R>
__device__ __forceinline__ Best two_best(const uint32_t (&key)[R], uint32_t picked) {
  Best b;
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const uint32_t k = (picked >> r & 1u) ? 0u : key[r];
    if (k > b.key) {
      b.next = b.key, b.next_at = b.at;
      b.key = k, b.at = r;
    } else if (k > b.next) {
      b.next = k, b.next_at = r;
    }
  }
  return b;
}

// The top_k largest keys of a warp, R contiguous ones a lane, the j-th in lane j
// (which keeps -1 where fewer are left), for kRows rows at once: a pick is a chain
// of warp-wide steps, and two rows' chains take little longer than one's.  Each
// lane keeps the two largest of its keys (`best` at first); a pick is a warp
// maximum, the lowest lane that holds it, and that lane's next key, for which it
// looks through its keys again only after two picks.  Lanes hold contiguous runs,
// so the lowest lane and the first place in it are the lowest index.
template <int kRows, int R>
__device__ __forceinline__ void pick(const uint32_t (&key)[kRows][R], Best (&best)[kRows], int top_k,
                                     int (&my_id)[kRows], uint32_t (&my_key)[kRows]) {
  static_assert(R <= 32, "a lane's picked keys are bits of a word");
  const int lane = threadIdx.x & 31;
  uint32_t picked[kRows] = {};
#pragma unroll 1
  for (int j = 0; j < top_k; ++j) {
    uint32_t m[kRows], some = 0;
#pragma unroll
    for (int i = 0; i < kRows; ++i) some |= m[i] = __reduce_max_sync(kFullWarp, best[i].key);
    if (some == 0u) break;
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      const int holder = __ffs(__ballot_sync(kFullWarp, best[i].key == m[i])) - 1;
      const int id = __shfl_sync(kFullWarp, lane * R + best[i].at, holder);
      if (lane == j && m[i] != 0u) my_id[i] = id, my_key[i] = m[i];
      if (lane == holder) {
        picked[i] |= 1u << best[i].at;
        best[i].key = best[i].next, best[i].at = best[i].next_at;
        best[i].next = 0u;
      }
      if (lane == holder && best[i].key == 0u) best[i] = two_best(key[i], picked[i]);
    }
    __syncwarp();
  }
}

}  // namespace dsmh
