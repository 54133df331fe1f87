// The weighted way back from grouped rows to tokens, and its gradients.
#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "dtypes.cuh"
#include "experts.h"

namespace dsmh {
namespace {

constexpr int kThreads = 256;
constexpr int kMostPieces = 65535;  // a grid's second extent; wider rows take more launches

// What one thread handles of a row at a time: 16 bytes, or (kWide false, where
// addresses allow none) two elements kThreads apart.  Rows of z, the outputs
// and dz go by once and pass the caches.
template <typename T, bool kWide>
struct Piece {
  static constexpr int kPairs = kWide ? Vector16<T>::kPairs : 1;
  static constexpr int kEach = 2 * kPairs;
  Vector16<T> wide;
  T single[kWide ? 1 : 2];

  // First column of a thread's piece, of those beginning at column `base`.
  __device__ __forceinline__ static int column(int base) {
    return base + static_cast<int>(threadIdx.x) * (kWide ? kEach : 1);
  }
  template <bool kOnce>
  __device__ __forceinline__ void load(const T* p, int left) {
    if constexpr (kWide) {
      const uint4* q = reinterpret_cast<const uint4*>(p);
      wide.words(kOnce ? __ldcs(q) : *q);
    } else {
      single[0] = p[0];
      single[1] = kThreads < left ? p[kThreads] : from_float<T>(0.0f);
    }
  }
  __device__ __forceinline__ float2 get(int i) const {
    if constexpr (kWide) return wide.get(i);
    else return make_float2(to_float(single[0]), to_float(single[1]));
  }
  __device__ __forceinline__ void set(int i, float2 v) {
    if constexpr (kWide) {
      wide.set(i, v);
    } else {
      single[0] = from_float<T>(v.x);
      single[1] = from_float<T>(v.y);
    }
  }
  __device__ __forceinline__ void store(T* p, int left) const {
    if constexpr (kWide) {
      __stcs(reinterpret_cast<uint4*>(p), wide.words());
    } else {
      p[0] = single[0];
      if (kThreads < left) p[kThreads] = single[1];
    }
  }
};

// The rows of a token are taken kAtOnce at a time: their positions first, then
// a piece of each in flight together.
constexpr int kAtOnce = 4;
constexpr int kCtas = 5;

// One CTA per token and kThreads pieces: out = sum_j w_j z[p_j], summed in 32
// bits in the order of j.  Bound by reading z: 16384 tokens x 8 rows of 2048
// bf16 in 90 us, 6.7 TB/s (eight rows in flight: 93; one: 102).
template <typename T, bool kWide>
__global__ void __launch_bounds__(kThreads, kCtas) combine_kernel(CombineArgs a) {
  using P = Piece<T, kWide>;
  const int64_t token = blockIdx.x;
  const int col = P::column((a.first_piece + blockIdx.y) * kThreads * P::kEach), left = a.width - col;
  if (left <= 0) return;
  const T* z = static_cast<const T*>(a.z) + col;
  float2 acc[P::kPairs];
#pragma unroll
  for (int q = 0; q < P::kPairs; ++q) acc[q] = make_float2(0.0f, 0.0f);
  for (int j0 = 0; j0 < a.top_k; j0 += kAtOnce) {
    int p[kAtOnce];
    float w[kAtOnce];
#pragma unroll
    for (int j = 0; j < kAtOnce; ++j) {
      const int64_t i = token * a.top_k + j0 + j;
      p[j] = j0 + j < a.top_k ? a.position[i] : -1;
      if (p[j] >= a.z_rows) p[j] = -1;
      w[j] = a.weights && j0 + j < a.top_k ? a.weights[i] : 1.0f;
    }
    P x[kAtOnce];
#pragma unroll
    for (int j = 0; j < kAtOnce; ++j)
      if (p[j] >= 0) x[j].template load<true>(z + p[j] * a.z_stride, left);
#pragma unroll
    for (int j = 0; j < kAtOnce; ++j)
      if (p[j] >= 0) {
#pragma unroll
        for (int q = 0; q < P::kPairs; ++q) acc[q] = fma2(make_float2(w[j], w[j]), x[j].get(q), acc[q]);
      }
  }
  P y;
#pragma unroll
  for (int q = 0; q < P::kPairs; ++q) y.set(q, acc[q]);
  y.store(static_cast<T*>(a.out) + token * a.width + col, left);
}

// One CTA per token: its dy row against each of its z rows.  dz is written on
// the way; the dot products are summed in 32 bits by thread, warp and CTA.
// The CTA also clears those of the rows [token * top_k, (token + 1) * top_k)
// that lie behind the last group.  Bound by reading z and writing dz: 174 us at
// that size, 6.6 TB/s.
template <typename T, bool kWide>
__global__ void __launch_bounds__(kThreads, kCtas) combine_backward_kernel(CombineArgs a) {
  using P = Piece<T, kWide>;
  __shared__ float part[kThreads / 32][kAtOnce];
  const int64_t token = blockIdx.x;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const T* dy = static_cast<const T*>(a.dy) + token * a.dy_stride;
  T* dz = static_cast<T*>(a.out);
  for (int j0 = 0; j0 < a.top_k; j0 += kAtOnce) {
    int p[kAtOnce];
    uint32_t behind = 0;
    float w[kAtOnce];
    float2 dot[kAtOnce];
#pragma unroll
    for (int j = 0; j < kAtOnce; ++j) {
      const int64_t i = token * a.top_k + j0 + j;
      const bool in = j0 + j < a.top_k;
      p[j] = in ? a.position[i] : -1;
      if (p[j] >= a.z_rows) p[j] = -1;
      w[j] = in ? a.weights[i] : 0.0f;
      if (in && a.order[i] < 0) behind |= 1u << j;
      dot[j] = make_float2(0.0f, 0.0f);
    }
    for (int base = 0; base < a.width; base += kThreads * P::kEach) {
      const int col = P::column(base), left = a.width - col;
      if (left <= 0) break;
      P g;
      g.template load<false>(dy + col, left);
      P x[kAtOnce];
#pragma unroll
      for (int j = 0; j < kAtOnce; ++j)
        if (p[j] >= 0) x[j].template load<true>(static_cast<const T*>(a.z) + p[j] * a.z_stride + col, left);
#pragma unroll
      for (int j = 0; j < kAtOnce; ++j)
        if (p[j] >= 0) {
#pragma unroll
          for (int q = 0; q < P::kPairs; ++q) {
            const float2 v = g.get(q);
            dot[j] = fma2(v, x[j].get(q), dot[j]);
            x[j].set(q, mul2(make_float2(w[j], w[j]), v));
          }
          x[j].store(dz + static_cast<int64_t>(p[j]) * a.width + col, left);
        }
      if (behind) {
#pragma unroll
        for (int q = 0; q < P::kPairs; ++q) g.set(q, make_float2(0.0f, 0.0f));
        for (int j = 0; j < kAtOnce; ++j)
          if (behind >> j & 1u) g.store(dz + (token * a.top_k + j0 + j) * a.width + col, left);
      }
    }
    float sum[kAtOnce];
#pragma unroll
    for (int j = 0; j < kAtOnce; ++j) {
      sum[j] = dot[j].x + dot[j].y;
#pragma unroll
      for (int d = 16; d > 0; d >>= 1) sum[j] += __shfl_xor_sync(0xffffffffu, sum[j], d);
      if (lane == j) part[warp][j] = sum[j];
    }
    __syncthreads();
    if (threadIdx.x < kAtOnce && j0 + static_cast<int>(threadIdx.x) < a.top_k) {
      float all = 0.0f;
#pragma unroll
      for (int k = 0; k < kThreads / 32; ++k) all += part[k][threadIdx.x];
      a.dweights[token * a.top_k + j0 + threadIdx.x] = all;
    }
    __syncthreads();
  }
}

bool wide(const void* p, int64_t stride, int size) {
  return reinterpret_cast<uintptr_t>(p) % 16 == 0 && stride * size % 16 == 0;
}

template <typename T, bool kWide>
cudaError_t launch(const CombineArgs& a, bool backward, cudaStream_t stream) {
  const unsigned tokens = static_cast<unsigned>(a.tokens);
  if (backward) {
    combine_backward_kernel<T, kWide><<<tokens, kThreads, 0, stream>>>(a);
    return cudaGetLastError();
  }
  const int columns = kThreads * Piece<T, kWide>::kEach, pieces = (a.width + columns - 1) / columns;
  cudaError_t e = cudaSuccess;
  CombineArgs part = a;
  for (; part.first_piece < pieces && e == cudaSuccess; part.first_piece += kMostPieces) {
    const unsigned here = static_cast<unsigned>(std::min(pieces - part.first_piece, kMostPieces));
    combine_kernel<T, kWide><<<dim3(tokens, here), kThreads, 0, stream>>>(part);
    e = cudaGetLastError();
  }
  return e;
}

// 16 bytes at a time where every base and row allows it.
template <typename T>
cudaError_t dispatch(const CombineArgs& a, bool backward, cudaStream_t stream) {
  const int s = sizeof(T);
  const bool ok = wide(a.z, a.z_stride, s) && wide(a.out, a.width, s) &&
                  (!backward || wide(a.dy, a.dy_stride, s));
  return ok ? launch<T, true>(a, backward, stream) : launch<T, false>(a, backward, stream);
}

cudaError_t dispatch_type(const CombineArgs& a, bool backward, cudaStream_t stream) {
  if (a.dtype == DSMEM_F32) return dispatch<float>(a, backward, stream);
  if (a.dtype == DSMEM_F16) return dispatch<__half>(a, backward, stream);
  return dispatch<__nv_bfloat16>(a, backward, stream);
}

}  // namespace

cudaError_t launch_combine(const CombineArgs& a, cudaStream_t stream) {
  return dispatch_type(a, false, stream);
}
cudaError_t launch_combine_backward(const CombineArgs& a, cudaStream_t stream) {
  return dispatch_type(a, true, stream);
}

}  // namespace dsmh
