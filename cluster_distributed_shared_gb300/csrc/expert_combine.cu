// The weighted way back from grouped rows to tokens, and its gradients.
#include <cuda_runtime.h>
#include <stdint.h>

#include "dtypes.cuh"
#include "experts.h"

namespace dsmh {
namespace {

constexpr int kThreads = 256;

// One CTA per token and kThreads * V columns: out = sum_j w_j z[p_j], summed in
// 32 bits in the order of j.
template <typename T, int V>
__global__ void __launch_bounds__(kThreads) combine_kernel(CombineArgs a) {
  const int64_t token = blockIdx.x;
  const int col = (blockIdx.y * kThreads + threadIdx.x) * V;
  if (col >= a.width) return;
  using P = Pack<T, V>;
  const T* z = static_cast<const T*>(a.z) + col;
  float acc[V];
#pragma unroll
  for (int v = 0; v < V; ++v) acc[v] = 0.0f;
  for (int j = 0; j < a.top_k; ++j) {
    const int64_t i = token * a.top_k + j;
    const int64_t p = a.position[i];
    if (p < 0 || p >= a.z_rows) continue;
    const float w = a.weights ? a.weights[i] : 1.0f;
    const P x = *reinterpret_cast<const P*>(z + p * a.z_stride);
#pragma unroll
    for (int v = 0; v < V; ++v) acc[v] += w * to_float(x.v[v]);
  }
  P y;
#pragma unroll
  for (int v = 0; v < V; ++v) y.v[v] = from_float<T>(acc[v]);
  *reinterpret_cast<P*>(static_cast<T*>(a.out) + token * a.width + col) = y;
}

// One CTA per token: its dy row against each of its z rows.  dz is written on
// the way; the dot products are summed in 32 bits by thread, warp and CTA.
// The CTA also clears those of the rows [token * top_k, (token + 1) * top_k)
// that lie behind the last group.
template <typename T, int V>
__global__ void __launch_bounds__(kThreads) combine_backward_kernel(CombineArgs a) {
  __shared__ float part[kThreads / 32];
  const int64_t token = blockIdx.x;
  using P = Pack<T, V>;
  const T* dy = static_cast<const T*>(a.dy) + token * a.dy_stride;
  for (int j = 0; j < a.top_k; ++j) {
    const int64_t i = token * a.top_k + j;
    const int64_t p = a.position[i];
    const bool found = p >= 0 && p < a.z_rows;
    float dot = 0.0f;
    if (found) {
      const float w = a.weights[i];
      const T* z = static_cast<const T*>(a.z) + p * a.z_stride;
      T* dz = static_cast<T*>(a.out) + p * a.width;
      for (int col = threadIdx.x * V; col < a.width; col += kThreads * V) {
        const P g = *reinterpret_cast<const P*>(dy + col);
        const P x = *reinterpret_cast<const P*>(z + col);
        P d;
#pragma unroll
        for (int v = 0; v < V; ++v) {
          const float gv = to_float(g.v[v]);
          dot += gv * to_float(x.v[v]);
          d.v[v] = from_float<T>(w * gv);
        }
        *reinterpret_cast<P*>(dz + col) = d;
      }
    }
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, d);
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = dot;
    __syncthreads();
    if (threadIdx.x == 0) {
      float sum = 0.0f;
      for (int k = 0; k < kThreads / 32; ++k) sum += part[k];
      a.dweights[i] = found ? sum : 0.0f;
    }
    __syncthreads();
    if (a.order[i] < 0) {
      P zero;
#pragma unroll
      for (int v = 0; v < V; ++v) zero.v[v] = from_float<T>(0.0f);
      T* dz = static_cast<T*>(a.out) + i * a.width;
      for (int col = threadIdx.x * V; col < a.width; col += kThreads * V)
        *reinterpret_cast<P*>(dz + col) = zero;
    }
  }
}

// Elements per access: 16 bytes where every base and row allows it, else one.
bool wide(const void* p, int64_t stride, int size) {
  return reinterpret_cast<uintptr_t>(p) % 16 == 0 && stride * size % 16 == 0;
}

template <typename T, int V>
cudaError_t launch(const CombineArgs& a, bool backward, cudaStream_t stream) {
  if (backward) {
    combine_backward_kernel<T, V><<<dim3(static_cast<unsigned>(a.tokens)), kThreads, 0, stream>>>(a);
  } else {
    const dim3 grid(static_cast<unsigned>(a.tokens), (a.width + kThreads * V - 1) / (kThreads * V));
    combine_kernel<T, V><<<grid, kThreads, 0, stream>>>(a);
  }
  return cudaGetLastError();
}

template <typename T>
cudaError_t dispatch(const CombineArgs& a, bool backward, cudaStream_t stream) {
  constexpr int kWide = 16 / sizeof(T);
  const int s = sizeof(T);
  const bool ok = wide(a.z, a.z_stride, s) && wide(a.out, a.width, s) &&
                  (!backward || wide(a.dy, a.dy_stride, s)) && a.width % kWide == 0;
  return ok ? launch<T, kWide>(a, backward, stream) : launch<T, 1>(a, backward, stream);
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
