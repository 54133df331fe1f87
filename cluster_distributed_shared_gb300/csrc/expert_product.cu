// Products grouped by key: the simple form, one 64 x 64 tile per CTA with
// 32-bit fused multiply-adds.
#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "dtypes.cuh"
#include "experts.h"

namespace dsmh {
namespace {

constexpr int kTile = 64, kDepth = 16, kThreads = 256;

__device__ __forceinline__ int64_t group_end(const ProductArgs& a, int g) {
  const int64_t e = a.offsets[g + 1];
  return e < 0 ? 0 : (e > a.n ? a.n : e);
}

template <typename T>
__device__ __forceinline__ float source(const ProductArgs& a, int64_t p, int c) {
  int64_t row = p;
  if (a.order) {
    const int64_t o = a.order[p];
    row = o < 0 ? -1 : o / a.fan;
  }
  if (row < 0 || row >= a.x_rows) return 0.0f;
  return to_float(static_cast<const T*>(a.x)[row * a.x_stride + c]);
}

// C[64 x 64] of A [64 x depth] times B [depth x 64], both staged in shared memory.
struct Tile {
  float a[kDepth][kTile + 1];
  float b[kDepth][kTile + 1];
};
__device__ __forceinline__ void multiply(const Tile& s, float (&acc)[4][4]) {
  const int ty = threadIdx.x / 16, tx = threadIdx.x % 16;
#pragma unroll
  for (int k = 0; k < kDepth; ++k) {
    float x[4], y[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = s.a[k][ty + 16 * i];
#pragma unroll
    for (int j = 0; j < 4; ++j) y[j] = s.b[k][tx + 16 * j];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) acc[i][j] = fmaf(x[i], y[j], acc[i][j]);
  }
}

template <typename T, typename O>
__global__ void __launch_bounds__(kThreads) rows_kernel(ProductArgs a) {
  __shared__ Tile s;
  const int cols = a.kind == kForward ? a.outer : a.inner;
  const int depth = a.kind == kForward ? a.inner : a.outer;
  // Row tile blockIdx.y of the groups' tiles laid end to end; the rows behind
  // the last group are one more group, of zeros.
  int64_t tile = blockIdx.y, begin = 0, end = 0;
  int g = 0;
  for (; g <= a.groups; ++g) {
    end = g < a.groups ? max(group_end(a, g), begin) : a.n;
    const int64_t tiles = (end - begin + kTile - 1) / kTile;
    if (tile < tiles) break;
    tile -= tiles;
    begin = end;
  }
  if (g > a.groups) return;
  const int64_t p0 = begin + tile * kTile;
  const int c0 = blockIdx.x * kTile;
  float acc[4][4] = {};
  if (g < a.groups) {
    const T* w = static_cast<const T*>(a.w) + g * a.w_group_stride;
    for (int k0 = 0; k0 < depth; k0 += kDepth) {
      for (int i = threadIdx.x; i < kTile * kDepth; i += kThreads) {
        const int r = i / kDepth, k = i % kDepth;
        s.a[k][r] = p0 + r < end && k0 + k < depth ? source<T>(a, p0 + r, k0 + k) : 0.0f;
        const int c = a.kind == kForward ? i / kDepth : i % kTile;
        const int kw = a.kind == kForward ? i % kDepth : i / kTile;
        const int64_t at = a.kind == kForward ? (c0 + c) * a.w_stride + k0 + kw
                                              : (k0 + kw) * a.w_stride + c0 + c;
        s.b[kw][c] = c0 + c < cols && k0 + kw < depth ? to_float(w[at]) : 0.0f;
      }
      __syncthreads();
      multiply(s, acc);
      __syncthreads();
    }
  }
  const int ty = threadIdx.x / 16, tx = threadIdx.x % 16;
  for (int i = 0; i < 4; ++i)
    for (int j = 0; j < 4; ++j) {
      const int64_t p = p0 + ty + 16 * i;
      const int c = c0 + tx + 16 * j;
      if (p < end && c < cols) static_cast<O*>(a.out)[p * cols + c] = from_float<O>(acc[i][j]);
    }
}

template <typename T, typename O>
__global__ void __launch_bounds__(kThreads) weight_grad_kernel(ProductArgs a) {
  __shared__ Tile s;
  const int g = blockIdx.z;
  int64_t begin = 0, end = 0;
  for (int i = 0; i <= g; ++i) {
    begin = end;
    end = max(group_end(a, i), begin);
  }
  const int n0 = blockIdx.y * kTile, k0 = blockIdx.x * kTile;
  float acc[4][4] = {};
  for (int64_t p0 = begin; p0 < end; p0 += kDepth) {
    for (int i = threadIdx.x; i < kTile * kDepth; i += kThreads) {
      const int c = i % kTile;
      const int64_t p = p0 + i / kTile;
      s.a[i / kTile][c] = p < end && n0 + c < a.outer
                              ? to_float(static_cast<const T*>(a.w)[p * a.w_stride + n0 + c]) : 0.0f;
      s.b[i / kTile][c] = p < end && k0 + c < a.inner ? source<T>(a, p, k0 + c) : 0.0f;
    }
    __syncthreads();
    multiply(s, acc);
    __syncthreads();
  }
  const int ty = threadIdx.x / 16, tx = threadIdx.x % 16;
  for (int i = 0; i < 4; ++i)
    for (int j = 0; j < 4; ++j) {
      const int n = n0 + ty + 16 * i, k = k0 + tx + 16 * j;
      if (n < a.outer && k < a.inner)
        static_cast<O*>(a.out)[(static_cast<int64_t>(g) * a.outer + n) * a.inner + k] =
            from_float<O>(acc[i][j]);
    }
}

template <typename T, typename O>
cudaError_t launch(const ProductArgs& a, cudaStream_t stream) {
  if (a.kind == kWeightGrad) {
    const dim3 grid((a.inner + kTile - 1) / kTile, (a.outer + kTile - 1) / kTile, a.groups);
    weight_grad_kernel<T, O><<<grid, kThreads, 0, stream>>>(a);
  } else {
    const int cols = a.kind == kForward ? a.outer : a.inner;
    const int64_t tiles = a.n / kTile + std::min<int64_t>(a.groups + 1, a.n);
    rows_kernel<T, O><<<dim3((cols + kTile - 1) / kTile, static_cast<unsigned>(tiles)), kThreads, 0,
                        stream>>>(a);
  }
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_product(const ProductArgs& a, cudaStream_t stream) {
  if (a.dtype == DSMEM_F16)
    return a.out_dtype == DSMEM_F32 ? launch<__half, float>(a, stream)
                                    : launch<__half, __half>(a, stream);
  return a.out_dtype == DSMEM_F32 ? launch<__nv_bfloat16, float>(a, stream)
                                  : launch<__nv_bfloat16, __nv_bfloat16>(a, stream);
}

}  // namespace dsmh
