// The global norm of many gradients, and clipping by it.
//
// Two passes over the gradients: squares, then scaling.  Tensors are cut into
// chunks of kChunk elements; CTA b of a launch takes chunks b, b + grid, ..
// The table of tensors travels as a kernel parameter, so nothing is copied to
// the device first and nothing is kept between calls.
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include <algorithm>

#include "dtypes.cuh"
#include "experts.h"

namespace dsmh {
namespace {

constexpr int kThreads = 256;
constexpr int kPerThread = 32;                    // elements of one thread in a chunk
constexpr int kChunk = kThreads * kPerThread;     // 8192
constexpr int kMaxTensors = 960;                  // per launch; the table stays under 32,764 bytes

struct Tensor {
  const void* grad;
  void* out;
  int64_t count : 60;
  int64_t dtype : 4;
};
struct Table {
  Tensor t[kMaxTensors];
  uint32_t first_chunk[kMaxTensors + 1];
  int32_t tensors;
  uint32_t chunks;
};
static_assert(sizeof(Table) + 64 <= 32764, "kernel parameters");

__device__ __forceinline__ int find_tensor(const Table& tab, uint32_t chunk) {
  int lo = 0, hi = tab.tensors - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (tab.first_chunk[mid] <= chunk) lo = mid; else hi = mid - 1;
  }
  return lo;
}

// One thread's elements of a chunk: vectors of V, interleaved over the CTA.
template <typename T, int V>
struct Slice {
  Pack<T, V> p[kPerThread / V];
  int64_t base;
  __device__ __forceinline__ static int64_t at(int64_t base, int k) {
    return base + (static_cast<int64_t>(k) * kThreads + threadIdx.x) * V;
  }
  __device__ __forceinline__ void load(const T* x, int64_t b, int64_t count) {
    base = b;
#pragma unroll
    for (int k = 0; k < kPerThread / V; ++k) {
      const int64_t i = at(base, k);
      if (i + V <= count) {
        p[k] = *reinterpret_cast<const Pack<T, V>*>(x + i);
      } else {
#pragma unroll
        for (int v = 0; v < V; ++v) p[k].v[v] = i + v < count ? x[i + v] : from_float<T>(0.0f);
      }
    }
  }
};

// Sum of squares of a slice.  32 squares are summed in 32 bits; where that
// left their range (a sum that overflowed, or so small that squares may have
// been lost) they are summed again in 64.
template <typename T, int V>
__device__ __forceinline__ double squares(const Slice<T, V>& s) {
  float sum = 0.0f, top = 0.0f;
#pragma unroll
  for (int k = 0; k < kPerThread / V; ++k)
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const float x = to_float(s.p[k].v[v]);
      sum = fmaf(x, x, sum);
      top = fmaxf(top, fabsf(x));
    }
  if ((sum > 1e-30f && sum < 1e37f) || (sum == 0.0f && top == 0.0f)) return sum;
  double exact = 0.0;
#pragma unroll
  for (int k = 0; k < kPerThread / V; ++k)
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const double x = to_float(s.p[k].v[v]);
      exact = fma(x, x, exact);
    }
  return exact;
}

template <typename T>
__device__ __forceinline__ bool wide(const Tensor& t) {
  return ((reinterpret_cast<uintptr_t>(t.grad) | reinterpret_cast<uintptr_t>(t.out)) & 15u) == 0;
}

template <typename T>
__device__ __forceinline__ double chunk_squares(const Tensor& t, int64_t base) {
  const T* x = static_cast<const T*>(t.grad);
  if (wide<T>(t)) {
    Slice<T, 16 / sizeof(T)> s;
    s.load(x, base, t.count);
    return squares(s);
  }
  Slice<T, 1> s;
  s.load(x, base, t.count);
  return squares(s);
}

template <typename T, int V>
__device__ __forceinline__ void scale_slice(const Tensor& t, int64_t base, float scale) {
  Slice<T, V> s;
  s.load(static_cast<const T*>(t.grad), base, t.count);
  T* out = static_cast<T*>(t.out);
#pragma unroll
  for (int k = 0; k < kPerThread / V; ++k) {
#pragma unroll
    for (int v = 0; v < V; ++v) s.p[k].v[v] = from_float<T>(to_float(s.p[k].v[v]) * scale);
    const int64_t i = Slice<T, V>::at(base, k);
    if (i + V <= t.count) {
      *reinterpret_cast<Pack<T, V>*>(out + i) = s.p[k];
    } else {
#pragma unroll
      for (int v = 0; v < V; ++v)
        if (i + v < t.count) out[i + v] = s.p[k].v[v];
    }
  }
}
template <typename T>
__device__ __forceinline__ void chunk_scale(const Tensor& t, int64_t base, float scale) {
  if (wide<T>(t)) scale_slice<T, 16 / sizeof(T)>(t, base, scale);
  else scale_slice<T, 1>(t, base, scale);
}

// Sum over the CTA in a fixed order (valid in every thread).
__device__ __forceinline__ double cta_sum(double v) {
  __shared__ double part[kThreads / 32];
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = v;
  __syncthreads();
  double sum = 0.0;
#pragma unroll
  for (int k = 0; k < kThreads / 32; ++k) sum += part[k];
  return sum;
}

__global__ void __launch_bounds__(kThreads) norm_kernel(const __grid_constant__ Table tab,
                                                        double* partial) {
  double sum = 0.0;
  for (uint32_t c = blockIdx.x; c < tab.chunks; c += gridDim.x) {
    const int i = find_tensor(tab, c);
    const Tensor& t = tab.t[i];
    const int64_t base = static_cast<int64_t>(c - tab.first_chunk[i]) * kChunk;
    if (t.dtype == DSMEM_F32) sum += chunk_squares<float>(t, base);
    else if (t.dtype == DSMEM_F16) sum += chunk_squares<__half>(t, base);
    else sum += chunk_squares<__nv_bfloat16>(t, base);
  }
  sum = cta_sum(sum);
  if (threadIdx.x == 0) partial[blockIdx.x] = sum;
}

__global__ void __launch_bounds__(kThreads) scale_kernel(const __grid_constant__ Table tab,
                                                         const double* partial, int partials,
                                                         float max_norm, float* norm) {
  double sum = 0.0;
  for (int i = threadIdx.x; i < partials; i += kThreads) sum += partial[i];
  const double total = sqrt(cta_sum(sum));
  if (norm && blockIdx.x == 0 && threadIdx.x == 0) *norm = static_cast<float>(total);
  const double ratio = max_norm / (total + 1e-6);
  const float scale = ratio > 1.0 ? 1.0f : static_cast<float>(ratio);  // NaN stays NaN
  for (uint32_t c = blockIdx.x; c < tab.chunks; c += gridDim.x) {
    const int i = find_tensor(tab, c);
    const Tensor& t = tab.t[i];
    const int64_t base = static_cast<int64_t>(c - tab.first_chunk[i]) * kChunk;
    if (t.dtype == DSMEM_F32) chunk_scale<float>(t, base, scale);
    else if (t.dtype == DSMEM_F16) chunk_scale<__half>(t, base, scale);
    else chunk_scale<__nv_bfloat16>(t, base, scale);
  }
}

// Fills a launch's table from grads[first..]; returns the next index.  A
// tensor too long for the chunk counter continues in the next launch.
struct Cursor {
  int tensor = 0;
  int64_t done = 0;  // elements of that tensor already taken
};
void fill(Table* tab, const dsmem_grad_t* grads, int num, Cursor* at) {
  tab->tensors = 0;
  uint32_t chunks = 0;
  constexpr uint32_t kMaxChunks = 1u << 30;
  while (at->tensor < num && tab->tensors < kMaxTensors && chunks < kMaxChunks) {
    const dsmem_grad_t& g = grads[at->tensor];
    const int64_t left = g.count - at->done;
    if (left > 0) {
      const int64_t room = static_cast<int64_t>(kMaxChunks - chunks) * kChunk;
      const int64_t take = std::min(left, room);
      Tensor& t = tab->t[tab->tensors];
      const int64_t skip = at->done * dtype_size(g.dtype);
      t.grad = static_cast<const char*>(g.grad) + skip;
      t.out = static_cast<char*>(g.out) + skip;
      t.count = take;
      t.dtype = g.dtype;
      tab->first_chunk[tab->tensors++] = chunks;
      chunks += static_cast<uint32_t>((take + kChunk - 1) / kChunk);
      at->done += take;
    }
    if (at->done == g.count) {
      ++at->tensor;
      at->done = 0;
    }
  }
  tab->first_chunk[tab->tensors] = chunks;
  tab->chunks = chunks;
}

}  // namespace

int run_grad_clip(const dsmem_grad_t* grads, int32_t num, float max_norm, float* norm,
                  const CallContext& ctx, cudaStream_t stream) {
  const int grid_max = ctx.sm_count * 8;
  int launches = 0;
  Table tab;
  for (Cursor at; at.tensor < num || launches == 0; ++launches) fill(&tab, grads, num, &at);
  double* partial = nullptr;
  int rc = pool_alloc(ctx, reinterpret_cast<void**>(&partial),
                      sizeof(double) * static_cast<size_t>(grid_max) * launches, stream);
  if (rc) return rc;
  cudaError_t e = cudaSuccess;
  int partials = 0;
  Cursor at;
  for (int l = 0; l < launches && e == cudaSuccess; ++l) {
    fill(&tab, grads, num, &at);
    const int grid = static_cast<int>(std::min<uint32_t>(std::max(tab.chunks, 1u), grid_max));
    norm_kernel<<<grid, kThreads, 0, stream>>>(tab, partial + partials);
    partials += grid;
    e = cudaGetLastError();
  }
  at = Cursor();
  for (int l = 0; l < launches && e == cudaSuccess; ++l) {
    if (launches > 1) fill(&tab, grads, num, &at);
    const int grid = static_cast<int>(std::min<uint32_t>(std::max(tab.chunks, 1u), grid_max));
    scale_kernel<<<grid, kThreads, 0, stream>>>(tab, partial, partials, max_norm,
                                                l == 0 ? norm : nullptr);
    e = cudaGetLastError();
  }
  rc = pool_free(partial, stream);
  if (e != cudaSuccess) return fail_with_cuda(e, "gradient clipping launch");
  return rc;
}

}  // namespace dsmh
