// The global norm of many gradients, and clipping by it.
//
// Two passes over the gradients: squares, then scaling.  Tensors are cut into
// chunks of 16 KB laid end to end, and every CTA takes an equal run of them in
// the first pass, so that the order of the sums depends on the sizes alone.
// The second pass goes through the runs backwards, so that it begins with what
// the first left in L2, and stores past the cache; a CTA scales the end of its
// own run and then pieces of any, as SMs differ in how fast they reach memory.
// The table of tensors travels as a kernel parameter: nothing is copied to the
// device first and nothing is kept between calls.
//
// Bound by memory: 1 GiB of bf16 takes 488 us, 6.6 TB/s over its two reads and
// one write (four CTAs an SM with four 16-byte vectors a thread; before the
// second pass shared its pieces 511, and with that six CTAs 541, eight vectors
// 533).
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include <algorithm>

#include "dtypes.cuh"
#include "experts.h"

namespace dsmh {
namespace {

constexpr int kThreads = 256;
constexpr int kCtasPerSm = 4;
constexpr int kVectors = 4;                            // 16-byte vectors of one thread in a chunk
constexpr int kChunkBytes = kThreads * kVectors * 16;  // 16 KB

struct Tensor {
  const void* grad;
  void* out;
  int64_t count : 60;
  int64_t dtype : 4;
};
// kTensors: 128 for short lists, else as many as 32,764 bytes of parameters hold.
constexpr int kFewTensors = 128, kMostTensors = 1100;
template <int kTensors>
struct Table {
  Tensor t[kTensors];
  uint32_t first_chunk[kTensors + 1];
  int32_t tensors;
  uint32_t chunks;
};
static_assert(sizeof(Table<kMostTensors>) + 64 <= 32764, "kernel parameters");

// The tensor of a chunk, from the chunks before or behind it.
template <typename Tab>
__device__ __forceinline__ int find_tensor(const Tab& tab, uint32_t chunk) {
  int lo = 0, hi = tab.tensors - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (tab.first_chunk[mid] <= chunk) lo = mid; else hi = mid - 1;
  }
  return lo;
}

// One thread's elements of a chunk: 16-byte vectors, or (kWide false, where
// the addresses allow none) single elements, interleaved over the CTA.
template <typename T, bool kWide>
struct Slice {
  static constexpr int kEach = kWide ? 16 / static_cast<int>(sizeof(T)) : 2;  // elements of a piece
  static constexpr int kPieces = kVectors * 16 / static_cast<int>(sizeof(T)) / kEach;
  static constexpr int kPairs = kEach / 2;
  Vector16<T> p[kWide ? kPieces : 1];
  T single[kWide ? 1 : kPieces][2];

  // The i-th element of piece k is element first(base, k) + i * kStep of the tensor.
  __device__ __forceinline__ static int64_t first(int64_t base, int k) {
    return kWide ? base + (k * kThreads + static_cast<int>(threadIdx.x)) * kEach
                 : base + k * 2 * kThreads + static_cast<int>(threadIdx.x);
  }
  static constexpr int kStep = kWide ? 1 : kThreads;

  __device__ __forceinline__ float2 get(int k, int pair) const {
    if constexpr (kWide) return p[k].get(pair);
    else return make_float2(to_float(single[k][0]), to_float(single[k][1]));
  }
  template <bool kLast>
  __device__ __forceinline__ void load(const T* x, int64_t base, int64_t count) {
#pragma unroll
    for (int k = 0; k < kPieces; ++k) {
      const int64_t i = first(base, k);
      if constexpr (kWide) {
        if (i + kEach <= count) {
          const uint4* q = reinterpret_cast<const uint4*>(x + i);
          p[k].words(kLast ? __ldcs(q) : __ldg(q));
        } else {
          alignas(16) T part[kEach];
#pragma unroll
          for (int v = 0; v < kEach; ++v) part[v] = i + v < count ? x[i + v] : from_float<T>(0.0f);
          p[k].words(*reinterpret_cast<const uint4*>(part));
        }
      } else {
#pragma unroll
        for (int v = 0; v < 2; ++v)
          single[k][v] = i + v * kStep < count ? x[i + v * kStep] : from_float<T>(0.0f);
      }
    }
  }
  // Stores every element times `scale`.
  __device__ __forceinline__ void store_scaled(T* out, int64_t base, int64_t count, float scale) {
#pragma unroll
    for (int k = 0; k < kPieces; ++k) {
      const int64_t i = first(base, k);
      if constexpr (kWide) {
#pragma unroll
        for (int q = 0; q < kPairs; ++q) p[k].set(q, mul2(p[k].get(q), make_float2(scale, scale)));
        if (i + kEach <= count) {
          __stcs(reinterpret_cast<uint4*>(out + i), p[k].words());
        } else {
          alignas(16) T part[kEach];
          *reinterpret_cast<uint4*>(part) = p[k].words();
#pragma unroll
          for (int v = 0; v < kEach; ++v)
            if (i + v < count) out[i + v] = part[v];
        }
      } else {
#pragma unroll
        for (int v = 0; v < 2; ++v)
          if (i + v * kStep < count) out[i + v * kStep] = from_float<T>(to_float(single[k][v]) * scale);
      }
    }
  }
};

// A sum held as two floats, hi + lo, with lo the rounding errors of hi
// (Knuth's two-sum), about 48 bits.  Doubles would do, but their adder takes
// 16 clocks for a warp here: sums in doubles cost a sixth of the norm pass.
struct Sum {
  float hi = 0.0f, lo = 0.0f;
  __device__ __forceinline__ void add(float x) {
    const float s = hi + x, b = s - hi;
    lo += (hi - (s - b)) + (x - b);
    hi = s;
  }
  __device__ __forceinline__ void add(const Sum& o) {
    add(o.hi);
    lo += o.lo;
  }
};
// What one thread, or one CTA, has seen: ordinary squares in `sum`, those
// outside its range in `rest`.
struct Squares {
  Sum sum;
  double rest = 0.0;
};

// Adds the squares of a slice.  Up to 32 squares are summed in 32 bits; where
// that leaves the range in which nothing overflows or is lost, they are summed
// again in 64.
template <typename S>
__device__ __forceinline__ void add_squares(const S& s, Squares* to) {
  float2 pair = make_float2(0.0f, 0.0f);
#pragma unroll
  for (int k = 0; k < S::kPieces; ++k)
#pragma unroll
    for (int q = 0; q < S::kPairs; ++q) {
      const float2 x = s.get(k, q);
      pair = fma2(x, x, pair);
    }
  const float sum = pair.x + pair.y;
  if (sum > 1e-30f && sum < 1e30f) {
    to->sum.add(sum);
    return;
  }
  float top = 0.0f;
#pragma unroll
  for (int k = 0; k < S::kPieces; ++k)
#pragma unroll
    for (int q = 0; q < S::kPairs; ++q) {
      const float2 x = s.get(k, q);
      top = fmaxf(top, fmaxf(fabsf(x.x), fabsf(x.y)));
    }
  if (sum == 0.0f && top == 0.0f) return;
  double exact = 0.0;
#pragma unroll
  for (int k = 0; k < S::kPieces; ++k)
#pragma unroll
    for (int q = 0; q < S::kPairs; ++q) {
      const float2 x = s.get(k, q);
      exact = fma(static_cast<double>(x.x), static_cast<double>(x.x), exact);
      exact = fma(static_cast<double>(x.y), static_cast<double>(x.y), exact);
    }
  to->rest += exact;
}

__device__ __forceinline__ bool wide(const Tensor& t) {
  return ((reinterpret_cast<uintptr_t>(t.grad) | reinterpret_cast<uintptr_t>(t.out)) & 15u) == 0;
}

template <typename T>
__device__ __forceinline__ void chunk_squares(const Tensor& t, int64_t chunk, Squares* to) {
  const int64_t base = chunk * (kChunkBytes / static_cast<int>(sizeof(T)));
  const T* x = static_cast<const T*>(t.grad);
  if (wide(t)) {
    Slice<T, true> s;
    s.template load<false>(x, base, t.count);
    add_squares(s, to);
  } else {
    Slice<T, false> s;
    s.template load<false>(x, base, t.count);
    add_squares(s, to);
  }
}

template <typename T>
__device__ __forceinline__ void chunk_scale(const Tensor& t, int64_t chunk, float scale) {
  const int64_t base = chunk * (kChunkBytes / static_cast<int>(sizeof(T)));
  const T* x = static_cast<const T*>(t.grad);
  if (wide(t)) {
    Slice<T, true> s;
    s.template load<true>(x, base, t.count);
    s.store_scaled(static_cast<T*>(t.out), base, t.count, scale);
  } else {
    Slice<T, false> s;
    s.template load<true>(x, base, t.count);
    s.store_scaled(static_cast<T*>(t.out), base, t.count, scale);
  }
}

// Sum over the CTA in a fixed order, valid in thread 0.
__device__ __forceinline__ double cta_sum(Squares v) {
  __shared__ double part[kThreads / 32];
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) {
    Sum o;
    o.hi = __shfl_xor_sync(0xffffffffu, v.sum.hi, d);
    o.lo = __shfl_xor_sync(0xffffffffu, v.sum.lo, d);
    v.sum.add(o);
  }
  if (__any_sync(0xffffffffu, !(v.rest == 0.0)))
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) v.rest += __shfl_xor_sync(0xffffffffu, v.rest, d);
  if ((threadIdx.x & 31) == 0)
    part[threadIdx.x >> 5] = static_cast<double>(v.sum.hi) + v.sum.lo + v.rest;
  __syncthreads();
  double sum = 0.0;
  if (threadIdx.x == 0)
    for (int k = 0; k < kThreads / 32; ++k) sum += part[k];
  return sum;
}

// A CTA's squares; `hi` and `lo` hold them too where they are in a float's
// ordinary range, else `hi` is NaN.
struct alignas(16) Partial {
  double exact;
  Sum sum;
};

// The run of a table's chunks that belongs to a CTA.
__device__ __forceinline__ void run_of(uint32_t cta, uint32_t chunks, uint32_t* begin, uint32_t* end) {
  *begin = static_cast<uint32_t>(static_cast<uint64_t>(chunks) * cta / gridDim.x);
  *end = static_cast<uint32_t>(static_cast<uint64_t>(chunks) * (cta + 1) / gridDim.x);
}

template <int kTensors>
__global__ void __launch_bounds__(kThreads, kCtasPerSm)
    norm_kernel(const __grid_constant__ Table<kTensors> tab, Partial* partial, uint32_t* taken) {
  uint32_t c, end;
  run_of(blockIdx.x, tab.chunks, &c, &end);
  Squares mine;
  int i = c < end ? find_tensor(tab, c) : 0;
  for (; c < end; ++c) {
    while (c >= tab.first_chunk[i + 1]) ++i;
    const Tensor& t = tab.t[i];
    const int64_t k = c - tab.first_chunk[i];
    if (t.dtype == DSMEM_F32) chunk_squares<float>(t, k, &mine);
    else if (t.dtype == DSMEM_F16) chunk_squares<__half>(t, k, &mine);
    else chunk_squares<__nv_bfloat16>(t, k, &mine);
  }
  const double sum = cta_sum(mine);
  if (threadIdx.x == 0) {
    Partial p;
    p.exact = sum;
    const bool ordinary = sum == 0.0 || (sum > 1e-25 && sum < 1e33);
    p.sum.hi = ordinary ? static_cast<float>(sum) : NAN;
    p.sum.lo = ordinary ? static_cast<float>(sum - p.sum.hi) : 0.0f;
    partial[blockIdx.x] = p;
    if (blockIdx.x == 0) *taken = 0;  // for the scaling
  }
}

template <int kTensors>
__device__ __forceinline__ void scale_chunks(const Table<kTensors>& tab, uint32_t begin, uint32_t c,
                                             float scale) {
  int i = begin < c ? find_tensor(tab, c - 1) : 0;
  while (c-- > begin) {
    while (c < tab.first_chunk[i]) --i;
    const Tensor& t = tab.t[i];
    const int64_t k = c - tab.first_chunk[i];
    if (t.dtype == DSMEM_F32) chunk_scale<float>(t, k, scale);
    else if (t.dtype == DSMEM_F16) chunk_scale<__half>(t, k, scale);
    else chunk_scale<__nv_bfloat16>(t, k, scale);
  }
}

// Of runs of kShared chunks and more a CTA scales the last quarter of its own,
// and pieces of kPiece chunks as `taken` hands them out: the first of every
// run, the second of every run and so on, from the end.  1 GiB of bf16, us: own
// quarter 488, half 490, none 490 (pieces of 8 chunks: 490, 492, 490), without
// pieces 505.  Shorter runs are mostly in L2 and gain nothing; without pieces /
// with: 128 MiB (13 chunks) 69.7 / 74.4, 256 MiB (26) 134.1 / 135.7, 384 MiB
// (40) 202.2 / 200.4, 512 MiB (53) 262.6 / 256.3.
// At its limit of 64 registers (four CTAs an SM) the kernel spills 40 bytes a
// thread, 44 read back.
constexpr uint32_t kShared = 32, kPiece = 4;

template <int kTensors>
__global__ void __launch_bounds__(kThreads, kCtasPerSm)
    scale_kernel(const __grid_constant__ Table<kTensors> tab, const Partial* partial, int partials,
                 uint32_t* taken, float max_norm, float* norm) {
  // Every CTA adds the partial sums, thread 0 turns them into the factor.
  __shared__ float factor;
  Squares mine;
  for (int i = threadIdx.x; i < partials; i += kThreads) {
    const Partial p = partial[i];
    if (p.sum.hi == p.sum.hi) mine.sum.add(p.sum);
    else mine.rest += p.exact;
  }
  const double squares = cta_sum(mine);
  if (threadIdx.x == 0) {
    const double total = sqrt(squares);
    if (norm && blockIdx.x == 0) *norm = static_cast<float>(total);
    const double ratio = max_norm / (total + 1e-6);
    factor = ratio > 1.0 ? 1.0f : static_cast<float>(ratio);  // NaN stays NaN
  }
  __syncthreads();
  const float scale = factor;
  uint32_t begin, end;
  run_of(blockIdx.x, tab.chunks, &begin, &end);
  const uint32_t shortest = tab.chunks / gridDim.x;  // the others have one more
  if (shortest < kShared) {
    scale_chunks(tab, begin, end, scale);
    return;
  }
  const uint32_t own = shortest / 4, pieces = (shortest + 1 - own + kPiece - 1) / kPiece;
  scale_chunks(tab, end - own, end, scale);
  __shared__ uint32_t next;
  for (;;) {
    __syncthreads();
    if (threadIdx.x == 0) next = atomicAdd(taken, 1u);
    __syncthreads();
    const uint32_t piece = next / gridDim.x;
    if (piece >= pieces) return;
    run_of(next - piece * gridDim.x, tab.chunks, &begin, &end);
    const uint32_t length = end - begin, from = own + piece * kPiece;
    if (from < length) scale_chunks(tab, end - min(from + kPiece, length), end - from, scale);
  }
}

// Fills a launch's table from the cursor on.  A tensor whose two addresses
// share a misalignment becomes its head up to the next 16 bytes and the rest;
// one too long for the chunk counter goes on in the next launch.
struct Cursor {
  int tensor = 0;
  int64_t done = 0;  // elements of that tensor already taken
};
template <int kTensors>
void fill(Table<kTensors>* tab, const dsmem_grad_t* grads, int num, Cursor* at) {
  int n = 0;
  uint32_t chunks = 0;
  constexpr uint32_t kMaxChunks = 1u << 30;
  while (at->tensor < num && n < kTensors && chunks < kMaxChunks) {
    const dsmem_grad_t& g = grads[at->tensor];
    const int size = dtype_size(g.dtype);
    const int64_t left = g.count - at->done, per_chunk = kChunkBytes / size;
    if (left > 0) {
      Tensor& t = tab->t[n];
      t.grad = static_cast<const char*>(g.grad) + at->done * size;
      t.out = static_cast<char*>(g.out) + at->done * size;
      const uintptr_t off = reinterpret_cast<uintptr_t>(t.grad) & 15u;
      int64_t take = std::min(left, static_cast<int64_t>(kMaxChunks - chunks) * per_chunk);
      if (off != 0 && off == (reinterpret_cast<uintptr_t>(t.out) & 15u))
        take = std::min<int64_t>(take, (16 - off) / size);
      t.count = take;
      t.dtype = g.dtype;
      tab->first_chunk[n++] = chunks;
      chunks += static_cast<uint32_t>((take + per_chunk - 1) / per_chunk);
      at->done += take;
    }
    if (at->done == g.count) {
      ++at->tensor;
      at->done = 0;
    }
  }
  tab->first_chunk[n] = chunks;
  tab->tensors = n;
  tab->chunks = chunks;
}

template <int kTensors>
int run(const dsmem_grad_t* grads, int32_t num, float max_norm, float* norm, const CallContext& ctx,
        cudaStream_t stream) {
  const uint32_t most = static_cast<uint32_t>(ctx.sm_count * kCtasPerSm);
  Table<kTensors> tab;
  // One launch of each kernel for every table the list takes.
  int launches = 0;
  for (Cursor at; at.tensor < num || launches == 0; ++launches) fill(&tab, grads, num, &at);
  Partial* partial = nullptr;
  int rc = pool_alloc(ctx, reinterpret_cast<void**>(&partial),
                      (sizeof(Partial) * most + sizeof(uint32_t)) * launches, stream);
  if (rc) return rc;
  uint32_t* const taken = reinterpret_cast<uint32_t*>(partial + static_cast<size_t>(most) * launches);
  cudaError_t e = cudaSuccess;
  int partials = 0;
  Cursor at;
  for (int l = 0; l < launches && e == cudaSuccess; ++l) {
    if (launches > 1) fill(&tab, grads, num, &at);
    const uint32_t grid = std::min(std::max(tab.chunks, 1u), most);
    norm_kernel<kTensors><<<grid, kThreads, 0, stream>>>(tab, partial + partials, taken + l);
    partials += static_cast<int>(grid);
    e = cudaGetLastError();
  }
  at = Cursor();
  for (int l = 0; l < launches && e == cudaSuccess; ++l) {
    if (launches > 1) fill(&tab, grads, num, &at);
    const uint32_t grid = std::min(std::max(tab.chunks, 1u), most);
    scale_kernel<kTensors><<<grid, kThreads, 0, stream>>>(tab, partial, partials, taken + l, max_norm,
                                                          l == 0 ? norm : nullptr);
    e = cudaGetLastError();
  }
  rc = pool_free(partial, stream);
  if (e != cudaSuccess) return fail_with_cuda(e, "gradient clipping launch");
  return rc;
}

}  // namespace

int run_grad_clip(const dsmem_grad_t* grads, int32_t num, float max_norm, float* norm,
                  const CallContext& ctx, cudaStream_t stream) {
  // Each tensor may take two entries (a misaligned head and the rest).
  if (2 * num <= kFewTensors) return run<kFewTensors>(grads, num, max_norm, norm, ctx, stream);
  return run<kMostTensors>(grads, num, max_norm, norm, ctx, stream);
}

}  // namespace dsmh
