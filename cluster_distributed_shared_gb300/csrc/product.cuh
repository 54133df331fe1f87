// What the kernels of products grouped by key share: bounded waits, matrix
// descriptors, the groups' tables, shared-memory accesses, tensor maps.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "bounded_wait.h"
#include "experts.h"
#include "ptx.cuh"
#include "tcgen.cuh"

namespace dsmh {
namespace {

using namespace ptx;

constexpr uint32_t kFull = 0xffffffffu;

__device__ uint32_t g_product_status;  // kStatusProduct once a bounded wait gave up

__device__ __forceinline__ uint32_t flag_set(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.volatile.shared.u32 %0, [%1];" : "=r"(v) : "r"(addr));
  return v;
}

// Waits for phase `parity` of an mbarrier, at most `limit` cycles or until
// another wait of this CTA has given up.
__device__ __noinline__ bool wait_slow(uint32_t mbar, uint32_t parity, uint32_t gave_up, long long limit,
                                       uint32_t* status) {
  const Waited how = bounded_wait([&] { return mbar_try_wait(mbar, parity); },
                                  [&] { return flag_set(gave_up) != 0u; }, [] { return clock64(); }, limit);
  if (how != Waited::kGaveUp) return how == Waited::kArrived;
  asm volatile("st.volatile.shared.u32 [%0], %1;" ::"r"(gave_up), "r"(1u) : "memory");
  atomicOr(&g_product_status, kStatusProduct);
  if (status) *reinterpret_cast<volatile uint32_t*>(status) = kStatusProduct;
  return false;
}
__device__ __forceinline__ bool wait_for(uint32_t mbar, uint32_t parity, uint32_t gave_up,
                                         long long limit, uint32_t* status) {
  return mbar_try_wait(mbar, parity) || wait_slow(mbar, parity, gave_up, limit, status);
}

// Reads (synchronously) and clears this file's status word.
inline cudaError_t take_product_status(uint32_t* out) {
  cudaError_t e = cudaMemcpyFromSymbol(out, g_product_status, sizeof(uint32_t));
  if (e != cudaSuccess) return e;
  const uint32_t zero = 0;
  return *out ? cudaMemcpyToSymbol(g_product_status, &zero, sizeof(uint32_t)) : cudaSuccess;
}

// Shared-memory matrix descriptors, 128-byte swizzle.  K-major: rows of 128
// bytes, groups of 8 rows 1024 bytes apart.  MN-major: boxes of 64 elements by
// 64 depth, 8192 bytes each, in them groups of 8 depth 1024 bytes apart.
constexpr uint64_t kDescBase = (uint64_t{1} << 46) | (uint64_t{2} << 61) | (uint64_t{1024 >> 4} << 32);
template <bool kMnMajor>
__device__ __forceinline__ uint64_t descriptor(uint32_t addr) {
  return kDescBase | (uint64_t{kMnMajor ? 8192 >> 4 : 1} << 16) | ((addr & 0x3ffffu) >> 4);
}

__device__ __forceinline__ uint4 ld_shared_16(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}
template <typename P>
__device__ __forceinline__ void st_shared_16(uint32_t addr, const P& p) {
  static_assert(sizeof(P) == 16, "one vector");
  const uint4 v = *reinterpret_cast<const uint4*>(&p);
  asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w)
               : "memory");
}
template <typename O>
__device__ __forceinline__ void st_shared_value(uint32_t addr, O v) {
  if constexpr (sizeof(O) == 2) {
    asm volatile("st.shared.u16 [%0], %1;" ::"r"(addr), "h"(*reinterpret_cast<const uint16_t*>(&v)) : "memory");
  } else {
    asm volatile("st.shared.f32 [%0], %1;" ::"r"(addr), "f"(static_cast<float>(v)) : "memory");
  }
}

template <typename O>
__device__ __forceinline__ O ld_shared_value(uint32_t addr) {
  O v;
  if constexpr (sizeof(O) == 2) {
    uint16_t bits;
    asm volatile("ld.shared.u16 %0, [%1];" : "=h"(bits) : "r"(addr) : "memory");
    *reinterpret_cast<uint16_t*>(&v) = bits;
  } else {
    float bits;
    asm volatile("ld.shared.f32 %0, [%1];" : "=f"(bits) : "r"(addr) : "memory");
    v = static_cast<O>(bits);
  }
  return v;
}

// A CTA's shared memory (227 KB) but for what lay_groups takes of it: a kernel's
// limit is on the sum.
constexpr int kMostShared = 227 * 1024 - 2 * 32 * static_cast<int>(sizeof(int));

// The groups' tables in shared memory, by all kThreads threads: begin[g], the
// first row of group g (begin[groups + 1] = n), from the offsets clamped into
// [0, n] and made monotone, and (where asked for) first[g], the first tile of
// each of `owners` groups laid end to end.  `meanwhile` runs before the first
// barrier.
template <int kThreads, typename TilesOf, typename Meanwhile>
__device__ __forceinline__ void lay_groups(const int32_t* offsets, int64_t n, int groups, int owners, int32_t* begin,
                                           int32_t* first, TilesOf tiles_of, Meanwhile meanwhile) {
  const int warp = __shfl_sync(kFull, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  for (int g = threadIdx.x; g < groups; g += kThreads) {
    const int64_t e = offsets[g + 1];
    begin[g + 1] = static_cast<int32_t>(e < 0 ? 0 : (e > n ? n : e));
  }
  if (threadIdx.x == 0) {
    begin[0] = 0;
    if (first) first[0] = 0;
    begin[groups + 1] = static_cast<int32_t>(n);
  }
  meanwhile();
  __syncthreads();
  // Each warp takes 32 groups of every kWarps * 32: the running maximum
  // of their ends, then the running sum of their tiles.
  constexpr int kWarps = kThreads / 32;
  __shared__ int of_warp[2][32];  // counted in kMostShared
  int end_before = 0, tiles_before = 0;
  for (int g0 = 0; g0 < owners; g0 += kWarps * 32) {
    const int g = g0 + warp * 32 + lane;
    const bool owner = g < owners;
    int end = owner ? begin[g + 1] : 0;
    const int most = __reduce_max_sync(kFull, end);
    if (lane == 0) of_warp[0][warp] = most;
    __syncthreads();
    const int other = lane < kWarps ? of_warp[0][lane] : 0;
    const int earlier = max(end_before, __reduce_max_sync(kFull, lane < warp ? other : 0));
    end_before = max(end_before, __reduce_max_sync(kFull, other));
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int up = __shfl_up_sync(kFull, end, d);
      if (lane >= d) end = max(end, up);
    }
    end = max(end, earlier);
    int start = __shfl_up_sync(kFull, end, 1);
    if (lane == 0) start = earlier;
    int tiles = owner ? tiles_of(end - start) : 0;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int up = __shfl_up_sync(kFull, tiles, d);
      if (lane >= d) tiles += up;
    }
    if (lane == 31) of_warp[1][warp] = tiles;
    __syncthreads();
    const int sum = lane < kWarps ? of_warp[1][lane] : 0;
    tiles += tiles_before + __reduce_add_sync(kFull, lane < warp ? sum : 0);
    tiles_before += __reduce_add_sync(kFull, sum);
    if (owner) {
      begin[g + 1] = end;
      if (first) first[g + 1] = tiles;
    }
  }
}

using EncodeFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                              const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                              CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
inline EncodeFn encoder() {
  static EncodeFn fn = [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult found;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &found) !=
            cudaSuccess || found != cudaDriverEntryPointSuccess)
      p = nullptr;
    return reinterpret_cast<EncodeFn>(p);
  }();
  return fn;
}

inline cudaLaunchAttribute cluster_of(int ctas) {
  cudaLaunchAttribute a = {};
  a.id = cudaLaunchAttributeClusterDimension;
  a.val.clusterDim.x = static_cast<unsigned>(ctas);
  a.val.clusterDim.y = a.val.clusterDim.z = 1;
  return a;
}

}  // namespace
}  // namespace dsmh
