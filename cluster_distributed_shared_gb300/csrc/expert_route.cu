// Routing: the choice of each token's experts with its gradient, and the
// stable grouping of keys that puts rows in expert order.
#include <cuda_runtime.h>
#include <stdint.h>

#include "dtypes.cuh"
#include "experts.h"
#include "launch_rules.h"
#include "ptx.cuh"
#include "route.cuh"

namespace dsmh {
namespace {

using namespace ptx;

constexpr uint32_t kFull = kFullWarp;
constexpr int kRouteWarps = 4;

// R logits of a row, contiguous ones, in lane l those from l * R on.  kVector:
// rows are 16-byte aligned and their length is a multiple of R.
template <typename T, int R, bool kVector>
__device__ __forceinline__ void load_row(const T* row, int experts, float (&v)[R]) {
  const int first = (threadIdx.x & 31) * R;
  constexpr int kEach = 16 / static_cast<int>(sizeof(T));
  if constexpr (kVector && R % kEach == 0) {
#pragma unroll
    for (int r = 0; r < R; r += kEach) {
      Vector16<T> p;
      p.words(first < experts ? *reinterpret_cast<const uint4*>(row + first + r) : make_uint4(0, 0, 0, 0));
#pragma unroll
      for (int q = 0; q < kEach / 2; ++q) {
        const float2 x = p.get(q);
        v[r + 2 * q] = first < experts ? x.x : -INFINITY;
        v[r + 2 * q + 1] = first < experts ? x.y : -INFINITY;
      }
    }
  } else {
#pragma unroll
    for (int r = 0; r < R; ++r) v[r] = first + r < experts ? to_float(row[first + r]) : -INFINITY;
  }
}

// One warp per token, the row in registers.  Softmax statistics are 32-bit.
// Bound by instructions: 16384 tokens, 256 experts, 8 picks in 10.5 us; with 32
// logits a lane, some lanes empty below 1024 experts, 384 take 32 us, 1024 27.
template <typename T, int R, bool kVector>
__global__ void __launch_bounds__(kRouteWarps * 32) route_kernel(RouteArgs a) {
  const int64_t token = static_cast<int64_t>(blockIdx.x) * kRouteWarps + (threadIdx.x >> 5);
  if (token >= a.tokens) return;
  const int lane = threadIdx.x & 31;
  uint32_t keys[1][R];
  const uint32_t(&key)[R] = keys[0];
  {
    float v[R];
    load_row<T, R, kVector>(static_cast<const T*>(a.logits) + token * a.row_stride, a.experts, v);
#pragma unroll
    for (int r = 0; r < R; ++r) keys[0][r] = rank_key(v[r]);
  }
  Best best[1] = {two_best(key, 0u)};
  const float top = rank_value(__reduce_max_sync(kFull, best[0].key));
  float all = 0.0f;
  if (!a.renormalize) {
#pragma unroll
    for (int r = 0; r < R; ++r)
      if (key[r]) all += raised(rank_value(key[r]), top);
    all = warp_sum(all);
  }
  int my_ids[1] = {-1};
  uint32_t my_keys[1] = {};
  pick(keys, best, a.top_k, my_ids, my_keys);
  const int my_id = my_ids[0];
  const uint32_t my_key = my_keys[0];
  const float mine = my_id >= 0 ? raised(rank_value(my_key), top) : 0.0f;
  if (a.renormalize) all = warp_sum(mine);
  if (lane < a.top_k) {
    a.ids[token * a.top_k + lane] = my_id;
    a.weights[token * a.top_k + lane] = my_id >= 0 ? mine / all : 0.0f;
  }
}

// The gradient, one warp per token.  With w the weights, g their gradient and
// s = sum_j w_j g_j:  renormalised, d logit[ids_j] = w_j (g_j - s) and 0
// elsewhere; else d logit[e] = [e = ids_j] w_j g_j - p_e s with the softmax p
// taken again from the row.  16384 tokens x 256 experts, 8 picks: 5.7 us.
template <typename T, int R, bool kVector>
__global__ void __launch_bounds__(kRouteWarps * 32) route_backward_kernel(RouteArgs a) {
  const int64_t token = static_cast<int64_t>(blockIdx.x) * kRouteWarps + (threadIdx.x >> 5);
  if (token >= a.tokens) return;
  const int lane = threadIdx.x & 31;
  int my_id = -1;
  float w = 0.0f, wg = 0.0f;
  if (lane < a.top_k) {
    my_id = a.ids[token * a.top_k + lane];
    if (my_id >= 0) {
      w = a.weights[token * a.top_k + lane];
      wg = w * a.grad_weights[token * a.top_k + lane];
    }
  }
  const float s = warp_sum(wg);
  const float mine = a.renormalize ? wg - w * s : wg;
  float grad[R];
#pragma unroll
  for (int r = 0; r < R; ++r) grad[r] = 0.0f;
  if (!a.renormalize) {
    float v[R];
    float top = -INFINITY, all = 0.0f;
    load_row<T, R, kVector>(static_cast<const T*>(a.logits) + token * a.row_stride, a.experts, v);
#pragma unroll
    for (int r = 0; r < R; ++r)
      if (v[r] > top) top = v[r];
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) top = fmaxf(top, __shfl_xor_sync(kFull, top, d));
#pragma unroll
    for (int r = 0; r < R; ++r) {
      grad[r] = v[r] > -INFINITY ? raised(v[r], top) : 0.0f;
      all += grad[r];
    }
    all = warp_sum(all);
    const float scale = all > 0.0f ? -s / all : 0.0f;
    // Masked logits keep their 0 where s is no finite number.
#pragma unroll
    for (int r = 0; r < R; ++r) grad[r] = v[r] > -INFINITY ? grad[r] * scale : 0.0f;
  }
  const int first = lane * R;
  for (int j = 0; j < a.top_k; ++j) {
    const int id = __shfl_sync(kFull, my_id, j);
    const float g = __shfl_sync(kFull, mine, j);
#pragma unroll
    for (int r = 0; r < R; ++r)
      if (first + r == id) grad[r] += g;
  }
  T* out = static_cast<T*>(a.grad_logits) + token * a.experts + first;
  constexpr int kEach = 16 / static_cast<int>(sizeof(T));
  if constexpr (kVector && R % kEach == 0) {
    if (first < a.experts) {
#pragma unroll
      for (int r = 0; r < R; r += kEach) {
        Vector16<T> p;
#pragma unroll
        for (int q = 0; q < kEach / 2; ++q) p.set(q, make_float2(grad[r + 2 * q], grad[r + 2 * q + 1]));
        *reinterpret_cast<uint4*>(out + r) = p.words();
      }
    }
  } else {
#pragma unroll
    for (int r = 0; r < R; ++r)
      if (first + r < a.experts) out[r] = from_float<T>(grad[r]);
  }
}

template <typename T>
cudaError_t launch_route_t(const RouteArgs& a, bool backward, cudaStream_t stream) {
  const int64_t blocks = (a.tokens + kRouteWarps - 1) / kRouteWarps;
  const dim3 grid(static_cast<unsigned>(blocks)), block(kRouteWarps * 32);
  const auto aligned = [&](const void* p, int64_t stride) {
    return reinterpret_cast<uintptr_t>(p) % 16 == 0 && stride * static_cast<int64_t>(sizeof(T)) % 16 == 0;
  };
  const bool vector = aligned(a.logits, a.row_stride) && (!backward || aligned(a.grad_logits, a.experts));
#define DSMH_ROUTE(R)                                                                 \
  if (a.experts <= 32 * R) {                                                          \
    if (vector && a.experts % R == 0) {                                               \
      if (backward) route_backward_kernel<T, R, true><<<grid, block, 0, stream>>>(a); \
      else route_kernel<T, R, true><<<grid, block, 0, stream>>>(a);                   \
    } else {                                                                          \
      if (backward) route_backward_kernel<T, R, false><<<grid, block, 0, stream>>>(a);\
      else route_kernel<T, R, false><<<grid, block, 0, stream>>>(a);                  \
    }                                                                                 \
    return cudaGetLastError();                                                        \
  }
  DSMH_ROUTE(2)
  DSMH_ROUTE(4)
  DSMH_ROUTE(8)
  DSMH_ROUTE(32)
#undef DSMH_ROUTE
  return cudaErrorInvalidValue;
}

cudaError_t dispatch_route(const RouteArgs& a, bool backward, cudaStream_t stream) {
  if (a.dtype == DSMEM_F32) return launch_route_t<float>(a, backward, stream);
  if (a.dtype == DSMEM_F16) return launch_route_t<__half>(a, backward, stream);
  return launch_route_t<__nv_bfloat16>(a, backward, stream);
}

// Grouping: a counting sort by one cluster of P CTAs of W warps.  Every warp
// owns a contiguous run of keys and a row of counters in its CTA's shared
// memory, one per group.
//   1. Each warp counts its keys into its row.
//   2. Per group, the rows of a CTA become exclusive prefixes over its warps
//      and the CTA's total; the totals of the cluster's CTAs are read through
//      distributed shared memory, so every CTA knows what precedes it in the
//      group and how large the group is; a scan over the groups gives the
//      offsets.  Row and base then say where a warp's next key of a group goes.
//   3. Each warp goes over its keys again, 32 at a time: lanes with equal
//      keys are found by one ballot per key bit, take consecutive places in
//      lane order and move the counter on.
// Order is by warp, step and lane, that is by index: the sort is stable and
// needs no atomics whose order could matter (the counts of step 1 commute).
// Bound by the latency of its steps: 4 keys 2.4 us, 131072 keys into 256
// groups 10.4 us (16 CTAs).
// More keys (group_shape) take three launches over all SMs: every CTA's counts,
// their prefixes over the CTAs, and the same kernel with these in place of the
// cluster's totals.
struct GroupArgs {
  const int32_t* keys;
  int64_t n;
  int groups, warps, bits;
  int shared_totals;  // one warp: its row is the CTA's totals and bases as well
  int32_t* offsets;
  int32_t* order;
  int32_t* position;
  // Many keys: the CTAs are no cluster, and an earlier launch has left each
  // group's size and, for each CTA, what precedes it in the group.
  const uint32_t* sizes;   // [groups], or null
  const uint32_t* before;  // [CTAs][groups]
};

__device__ __forceinline__ uint32_t ld_cluster_u32(uint32_t cluster_addr) {
  uint32_t v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(cluster_addr) : "memory");
  return v;
}

constexpr int kGroupBatch = 8;  // keys of a lane that are loaded together

// The batch of a warp's run that begins at `i0`; ~0 behind the run's end.
__device__ __forceinline__ void load_keys(const GroupArgs& a, int64_t i0, int64_t end,
                                          uint32_t (&key)[kGroupBatch]) {
#pragma unroll
  for (int u = 0; u < kGroupBatch; ++u) {
    const int64_t i = i0 + u * 32 + (threadIdx.x & 31);
    key[u] = i < end ? static_cast<uint32_t>(a.keys[i]) : 0xffffffffu;
  }
}

__global__ void __launch_bounds__(1024) group_kernel(GroupArgs a) {
  extern __shared__ uint32_t smem[];  // rows [warps][groups], totals and bases [groups], scan [32]
  const uint32_t rank = blockIdx.x, ctas = gridDim.x, P = cluster_nctarank();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const uint32_t G = static_cast<uint32_t>(a.groups);
  uint32_t* total = smem + (a.shared_totals ? 0 : static_cast<size_t>(a.warps) * G);
  uint32_t* base = total + (a.shared_totals ? 0 : G);
  uint32_t* scan = base + G;
  uint32_t* mine = smem + static_cast<size_t>(warp) * G;

  // Each warp's run of keys, a multiple of 32 long; its first batch stays in
  // registers for both passes.
  const int64_t parts = static_cast<int64_t>(ctas) * a.warps;
  const int64_t run = ((a.n + parts - 1) / parts + 31) / 32 * 32;
  int64_t begin = (static_cast<int64_t>(rank) * a.warps + warp) * run;
  int64_t end = begin + run;
  if (begin > a.n) begin = a.n;
  if (end > a.n) end = a.n;
  uint32_t key[kGroupBatch];
  load_keys(a, begin, end, key);

  for (uint32_t i = threadIdx.x; i < a.warps * G; i += blockDim.x) smem[i] = 0;
  __syncthreads();
  for (int64_t i0 = begin; i0 < end; i0 += 32 * kGroupBatch) {
    if (i0 != begin) load_keys(a, i0, end, key);
#pragma unroll
    for (int u = 0; u < kGroupBatch; ++u)
      if (key[u] < G) atomicAdd(mine + key[u], 1u);
  }
  __syncthreads();
  for (uint32_t g = threadIdx.x; g < G && !a.shared_totals; g += blockDim.x) {
    uint32_t sum = 0;
    for (int w0 = 0; w0 < a.warps; w0 += 8) {
      uint32_t c[8];
#pragma unroll
      for (int w = 0; w < 8; ++w) c[w] = w0 + w < a.warps ? smem[static_cast<size_t>(w0 + w) * G + g] : 0u;
#pragma unroll
      for (int w = 0; w < 8; ++w) {
        if (w0 + w < a.warps) smem[static_cast<size_t>(w0 + w) * G + g] = sum;
        sum += c[w];
      }
    }
    total[g] = sum;
  }
  if (P > 1) cluster_barrier();
  else __syncthreads();
  // Scan over the groups, blockDim.x at a time, carrying the sum so far.
  uint32_t carry = 0;
  for (uint32_t g0 = 0; g0 < G; g0 += blockDim.x) {
    const uint32_t g = g0 + threadIdx.x;
    uint32_t before = 0, size = 0;
    if (g < G) {
      if (a.sizes) {
        size = a.sizes[g];
        before = a.before[static_cast<size_t>(rank) * G + g];
      } else if (P > 1) {
        const uint32_t addr = smem_u32(total + g);
        uint32_t c[16];
#pragma unroll
        for (uint32_t r = 0; r < 16; ++r) c[r] = r < P ? ld_cluster_u32(map_rank(addr, r)) : 0u;
#pragma unroll
        for (uint32_t r = 0; r < 16; ++r) {
          if (r < rank) before += c[r];
          size += c[r];
        }
      } else {
        size = total[g];
      }
    }
    uint32_t incl = size;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const uint32_t up = __shfl_up_sync(kFull, incl, d);
      if (lane >= d) incl += up;
    }
    if (lane == 31) scan[warp] = incl;
    __syncthreads();
    uint32_t ahead = lane < a.warps ? scan[lane] : 0u;
    const uint32_t block = __reduce_add_sync(kFull, ahead);
    ahead = __reduce_add_sync(kFull, lane < warp ? ahead : 0u);
    const uint32_t offset = carry + ahead + incl - size;
    if (g < G) {
      base[g] = offset + before;
      if (rank == 0) a.offsets[g] = static_cast<int32_t>(offset);
    }
    carry += block;
    __syncthreads();
  }
  if (rank == 0 && threadIdx.x == 0) a.offsets[G] = static_cast<int32_t>(carry);
  // No CTA leaves while others still read its totals: the arrival here, the
  // wait at the end.
  if (P > 1) cluster_arrive_relaxed();

  const uint32_t below = (1u << lane) - 1u;
  for (int64_t i0 = begin; i0 < end; i0 += 32 * kGroupBatch) {
    if (run > 32 * kGroupBatch) load_keys(a, i0, end, key);
#pragma unroll
    for (int u = 0; u < kGroupBatch; ++u) {
      const int64_t i = i0 + u * 32 + lane;
      if (i0 + u * 32 >= end) break;
      const bool valid = key[u] < G;
      uint32_t peers = __ballot_sync(kFull, valid);
      for (int b = 0; b < a.bits; ++b) {
        const bool bit = (key[u] >> b) & 1u;
        const uint32_t with = __ballot_sync(kFull, bit);
        peers &= bit ? with : ~with;
      }
      uint32_t place = 0xffffffffu;
      if (valid) {
        // With shared totals the row holds the places themselves.
        place = mine[key[u]] + __popc(peers & below);
        if (!a.shared_totals) place += base[key[u]];
      }
      __syncwarp();
      if (valid && lane == 31 - __clz(peers)) mine[key[u]] += __popc(peers);
      __syncwarp();
      if (i < end) a.position[i] = static_cast<int32_t>(place);
      if (valid) a.order[place] = static_cast<int32_t>(i);
    }
  }
  // Places behind the last group.
  for (int64_t p = carry + static_cast<int64_t>(rank) * blockDim.x + threadIdx.x; p < a.n;
       p += static_cast<int64_t>(ctas) * blockDim.x)
    a.order[p] = -1;
  if (P > 1) cluster_wait();
}

// The CTAs' counts of their keys, [CTAs][groups]; CTAs and their keys are
// those of group_kernel.
__global__ void __launch_bounds__(1024) group_count_kernel(const int32_t* keys, int64_t n, int groups,
                                                           int64_t run, uint32_t* counts) {
  extern __shared__ uint32_t smem[];
  const uint32_t G = static_cast<uint32_t>(groups);
  for (uint32_t g = threadIdx.x; g < G; g += blockDim.x) smem[g] = 0;
  __syncthreads();
  const int64_t begin = static_cast<int64_t>(blockIdx.x) * run;
  const int64_t end = begin + run < n ? begin + run : n;
  for (int64_t i0 = begin + threadIdx.x; i0 < end; i0 += 4 * blockDim.x) {
    uint32_t key[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int64_t i = i0 + static_cast<int64_t>(u) * blockDim.x;
      key[u] = i < end ? static_cast<uint32_t>(keys[i]) : 0xffffffffu;
    }
#pragma unroll
    for (int u = 0; u < 4; ++u)
      if (key[u] < G) atomicAdd(smem + key[u], 1u);
  }
  __syncthreads();
  for (uint32_t g = threadIdx.x; g < G; g += blockDim.x)
    counts[static_cast<size_t>(blockIdx.x) * G + g] = smem[g];
}

// counts[c][g] -> the sum of counts[c'][g] over c' < c, and the groups' sizes.
// A CTA has 32 groups, each of its 8 warps a run of the CTAs' rows.
__global__ void __launch_bounds__(256) group_prefix_kernel(uint32_t* counts, int ctas, int groups,
                                                           uint32_t* sizes) {
  __shared__ uint32_t part[8][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = blockIdx.x * 32 + lane;
  const int begin = ctas * warp / 8, end = ctas * (warp + 1) / 8;
  uint32_t sum = 0;
  if (g < groups)
#pragma unroll 8
    for (int c = begin; c < end; ++c) sum += counts[static_cast<size_t>(c) * groups + g];
  part[warp][lane] = sum;
  __syncthreads();
  if (g >= groups) return;
  uint32_t before = 0;
  for (int w = 0; w < warp; ++w) before += part[w][lane];
#pragma unroll 8
  for (int c = begin; c < end; ++c) {
    const uint32_t count = counts[static_cast<size_t>(c) * groups + g];
    counts[static_cast<size_t>(c) * groups + g] = before;
    before += count;
  }
  if (warp == 7) sizes[g] = before;
}

}  // namespace

cudaError_t launch_route(const RouteArgs& a, cudaStream_t stream) {
  return dispatch_route(a, false, stream);
}
cudaError_t launch_route_backward(const RouteArgs& a, cudaStream_t stream) {
  return dispatch_route(a, true, stream);
}

int run_group(const int32_t* keys, int64_t n, int num_groups, int32_t* offsets, int32_t* order,
              int32_t* position, const CallContext& ctx, cudaStream_t stream) {
  GroupArgs a{};
  a.keys = keys, a.n = n, a.groups = num_groups;
  a.offsets = offsets, a.order = order, a.position = position;
  while ((int64_t{1} << a.bits) < num_groups) ++a.bits;
  const GroupShape shape = group_shape(n, num_groups, ctx.sm_count);
  a.shared_totals = shape.shared_totals;
  a.warps = shape.warps;
  const size_t smem = shape.smem_bytes;

  static SmemLimit limit, count_limit;
  cudaError_t e = limit.need(reinterpret_cast<const void*>(group_kernel), ctx.device, kGroupSmemLimit, true);
  if (e != cudaSuccess) return fail_with_cuda(e, "cudaFuncSetAttribute");
  uint32_t* scratch = nullptr;
  const int ctas = shape.ctas;
  if (!shape.one_cluster) {
    const size_t counts = static_cast<size_t>(ctas) * num_groups;
    int rc = pool_alloc(ctx, reinterpret_cast<void**>(&scratch), (counts + num_groups) * 4, stream);
    if (rc) return rc;
    uint32_t* sizes = scratch + counts;
    a.sizes = sizes, a.before = scratch;
    // The keys of a CTA as group_kernel gives them to its warps.
    const int64_t parts = static_cast<int64_t>(ctas) * a.warps;
    const int64_t run = ((n + parts - 1) / parts + 31) / 32 * 32 * a.warps;
    e = count_limit.need(reinterpret_cast<const void*>(group_count_kernel), ctx.device, num_groups * 4);
    if (e == cudaSuccess) {
      group_count_kernel<<<ctas, 1024, num_groups * 4, stream>>>(keys, n, num_groups, run, scratch);
      group_prefix_kernel<<<(num_groups + 31) / 32, 256, 0, stream>>>(scratch, ctas, num_groups, sizes);
      e = cudaGetLastError();
    }
  }
  if (e == cudaSuccess) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(ctas);
    cfg.blockDim = dim3(a.warps * 32);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = shape.one_cluster ? ctas : 1;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, group_kernel, a);
  }
  const int rc = scratch ? pool_free(scratch, stream) : DSMEM_HIST_OK;
  return e == cudaSuccess ? rc : fail_with_cuda(e, "group launch");
}

}  // namespace dsmh
