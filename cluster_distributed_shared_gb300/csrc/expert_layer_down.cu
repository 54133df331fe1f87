// The expert layer's down kernel.
#include "expert_layer.cuh"

namespace dsmh {
namespace {

using namespace layer;

// Each CTA an equal share of y's channels, 16 at a time, over all active
// experts: with their rows of h end to end the layer's second half is one
// product of great depth, so no two CTAs add to one sum.  The warps split that
// depth evenly; each adds an expert's columns to its tokens' sums in shared
// memory when it has passed the expert, and at the end the warps' sums are
// added in order.
template <int kHeld, int kTiles, bool kWide>
__global__ void __launch_bounds__(kLayerThreads, 1) down_kernel(const __grid_constant__ LayerArgs a) {
  __shared__ Routing routing;
  extern __shared__ float sums[];  // [warp][token][16]
  route_all(a, routing);

  const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3, warp = threadIdx.x >> 5;
  const int steps = (a.hidden + kDepth<kHeld> - 1) / kDepth<kHeld>, batches = (steps + kSteps - 1) / kSteps;
  const int total = routing.count * batches;
  const int begin = static_cast<int>(static_cast<int64_t>(total) * warp / kLayerWarps);
  const int end = static_cast<int>(static_cast<int64_t>(total) * (warp + 1) / kLayerWarps);
  const int64_t width = a.width;
  const int first = static_cast<int>(width * blockIdx.x / gridDim.x);
  const int last = static_cast<int>(width * (blockIdx.x + 1) / gridDim.x);
  const FromH from{a.h, a.h_pitch};
  float* mine = sums + warp * a.tokens * 16;

  for (int channel = first; channel < last; channel += 16) {
    const int count = min(16, last - channel);
    for (int i = lane; i < a.tokens * 16; i += 32) mine[i] = 0.0f;
    __syncwarp();
    int ahead = begin / batches, ahead_batch = begin % batches, left = end - begin;
    TwoRows at;
    // Channels beyond the tile's are read as its last one and left out of y.
    const auto point = [&] {
      const int e = routing.active[ahead], last_channel = channel + count - 1;
      point_at<kHeld>(a.down, e, min(channel + g, last_channel), ahead_batch * kSteps, at, 0);
      point_at<kHeld>(a.down, e, min(channel + 8 + g, last_channel), ahead_batch * kSteps, at, 1);
    };
    const auto batch_at = [&](int b) { return Batch{b * kSteps, (b + 1) * kSteps * kDepth<kHeld> <= a.hidden}; };
    Batch next = batch_at(ahead_batch);
    Slot slot[kSteps];
    if (left > 0) {
      point();
#pragma unroll
      for (int d = 0; d < kSteps; ++d) load_slot<kHeld, kWide>(slot[d], at, d, next, steps, a.hidden);
    }
    if (channel == first) wait_for_previous();
    while (left > 0) {
      const int expert = ahead, columns = routing.rows_of[expert], first_row = routing.start[expert];
      const int tiles = (columns + 7) >> 3;
      int column[kTiles];
#pragma unroll
      for (int n = 0; n < kTiles; ++n) column[n] = first_row + min(n * 8 + g, columns - 1);
      float sum[kTiles][4];
#pragma unroll
      for (int n = 0; n < kTiles; ++n) sum[n][0] = sum[n][1] = sum[n][2] = sum[n][3] = 0.0f;
      do {
        const Batch now = next;
        if (--left > 0) {
          if (++ahead_batch < batches) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              at.row[i] += kSteps * 64;
              if (kIsMx4<kHeld>) at.scale[i] += kSteps * 4;
            }
          } else {
            ahead_batch = 0;
            ++ahead;
            point();
          }
          next = batch_at(ahead_batch);
        }
        multiply<kHeld, kTiles>(slot, now, steps, tiles, column, from, sum, [&](int d) {
          if (left > 0) load_slot<kHeld, kWide>(slot[d], at, d, next, steps, a.hidden);
        });
      } while (left > 0 && ahead == expert);
#pragma unroll
      for (int n = 0; n < kTiles; ++n) {
        if (kTiles > 1 && n >= tiles) break;
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const int col = n * 8 + t * 2 + j;
          if (col < columns) {
            float* p = mine + routing.token[first_row + col] * 16 + g;
            p[0] += sum[n][j];
            p[8] += sum[n][j + 2];
          }
        }
      }
      __syncwarp();
    }
    __syncthreads();
    for (int i = threadIdx.x; i < a.tokens * 16; i += kLayerThreads) {
      float v = sums[i];
      for (int w = 1; w < kLayerWarps; ++w) v += sums[w * a.tokens * 16 + i];
      const int token = i >> 4, c = i & 15;
      if (c >= count) continue;
      const int64_t at = token * width + channel + c;
      if (a.dtype == DSMEM_F16) static_cast<__half*>(a.out)[at] = from_float<__half>(v);
      else static_cast<__nv_bfloat16*>(a.out)[at] = from_float<__nv_bfloat16>(v);
    }
    __syncthreads();
  }
}

template <int kHeld, int kTiles, bool kWide>
cudaError_t launch(const LayerArgs& a, const CallContext& ctx, cudaStream_t stream) {
  static SmemLimit limit;
  const auto kernel = down_kernel<kHeld, kTiles, kWide>;
  const int bytes = kLayerWarps * a.tokens * 16 * static_cast<int>(sizeof(float));
  const cudaError_t e = limit.need(reinterpret_cast<const void*>(kernel), ctx.device, bytes);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(std::min(a.width, ctx.sm_count)));
  cfg.blockDim = dim3(kLayerThreads);
  cfg.dynamicSmemBytes = static_cast<size_t>(bytes);
  cfg.stream = stream;
  cudaLaunchAttribute attr = {};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, a);
}

template <int kHeld>
cudaError_t launch_held(const LayerArgs& a, const CallContext& ctx, cudaStream_t stream) {
  if constexpr (!kIsMx4<kHeld>) {
    if (!whole_vectors(a.down, a.hidden)) return launch<kHeld, kMaxTokens / 8, false>(a, ctx, stream);
  }
  if (a.tokens <= 8) return launch<kHeld, 1, true>(a, ctx, stream);
  if (a.tokens <= 32) return launch<kHeld, 4, true>(a, ctx, stream);
  return launch<kHeld, kMaxTokens / 8, true>(a, ctx, stream);
}

}  // namespace

// h is in bf16 parts beside 4-bit matrices, whatever x's type.
cudaError_t launch_layer_down(const LayerArgs& a, const CallContext& ctx, cudaStream_t stream) {
  if (a.mx4) return launch_held<kMx4Bf16>(a, ctx, stream);
  return a.dtype == DSMEM_F16 ? launch_held<kF16>(a, ctx, stream) : launch_held<kBf16>(a, ctx, stream);
}

}  // namespace dsmh
