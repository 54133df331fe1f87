// The expert layer's up kernel, and the layer's two launches.
#include "expert_layer.cuh"

namespace dsmh {
namespace {

using namespace layer;

// The rows of h of all active experts laid end to end, each CTA an equal share
// of them.  A tile is 16 rows of weights: 8 rows of h with a gate (rows g of
// the gate beside rows g of up, so one lane ends up with both), 16 without.  A
// team of warps splits a tile's depth, as many as leave each kSteps steps, and
// adds its sums through shared memory; teams take tiles in turn.
template <int kHeld, int kTiles, bool kWide>
__global__ void __launch_bounds__(kLayerThreads, 1) up_kernel(const __grid_constant__ LayerArgs a) {
  __shared__ Routing routing;
  extern __shared__ float2 parts[];  // [team][warp][tile][half][lane]
  launch_dependents();
  route_all(a, routing);

  const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int warp = threadIdx.x >> 5, team = warp / a.team, member = warp % a.team, teams = kLayerWarps / a.team;
  const int high = a.gated ? 8 : 16;  // rows of h of a tile
  const int steps = (a.width + kDepth<kHeld> - 1) / kDepth<kHeld>;
  const int each = (steps + a.team - 1) / a.team;            // of a warp
  const int batches = (each + kSteps - 1) / kSteps;          // of a tile
  const int first_step = member * each, end_step = min(steps, first_step + each);
  const int64_t rows = static_cast<int64_t>(routing.count) * a.hidden;
  const int64_t begin = rows * blockIdx.x / gridDim.x, end = rows * (blockIdx.x + 1) / gridDim.x;
  const FromX<kHeld, kWide> from{static_cast<const uint16_t*>(a.x), a.x_stride, a.width};
  float2* mine = parts + team * a.team * kTiles * 64;

  // A place among the tiles: the active expert, the tile's first row of h, its rows.
  struct Place {
    int expert, row, count;
  };
  int64_t left = end - begin;
  Place next{static_cast<int>(begin / a.hidden), static_cast<int>(begin % a.hidden), 0};
  const auto fit = [&] { next.count = static_cast<int>(min(static_cast<int64_t>(min(high, a.hidden - next.row)), left)); };
  const auto advance = [&] {
    left -= next.count;
    next.row += next.count;
    if (next.row == a.hidden) next.row = 0, ++next.expert;
    fit();
  };
  fit();
  for (int i = 0; i < team && next.count > 0; ++i) advance();

  TwoRows rows_next = {};
  const auto point = [&] {
    const bool some = next.count > 0;
    const int e = some ? routing.active[next.expert] : 0;
    if (a.gated) {
      point_at<kHeld>(a.gate, e, next.row + g, some && g < next.count, rows_next, 0);
      point_at<kHeld>(a.up, e, next.row + g, some && g < next.count, rows_next, 1);
    } else {
      point_at<kHeld>(a.up, e, next.row + g, some && g < next.count, rows_next, 0);
      point_at<kHeld>(a.up, e, next.row + 8 + g, some && g + 8 < next.count, rows_next, 1);
    }
  };
  point();
  Slot slot[kSteps];
#pragma unroll
  for (int d = 0; d < kSteps; ++d) load_slot<kHeld, kWide>(slot[d], rows_next, first_step + d, end_step, a.width);

  while (next.count > 0) {
    const Place here = next;
    const int first_row = routing.start[here.expert], columns = routing.rows_of[here.expert];
    const int tiles = (columns + 7) >> 3;
    int column[kTiles];
#pragma unroll
    for (int n = 0; n < kTiles; ++n) column[n] = n * 8 + g < columns ? routing.token[first_row + n * 8 + g] : -1;
    float sum[kTiles][4];
#pragma unroll
    for (int n = 0; n < kTiles; ++n) sum[n][0] = sum[n][1] = sum[n][2] = sum[n][3] = 0.0f;
    for (int b = 0; b < batches; ++b) {
      int ahead = first_step + (b + 1) * kSteps;
      if (b + 1 == batches) {
        for (int i = 0; i < teams && next.count > 0; ++i) advance();
        point();
        ahead = first_step;
      }
#pragma unroll
      for (int d = 0; d < kSteps; ++d) {
        const int step = first_step + b * kSteps + d;
        if (step < end_step) multiply<kHeld, kTiles>(slot[d], step, tiles, column, from, sum);
        load_slot<kHeld, kWide>(slot[d], rows_next, ahead + d, end_step, a.width);
      }
    }
    // The team's sums, then h.
    if (a.team > 1) team_barrier(team, a.team);
#pragma unroll
    for (int n = 0; n < kTiles; ++n) {
      if (kTiles > 1 && n >= tiles) break;
      float2* p = mine + (member * kTiles + n) * 64 + lane;
      p[0] = make_float2(sum[n][0], sum[n][2]);
      p[32] = make_float2(sum[n][1], sum[n][3]);
    }
    if (a.team > 1) team_barrier(team, a.team);
    else __syncwarp();
    for (int i = member * 32 + lane; i < tiles * 64; i += a.team * 32) {
      float2 v = mine[i];
      for (int w = 1; w < a.team; ++w) {
        const float2 o = mine[w * kTiles * 64 + i];
        v.x += o.x, v.y += o.y;
      }
      // Columns 2t and 2t + 1 of tile i / 64, rows g and g + 8 of the weights.
      const int col = (i >> 6) * 8 + (i & 3) * 2 + ((i >> 5) & 1), r = (i & 31) >> 2;
      if (col >= columns) continue;
      const int row = first_row + col;
      const float w = routing.weight[row];
      const auto act = [&](float f) { return a.silu ? f / (1.0f + expf(-f)) : (f > 0.0f || f != f ? f : 0.0f); };
      uint16_t* h = a.h + static_cast<int64_t>(row) * 2 * a.h_pitch;
      const auto put = [&](int k, float f) {
        // Two 16-bit numbers hold h to 16 bits or more: what they leave out is
        // far below the output's rounding.  4-bit fragments pair elements 4 apart.
        const int at = kIsMx4<kHeld> ? (k & ~7) | ((k & 3) << 1) | ((k >> 2) & 1) : k;
        uint16_t big, rest;
        if constexpr (kHeld == kF16) {
          const __half b = __float2half_rn(f);
          const __half s = __hisinf(b) ? __half(0.0f) : __float2half_rn(f - __half2float(b));
          big = __half_as_ushort(b), rest = __half_as_ushort(s);
        } else {
          const __nv_bfloat16 b = __float2bfloat16_rn(f);
          const __nv_bfloat16 s = __hisinf(b) ? __nv_bfloat16(0.0f) : __float2bfloat16_rn(f - __bfloat162float(b));
          big = __bfloat16_as_ushort(b), rest = __bfloat16_as_ushort(s);
        }
        h[at] = big;
        h[a.h_pitch + at] = rest;
      };
      if (a.gated) {
        if (r < here.count) put(here.row + r, w * (act(v.x) * v.y));
      } else {
        if (r < here.count) put(here.row + r, w * act(v.x));
        if (r + 8 < here.count) put(here.row + r + 8, w * act(v.y));
      }
      // Zeros behind the end of each row, up to a whole step.
      if (r == 0 && here.row + here.count == a.hidden)
        for (int k = a.hidden; k < a.h_pitch; ++k) put(k, 0.0f);
    }
    if (a.team == 1) __syncwarp();
  }
}

template <int kHeld, int kTiles, bool kWide>
cudaError_t launch(const LayerArgs& a, const CallContext& ctx, cudaStream_t stream) {
  static SmemLimit limit;
  const auto kernel = up_kernel<kHeld, kTiles, kWide>;
  const int bytes = kLayerWarps * kTiles * 64 * static_cast<int>(sizeof(float2));
  const cudaError_t e = limit.need(reinterpret_cast<const void*>(kernel), ctx.device, bytes);
  if (e != cudaSuccess) return e;
  kernel<<<ctx.sm_count, kLayerThreads, bytes, stream>>>(a);
  return cudaGetLastError();
}

template <int kHeld>
cudaError_t launch_up(const LayerArgs& a, const CallContext& ctx, cudaStream_t stream) {
  const bool wide = reinterpret_cast<uintptr_t>(a.x) % 16 == 0 && a.x_stride % 8 == 0 && a.width % 8 == 0 &&
                    (kIsMx4<kHeld> || (whole_vectors(a.up, a.width) && (!a.gated || whole_vectors(a.gate, a.width))));
  if (!wide) return launch<kHeld, kMaxTokens / 8, false>(a, ctx, stream);
  if (a.tokens <= 8) return launch<kHeld, 1, true>(a, ctx, stream);
  return launch<kHeld, kMaxTokens / 8, true>(a, ctx, stream);
}

}  // namespace

int run_expert_layer(const LayerArgs& args, const CallContext& ctx, cudaStream_t stream) {
  LayerArgs a = args;
  const int depth = a.mx4 ? kDepth<kMx4Bf16> : kDepth<kBf16>;
  const int steps = (a.width + depth - 1) / depth;
  a.team = 1;
  while (a.team < kLayerWarps && steps > a.team * kSteps) a.team *= 2;
  a.h_pitch = (a.hidden + depth - 1) / depth * depth;
  const int64_t rows = static_cast<int64_t>(a.tokens) * a.top_k;
  void* scratch = nullptr;
  const int rc = pool_alloc(ctx, &scratch, static_cast<size_t>(rows * a.h_pitch * 4), stream);
  if (rc) return rc;
  a.h = static_cast<uint16_t*>(scratch);
  const bool half = a.dtype == DSMEM_F16;
  cudaError_t e = a.mx4 ? (half ? launch_up<kMx4F16>(a, ctx, stream) : launch_up<kMx4Bf16>(a, ctx, stream))
                        : (half ? launch_up<kF16>(a, ctx, stream) : launch_up<kBf16>(a, ctx, stream));
  if (e == cudaSuccess) e = launch_layer_down(a, ctx, stream);
  const int freed = pool_free(scratch, stream);
  return e == cudaSuccess ? freed : fail_with_cuda(e, "expert layer launch");
}

}  // namespace dsmh
