// The expert layer's up kernel, and the layer's two launches.
#include "expert_layer.cuh"

namespace dsmh {
namespace {

using namespace layer;

// The rows of h of all active experts laid end to end, each CTA an equal share
// of them.  A tile is 16 rows of weights: 8 rows of h with a gate (rows g of the
// gate beside rows g of up, so one lane ends up with both), 16 without.  The
// tiles' batches of steps are again laid end to end, and each warp takes an
// equal share of these: whole tiles go from its fragments to h, parts of tiles
// to shared memory, where they are joined in order when all warps are done.
template <int kHeld, int kTiles, bool kWide>
__global__ void __launch_bounds__(kLayerThreads, 1) up_kernel(const __grid_constant__ LayerArgs a) {
  __shared__ Routing routing;
  extern __shared__ float4 parts[];  // [warp][first, last][tile of columns][lane]
  launch_dependents();
  route_all(a, routing);

  const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3, warp = threadIdx.x >> 5;
  const int high = a.gated ? 8 : 16;  // rows of h of a tile
  const int steps = (a.width + kDepth<kHeld> - 1) / kDepth<kHeld>, batches = (steps + kSteps - 1) / kSteps;
  const int64_t rows = static_cast<int64_t>(routing.count) * a.hidden;
  const int64_t begin = rows * blockIdx.x / gridDim.x, end = rows * (blockIdx.x + 1) / gridDim.x;
  if (begin == end) return;
  const FromX<kHeld, kWide> from{static_cast<const uint16_t*>(a.x), a.x_stride, a.width};

  // Tiles do not reach over the end of an expert: those of the first expert
  // here, then as many of each other one.
  const int expert0 = static_cast<int>(begin / a.hidden), row0 = static_cast<int>(begin % a.hidden);
  const int per_expert = (a.hidden + high - 1) / high;
  const int in_first = static_cast<int>((min(static_cast<int64_t>(a.hidden - row0), end - begin) + high - 1) / high);
  const int64_t behind = end - begin - min(static_cast<int64_t>(a.hidden - row0), end - begin);
  const int tiles_here = in_first + static_cast<int>(behind / a.hidden) * per_expert +
                         static_cast<int>(behind % a.hidden + high - 1) / high;
  struct Place {
    int expert, row, count;  // the active expert, the tile's first row of h, its rows
  };
  const auto place = [&](int tile) {
    Place p{expert0, row0 + tile * high, 0};
    if (tile >= in_first) {
      const int other = (tile - in_first) / per_expert;
      p.expert = expert0 + 1 + other;
      p.row = (tile - in_first - other * per_expert) * high;
    }
    const int64_t left = end - (static_cast<int64_t>(p.expert) * a.hidden + p.row);
    p.count = static_cast<int>(min(static_cast<int64_t>(min(high, a.hidden - p.row)), left));
    return p;
  };
  // A tile's sums, columns 2t and 2t + 1 of tile n of columns, rows g and g + 8 of
  // the weights, to h.
  const auto finish = [&](const Place& p, int first_row, int columns, int n, const float (&sum)[4]) {
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int col = n * 8 + t * 2 + j;
      if (col >= columns) continue;
      const int row = first_row + col;
      const float w = routing.weight[row];
      const auto act = [&](float f) { return a.silu ? f / (1.0f + expf(-f)) : (f > 0.0f || f != f ? f : 0.0f); };
      uint16_t* h = a.h + static_cast<int64_t>(row) * 2 * a.h_pitch;
      const auto put = [&](int k, float f) {
        // Two 16-bit numbers hold h to 16 bits or more: what they leave out is
        // far below the output's rounding.  4-bit fragments pair elements 4 apart.
        const int at = kIsMx4<kHeld> ? (k & ~7) | ((k & 3) << 1) | ((k >> 2) & 1) : k;
        if constexpr (kHeld == kF16) {
          const __half b = __float2half_rn(f);
          h[at] = __half_as_ushort(b);
          h[a.h_pitch + at] = __half_as_ushort(__float2half_rn(__hisinf(b) ? 0.0f : f - __half2float(b)));
        } else {
          const __nv_bfloat16 b = __float2bfloat16_rn(f);
          h[at] = __bfloat16_as_ushort(b);
          h[a.h_pitch + at] = __bfloat16_as_ushort(__float2bfloat16_rn(__hisinf(b) ? 0.0f : f - __bfloat162float(b)));
        }
      };
      if (a.gated) {
        if (g < p.count) put(p.row + g, w * (act(sum[j]) * sum[j + 2]));
      } else {
        if (g < p.count) put(p.row + g, w * act(sum[j]));
        if (g + 8 < p.count) put(p.row + g + 8, w * act(sum[j + 2]));
      }
      // Zeros behind the end of each row, up to a whole step.
      if (g == 0 && p.row + p.count == a.hidden)
        for (int k = a.hidden; k < a.h_pitch; ++k) put(k, 0.0f);
    }
  };

  const int64_t total = static_cast<int64_t>(tiles_here) * batches;
  const auto share = [&](int w) { return total * w / kLayerWarps; };
  const int64_t mine = share(warp), my_end = share(warp + 1);
  if (mine < my_end) {
    int tile = static_cast<int>(mine / batches), batch = static_cast<int>(mine - static_cast<int64_t>(tile) * batches);
    int left = static_cast<int>(my_end - mine);  // batches, the one at hand included
    Place next = place(tile);
    TwoRows at;
    // Rows beyond the tile's are read as its last one and left out of h.
    const auto point = [&](int step) {
      const int e = routing.active[next.expert], last = next.row + next.count - 1;
      point_at<kHeld>(a.gated ? a.gate : a.up, e, min(next.row + g, last), step, at, 0);
      point_at<kHeld>(a.up, e, min(next.row + (a.gated ? g : 8 + g), last), step, at, 1);
    };
    const auto batch_at = [&](int b) { return Batch{b * kSteps, (b + 1) * kSteps * kDepth<kHeld> <= a.width}; };
    Batch ahead = batch_at(batch);
    point(ahead.step);
    Slot slot[kSteps];
#pragma unroll
    for (int d = 0; d < kSteps; ++d) load_slot<kHeld, kWide>(slot[d], at, d, ahead, steps, a.width);
    do {
      const Place here = next;
      const int first_batch = batch;
      const int first_row = routing.start[here.expert], columns = routing.rows_of[here.expert];
      const int tiles = (columns + 7) >> 3;
      int column[kTiles];
#pragma unroll
      for (int n = 0; n < kTiles; ++n) column[n] = routing.token[first_row + min(n * 8 + g, columns - 1)];
      float sum[kTiles][4];
#pragma unroll
      for (int n = 0; n < kTiles; ++n) sum[n][0] = sum[n][1] = sum[n][2] = sum[n][3] = 0.0f;
      bool more;
      do {
        const Batch now = ahead;
        more = ++batch < batches;
        --left;
        if (left > 0) {
          ahead = batch_at(more ? batch : 0);
          if (more) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              at.row[i] += kSteps * 64;
              if (kIsMx4<kHeld>) at.scale[i] += kSteps * 4;
            }
          } else {
            next = place(++tile);
            point(0);
          }
        }
        multiply<kHeld, kTiles>(slot, now, steps, tiles, column, from, sum, [&](int d) {
          if (left > 0) load_slot<kHeld, kWide>(slot[d], at, d, ahead, steps, a.width);
        });
      } while (more && left > 0);
      const bool whole = first_batch == 0 && !more;
#pragma unroll
      for (int n = 0; n < kTiles; ++n) {
        if (kTiles > 1 && n >= tiles) break;
        if (whole) finish(here, first_row, columns, n, sum[n]);
        else parts[((warp * 2 + (first_batch == 0)) * kTiles + n) * 32 + lane] =
                 make_float4(sum[n][0], sum[n][1], sum[n][2], sum[n][3]);
      }
      batch = 0;
    } while (left > 0);
  }
  __syncthreads();
  // Warp w joins the tile that ends in its share having begun before it, from the
  // parts of the warps before (whose last part it is) in their order.
  if (mine < my_end) {
    const int tile = static_cast<int>(mine / batches);
    const int64_t tile_begin = static_cast<int64_t>(tile) * batches, tile_end = tile_begin + batches;
    if (tile_begin < mine && tile_end <= my_end) {
      const Place p = place(tile);
      const int first_row = routing.start[p.expert], columns = routing.rows_of[p.expert];
      int from_warp = warp;
      while (share(from_warp) > tile_begin) --from_warp;
      for (int n = 0; n * 8 < columns; ++n) {
        float sum[4] = {0.0f, 0.0f, 0.0f, 0.0f};
        for (int w = from_warp; w <= warp; ++w) {
          if (share(w) == share(w + 1)) continue;
          const float4 v = parts[((w * 2 + (share(w) <= tile_begin)) * kTiles + n) * 32 + lane];
          sum[0] += v.x, sum[1] += v.y, sum[2] += v.z, sum[3] += v.w;
        }
        finish(p, first_row, columns, n, sum);
      }
    }
  }
}

template <int kHeld, int kTiles, bool kWide>
cudaError_t launch(const LayerArgs& a, const CallContext& ctx, cudaStream_t stream) {
  static SmemLimit limit;
  const auto kernel = up_kernel<kHeld, kTiles, kWide>;
  const int bytes = kLayerWarps * 2 * kTiles * 32 * static_cast<int>(sizeof(float4));
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
  if (a.tokens <= 32) return launch<kHeld, 4, true>(a, ctx, stream);
  return launch<kHeld, kMaxTokens / 8, true>(a, ctx, stream);
}

}  // namespace

int run_expert_layer(const LayerArgs& args, const CallContext& ctx, cudaStream_t stream) {
  LayerArgs a = args;
  const int depth = a.mx4 ? kDepth<kMx4Bf16> : kDepth<kBf16>;
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
