// The expert layer with 16-bit matrices, and the call.
#include "expert_layer.cuh"

namespace dsmh {

int run_expert_layer(const LayerArgs& args, const CallContext& ctx, cudaStream_t stream) {
  LayerArgs a = args;
  const int depth = a.mx4 ? kDepth<kMx4Bf16> : kDepth<kBf16>;
  const int batch = depth * (a.mx4 ? kSteps<kMx4Bf16> : kSteps<kBf16>);
  a.h_pitch = (a.hidden + depth - 1) / depth * depth;
  a.by_ctas = Divisor(static_cast<uint32_t>(ctx.sm_count));
  a.by_hidden = Divisor(static_cast<uint32_t>(a.hidden));
  a.by_tiles = Divisor(static_cast<uint32_t>((a.hidden + (a.gated ? 7 : 15)) / (a.gated ? 8 : 16)));
  const auto batches = [&](int of) { return static_cast<uint32_t>((of + batch - 1) / batch); };
  a.by_up_batches = Divisor(batches(a.width));
  a.by_down_batches = Divisor(batches(a.hidden));
  const int64_t rows = static_cast<int64_t>(a.tokens) * a.top_k;
  void* scratch = nullptr;
  const int rc = pool_alloc(ctx, &scratch, sizeof(Routing) + static_cast<size_t>(rows * a.h_pitch * 4), stream);
  if (rc) return rc;
  a.routing = scratch;
  a.h = reinterpret_cast<uint16_t*>(static_cast<uint8_t*>(scratch) + sizeof(Routing));
  cudaError_t e;
  if (a.mx4) e = launch_layer_mx4(a, ctx, stream);
  else if (a.dtype == DSMEM_F16) e = launch_both<kF16, kF16>(a, ctx, stream);
  else e = launch_both<kBf16, kBf16>(a, ctx, stream);
  const int freed = pool_free(scratch, stream);
  return e == cudaSuccess ? freed : fail_with_cuda(e, "expert layer launch");
}

}  // namespace dsmh
