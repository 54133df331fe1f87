// The expert layer with 4-bit matrices.
#include "expert_layer.cuh"

namespace dsmh {

// h is in bf16 parts, whatever x's type.
cudaError_t launch_layer_mx4(const LayerArgs& a, const CallContext& ctx, cudaStream_t stream) {
  return a.dtype == DSMEM_F16 ? launch_both<kMx4F16, kMx4Bf16>(a, ctx, stream)
                              : launch_both<kMx4Bf16, kMx4Bf16>(a, ctx, stream);
}

}  // namespace dsmh
