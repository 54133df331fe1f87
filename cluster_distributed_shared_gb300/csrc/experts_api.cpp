// C ABI of the expert-layer operators: argument checks, then one launch
// sequence each (see dsmem_experts.h).
#include <math.h>
#include <stdint.h>

#include <algorithm>

#include <cuda_runtime_api.h>

#include "dsmem_experts.h"
#include "experts.h"

namespace dsmh {
namespace {

constexpr int64_t kMaxRows = INT32_MAX;

bool known_dtype(int32_t d) { return d == DSMEM_F32 || d == DSMEM_F16 || d == DSMEM_BF16; }
bool misaligned(const void* p, int size) {
  return reinterpret_cast<uintptr_t>(p) % static_cast<uintptr_t>(size) != 0;
}
int null_pointer(const char* name) { return fail_with(DSMEM_HIST_EINVAL, "%s is NULL", name); }
int bad_alignment(const char* name) {
  return fail_with(DSMEM_HIST_EINVAL, "%s must be aligned to its element size", name);
}

#define DSMH_REQUIRE(cond, ...) \
  if (!(cond)) return fail_with(DSMEM_HIST_EINVAL, __VA_ARGS__)
#define DSMH_POINTER(p, size)              \
  if (!(p)) return null_pointer(#p);       \
  if (misaligned(p, size)) return bad_alignment(#p)

int finish(cudaError_t e, const char* what) {
  return e == cudaSuccess ? DSMEM_HIST_OK : fail_with_cuda(e, what);
}

int check_route(int32_t dtype, int64_t tokens, int32_t experts, int64_t row_stride, int32_t top_k) {
  DSMH_REQUIRE(known_dtype(dtype), "dtype must be DSMEM_F32, DSMEM_F16 or DSMEM_BF16 (got %d)", dtype);
  DSMH_REQUIRE(tokens >= 0 && tokens <= kMaxRows, "tokens must be in [0, 2^31) (got %lld)",
               static_cast<long long>(tokens));
  DSMH_REQUIRE(experts >= 1 && experts <= DSMEM_ROUTE_MAX_EXPERTS, "experts must be in [1, %d] (got %d)",
               DSMEM_ROUTE_MAX_EXPERTS, experts);
  DSMH_REQUIRE(top_k >= 1 && top_k <= std::min<int32_t>(experts, DSMEM_ROUTE_MAX_TOP_K),
               "top_k must be in [1, min(experts, %d)] (got %d)", DSMEM_ROUTE_MAX_TOP_K, top_k);
  DSMH_REQUIRE(row_stride >= experts, "row_stride must be >= experts");
  return DSMEM_HIST_OK;
}

int run_route(const void* logits, int32_t dtype, int64_t tokens, int32_t experts, int64_t row_stride,
              int32_t top_k, int32_t renormalize, int32_t* ids, float* weights, cudaStream_t stream) {
  int rc = check_route(dtype, tokens, experts, row_stride, top_k);
  if (rc) return rc;
  if (tokens == 0) return DSMEM_HIST_OK;
  DSMH_POINTER(logits, dtype_size(dtype));
  DSMH_POINTER(ids, 4);
  DSMH_POINTER(weights, 4);
  CallContext ctx;
  if ((rc = begin_call(stream, &ctx))) return rc;
  RouteArgs a{logits, tokens, row_stride, experts, top_k, renormalize != 0, dtype,
              ids,    weights, nullptr,   nullptr};
  return finish(launch_route(a, stream), "route launch");
}

int run_route_backward(const void* logits, int32_t dtype, int64_t tokens, int32_t experts,
                       int64_t row_stride, int32_t top_k, int32_t renormalize, const int32_t* ids,
                       const float* weights, const float* grad_weights, void* grad_logits,
                       cudaStream_t stream) {
  int rc = check_route(dtype, tokens, experts, row_stride, top_k);
  if (rc) return rc;
  if (tokens == 0) return DSMEM_HIST_OK;
  DSMH_POINTER(logits, dtype_size(dtype));
  DSMH_POINTER(ids, 4);
  DSMH_POINTER(weights, 4);
  DSMH_POINTER(grad_weights, 4);
  DSMH_POINTER(grad_logits, dtype_size(dtype));
  CallContext ctx;
  if ((rc = begin_call(stream, &ctx))) return rc;
  RouteArgs a{logits,
              tokens,
              row_stride,
              experts,
              top_k,
              renormalize != 0,
              dtype,
              const_cast<int32_t*>(ids),
              const_cast<float*>(weights),
              grad_weights,
              grad_logits};
  return finish(launch_route_backward(a, stream), "route_backward launch");
}

int group(const int32_t* keys, int64_t n, int32_t num_groups, int32_t* offsets, int32_t* order,
          int32_t* position, cudaStream_t stream) {
  DSMH_REQUIRE(n >= 0 && n <= kMaxRows, "n must be in [0, 2^31) (got %lld)", static_cast<long long>(n));
  DSMH_REQUIRE(num_groups >= 1 && num_groups <= DSMEM_GROUP_MAX_GROUPS,
               "num_groups must be in [1, %d] (got %d)", DSMEM_GROUP_MAX_GROUPS, num_groups);
  DSMH_POINTER(offsets, 4);
  if (n > 0) {
    DSMH_POINTER(keys, 4);
    DSMH_POINTER(order, 4);
    DSMH_POINTER(position, 4);
  }
  CallContext ctx;
  int rc = begin_call(stream, &ctx);
  if (rc) return rc;
  return run_group(keys, n, num_groups, offsets, order, position, ctx, stream);
}

int check_product(int64_t x_rows, int32_t groups, int32_t fan, int64_t n, int32_t outer, int32_t inner,
                  int32_t dtype, int32_t out_dtype) {
  DSMH_REQUIRE(dtype == DSMEM_F16 || dtype == DSMEM_BF16, "dtype must be DSMEM_F16 or DSMEM_BF16 (got %d)",
               dtype);
  DSMH_REQUIRE(out_dtype == dtype || out_dtype == DSMEM_F32, "out_dtype must be dtype or DSMEM_F32 (got %d)",
               out_dtype);
  DSMH_REQUIRE(groups >= 1 && groups <= DSMEM_PRODUCT_MAX_GROUPS, "groups must be in [1, %d] (got %d)",
               DSMEM_PRODUCT_MAX_GROUPS, groups);
  DSMH_REQUIRE(n >= 0 && n <= kMaxRows - 512 && x_rows >= 0 && x_rows <= kMaxRows - 512,
               "n and x_rows must be in [0, 2^31 - 512)");
  // Tiles end at most 256 past these extents, in 32 bits.
  DSMH_REQUIRE(outer >= 1 && inner >= 1 && outer <= kMaxRows - 512 && inner <= kMaxRows - 512,
               "outer and inner must be in [1, 2^31 - 512) (got %d and %d)", outer, inner);
  DSMH_REQUIRE(fan >= 1, "fan must be >= 1 (got %d)", fan);
  return DSMEM_HIST_OK;
}

int multiply(const ProductArgs& a, int64_t out_elements, cudaStream_t stream) {
  CallContext ctx;
  int rc = begin_call(stream, &ctx);
  if (rc) return rc;
  // Without rows there is nothing to multiply: the gradient of the weights
  // is 0 and the other products are empty.
  if (a.n == 0 || a.x_rows == 0) {
    if (out_elements == 0) return DSMEM_HIST_OK;
    return finish(cudaMemsetAsync(a.out, 0, static_cast<size_t>(out_elements) * dtype_size(a.out_dtype),
                                  stream), "cudaMemsetAsync");
  }
  return run_product(a, ctx, stream);
}

int run_grouped_matmul(const void* x, int64_t x_rows, int64_t x_stride, const void* weight,
                       int64_t weight_row_stride, int64_t weight_group_stride, const int32_t* offsets,
                       int32_t groups, const int32_t* order, int32_t fan, int64_t n, int32_t outer,
                       int32_t inner, int32_t transpose, int32_t dtype, void* out, int32_t out_dtype,
                       cudaStream_t stream) {
  int rc = check_product(x_rows, groups, fan, n, outer, inner, dtype, out_dtype);
  if (rc) return rc;
  const int32_t depth = transpose ? outer : inner, cols = transpose ? inner : outer;
  DSMH_REQUIRE(x_stride >= depth, "x_stride must be >= %d", depth);
  DSMH_REQUIRE(weight_row_stride >= inner, "weight_row_stride must be >= inner");
  DSMH_REQUIRE(groups == 1 || weight_group_stride >= 1, "weight_group_stride must be >= 1");
  if (n == 0) return DSMEM_HIST_OK;
  if (x_rows > 0) { DSMH_POINTER(x, 2); }
  DSMH_POINTER(weight, 2);
  DSMH_POINTER(offsets, 4);
  DSMH_POINTER(out, dtype_size(out_dtype));
  if (misaligned(order, 4)) return bad_alignment("order");
  ProductArgs a{};
  a.kind = transpose ? kInputGrad : kForward;
  a.x = x, a.x_rows = x_rows, a.x_stride = x_stride;
  a.w = weight, a.w_stride = weight_row_stride, a.w_group_stride = weight_group_stride;
  a.offsets = offsets, a.order = order, a.groups = groups, a.fan = fan, a.n = n;
  a.outer = outer, a.inner = inner, a.dtype = dtype, a.out_dtype = out_dtype, a.out = out;
  return multiply(a, n * cols, stream);
}

int run_wgrad(const void* dy, int64_t dy_stride, const void* x, int64_t x_rows, int64_t x_stride,
              const int32_t* offsets, int32_t groups, const int32_t* order, int32_t fan, int64_t n,
              int32_t outer, int32_t inner, int32_t dtype, void* out, int32_t out_dtype,
              cudaStream_t stream) {
  int rc = check_product(x_rows, groups, fan, n, outer, inner, dtype, out_dtype);
  if (rc) return rc;
  DSMH_REQUIRE(x_stride >= inner, "x_stride must be >= inner");
  DSMH_REQUIRE(dy_stride >= outer, "dy_stride must be >= outer");
  if (n > 0) {
    DSMH_POINTER(dy, 2);
    if (x_rows > 0) { DSMH_POINTER(x, 2); }
  }
  DSMH_POINTER(offsets, 4);
  DSMH_POINTER(out, dtype_size(out_dtype));
  if (misaligned(order, 4)) return bad_alignment("order");
  ProductArgs a{};
  a.kind = kWeightGrad;
  a.x = x, a.x_rows = x_rows, a.x_stride = x_stride;
  a.w = dy, a.w_stride = dy_stride, a.w_group_stride = 0;
  a.offsets = offsets, a.order = order, a.groups = groups, a.fan = fan, a.n = n;
  a.outer = outer, a.inner = inner, a.dtype = dtype, a.out_dtype = out_dtype, a.out = out;
  return multiply(a, static_cast<int64_t>(groups) * outer * inner, stream);
}

int check_combine(int64_t tokens, int32_t top_k, int32_t width, int32_t dtype) {
  DSMH_REQUIRE(known_dtype(dtype), "dtype must be DSMEM_F32, DSMEM_F16 or DSMEM_BF16 (got %d)", dtype);
  DSMH_REQUIRE(tokens >= 0 && top_k >= 1 && width >= 1 && tokens <= kMaxRows / top_k,
               "tokens must be >= 0, top_k and width >= 1, and tokens * top_k < 2^31");
  // Columns step past a row's end by less than the 2048 that a CTA takes at once.
  DSMH_REQUIRE(width <= kMaxRows - 2048, "width must be < 2^31 - 2048 (got %d)", width);
  return DSMEM_HIST_OK;
}

int run_combine(const void* z, int64_t z_rows, int64_t z_stride, const int32_t* position,
                const float* weights, int64_t tokens, int32_t top_k, int32_t width, int32_t dtype,
                void* out, cudaStream_t stream) {
  int rc = check_combine(tokens, top_k, width, dtype);
  if (rc) return rc;
  DSMH_REQUIRE(z_rows >= 0 && z_rows <= kMaxRows, "z_rows must be in [0, 2^31)");
  DSMH_REQUIRE(z_stride >= width, "z_stride must be >= width");
  if (tokens == 0) return DSMEM_HIST_OK;
  if (z_rows > 0) { DSMH_POINTER(z, dtype_size(dtype)); }
  DSMH_POINTER(position, 4);
  DSMH_POINTER(out, dtype_size(dtype));
  if (misaligned(weights, 4)) return bad_alignment("weights");
  CallContext ctx;
  if ((rc = begin_call(stream, &ctx))) return rc;
  CombineArgs a{};
  a.z = z, a.z_rows = z_rows, a.z_stride = z_stride, a.position = position, a.weights = weights;
  a.tokens = tokens, a.top_k = top_k, a.width = width, a.dtype = dtype, a.out = out;
  return finish(launch_combine(a, stream), "combine launch");
}

int run_combine_backward(const void* dy, int64_t dy_stride, const void* z, int64_t z_stride,
                         const int32_t* position, const int32_t* order, const float* weights,
                         int64_t tokens, int32_t top_k, int32_t width, int32_t dtype, void* dz,
                         float* dweights, cudaStream_t stream) {
  int rc = check_combine(tokens, top_k, width, dtype);
  if (rc) return rc;
  DSMH_REQUIRE(dy_stride >= width && z_stride >= width, "dy_stride and z_stride must be >= width");
  if (tokens == 0) return DSMEM_HIST_OK;
  const int size = dtype_size(dtype);
  DSMH_POINTER(dy, size);
  DSMH_POINTER(z, size);
  DSMH_POINTER(position, 4);
  DSMH_POINTER(order, 4);
  DSMH_POINTER(weights, 4);
  DSMH_POINTER(dz, size);
  DSMH_POINTER(dweights, 4);
  CallContext ctx;
  if ((rc = begin_call(stream, &ctx))) return rc;
  CombineArgs a{};
  a.z = z, a.z_rows = tokens * top_k, a.z_stride = z_stride, a.dy = dy, a.dy_stride = dy_stride;
  a.position = position, a.order = order, a.weights = weights;
  a.tokens = tokens, a.top_k = top_k, a.width = width, a.dtype = dtype, a.out = dz;
  a.dweights = dweights;
  return finish(launch_combine_backward(a, stream), "combine_backward launch");
}

int run_clip(const dsmem_grad_t* grads, int32_t num_grads, float max_norm, float* norm,
             cudaStream_t stream) {
  DSMH_REQUIRE(num_grads >= 0, "num_grads must be >= 0 (got %d)", num_grads);
  DSMH_REQUIRE(isfinite(max_norm) && max_norm > 0.0f, "max_norm must be positive and finite");
  DSMH_POINTER(norm, 4);
  if (num_grads > 0 && !grads) return null_pointer("grads");
  for (int32_t i = 0; i < num_grads; ++i) {
    const dsmem_grad_t& g = grads[i];
    DSMH_REQUIRE(known_dtype(g.dtype), "grads[%d]: unknown dtype %d", i, g.dtype);
    DSMH_REQUIRE(g.count >= 0 && g.count < (int64_t{1} << 48), "grads[%d]: count out of range", i);
    if (g.count == 0) continue;
    DSMH_REQUIRE(g.grad && g.out, "grads[%d]: NULL pointer", i);
    const int size = dtype_size(g.dtype);
    DSMH_REQUIRE(!misaligned(g.grad, size) && !misaligned(g.out, size),
                 "grads[%d]: pointers must be aligned to the element size", i);
  }
  CallContext ctx;
  int rc = begin_call(stream, &ctx);
  if (rc) return rc;
  return run_grad_clip(grads, num_grads, max_norm, norm, ctx, stream);
}

}  // namespace
}  // namespace dsmh

extern "C" {

int dsmem_route(const void* logits, int32_t dtype, int64_t tokens, int32_t experts, int64_t row_stride,
                int32_t top_k, int32_t renormalize, int32_t* ids, float* weights, cudaStream_t stream) {
  return dsmh::guarded([&] {
    return dsmh::run_route(logits, dtype, tokens, experts, row_stride, top_k, renormalize, ids, weights,
                           stream);
  });
}

int dsmem_route_backward(const void* logits, int32_t dtype, int64_t tokens, int32_t experts,
                         int64_t row_stride, int32_t top_k, int32_t renormalize, const int32_t* ids,
                         const float* weights, const float* grad_weights, void* grad_logits,
                         cudaStream_t stream) {
  return dsmh::guarded([&] {
    return dsmh::run_route_backward(logits, dtype, tokens, experts, row_stride, top_k, renormalize, ids,
                                    weights, grad_weights, grad_logits, stream);
  });
}

int dsmem_group(const int32_t* keys, int64_t n, int32_t num_groups, int32_t* offsets, int32_t* order,
                int32_t* position, cudaStream_t stream) {
  return dsmh::guarded([&] {
    return dsmh::group(keys, n, num_groups, offsets, order, position, stream);
  });
}

int dsmem_grouped_matmul(const void* x, int64_t x_rows, int64_t x_stride, const void* weight,
                         int64_t weight_row_stride, int64_t weight_group_stride, const int32_t* offsets,
                         int32_t groups, const int32_t* order, int32_t fan, int64_t n, int32_t outer,
                         int32_t inner, int32_t transpose, int32_t dtype, void* out, int32_t out_dtype,
                         cudaStream_t stream) {
  return dsmh::guarded([&] {
    return dsmh::run_grouped_matmul(x, x_rows, x_stride, weight, weight_row_stride, weight_group_stride,
                                    offsets, groups, order, fan, n, outer, inner, transpose, dtype, out,
                                    out_dtype, stream);
  });
}

int dsmem_grouped_matmul_wgrad(const void* dy, int64_t dy_stride, const void* x, int64_t x_rows,
                               int64_t x_stride, const int32_t* offsets, int32_t groups,
                               const int32_t* order, int32_t fan, int64_t n, int32_t outer,
                               int32_t inner, int32_t dtype, void* out, int32_t out_dtype,
                               cudaStream_t stream) {
  return dsmh::guarded([&] {
    return dsmh::run_wgrad(dy, dy_stride, x, x_rows, x_stride, offsets, groups, order, fan, n, outer,
                           inner, dtype, out, out_dtype, stream);
  });
}

int dsmem_combine(const void* z, int64_t z_rows, int64_t z_stride, const int32_t* position,
                  const float* weights, int64_t tokens, int32_t top_k, int32_t width, int32_t dtype,
                  void* out, cudaStream_t stream) {
  return dsmh::guarded([&] {
    return dsmh::run_combine(z, z_rows, z_stride, position, weights, tokens, top_k, width, dtype, out,
                             stream);
  });
}

int dsmem_combine_backward(const void* dy, int64_t dy_stride, const void* z, int64_t z_stride,
                           const int32_t* position, const int32_t* order, const float* weights,
                           int64_t tokens, int32_t top_k, int32_t width, int32_t dtype, void* dz,
                           float* dweights, cudaStream_t stream) {
  return dsmh::guarded([&] {
    return dsmh::run_combine_backward(dy, dy_stride, z, z_stride, position, order, weights, tokens, top_k,
                                      width, dtype, dz, dweights, stream);
  });
}

int dsmem_grad_clip(const dsmem_grad_t* grads, int32_t num_grads, float max_norm, float* norm,
                    cudaStream_t stream) {
  return dsmh::guarded([&] { return dsmh::run_clip(grads, num_grads, max_norm, norm, stream); });
}

}  // extern "C"
