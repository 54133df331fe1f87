// Internal interfaces between the expert-layer kernels and their host layer.
// Not installed; the public C ABI is include/dsmem_experts.h.
#pragma once

#include <stdint.h>

#include <atomic>
#include <mutex>

#include <cuda_runtime_api.h>

#include "dsmem_experts.h"
#include "internal.h"

namespace dsmh {

inline int dtype_size(int dtype) { return dtype == DSMEM_F32 ? 4 : 2; }

// Status-word value of a launch of the product kernels whose wait gave up
// (the ship kernel writes 1).
constexpr uint32_t kStatusProduct = 2;

// Host layer of api.cpp: reports an earlier launch's timeout on this stream
// and hands out what a launch needs of the current device.
constexpr int kMaxDevices = 64;
struct CallContext {
  int device = 0;
  uint32_t* status = nullptr;  // the stream's host-mapped status word
  cudaMemPool_t pool = nullptr;
  int sm_count = 0;
};
int begin_call(cudaStream_t stream, CallContext* out);
// The bound of one device-side wait, and the test hook that leaves out the
// copies of a last stage (both from the environment, read at every call).
long long call_wait_cycles();
bool call_withholds();
// Scratch from the device's stream-ordered pool; given back on the same stream.
int pool_alloc(const CallContext& ctx, void** out, size_t bytes, cudaStream_t stream);
int pool_free(void* p, cudaStream_t stream);
int fail_with(int code, const char* fmt, ...) __attribute__((format(printf, 2, 3)));
int fail_with_cuda(cudaError_t e, const char* what);

// Runs a C entry's body; a C++ exception becomes an error code.
template <typename F>
int guarded(F&& body) noexcept {
  try {
    return body();
  } catch (...) {
    return record_error(DSMEM_HIST_ENOMEM, "out of host memory");
  }
}

// A kernel's largest dynamic shared memory so far on each device.  need()
// raises the kernel's limit where a launch wants more (and, once, allows
// clusters of 16).
class SmemLimit {
 public:
  cudaError_t need(const void* kernel, int device, int bytes, bool wide_clusters = false) {
    std::atomic<int>& set = set_[device];
    if (set.load(std::memory_order_acquire) >= bytes) return cudaSuccess;
    std::lock_guard<std::mutex> guard(mutex_);  // never lowers another thread's limit
    if (set.load(std::memory_order_relaxed) >= bytes) return cudaSuccess;
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e == cudaSuccess && wide_clusters)
      e = cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e == cudaSuccess) set.store(bytes, std::memory_order_release);
    return e;
  }

 private:
  std::atomic<int> set_[kMaxDevices] = {};
  std::mutex mutex_;
};

struct RouteArgs {
  const void* logits;
  int64_t tokens, row_stride;
  int experts, top_k, renormalize, dtype;
  int32_t* ids;
  float* weights;
  const float* grad_weights;  // backward only
  void* grad_logits;
};
cudaError_t launch_route(const RouteArgs& a, cudaStream_t stream);
cudaError_t launch_route_backward(const RouteArgs& a, cudaStream_t stream);

int run_group(const int32_t* keys, int64_t n, int num_groups, int32_t* offsets, int32_t* order,
              int32_t* position, const CallContext& ctx, cudaStream_t stream);

enum ProductKind { kForward = 0, kInputGrad = 1, kWeightGrad = 2 };
struct ProductArgs {
  int kind;
  const void* x;       // rows' source: [x_rows, inner] (kInputGrad: [x_rows, outer])
  int64_t x_rows, x_stride;
  const void* w;       // [groups, outer, inner]; kWeightGrad: dy [n, outer]
  int64_t w_stride, w_group_stride;
  const int32_t* offsets;
  const int32_t* order;  // may be null
  int groups, fan;
  int64_t n;
  int outer, inner;
  int dtype, out_dtype;
  void* out;
};
int run_product(const ProductArgs& a, const CallContext& ctx, cudaStream_t stream);
// Reads (synchronously) and clears the product kernels' device status word.
cudaError_t read_and_clear_product_status(uint32_t* out);

struct CombineArgs {
  const void* z;
  int64_t z_rows, z_stride;
  const void* dy;
  int64_t dy_stride;
  const int32_t* position;
  const int32_t* order;
  const float* weights;  // may be null (forward)
  int64_t tokens;
  int top_k, width, dtype;
  int first_piece;  // forward: the launch's first kThreads pieces of a row
  void* out;  // forward: [tokens, width]; backward: dz
  float* dweights;
};
cudaError_t launch_combine(const CombineArgs& a, cudaStream_t stream);
cudaError_t launch_combine_backward(const CombineArgs& a, cudaStream_t stream);

int run_grad_clip(const dsmem_grad_t* grads, int32_t num_grads, float max_norm, float* norm,
                  const CallContext& ctx, cudaStream_t stream);

}  // namespace dsmh
