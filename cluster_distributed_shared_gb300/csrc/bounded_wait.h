// A wait that ends: what the product kernels' waits on mbarriers do beyond
// their first probe.  Free of CUDA calls, so that the CPU tests can drive it
// with made-up clocks.
#pragma once

#ifdef __CUDACC__
#define DSMH_HOST_DEVICE __host__ __device__
#else
#define DSMH_HOST_DEVICE
#endif

namespace dsmh {

enum class Waited { kArrived, kLeft, kGaveUp };

// Probes until `arrived()`, until `left()` (another wait has given up), or for
// `limit` units of `clock()`.  The clock is read before a probe, never between
// a probe and giving up: a thread that was switched out for longer than the
// limit looks once more at what has arrived meanwhile.
template <typename Arrived, typename Left, typename Clock>
DSMH_HOST_DEVICE inline Waited bounded_wait(Arrived arrived, Left left, Clock clock, long long limit) {
  const long long deadline = clock() + limit;
  for (;;) {
    const bool late = clock() >= deadline;
    if (arrived()) return Waited::kArrived;
    if (left()) return Waited::kLeft;
    if (late) return Waited::kGaveUp;
  }
}

}  // namespace dsmh
