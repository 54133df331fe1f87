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
// `limit` units of `clock()`, and once more before it gives up: a thread that was
// switched out for longer than the limit sees what has arrived meanwhile.  The
// clock is read once before the first probe (it takes long enough that a second
// reading there made a weight gradient of 16384 rows 14% slower).
template <typename Arrived, typename Left, typename Clock>
DSMH_HOST_DEVICE inline Waited bounded_wait(Arrived arrived, Left left, Clock clock, long long limit) {
  const long long deadline = clock() + limit;
  do {
    if (arrived()) return Waited::kArrived;
    if (left()) return Waited::kLeft;
  } while (clock() < deadline);
  return arrived() ? Waited::kArrived : Waited::kGaveUp;
}

}  // namespace dsmh
