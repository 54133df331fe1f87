// Division by a divisor that a launch knows.
#pragma once

#include <stdint.h>

namespace dsmh {

// Division of 31-bit values by a fixed divisor: with l = ceil(log2 d) and
// m = floor(2^32 (2^l - d) / d) + 1, the quotient is (mulhi(m, v) + v) >> l.
struct Divisor {
  uint32_t m, l;
  Divisor(uint32_t d = 1) : m(0), l(0) {
    while ((uint64_t{1} << l) < d) ++l;
    m = static_cast<uint32_t>((uint64_t{1} << 32) * ((uint64_t{1} << l) - d) / d + 1);
  }
#ifdef __CUDACC__
  __device__ __forceinline__ int quotient(int v) const {
    return static_cast<int>((__umulhi(m, static_cast<uint32_t>(v)) + static_cast<uint32_t>(v)) >> l);
  }
#endif
};

}  // namespace dsmh
