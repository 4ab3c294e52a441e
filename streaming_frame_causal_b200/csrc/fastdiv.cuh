// fastdiv.cuh -- division of 31-bit numbers by a divisor that is the same for a whole
// launch: the host forms a multiplier m and a shift with m / 2^(31 + shift) just above
// 1 / d, and n / d is the upper part of one product.  With shift = ceil(log2 d) and
// m = ceil(2^(31 + shift) / d) the error m d - 2^(31 + shift) is below d <= 2^shift, so the
// quotient is exact for every n < 2^31 (T. Granlund and P. Montgomery, "Division by
// Invariant Integers using Multiplication", 1994).
#pragma once
#include <cstdint>

#include "ptx.cuh"

namespace swa {

struct FastDiv {
  uint32_t d, m, shift;
  FastDiv() = default;
  explicit FastDiv(uint32_t divisor) : d(divisor), shift(31) {
    uint32_t s = 0;
    while ((1ull << s) < divisor) ++s;
    shift += s;
    m = static_cast<uint32_t>(((1ull << shift) + divisor - 1) / divisor);
  }
#ifdef __CUDACC__
  SWA_DEV int div(int n) const {
    return static_cast<int>((static_cast<uint64_t>(static_cast<uint32_t>(n)) * m) >> shift);
  }
  SWA_DEV int divmod(int n, int& rest) const {
    const int q = div(n);
    rest = n - q * static_cast<int>(d);
    return q;
  }
#endif
};

}  // namespace swa
