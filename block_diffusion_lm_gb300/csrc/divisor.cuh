// Division by a number that a whole launch shares, without a divide.
#pragma once

#include <cstdint>

namespace csbp {

// Division of 0 <= n < 2^31 by an invariant d >= 1 (Granlund and Montgomery,
// "Division by invariant integers using multiplication").
struct Divisor {
  uint32_t mul, shift;
  static Divisor of(uint32_t d) {
    Divisor r{0, 0};
    while ((uint64_t(1) << r.shift) < d) ++r.shift;
    r.mul = static_cast<uint32_t>((((uint64_t(1) << r.shift) - d) << 32) / d + 1);
    return r;
  }
  __host__ __device__ __forceinline__ uint32_t operator()(uint32_t n) const {
    return (static_cast<uint32_t>((static_cast<uint64_t>(mul) * n) >> 32) + n) >> shift;
  }
};

}  // namespace csbp
