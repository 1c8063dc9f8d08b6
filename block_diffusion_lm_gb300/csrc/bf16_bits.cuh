// Magnitudes of packed bf16 pairs as integers: with the sign bits cleared, bit
// patterns order as the values do, infinities and NaN above all.
#pragma once

#include <cstdint>

namespace csbp {

// Larger of each 16-bit half, in one instruction.
__device__ __forceinline__ uint32_t max_u16x2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("max.u16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}

}  // namespace csbp
