// Internal declarations shared by the generation operators (csbp_generate.h).
#pragma once

#include <cstdint>

#include "csbp_internal.h"

namespace csbp {

// Timer kinds (csbp_kernel_timing) after those of csbp_internal.h: 11 cache
// write and append, 12 cache read, 13 prefix and paged attention, 14 the joining
// of their pieces in a kernel of its own, 15 draft verification.
constexpr int kAllTimerKinds = kTimerKinds + 5;

// Encode a 3-D TMA descriptor (a CUtensorMap at `map`) over a bf16 tensor,
// innermost dimension first: strides[i] is the byte stride of dimension i + 1;
// box[0] = 64 elements, 128-byte swizzle; out-of-range elements read as zero.
bool encode_map_3d(void* map, const void* base, const uint64_t dims[3], const uint64_t strides[2],
                   const uint32_t box[3]);

}  // namespace csbp
