// unaligned.hpp -- groups of 8 values read from any element on, for the log
// probabilities and the cache (the row pass reads aligned groups, in
// device_common.hpp).
#pragma once

#include "device_common.hpp"

namespace specv {

// 8 values from any element on: the hardware's 16-byte loads need no
// alignment, so rows of any length and stride can take one path.
typedef uint32_t u32x4_any __attribute__((ext_vector_type(4), aligned(2)));
typedef float f32x4_any __attribute__((ext_vector_type(4), aligned(4)));
template <int ES>
__device__ __forceinline__ RawGroup<ES, true> load_any(const char* __restrict__ row, int64_t e0) {
  RawGroup<ES, true> r;
  if constexpr (ES == 2) {
    r.v = __builtin_nontemporal_load(reinterpret_cast<const u32x4_any*>(row + e0 * 2));
  } else {
    r.a = __builtin_nontemporal_load(reinterpret_cast<const f32x4_any*>(row + e0 * 4));
    r.b = __builtin_nontemporal_load(reinterpret_cast<const f32x4_any*>(row + e0 * 4 + 16));
  }
  return r;
}

}  // namespace specv
