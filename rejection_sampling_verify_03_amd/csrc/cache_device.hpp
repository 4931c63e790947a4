// cache_device.hpp -- addressing and 8-bit conversion of the paged KV cache,
// shared by its write, its read and the attention over it.
#pragma once

#include "device_common.hpp"
#include "ops_kernels.hpp"

namespace specv {

typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));

constexpr int kScaleBias = 127;
// The smallest exponent a written group gets: the smallest code, 2^-9, is
// then still a normal number in bf16 and fp32, so values read back exactly.
constexpr int kScaleMin = -117;

// 2^(byte - 127); a byte of 0, which only memory never written has, as 0 (its
// codes, which may be NaN, are taken as 0 too).
__device__ __forceinline__ float scale_of(uint32_t byte) { return __uint_as_float(byte << 23); }

// 2^e for e in [-126, 127].
__device__ __forceinline__ float two_to(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }

// The smallest e with amax <= 448 * 2^e (448 = 1.75 * 2^8, the largest
// code), at least kScaleMin; amax finite and not negative.
__device__ __forceinline__ int group_exponent(float amax) {
  const uint32_t u = __float_as_uint(amax);
  const int e = (int)(u >> 23) - 127 - 8 + ((u & 0x7fffffu) > 0x600000u ? 1 : 0);
  return max(e, kScaleMin);
}

__device__ __forceinline__ float finite_or_nan(float x) { return fabsf(x) <= FLT_MAX ? x : __builtin_nanf(""); }

// Four values (magnitudes at most 448, or NaN) as e4m3 codes, rounded to
// nearest even.
__device__ __forceinline__ uint32_t encode4(float a, float b, float c, float d) {
  int w = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false);
  return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(c, d, w, true);
}

__device__ __forceinline__ void decode4(uint32_t w, float x[4]) {
  const f32x2 lo = __builtin_amdgcn_cvt_pk_f32_fp8((int)w, false);
  const f32x2 hi = __builtin_amdgcn_cvt_pk_f32_fp8((int)w, true);
  x[0] = lo.x;
  x[1] = lo.y;
  x[2] = hi.x;
  x[3] = hi.y;
}

// Two fp32 values as bf16, rounded to nearest even, the first in the low half.
__device__ __forceinline__ uint32_t round_bf16x2(float a, float b) {
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2{a, b}, bf16x2));
}

// Byte SEL of a word of e2m1 codes as two bf16 values, the scale's exponent
// applied: exact down to the subnormal ones; an exponent byte of 255 gives NaN
// whatever the codes.
template <int SEL>
__device__ __forceinline__ uint32_t widen4(uint32_t codes, float scale) {
  return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, SEL));
}

// (byte b, a constant after unrolling)
__device__ __forceinline__ uint32_t widen4_at(uint32_t codes, float scale, int b) {
  return b == 0 ? widen4<0>(codes, scale)
                : b == 1 ? widen4<1>(codes, scale) : b == 2 ? widen4<2>(codes, scale) : widen4<3>(codes, scale);
}

}  // namespace specv
