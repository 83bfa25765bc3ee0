// One-byte codes (e4m3, int8) of block-scaled caches: 4 or 16 values at a
// time to and from fp32.
#pragma once

#include "kvc_device.cuh"
#include "kvc_internal.h"

namespace kvc {

// Reciprocal of the largest code, and the smallest scale that counts (the
// smallest normal number: its reciprocal is finite; a smaller scale is taken
// as 0 and its codes as 0).
template <bool INT8>
struct Code8 {
  static constexpr float kInvMax = 1.0f / (INT8 ? 127.0f : 448.0f);
};
constexpr float kTinyScale = 1.17549435e-38f;

// Four values rounded to codes (nearest, ties to even, saturating), a in the low byte.
template <bool INT8>
__device__ __forceinline__ uint32_t encode4(float a, float b, float c, float d) {
  if constexpr (INT8) {
    const uint32_t ab = (float_to_s8(a) & 0xff) | ((float_to_s8(b) & 0xff) << 8);
    return ab | ((float_to_s8(c) & 0xff) << 16) | (static_cast<uint32_t>(float_to_s8(d)) << 24);
  } else {
    return static_cast<uint32_t>(float2_to_fp8x2(a, b)) | (static_cast<uint32_t>(float2_to_fp8x2(c, d)) << 16);
  }
}

// encode4 for values known to be finite and, rounded, within the codes' range:
// int8 codes come out of the low mantissa bits of 1.5 x 2^23 + x (the addition
// rounds to the nearest integer, ties to even).
template <bool INT8>
__device__ __forceinline__ uint32_t encode4_in_range(float2 a, float2 b) {
  if constexpr (INT8) {
    constexpr float k = 12582912.0f;
    const uint32_t lo = __byte_perm(__float_as_uint(__fadd_rn(a.x, k)), __float_as_uint(__fadd_rn(a.y, k)), 0x0040u);
    const uint32_t hi = __byte_perm(__float_as_uint(__fadd_rn(b.x, k)), __float_as_uint(__fadd_rn(b.y, k)), 0x0040u);
    return __byte_perm(lo, hi, 0x5410u);
  } else {
    return encode4<false>(a.x, a.y, b.x, b.y);
  }
}

// The codes of one word times f, rounded to codes again.
template <bool INT8>
__device__ __forceinline__ uint32_t rescale4(uint32_t w, float f) {
  float2 lo, hi;
  if constexpr (INT8) {
    lo = s8x2_to_float2(w & 0xffffu);
    hi = s8x2_to_float2(w >> 16);
  } else {
    lo = fp8x2_to_float2(w & 0xffffu);
    hi = fp8x2_to_float2(w >> 16);
  }
  return encode4<INT8>(lo.x * f, lo.y * f, hi.x * f, hi.y * f);
}

template <bool INT8>
__device__ __forceinline__ uint4 rescale16(const uint4& u, float f) {
  return make_uint4(rescale4<INT8>(u.x, f), rescale4<INT8>(u.y, f), rescale4<INT8>(u.z, f), rescale4<INT8>(u.w, f));
}

}  // namespace kvc
