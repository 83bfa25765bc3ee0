// Four-bit codes (e2m1) in groups of 16 with an e4m3 scale: conversions.
#pragma once

#include "kvc_device.cuh"

namespace kvc {

constexpr int kGroup4 = 16;  // elements of a row that share a scale

// Eight values in units of their scale rounded to e2m1 (nearest, ties to even,
// saturating at +-6), the first in the lowest bits.
__device__ __forceinline__ uint32_t encode8_e2m1(const float* y) {
  uint32_t r;
  asm("{\n\t.reg .b8 a, b, c, d;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
      "mov.b32 %0, {a, b, c, d};\n\t}"
      : "=r"(r)
      : "f"(y[0]), "f"(y[1]), "f"(y[2]), "f"(y[3]), "f"(y[4]), "f"(y[5]), "f"(y[6]), "f"(y[7]));
  return r;
}

// The eight codes of a word as four f16 pairs (exact).
__device__ __forceinline__ void decode8_e2m1(uint32_t w, uint32_t (&h)[4]) {
  asm("{\n\t.reg .b8 a, b, c, d;\n\t"
      "mov.b32 {a, b, c, d}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, a;\n\t"
      "cvt.rn.f16x2.e2m1x2 %1, b;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, c;\n\t"
      "cvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
      : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
      : "r"(w));
}

// e4m3 nearest to a / 6 (ties to even, saturating at 448) for a finite a >= 0.
// EXACT: the quotient is rounded to odd first (cut, the last bit set if
// anything was cut), so that it cannot land on a midpoint by its own rounding.
// 16-bit inputs need none of it: their quotients keep 2^-12 from every midpoint
// that they do not hit.
template <bool EXACT>
__device__ __forceinline__ uint32_t scale_of(float a) {
  float t = __fdiv_rn(a, 6.0f);
  if constexpr (EXACT) {
    const float r = fmaf(-6.0f, t, a);
    uint32_t b = __float_as_uint(t);
    if (r < 0.f) --b;
    if (r != 0.f) b |= 1u;
    t = __uint_as_float(b);
  }
  return float2_to_fp8x2(t, 0.f) & 0xffu;
}

__device__ __forceinline__ float scale_value(uint32_t code) { return fp8x2_to_float2(code).x; }

}  // namespace kvc
