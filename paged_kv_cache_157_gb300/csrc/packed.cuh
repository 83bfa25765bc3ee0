// Packed fp32 addition of sm_100+, beside the products of kvc_device.cuh.
#pragma once

#include "kvc_device.cuh"

namespace kvc {

__device__ __forceinline__ float2 fadd2(float2 a, float2 b) {
  F2U64 x, y, r;
  x.f = a;
  y.f = b;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r.u) : "l"(x.u), "l"(y.u));
  return r.f;
}

}  // namespace kvc
