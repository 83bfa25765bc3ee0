// Attention of one query over the cached rows it sees, by one warp.
//
// The query at position pos sees row r if r <= pos and (r > pos - window or
// r < sinks): o = sum_r p_r v_r / sum_r p_r with p_r = 2^(x_r - m), x_r =
// scale * log2(e) * q . k_r and m the running maximum. Lane l holds the
// dims l * D / 32 on; every product and sum is fp32. Only visible rows are read.
//
// An infinity or NaN in V of a visible row is the output there, however small
// the row's weight: weights and rescalings are kept at or above the smallest
// normal number, which changes no finite output in fp32.
#pragma once

#include <type_traits>

#include "code4.cuh"
#include "decode_scored.h"
#include "kvc_internal.h"

namespace kvc {

struct RowParams {
  const void* k_cache;
  const void* v_cache;
  const unsigned char* k_scale;  // four-bit caches: e4m3 [num_blocks, n_kv_heads, block_size, D / 16]
  const unsigned char* v_scale;
  int64_t num_blocks;
  int n_kv_heads, block_size;
  int window, sinks;
  float qscale;  // scale * log2(e)
};

// Dims [lane * D / 32, + D / 32) of pool row `row`.
template <typename CT, int D>
__device__ __forceinline__ void load_dims(const void* cache, const unsigned char* scale, int64_t row, int lane,
                                          float (&x)[D / 32]) {
  constexpr int N = D / 32;
  if constexpr (std::is_same<CT, fp4e2m1>::value) {
    const unsigned char* p = static_cast<const unsigned char*>(cache) + row * (D / 2) + lane * (N / 2);
    uint32_t w = 0;
#pragma unroll
    for (int i = 0; i < N / 2; ++i) w |= static_cast<uint32_t>(__ldg(p + i)) << (8 * i);
    uint32_t h[4];
    decode8_e2m1(w, h);
    const float s = scale_value(__ldg(scale + row * (D / 16) + lane * N / 16));
#pragma unroll
    for (int i = 0; i < N / 2; ++i) {
      const float2 f = __half22float2(*reinterpret_cast<__half2*>(&h[i]));
      x[2 * i] = f.x * s;
      x[2 * i + 1] = f.y * s;
    }
  } else {
    const CT* p = static_cast<const CT*>(cache) + row * D + lane * N;
#pragma unroll
    for (int i = 0; i < N; ++i) x[i] = Elem<CT>::to_float(p[i]);
  }
}

// q: the query's dims of this lane; table: the sequence's row of the block
// table. Writes the outputs' dims of this lane. Returns false if a block lies
// outside the pool (its rows get no weight).
template <typename CT, int D>
__device__ bool attend_row(const RowParams& p, const float (&q)[D / 32], const int32_t* table, int kvh, int pos,
                           float (&o)[D / 32]) {
  constexpr int N = D / 32;
  constexpr float kTiny = 1.17549435e-38f;
  const int lane = threadIdx.x & 31;
  const int low = pos >= p.window ? pos - p.window + 1 : 0;  // first row of the window
  const int front = min(p.sinks, low);
  float m = -1e30f, l = 0.f;
  bool good = true;
#pragma unroll
  for (int i = 0; i < N; ++i) o[i] = 0.f;
  for (int i = 0; i < front + (pos - low + 1); ++i) {
    const int r = i < front ? i : i - front + low;
    const int b = r / p.block_size;
    const int phys = __ldg(table + b);
    if (phys < 0 || phys >= p.num_blocks) {
      good = false;
      continue;
    }
    const int64_t row = (static_cast<int64_t>(phys) * p.n_kv_heads + kvh) * p.block_size + (r - b * p.block_size);
    float x[N];
    load_dims<CT, D>(p.k_cache, p.k_scale, row, lane, x);
    float s = 0.f;
#pragma unroll
    for (int j = 0; j < N; ++j) s = fmaf(q[j], x[j], s);
    s = warp_sum(s) * p.qscale;
    if (s > m) {
      const float f = fmaxf(fast_exp2(m - s), kTiny);
      l *= f;
#pragma unroll
      for (int j = 0; j < N; ++j) o[j] *= f;
      m = s;
    }
    const float w = s - m == -__builtin_huge_valf() ? 0.f : fast_exp2(s - m);
    l += w;
    load_dims<CT, D>(p.v_cache, p.v_scale, row, lane, x);
#pragma unroll
    for (int j = 0; j < N; ++j) o[j] = fmaf(w >= 0.f ? fmaxf(w, kTiny) : w, x[j], o[j]);
  }
  const float inv = l == 0.f ? 0.f : 1.0f / l;
#pragma unroll
  for (int j = 0; j < N; ++j) o[j] *= inv;
  return good;
}

}  // namespace kvc
