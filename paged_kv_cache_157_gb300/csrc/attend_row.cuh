// Attention of one query over the cached rows (16-bit) that it sees, by one warp: for
// the few outputs that the tensor-core kernels cannot give, U rows in flight.
//
// The query at position pos sees row r if r <= pos and (r > pos - window or
// r < sinks): o = sum_r p_r v_r / sum_r p_r with p_r = 2^(x_r - m), x_r =
// scale * log2(e) * q . k_r and m the running maximum. Lane l holds the
// dims l * D / 32 on; every product and sum is fp32. Only visible rows are read.
//
// An infinity or NaN in V of a visible row is the output there, however small
// the row's weight: what is not finite is weighed and rescaled by the smallest normal
// number at least. Finite values take weights as they are (bf16 ends at 3.4e38, where
// a weight of 1.2e-38 in place of 0 would be seen).
#pragma once

#include <type_traits>

#include "kvc_device.cuh"
#include "kvc_internal.h"

namespace kvc {

struct RowParams {
  const void* k_cache;
  const void* v_cache;
  int64_t num_blocks;
  int n_kv_heads, block_size;
  int window, sinks;
  float qscale;  // scale * log2(e)
};

// Dims [lane * D / 32, + D / 32) of pool row `row`.
template <typename CT, int D>
__device__ __forceinline__ void load_dims(const void* cache, int64_t row, int lane, float (&x)[D / 32]) {
  constexpr int N = D / 32;
  const CT* p = static_cast<const CT*>(cache) + row * D + lane * N;
#pragma unroll
  for (int i = 0; i < N; ++i) x[i] = Elem<CT>::to_float(p[i]);
}

// q: the query's dims of this lane; table: the sequence's row of the block
// table. Writes the outputs' dims of this lane. Returns false if a block lies
// outside the pool (its rows get no weight).
template <typename CT, int D, int U>
__device__ bool attend_row(const RowParams& p, const float (&q)[D / 32], const int32_t* table, int kvh, int pos,
                           float (&o)[D / 32]) {
  constexpr int N = D / 32;
  constexpr float kTiny = 1.17549435e-38f;
  auto finite = [](float a) { return fabsf(a) < __builtin_huge_valf(); };
  const int lane = threadIdx.x & 31;
  const int low = pos >= p.window ? pos - p.window + 1 : 0;  // first row of the window
  const int front = min(p.sinks, low);
  float m = -1e30f, l = 0.f;
  bool good = true;
#pragma unroll
  for (int i = 0; i < N; ++i) o[i] = 0.f;
  const int count = front + (pos - low + 1);
  for (int i0 = 0; i0 < count; i0 += U) {
    int64_t row[U];
    float s[U], x[U][N];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int i = i0 + u, r = i < front ? i : i - front + low;
      row[u] = -1;
      if (i >= count) continue;
      const int b = r / p.block_size;
      const int phys = __ldg(table + b);
      if (phys < 0 || phys >= p.num_blocks) {
        good = false;
        continue;
      }
      row[u] = (static_cast<int64_t>(phys) * p.n_kv_heads + kvh) * p.block_size + (r - b * p.block_size);
    }
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (row[u] >= 0) load_dims<CT, D>(p.k_cache, row[u], lane, x[u]);
    float top = -__builtin_huge_valf();
#pragma unroll
    for (int u = 0; u < U; ++u) {
      s[u] = 0.f;
      if (row[u] < 0) continue;
#pragma unroll
      for (int j = 0; j < N; ++j) s[u] = fmaf(q[j], x[u][j], s[u]);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      s[u] = warp_sum(s[u]) * p.qscale;
      if (row[u] >= 0) top = fmaxf(top, s[u]);
    }
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (row[u] >= 0) load_dims<CT, D>(p.v_cache, row[u], lane, x[u]);
    if (top > m) {
      const float f = fast_exp2(m - top);
      l *= f;
#pragma unroll
      for (int j = 0; j < N; ++j) o[j] *= finite(o[j]) ? f : fmaxf(f, kTiny);
      m = top;
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (row[u] < 0) continue;
      const float w = s[u] == -__builtin_huge_valf() ? 0.f : fast_exp2(s[u] - m);
      l += w;
#pragma unroll
      for (int j = 0; j < N; ++j) o[j] = fmaf(finite(x[u][j]) || w != w ? w : fmaxf(w, kTiny), x[u][j], o[j]);
    }
  }
  const float inv = l == 0.f ? 0.f : 1.0f / l;
#pragma unroll
  for (int j = 0; j < N; ++j) o[j] *= inv;
  return good;
}

}  // namespace kvc
