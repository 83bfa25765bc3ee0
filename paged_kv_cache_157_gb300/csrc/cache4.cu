// Four-bit caches: append (kvc_append_fp4) and reading rows back
// (kvc_read_fp4).
//
// A row of head_dim elements is cut into groups of 16. With A the largest
// finite |x| of a group:
//   scale = e4m3(A / 6),  code_i = e2m1(x_i / scale),  x_i ~ code_i * scale
// both rounded to nearest, ties to even, from the exact quotient. 6 is the
// largest e2m1 value. A row of 128 elements takes 64 + 8 bytes against 256 in
// bf16. code * scale has at most 6 significant bits, so it is exact in f16,
// bf16 and f32, and reading back does not round.
//
// Bound by HBM: one pass, every element read once and its code written once.
// One thread has one group of K and the same one of V: 64 bytes of bf16 in
// flight per thread. What the exact rounding costs: a 16-bit x
// times the rounded reciprocal of the scale is off by at most 2^-22, while it
// keeps 2^-11 from every midpoint that it does not hit; so the product is
// rounded to 17 bits (two integer instructions), which restores the hits, and
// goes to the hardware's conversion. f32 inputs can lie closer and take the
// quotient with its remainder.
//
// Source: "KV-Cache——为什么AI回复越来越快" section 08 (KV-Cache quantisation);
// the format is this library's choice for this GPU, which converts e2m1 and
// e4m3 in hardware.
#include <type_traits>

#include "code4.cuh"
#include "kvc_internal.h"

namespace kvc {

namespace {

constexpr int kThreads4 = 256;

template <typename T>
__device__ __forceinline__ void load16(const T* p, float (&x)[kGroup4]) {
  constexpr int N = Elem<T>::kVec;
  uint4 u[kGroup4 / N];
#pragma unroll
  for (int i = 0; i < kGroup4 / N; ++i) u[i] = __ldg(reinterpret_cast<const uint4*>(p) + i);
#pragma unroll
  for (int i = 0; i < kGroup4 / N; ++i) Elem<T>::unpack(u[i], x + i * N);
}

// Codes (8 bytes) and the scale's code of one group.
template <bool F32>
__device__ __forceinline__ uint2 quantise(float (&x)[kGroup4], uint32_t& scale) {
  float a = 0.f;
  bool odd = false;
#pragma unroll
  for (int i = 0; i < kGroup4; ++i) {
    a = fmaxf(a, fabsf(x[i]));
    odd |= x[i] != x[i];
  }
  if (odd || a == __builtin_huge_valf()) {
    // NaN becomes 0; infinities take the largest finite number, which
    // saturates, and do not count for the scale
    a = 0.f;
#pragma unroll
    for (int i = 0; i < kGroup4; ++i) {
      if (x[i] != x[i]) x[i] = 0.f;
      if (fabsf(x[i]) == __builtin_huge_valf())
        x[i] = copysignf(3.4028234e38f, x[i]);
      else
        a = fmaxf(a, fabsf(x[i]));
    }
  }
  scale = scale_of<F32>(a);
  const float s = scale_value(scale);
  const float inv = s > 0.f ? __frcp_rn(s) : 0.f;
  float y[kGroup4];
#pragma unroll
  for (int i = 0; i < kGroup4; ++i) {
    if constexpr (F32) {
      const float m = fabsf(x[i]);
      float q = s > 0.f ? __fdiv_rn(m, s) : 0.f;
      const float r = fmaf(-q, s, m);
      uint32_t b = __float_as_uint(q);
      if (s > 0.f && q < 8.f) {  // beyond, it saturates anyway
        if (r < 0.f) --b;
        if (r != 0.f) b |= 1u;
      }
      y[i] = copysignf(__uint_as_float(b), x[i]);
    } else {
      y[i] = __uint_as_float((__float_as_uint(x[i] * inv) + 64u) & ~127u);
    }
  }
  return make_uint2(encode8_e2m1(y), encode8_e2m1(y + 8));
}

// Where a token's group lives: (block, head, row) of its slot, then the group.
struct Place4 {
  int64_t row;  // row of the pool, [num_blocks, n_heads, block_size]
  int g;        // group of the row
};

// i: (token, head, group). False: the token is skipped.
__device__ __forceinline__ bool place(int64_t i, const int64_t* slots, int64_t num_slots, int n_heads, int block_size,
                                      int groups, unsigned int* err, Place4& at) {
  const uint32_t per = static_cast<uint32_t>(n_heads) * groups;
  const int64_t t = i / per;
  const uint32_t r = static_cast<uint32_t>(i - t * per);
  const uint32_t h = r / groups;
  at.g = static_cast<int>(r - h * groups);
  const int64_t slot = __ldg(slots + t);
  if (slot < 0) return false;
  if (slot >= num_slots) {
    if (r == 0) set_flag(err, KVC_FLAG_BAD_SLOT);
    return false;
  }
  const int64_t blk = slot / block_size;
  at.row = (blk * n_heads + h) * block_size + (slot - blk * block_size);
  return true;
}

template <typename T>
__global__ void __launch_bounds__(kThreads4)
    append4_kernel(const T* __restrict__ k, const T* __restrict__ v, const int64_t* __restrict__ slots, int64_t total,
                   int64_t num_slots, int n_heads, int block_size, int groups, uint2* __restrict__ kc,
                   uint2* __restrict__ vc, unsigned char* __restrict__ ks, unsigned char* __restrict__ vs,
                   unsigned int* err) {
  constexpr bool F32 = sizeof(T) == 4;
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * kThreads4 + threadIdx.x; i < total;
       i += static_cast<int64_t>(gridDim.x) * kThreads4) {
    Place4 at;
    if (!place(i, slots, num_slots, n_heads, block_size, groups, err, at)) continue;
    float x[kGroup4], y[kGroup4];
    load16(k + i * kGroup4, x);
    load16(v + i * kGroup4, y);
    const int64_t to = at.row * groups + at.g;
    uint32_t s;
    kc[to] = quantise<F32>(x, s);
    ks[to] = static_cast<unsigned char>(s);
    vc[to] = quantise<F32>(y, s);
    vs[to] = static_cast<unsigned char>(s);
  }
}

template <typename T>
__device__ __forceinline__ void store16(T* p, const uint2 code, float s) {
  uint32_t h[2][4];
  decode8_e2m1(code.x, h[0]);
  decode8_e2m1(code.y, h[1]);
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    float x[8];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float2 f = __half22float2(*reinterpret_cast<__half2*>(&h[i][j]));
      x[2 * j] = f.x * s;
      x[2 * j + 1] = f.y * s;
    }
    constexpr int kind = sizeof(T) == 4 ? KVC_F32 : std::is_same<T, __half>::value ? KVC_F16 : KVC_BF16;
    if constexpr (kind == KVC_F32) {
      store_out_vec<4>(p, 8 * i, x, kind);
      store_out_vec<4>(p, 8 * i + 4, x + 4, kind);
    } else {
      store_out_vec<8>(p, 8 * i, x, kind);
    }
  }
}

template <typename T>
__global__ void __launch_bounds__(kThreads4)
    read4_kernel(const int64_t* __restrict__ slots, int64_t total, int64_t num_slots, int n_heads, int block_size,
                 int groups, const uint2* __restrict__ kc, const uint2* __restrict__ vc,
                 const unsigned char* __restrict__ ks, const unsigned char* __restrict__ vs, T* __restrict__ k,
                 T* __restrict__ v, unsigned int* err) {
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * kThreads4 + threadIdx.x; i < total;
       i += static_cast<int64_t>(gridDim.x) * kThreads4) {
    Place4 at;
    if (!place(i, slots, num_slots, n_heads, block_size, groups, err, at)) continue;
    const int64_t from = at.row * groups + at.g;
    const uint2 a = __ldg(kc + from), b = __ldg(vc + from);
    const uint32_t sa = __ldg(ks + from), sb = __ldg(vs + from);
    store16(k + i * kGroup4, a, scale_value(sa));
    store16(v + i * kGroup4, b, scale_value(sb));
  }
}

// Checks shared by both calls. *total: groups of the call, 0 for no tokens.
kvc_status check4(const void* k, const void* v, const int64_t* slots, int64_t num_tokens, const void* kc,
                  const void* vc, const uint8_t* ks, const uint8_t* vs, int64_t num_blocks, int block_size,
                  int n_kv_heads, int head_dim, kvc_dtype dtype, int64_t* total) {
  if (!dtype_ok(dtype)) return fail(KVC_ERR_INVALID_ARG, "unknown dtype %d", static_cast<int>(dtype));
  if (num_tokens < 0 || num_blocks < 1 || block_size < 1 || n_kv_heads < 1 || head_dim < 1)
    return fail(KVC_ERR_INVALID_ARG, "sizes must be positive (num_tokens >= 0)");
  if (head_dim != 64 && head_dim != 128 && head_dim != 256)
    return fail(KVC_ERR_UNSUPPORTED, "head_dim %d (supported: 64, 128, 256)", head_dim);
  if (block_size % 16 != 0 || block_size > 128)
    return fail(KVC_ERR_UNSUPPORTED, "block_size %d (supported: multiples of 16 up to 128)", block_size);
  if (n_kv_heads > (1 << 24) || num_blocks > (1ll << 55) / block_size / n_kv_heads / head_dim ||
      num_tokens > (1ll << 55) / n_kv_heads / head_dim)
    return fail(KVC_ERR_UNSUPPORTED, "num_blocks, num_tokens or n_kv_heads too large");
  *total = num_tokens * n_kv_heads * (head_dim / kGroup4);
  if (num_tokens == 0) return KVC_OK;
  if (k == nullptr || v == nullptr || slots == nullptr || kc == nullptr || vc == nullptr || ks == nullptr ||
      vs == nullptr)
    return fail(KVC_ERR_INVALID_ARG, "NULL pointer");
  if (!aligned16(k) || !aligned16(v) || !aligned16(kc) || !aligned16(vc) || !aligned16(ks) || !aligned16(vs))
    return fail(KVC_ERR_INVALID_ARG, "k, v, the caches and the scales must be 16-byte aligned");
  return KVC_OK;
}

int grid4(int64_t total, int num_sms) {
  const int64_t want = (total + kThreads4 - 1) / kThreads4;
  return static_cast<int>(want < num_sms * 64ll ? want : num_sms * 64ll);
}

}  // namespace
}  // namespace kvc

extern "C" {

kvc_status kvc_append_fp4(const void* k, const void* v, const int64_t* slot_mapping, int64_t num_tokens,
                          void* k_cache, void* v_cache, uint8_t* k_scale, uint8_t* v_scale, int64_t num_blocks,
                          int block_size, int n_kv_heads, int head_dim, kvc_dtype dtype, kvc_stream stream) {
  using namespace kvc;
  clear_error();
  int64_t total = 0;
  kvc_status st = check4(k, v, slot_mapping, num_tokens, k_cache, v_cache, k_scale, v_scale, num_blocks, block_size,
                         n_kv_heads, head_dim, dtype, &total);
  if (st != KVC_OK || total == 0) return st;
  DeviceInfo* dev = nullptr;
  if ((st = current_device(&dev)) != KVC_OK) return st;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  auto launch = [&](auto* kernel, auto zero) {
    using T = decltype(zero);
    kernel<<<grid4(total, dev->num_sms), kThreads4, 0, s>>>(
        static_cast<const T*>(k), static_cast<const T*>(v), slot_mapping, total, num_blocks * block_size, n_kv_heads,
        block_size, head_dim / kGroup4, static_cast<uint2*>(k_cache), static_cast<uint2*>(v_cache), k_scale, v_scale,
        dev->error_word);
  };
  if (dtype == KVC_F32) launch(append4_kernel<float>, float());
  else if (dtype == KVC_F16) launch(append4_kernel<__half>, __half());
  else launch(append4_kernel<__nv_bfloat16>, __nv_bfloat16());
  return finish_call(s);
}

kvc_status kvc_read_fp4(const int64_t* slot_mapping, int64_t num_tokens, const void* k_cache, const void* v_cache,
                        const uint8_t* k_scale, const uint8_t* v_scale, int64_t num_blocks, int block_size,
                        int n_kv_heads, int head_dim, void* k, void* v, kvc_dtype dtype, kvc_stream stream) {
  using namespace kvc;
  clear_error();
  int64_t total = 0;
  kvc_status st = check4(k, v, slot_mapping, num_tokens, k_cache, v_cache, k_scale, v_scale, num_blocks, block_size,
                         n_kv_heads, head_dim, dtype, &total);
  if (st != KVC_OK || total == 0) return st;
  DeviceInfo* dev = nullptr;
  if ((st = current_device(&dev)) != KVC_OK) return st;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  auto launch = [&](auto* kernel, auto zero) {
    using T = decltype(zero);
    kernel<<<grid4(total, dev->num_sms), kThreads4, 0, s>>>(
        slot_mapping, total, num_blocks * block_size, n_kv_heads, block_size, head_dim / kGroup4,
        static_cast<const uint2*>(k_cache), static_cast<const uint2*>(v_cache), k_scale, v_scale, static_cast<T*>(k),
        static_cast<T*>(v), dev->error_word);
  };
  if (dtype == KVC_F32) launch(read4_kernel<float>, float());
  else if (dtype == KVC_F16) launch(read4_kernel<__half>, __half());
  else launch(read4_kernel<__nv_bfloat16>, __nv_bfloat16());
  return finish_call(s);
}

}  // extern "C"
