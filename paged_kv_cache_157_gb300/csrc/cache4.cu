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
// One pass: every element is read once and its code written once. Bound by the
// instructions for it before HBM: in the append 70 % of the cycles issue one and DRAM
// moves 3.9 TB/s, reading back 71 % and 1.6 (much of what is written stays in L2 at first). In the
// append a thread has a group of K and the same one of V (64 bytes of bf16 in
// flight; 17.2 us for 16384 tokens of 8 heads and 128 dims in 16 bits, 86 MB: half
// a group per thread reads whole lines but finds every scale twice, 21.6 us; two
// groups, 20.7 us). Reading back it has half a group, so that a warp's stores are
// whole lines (15.2 us; whole groups 19.7 us). A CTA has the rows of one kv
// head and some neighbouring tokens, because a prompt's rows lie one behind the other
// in its blocks: it writes their codes and scales side by side (head by head within a
// token, each row's 8 bytes of scales lay alone).
//
// What the exact rounding costs: a 16-bit x times the rounded reciprocal of the scale
// is off by at most 2^-22, while it keeps 2^-11 from every midpoint that it does not
// hit; so the product is rounded to 17 bits (two integer instructions), which restores
// the hits, and goes to the hardware's conversion. f32 inputs can lie closer and take
// the quotient with its remainder.
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
constexpr int kHalf4 = kGroup4 / 2;

template <typename T>
__device__ __forceinline__ T from_bits(unsigned short x) {
  T r;
  *reinterpret_cast<unsigned short*>(&r) = x;
  return r;
}

// A group as it lies in memory.
template <typename T>
struct Group {
  static constexpr int N = Elem<T>::kVec;
  uint4 u[kGroup4 / N];
  __device__ __forceinline__ void load(const T* p) {
#pragma unroll
    for (int i = 0; i < kGroup4 / N; ++i) u[i] = __ldg(reinterpret_cast<const uint4*>(p) + i);
  }
  __device__ __forceinline__ void unpack(float (&x)[kGroup4]) const {
#pragma unroll
    for (int i = 0; i < kGroup4 / N; ++i) Elem<T>::unpack(u[i], x + i * N);
  }
  // The largest magnitude: the order of magnitudes is that of their bits, NaN above
  // infinity, and 16-bit elements go two at a time.
  __device__ __forceinline__ float largest() const {
    if constexpr (sizeof(T) == 4) {
      uint32_t m = 0;
#pragma unroll
      for (int i = 0; i < kGroup4 / N; ++i)
        m = max(max(max(u[i].x & 0x7fffffffu, u[i].y & 0x7fffffffu),
                    max(u[i].z & 0x7fffffffu, u[i].w & 0x7fffffffu)), m);
      return __uint_as_float(m);
    } else {
      uint32_t m = 0;
#pragma unroll
      for (int i = 0; i < kGroup4 / N; ++i) {
        m = __vmaxu2(m, __vmaxu2(u[i].x & 0x7fff7fffu, u[i].y & 0x7fff7fffu));
        m = __vmaxu2(m, __vmaxu2(u[i].z & 0x7fff7fffu, u[i].w & 0x7fff7fffu));
      }
      m = max(m & 0xffffu, m >> 16);
      return Elem<T>::to_float(from_bits<T>(static_cast<unsigned short>(m)));
    }
  }
};

// Codes (8 bytes) of a group and its scale's code.
template <typename T>
__device__ __forceinline__ uint2 quantise(const Group<T>& u, uint32_t& scale) {
  constexpr bool F32 = sizeof(T) == 4;
  float x[kGroup4];
  u.unpack(x);
  float a = u.largest();
  if (!(a < __builtin_huge_valf())) {
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

// What a call's threads have: CTA (x, y) some tokens of kv head y, thread i token
// i / lanes of them and piece i % lanes of its row: a group (append) or half of one
// (reading back).
struct Rows4 {
  const int64_t* slots;
  int64_t num_tokens, num_slots;
  int n_heads, block_size;
  int lanes_log2;
  unsigned int* err;
};

// in: piece of [num_tokens, n_heads, lanes]; pool: piece of the pool. False:
// the token is skipped, or there is none.
__device__ __forceinline__ bool place(const Rows4& p, int64_t& in, int64_t& pool) {
  const int g = threadIdx.x & ((1 << p.lanes_log2) - 1);
  const int64_t t = static_cast<int64_t>(blockIdx.x) * (kThreads4 >> p.lanes_log2) + (threadIdx.x >> p.lanes_log2);
  const int h = blockIdx.y;
  in = pool = 0;
  if (t >= p.num_tokens) return false;
  const int64_t slot = __ldg(p.slots + t);
  if (slot < 0) return false;
  if (slot >= p.num_slots) {
    if (h == 0 && g == 0) set_flag(p.err, KVC_FLAG_BAD_SLOT);
    return false;
  }
  int64_t blk;
  int row;
  if (p.num_slots < (1ll << 31)) {  // (the same in every thread; a 64-bit division takes four times as long)
    const uint32_t b = static_cast<uint32_t>(slot) / static_cast<uint32_t>(p.block_size);
    row = static_cast<int>(static_cast<uint32_t>(slot) - b * p.block_size);
    blk = b;
  } else {
    blk = slot / p.block_size;
    row = static_cast<int>(slot - blk * p.block_size);
  }
  in = ((t * p.n_heads + h) << p.lanes_log2) + g;
  pool = (((blk * p.n_heads + h) * p.block_size + row) << p.lanes_log2) + g;
  return true;
}

template <typename T>
__global__ void __launch_bounds__(kThreads4)
    append4_kernel(const T* __restrict__ k, const T* __restrict__ v, const Rows4 p, uint2* __restrict__ kc,
                   uint2* __restrict__ vc, unsigned char* __restrict__ ks, unsigned char* __restrict__ vs) {
  // a decode launched behind this kernel may start its prologue now; it waits for
  // this grid to finish before it reads any cached row
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  int64_t from, to;
  if (!place(p, from, to)) return;
  Group<T> x, y;
  x.load(k + from * kGroup4);
  y.load(v + from * kGroup4);
  uint32_t s;
  kc[to] = quantise<T>(x, s);
  ks[to] = static_cast<unsigned char>(s);
  vc[to] = quantise<T>(y, s);
  vs[to] = static_cast<unsigned char>(s);
}

template <typename T>
__device__ __forceinline__ void store8(T* p, uint32_t code, float s) {
  uint32_t h[4];
  decode8_e2m1(code, h);
  float x[8];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float2 f = __half22float2(*reinterpret_cast<__half2*>(&h[j]));
    x[2 * j] = f.x * s;
    x[2 * j + 1] = f.y * s;
  }
  constexpr int kind = sizeof(T) == 4 ? KVC_F32 : std::is_same<T, __half>::value ? KVC_F16 : KVC_BF16;
  if constexpr (kind == KVC_F32) {
    store_out_vec<4>(p, 0, x, kind);
    store_out_vec<4>(p, 4, x + 4, kind);
  } else {
    store_out_vec<8>(p, 0, x, kind);
  }
}

template <typename T>
__global__ void __launch_bounds__(kThreads4)
    read4_kernel(const Rows4 p, const uint32_t* __restrict__ kc, const uint32_t* __restrict__ vc,
                 const unsigned char* __restrict__ ks, const unsigned char* __restrict__ vs, T* __restrict__ k,
                 T* __restrict__ v) {
  int64_t to, from;
  if (!place(p, to, from)) return;
  const uint32_t a = __ldg(kc + from), b = __ldg(vc + from);
  const uint32_t sa = __ldg(ks + (from >> 1)), sb = __ldg(vs + (from >> 1));
  store8(k + to * kHalf4, a, scale_value(sa));
  store8(v + to * kHalf4, b, scale_value(sb));
}

// Checks shared by both calls.
kvc_status check4(const void* k, const void* v, const int64_t* slots, int64_t num_tokens, const void* kc,
                  const void* vc, const uint8_t* ks, const uint8_t* vs, int64_t num_blocks, int block_size,
                  int n_kv_heads, int head_dim, kvc_dtype dtype) {
  if (!dtype_ok(dtype)) return fail(KVC_ERR_INVALID_ARG, "unknown dtype %d", static_cast<int>(dtype));
  if (num_tokens < 0 || num_blocks < 1 || block_size < 1 || n_kv_heads < 1 || head_dim < 1)
    return fail(KVC_ERR_INVALID_ARG, "sizes must be positive (num_tokens >= 0)");
  if (head_dim != 64 && head_dim != 128 && head_dim != 256)
    return fail(KVC_ERR_UNSUPPORTED, "head_dim %d (supported: 64, 128, 256)", head_dim);
  if (block_size % 16 != 0 || block_size > 128)
    return fail(KVC_ERR_UNSUPPORTED, "block_size %d (supported: multiples of 16 up to 128)", block_size);
  if (n_kv_heads > 65535 || num_blocks > (1ll << 55) / block_size / n_kv_heads / head_dim ||
      num_tokens > (1ll << 31) * (kThreads4 * kHalf4 / head_dim) - (1 << 20))
    return fail(KVC_ERR_UNSUPPORTED, "num_blocks, num_tokens or n_kv_heads too large");
  if (num_tokens == 0) return KVC_OK;
  if (k == nullptr || v == nullptr || slots == nullptr || kc == nullptr || vc == nullptr || ks == nullptr ||
      vs == nullptr)
    return fail(KVC_ERR_INVALID_ARG, "NULL pointer");
  if (!aligned16(k) || !aligned16(v) || !aligned16(kc) || !aligned16(vc) || !aligned16(ks) || !aligned16(vs))
    return fail(KVC_ERR_INVALID_ARG, "k, v, the caches and the scales must be 16-byte aligned");
  return KVC_OK;
}

Rows4 rows4(const int64_t* slots, int64_t num_tokens, int64_t num_blocks, int block_size, int n_kv_heads,
            int lanes, unsigned int* err) {
  int log2 = 0;
  while ((1 << log2) < lanes) ++log2;
  return {slots, num_tokens, num_blocks * block_size, n_kv_heads, block_size, log2, err};
}
dim3 grid4(const Rows4& p) {
  const int64_t per = kThreads4 >> p.lanes_log2;
  return dim3(static_cast<unsigned>((p.num_tokens + per - 1) / per), static_cast<unsigned>(p.n_heads));
}

}  // namespace
}  // namespace kvc

extern "C" {

kvc_status kvc_append_fp4(const void* k, const void* v, const int64_t* slot_mapping, int64_t num_tokens,
                          void* k_cache, void* v_cache, uint8_t* k_scale, uint8_t* v_scale, int64_t num_blocks,
                          int block_size, int n_kv_heads, int head_dim, kvc_dtype dtype, kvc_stream stream) {
  using namespace kvc;
  clear_error();
  kvc_status st = check4(k, v, slot_mapping, num_tokens, k_cache, v_cache, k_scale, v_scale, num_blocks, block_size,
                         n_kv_heads, head_dim, dtype);
  if (st != KVC_OK || num_tokens == 0) return st;
  DeviceInfo* dev = nullptr;
  if ((st = current_device(&dev)) != KVC_OK) return st;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const Rows4 p =
      rows4(slot_mapping, num_tokens, num_blocks, block_size, n_kv_heads, head_dim / kGroup4, dev->error_word);
  auto launch = [&](auto* kernel, auto zero) {
    using T = decltype(zero);
    kernel<<<grid4(p), kThreads4, 0, s>>>(static_cast<const T*>(k), static_cast<const T*>(v), p,
                                          static_cast<uint2*>(k_cache), static_cast<uint2*>(v_cache), k_scale,
                                          v_scale);
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
  kvc_status st = check4(k, v, slot_mapping, num_tokens, k_cache, v_cache, k_scale, v_scale, num_blocks, block_size,
                         n_kv_heads, head_dim, dtype);
  if (st != KVC_OK || num_tokens == 0) return st;
  DeviceInfo* dev = nullptr;
  if ((st = current_device(&dev)) != KVC_OK) return st;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const Rows4 p =
      rows4(slot_mapping, num_tokens, num_blocks, block_size, n_kv_heads, head_dim / kHalf4, dev->error_word);
  auto launch = [&](auto* kernel, auto zero) {
    using T = decltype(zero);
    kernel<<<grid4(p), kThreads4, 0, s>>>(p, static_cast<const uint32_t*>(k_cache), static_cast<const uint32_t*>(v_cache),
                                          k_scale, v_scale, static_cast<T*>(k), static_cast<T*>(v));
  };
  if (dtype == KVC_F32) launch(read4_kernel<float>, float());
  else if (dtype == KVC_F16) launch(read4_kernel<__half>, __half());
  else launch(read4_kernel<__nv_bfloat16>, __nv_bfloat16());
  return finish_call(s);
}

}  // extern "C"
