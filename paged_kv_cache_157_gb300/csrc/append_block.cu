// Append into a one-byte cache that has one scale for each (block, kv head).
//
// The tokens of a call that fall into one block are adjacent in the slot
// mapping: a run. For a run with lowest row `first` and each kv head,
//   A = max |x| over the run's finite entries
//   s = max(s_old, A * (1 / Q))    s_old = 0 when the run starts the block (first == 0); Q = 448 or 127
//   rows below first: c = q(c * (s_old / s)) when the scale grew
//   the run's rows:   c = q(x * (1 / s))
// in fp32, each operation rounded once, q to the nearest code (ties to even,
// saturating). The scale of a block never shrinks while the block fills, so
// earlier rows are rounded again only when a louder token arrives.
//
// One warp per (run, kv head, K or V). A warp looks at a stretch of tokens,
// finds the runs that begin in it and takes them one by one: two sweeps over
// the rows in 16-byte loads, the second (the codes) out of L1/L2. Bound by
// HBM for prompts; by the chain slot -> scale -> row -> code of four dependent
// accesses for a decode step, which is why a step's warps get one token each.
#include <algorithm>

#include "code8.cuh"

namespace kvc {

namespace {

// Largest finite |x| among the values of one 16-byte chunk of T.
template <typename T>
__device__ __forceinline__ float chunk_max(const uint4& u) {
  float m = 0.f;
#pragma unroll
  for (int i = 0; i < 16 / static_cast<int>(sizeof(T)) / 2; ++i) {
    const float2 x = Elem<T>::pair(u, i);
    const float a = fabsf(x.x), b = fabsf(x.y);
    m = fmaxf(m, a < INFINITY ? a : 0.f);
    m = fmaxf(m, b < INFINITY ? b : 0.f);
  }
  return m;
}

struct AppendBlockParams {
  const void *k, *v;  // [num_tokens, n_heads, D]
  const int64_t* slots;
  unsigned char *k_codes, *v_codes;  // [num_blocks, n_heads, block_size, D]
  float *k_scale, *v_scale;          // [num_blocks, n_heads]
  int64_t num_tokens, num_slots;
  int n_heads, block_size;
  int stretch;  // tokens a warp looks at (1 .. 32)
  unsigned int* err;
};

// Block of a slot, -1 if the token is not written.
__device__ __forceinline__ int64_t block_of(int64_t slot, const AppendBlockParams& p) {
  if (slot < 0 || slot >= p.num_slots) return -1;
  return ((slot | p.block_size) >> 32) == 0 ? static_cast<uint32_t>(slot) / static_cast<uint32_t>(p.block_size)
                                            : slot / p.block_size;
}

constexpr int kAppendWarps = 4;

template <typename T, bool INT8, int D>
__global__ void __launch_bounds__(32 * kAppendWarps) append_block_kernel(const AppendBlockParams p) {
  constexpr int VEC = 16 / sizeof(T);  // values per 16-byte chunk
  constexpr int CPR = D / VEC;         // chunks per row
  constexpr int U = 8;                 // chunks in flight per lane
  constexpr uint32_t full = 0xffffffffu;
  // a decode launched behind this kernel may set itself up meanwhile; it waits
  // for this grid to end before it reads any cached row
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int lane = threadIdx.x & 31;
  const int64_t wi = static_cast<int64_t>(blockIdx.x) * kAppendWarps + (threadIdx.x >> 5);
  const int kv = static_cast<int>(wi % 2);
  const int h = static_cast<int>((wi / 2) % p.n_heads);
  const int64_t t0 = wi / 2 / p.n_heads * p.stretch;
  if (t0 >= p.num_tokens) return;
  const T* x = static_cast<const T*>(kv ? p.v : p.k);
  const int bs = p.block_size;

  int64_t mine = -1;  // this lane's token's block
  bool leads = false;
  if (lane < p.stretch && t0 + lane < p.num_tokens) {
    const int64_t slot = __ldg(p.slots + t0 + lane);
    mine = block_of(slot, p);
    if (slot >= p.num_slots && h == 0 && kv == 0) set_flag(p.err, KVC_FLAG_BAD_SLOT);
    leads = mine >= 0 && (t0 + lane == 0 || block_of(__ldg(p.slots + t0 + lane - 1), p) != mine);
  }
  for (uint32_t todo = __ballot_sync(full, leads); todo != 0; todo &= todo - 1) {
    const int at = __ffs(todo) - 1;
    const int64_t blk = __shfl_sync(full, mine, at);
    const int64_t a = t0 + at;  // the run's first token
    // its end, and the lowest row it writes
    int64_t e = a;
    int first = bs;
    for (;;) {
      bool in = false;
      int row = bs;
      if (e + lane < p.num_tokens) {
        const int64_t slot = __ldg(p.slots + e + lane);
        in = block_of(slot, p) == blk;
        if (in) row = static_cast<int>(slot - blk * bs);
      }
      const uint32_t got = __ballot_sync(full, in);
      const int len = got == full ? 32 : __ffs(~got) - 1;
      first = min(first, static_cast<int>(__reduce_min_sync(full, lane < len ? row : bs)));
      e += len;
      if (len < 32) break;
    }
    float* scale = (kv ? p.v_scale : p.k_scale) + blk * p.n_heads + h;
    const float old = first == 0 ? 0.f : *scale;
    const int64_t chunks = (e - a) * CPR;
    auto src = [&](int64_t i) {  // chunk i of the run
      return reinterpret_cast<const uint4*>(x + ((a + i / CPR) * p.n_heads + h) * D) + i % CPR;
    };
    float m = 0.f;
    for (int64_t i0 = lane; i0 < chunks; i0 += 32 * U) {
      uint4 u[U];
#pragma unroll
      for (int j = 0; j < U; ++j) u[j] = i0 + 32 * j < chunks ? *src(i0 + 32 * j) : make_uint4(0, 0, 0, 0);
#pragma unroll
      for (int j = 0; j < U; ++j) m = fmaxf(m, chunk_max<T>(u[j]));
    }
    m = warp_max(m);
    float s = fmaxf(old, m * Code8<INT8>::kInvMax);
    if (!(s >= kTinyScale)) s = 0.f;
    const float inv = s > 0.f ? __fdiv_rn(1.0f, s) : 0.f;
    unsigned char* dst = (kv ? p.v_codes : p.k_codes) + (blk * p.n_heads + h) * static_cast<int64_t>(bs) * D;
    if (first > 0 && s != old) {
      const float f = s > 0.f ? __fdiv_rn(old, s) : 0.f;
      uint4* rows = reinterpret_cast<uint4*>(dst);
      for (int i = lane; i < first * (D / 16); i += 32) rows[i] = rescale16<INT8>(rows[i], f);
    }
    for (int64_t i0 = lane; i0 < chunks; i0 += 32 * U) {
      uint4 u[U];
      int row[U];
#pragma unroll
      for (int j = 0; j < U; ++j) {
        const int64_t i = i0 + 32 * j;
        row[j] = -1;
        if (i < chunks) {
          u[j] = *src(i);
          row[j] = static_cast<int>(__ldg(p.slots + a + i / CPR) - blk * bs);
        }
      }
#pragma unroll
      for (int j = 0; j < U; ++j) {
        if (row[j] < 0) continue;
        unsigned char* to = dst + row[j] * D + static_cast<int>((i0 + 32 * j) % CPR) * VEC;
        float2 v[VEC / 2];
#pragma unroll
        for (int k = 0; k < VEC / 2; ++k) {
          v[k] = Elem<T>::pair(u[j], k);
          // scale 0: every finite entry is 0 (or too small to count), and 0 x inf would not be
          v[k].x = s > 0.f ? v[k].x * inv : 0.f;
          v[k].y = s > 0.f ? v[k].y * inv : 0.f;
        }
        if constexpr (VEC == 8)
          *reinterpret_cast<uint2*>(to) = make_uint2(encode4<INT8>(v[0].x, v[0].y, v[1].x, v[1].y),
                                                     encode4<INT8>(v[2].x, v[2].y, v[3].x, v[3].y));
        else
          *reinterpret_cast<uint32_t*>(to) = encode4<INT8>(v[0].x, v[0].y, v[1].x, v[1].y);
      }
    }
    __syncwarp();
    if (lane == 0) *scale = s;
  }
}

template <typename T, bool INT8>
void launch(const AppendBlockParams& p, int D, int64_t grid, cudaStream_t s) {
  const dim3 g(static_cast<unsigned>(grid)), b(32 * kAppendWarps);
  if (D == 64) append_block_kernel<T, INT8, 64><<<g, b, 0, s>>>(p);
  else if (D == 128) append_block_kernel<T, INT8, 128><<<g, b, 0, s>>>(p);
  else append_block_kernel<T, INT8, 256><<<g, b, 0, s>>>(p);
}

template <typename T>
void launch(const AppendBlockParams& p, int D, kvc_code code, int64_t grid, cudaStream_t s) {
  if (code == KVC_INT8) launch<T, true>(p, D, grid, s);
  else launch<T, false>(p, D, grid, s);
}

}  // namespace
}  // namespace kvc

extern "C" kvc_status kvc_append_block8(const void* k, const void* v, const int64_t* slot_mapping, int64_t num_tokens,
                                        void* k_cache, void* v_cache, float* k_scale, float* v_scale, kvc_code code,
                                        int64_t num_blocks, int block_size, int n_kv_heads, int head_dim,
                                        kvc_dtype dtype, kvc_stream stream) {
  using namespace kvc;
  clear_error();
  if (code != KVC_E4M3 && code != KVC_INT8)
    return fail(KVC_ERR_INVALID_ARG, "unknown code format %d", static_cast<int>(code));
  if (!dtype_ok(dtype)) return fail(KVC_ERR_INVALID_ARG, "unknown dtype %d", static_cast<int>(dtype));
  if (num_tokens < 0 || num_blocks < 1 || block_size < 1 || n_kv_heads < 1 || head_dim < 1)
    return fail(KVC_ERR_INVALID_ARG, "sizes must be positive (num_tokens >= 0)");
  if (head_dim != 64 && head_dim != 128 && head_dim != 256)
    return fail(KVC_ERR_UNSUPPORTED, "head_dim %d (supported: 64, 128, 256)", head_dim);
  if (block_size % 16 != 0 || block_size > 128)
    return fail(KVC_ERR_UNSUPPORTED, "block_size %d (supported: multiples of 16 up to 128)", block_size);
  if (num_tokens == 0) return KVC_OK;
  if (k == nullptr || v == nullptr || slot_mapping == nullptr || k_cache == nullptr || v_cache == nullptr ||
      k_scale == nullptr || v_scale == nullptr)
    return fail(KVC_ERR_INVALID_ARG, "NULL pointer");
  if (!aligned16(k) || !aligned16(v) || !aligned16(k_cache) || !aligned16(v_cache))
    return fail(KVC_ERR_INVALID_ARG, "k, v and the caches must be 16-byte aligned");
  DeviceInfo* dev = nullptr;
  kvc_status st = current_device(&dev);
  if (st != KVC_OK) return st;
  AppendBlockParams p{};
  p.k = k;
  p.v = v;
  p.slots = slot_mapping;
  p.k_codes = static_cast<unsigned char*>(k_cache);
  p.v_codes = static_cast<unsigned char*>(v_cache);
  p.k_scale = k_scale;
  p.v_scale = v_scale;
  p.num_tokens = num_tokens;
  p.num_slots = num_blocks * block_size;
  p.n_heads = n_kv_heads;
  p.block_size = block_size;
  p.err = dev->error_word;
  // one token per warp while the warps fit the GPU at once, longer stretches
  // beyond: most warps of a prompt find no run that begins in theirs
  const int64_t items = 2 * num_tokens * n_kv_heads, resident = 64LL * dev->num_sms;
  p.stretch = static_cast<int>(std::min<int64_t>(32, (items + resident - 1) / resident));
  const int64_t warps = (num_tokens + p.stretch - 1) / p.stretch * n_kv_heads * 2;
  const int64_t grid = (warps + kAppendWarps - 1) / kAppendWarps;
  if (grid >= (1ll << 31)) return fail(KVC_ERR_UNSUPPORTED, "num_tokens x n_kv_heads too large");
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  switch (dtype) {
    case KVC_F32: launch<float>(p, head_dim, code, grid, s); break;
    case KVC_F16: launch<__half>(p, head_dim, code, grid, s); break;
    case KVC_BF16: launch<__nv_bfloat16>(p, head_dim, code, grid, s); break;
  }
  return finish_call(s);
}
