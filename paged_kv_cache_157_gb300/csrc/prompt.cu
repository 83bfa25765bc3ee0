// Prompt attention over a paged 16-bit cache (kvc_prompt_attention): a ragged
// batch of new tokens, each attending its sequence's cached rows up to its own,
// optionally only a window of them and the sequence's first rows.
//
// Sources: the chunk mask of "单请求 KV Cache" (query row i of a chunk sees
// columns up to past_len + i) and the block table of "KV Cache（键值缓存）" section
// 2.3; Window Attention of "KV-Cache——为什么AI回复越来越快" section 08.
#include <algorithm>

#include "attend_row.cuh"
#include "kvc_internal.h"

namespace kvc {

namespace {

constexpr int kPromptMaxBatch = 4096;

struct PromptShape {
  int batch;
  int64_t num_tokens;
  int n_q_heads, n_kv_heads, D, block_size, max_blocks;
};

struct PromptParams {
  RowParams row;
  const void* q;  // [num_tokens, n_q_heads, D]
  void* out;
  const int32_t* block_tables;
  const int32_t* query_starts;  // [batch + 1]
  const int32_t* context_lens;
  unsigned int* err;
  int batch, num_tokens, n_q_heads, group, max_blocks, rows;
};

// Sequence i's first new token, their number and its rows. Tokens of a
// sequence whose starts are out of order or range are none; rows 0: the length
// is invalid, its outputs are zeros.
struct Span {
  int first, count, rows;
};
__device__ __forceinline__ Span span_of(const PromptParams& p, int i, bool flag) {
  Span s;
  s.first = __ldg(p.query_starts + i);
  const int end = __ldg(p.query_starts + i + 1);
  s.rows = __ldg(p.context_lens + i);
  s.count = end - s.first;
  bool bad = false;
  if (s.first < 0 || end < s.first || end > p.num_tokens) {
    s.count = s.first = 0;
    bad = true;
  } else if (s.count > 0 && (s.rows < s.count || s.rows > p.rows)) {
    s.rows = 0;
    bad = true;
  }
  if (flag && bad) set_flag(p.err, KVC_FLAG_BAD_LEN);
  return s;
}

template <typename CT, int D>
__global__ void __launch_bounds__(256) prompt_rows_kernel(const PromptParams p) {
  const int lane = threadIdx.x & 31;
  const int64_t warp = (static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x) >> 5;
  if (blockIdx.x == 0)
    for (int i = threadIdx.x; i < p.batch; i += 256) (void)span_of(p, i, true);
  if (warp >= static_cast<int64_t>(p.num_tokens) * p.n_q_heads) return;
  const int t = static_cast<int>(warp / p.n_q_heads), h = static_cast<int>(warp - static_cast<int64_t>(t) * p.n_q_heads);
  int a = 0, b = p.batch - 1;  // the last sequence that starts at or before t
  while (a < b) {
    const int mid = (a + b + 1) >> 1;
    if (__ldg(p.query_starts + mid) <= t) a = mid; else b = mid - 1;
  }
  const Span s = span_of(p, a, false);
  if (t < s.first || t >= s.first + s.count) return;
  constexpr int N = D / 32;
  float q[N], o[N];
#pragma unroll
  for (int j = 0; j < N; ++j) o[j] = 0.f;
  if (s.rows > 0) {
    const CT* qr = static_cast<const CT*>(p.q) + warp * D + lane * N;
#pragma unroll
    for (int j = 0; j < N; ++j) q[j] = Elem<CT>::to_float(qr[j]);
    if (!attend_row<CT, D>(p.row, q, p.block_tables + static_cast<int64_t>(a) * p.max_blocks, h / p.group,
                           s.rows - s.count + t - s.first, o) && lane == 0)
      set_flag(p.err, KVC_FLAG_BAD_BLOCK);
  }
  store_out_vec<N>(p.out, warp * D + lane * N, o, std::is_same<CT, __half>::value ? KVC_F16 : KVC_BF16);
}

kvc_status check_shape(const PromptShape& s) {
  if (s.batch < 1 || s.num_tokens < 0 || s.n_q_heads < 1 || s.n_kv_heads < 1 || s.D < 1 || s.block_size < 1 ||
      s.max_blocks < 1)
    return fail(KVC_ERR_INVALID_ARG,
                "batch, heads, head_dim, block_size and max_blocks_per_seq must be >= 1, num_tokens >= 0");
  if (s.n_q_heads % s.n_kv_heads != 0)
    return fail(KVC_ERR_INVALID_ARG, "n_q_heads (%d) must be a multiple of n_kv_heads (%d)", s.n_q_heads,
                s.n_kv_heads);
  if (s.D != 64 && s.D != 128) return fail(KVC_ERR_UNSUPPORTED, "head_dim %d (supported: 64, 128)", s.D);
  if (s.block_size % 16 != 0 || s.block_size > 128)
    return fail(KVC_ERR_UNSUPPORTED, "block_size %d (supported: multiples of 16 up to 128)", s.block_size);
  if (s.batch > kPromptMaxBatch) return fail(KVC_ERR_UNSUPPORTED, "batch %d > %d", s.batch, kPromptMaxBatch);
  if (s.n_q_heads / s.n_kv_heads > 128)
    return fail(KVC_ERR_UNSUPPORTED, "at most 128 query heads per kv head");
  if (static_cast<int64_t>(s.max_blocks) * s.block_size > (1ll << 30))
    return fail(KVC_ERR_UNSUPPORTED, "max_blocks_per_seq x block_size too large");
  if (s.num_tokens >= (1ll << 31) / s.n_q_heads)
    return fail(KVC_ERR_UNSUPPORTED, "num_tokens x n_q_heads must be below 2^31");
  return KVC_OK;
}

}  // namespace
}  // namespace kvc

extern "C" {

kvc_status kvc_prompt_workspace_size(int batch, int64_t num_tokens, int n_q_heads, int n_kv_heads, int head_dim,
                                     int block_size, int max_blocks_per_seq, size_t* bytes) {
  using namespace kvc;
  clear_error();
  if (bytes == nullptr) return fail(KVC_ERR_INVALID_ARG, "bytes is NULL");
  const kvc_status st =
      check_shape({batch, num_tokens, n_q_heads, n_kv_heads, head_dim, block_size, max_blocks_per_seq});
  if (st != KVC_OK) return st;
  DeviceInfo* dev = nullptr;
  const kvc_status sd = current_device(&dev);
  if (sd != KVC_OK) return sd;
  *bytes = 256;
  return KVC_OK;
}

kvc_status kvc_prompt_attention(const void* q, const void* k_cache, const void* v_cache, const int32_t* block_tables,
                                int max_blocks_per_seq, const int32_t* query_starts, const int32_t* context_lens,
                                int batch, int64_t num_tokens, float scale, int n_q_heads, int n_kv_heads,
                                int head_dim, int block_size, int64_t num_blocks, int window, int sinks,
                                kvc_dtype dtype, void* out, void* workspace, size_t workspace_bytes,
                                kvc_stream stream) {
  using namespace kvc;
  clear_error();
  kvc_status st = check_shape({batch, num_tokens, n_q_heads, n_kv_heads, head_dim, block_size, max_blocks_per_seq});
  if (st != KVC_OK) return st;
  if (!dtype_ok(dtype)) return fail(KVC_ERR_INVALID_ARG, "unknown dtype %d", static_cast<int>(dtype));
  if (dtype == KVC_F32) return fail(KVC_ERR_UNSUPPORTED, "16-bit elements only (F16, BF16)");
  if (window < 1 || sinks < 0) return fail(KVC_ERR_INVALID_ARG, "window must be >= 1 and sinks >= 0");
  if (num_blocks < 1) return fail(KVC_ERR_INVALID_ARG, "num_blocks must be >= 1");
  if (num_blocks > ((1ll << 31) - 1) / block_size / n_kv_heads)
    return fail(KVC_ERR_UNSUPPORTED, "num_blocks x n_kv_heads x block_size must be below 2^31");
  if (num_tokens == 0) return KVC_OK;
  if (q == nullptr || k_cache == nullptr || v_cache == nullptr || block_tables == nullptr ||
      query_starts == nullptr || context_lens == nullptr || out == nullptr)
    return fail(KVC_ERR_INVALID_ARG, "NULL pointer");
  if (!aligned16(q) || !aligned16(k_cache) || !aligned16(v_cache) || !aligned16(out))
    return fail(KVC_ERR_INVALID_ARG, "q, out, k_cache and v_cache must be 16-byte aligned");
  DeviceInfo* dev = nullptr;
  if ((st = current_device(&dev)) != KVC_OK) return st;
  size_t needed = 0;
  if ((st = kvc_prompt_workspace_size(batch, num_tokens, n_q_heads, n_kv_heads, head_dim, block_size,
                                      max_blocks_per_seq, &needed)) != KVC_OK)
    return st;
  if (workspace == nullptr || workspace_bytes < needed)
    return fail(KVC_ERR_WORKSPACE, "workspace of %zu bytes, %zu needed", workspace == nullptr ? 0 : workspace_bytes,
                needed);
  if ((reinterpret_cast<uintptr_t>(workspace) & 255u) != 0)
    return fail(KVC_ERR_INVALID_ARG, "workspace must be 256-byte aligned");
  PromptParams p{};
  p.row = {k_cache, v_cache, nullptr, nullptr, num_blocks, n_kv_heads, block_size, window, sinks,
           scale * 1.4426950408889634f};
  p.q = q;
  p.out = out;
  p.block_tables = block_tables;
  p.query_starts = query_starts;
  p.context_lens = context_lens;
  p.err = dev->error_word;
  p.batch = batch;
  p.num_tokens = static_cast<int>(num_tokens);
  p.n_q_heads = n_q_heads;
  p.group = n_q_heads / n_kv_heads;
  p.max_blocks = max_blocks_per_seq;
  p.rows = max_blocks_per_seq * block_size;
  const unsigned grid = static_cast<unsigned>((num_tokens * n_q_heads + 7) / 8);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  auto* kernel = dtype == KVC_F16 ? (head_dim == 64 ? prompt_rows_kernel<__half, 64> : prompt_rows_kernel<__half, 128>)
                                  : (head_dim == 64 ? prompt_rows_kernel<__nv_bfloat16, 64>
                                                    : prompt_rows_kernel<__nv_bfloat16, 128>);
  kernel<<<grid, 256, 0, s>>>(p);
  return finish_call(s);
}

}  // extern "C"
