// Host side of kvc_decode_attention_scored and kvc_decode_attention_block8:
// argument checks, workspace layout, tensor maps and launch.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>
#include <mutex>

#include "decode_scored.h"
#include "kvc_device.cuh"

namespace kvc {

namespace {

// Tiles (16 cached rows of one kv head) a warp takes at least: below that the
// records and their merge cost more than the extra warps bring.
constexpr int kMinTiles = 2;

struct ScoredShape {
  int batch, n_tok, n_q_heads, n_kv_heads, D, block_size, max_blocks;
  int64_t rows() const { return static_cast<int64_t>(max_blocks) * block_size; }
  int group() const { return n_q_heads / n_kv_heads; }
  int qn() const { return n_tok * group(); }
};

kvc_status check_shape(const ScoredShape& s) {
  if (s.batch < 1 || s.n_tok < 1 || s.n_q_heads < 1 || s.n_kv_heads < 1 || s.D < 1 || s.block_size < 1 ||
      s.max_blocks < 1)
    return fail(KVC_ERR_INVALID_ARG,
                "batch, n_tokens, heads, head_dim, block_size and max_blocks_per_seq must be >= 1");
  if (s.n_q_heads % s.n_kv_heads != 0)
    return fail(KVC_ERR_INVALID_ARG, "n_q_heads (%d) must be a multiple of n_kv_heads (%d)", s.n_q_heads,
                s.n_kv_heads);
  if (s.D != 64 && s.D != 128 && s.D != 256)
    return fail(KVC_ERR_UNSUPPORTED, "head_dim %d (supported: 64, 128, 256)", s.D);
  if (s.block_size % 16 != 0 || s.block_size > 128)
    return fail(KVC_ERR_UNSUPPORTED, "block_size %d (supported: multiples of 16 up to 128)", s.block_size);
  if (s.batch > kScoredMaxBatch) return fail(KVC_ERR_UNSUPPORTED, "batch %d > %d", s.batch, kScoredMaxBatch);
  if (s.n_tok > kScoredMaxTokens)
    return fail(KVC_ERR_UNSUPPORTED, "n_tokens %d > %d", s.n_tok, kScoredMaxTokens);
  if (static_cast<int64_t>(s.n_tok) * s.group() > kScoredMaxQueries)
    return fail(KVC_ERR_UNSUPPORTED, "n_tokens x query heads per kv head must be at most %d", kScoredMaxQueries);
  if (s.rows() > (1ll << 30)) return fail(KVC_ERR_UNSUPPORTED, "max_blocks_per_seq x block_size too large");
  // the kernel's tile positions and unit numbers are 32-bit
  const int nc = 8 * scored_nt(s.D, s.qn()), n_hsub = (s.qn() + nc - 1) / nc;
  const int64_t units = static_cast<int64_t>(s.batch) * s.n_kv_heads * n_hsub;
  if (units >= (1ll << 27) || units * ((s.rows() + kTileRows - 1) / kTileRows) >= (1ll << 31) ||
      static_cast<int64_t>(s.batch) * s.n_tok * s.n_q_heads >= (1ll << 31))
    return fail(KVC_ERR_UNSUPPORTED, "batch x heads x queries x rows too large");
  return KVC_OK;
}

// Workspace: [records' outputs][records' maxima and sums][units][denominators]
// [scaled scores], each 256-byte aligned. Nothing in it has to be cleared.
struct ScoredLayout {
  size_t rec_o, rec_ml, units, lse, logits, total;
  int workers, grid, nt, n_hsub, qns;
};

inline size_t up256(size_t x) { return (x + 255) / 256 * 256; }

ScoredLayout layout(const ScoredShape& s, int elt, bool scored, int num_sms) {
  ScoredLayout l;
  const int qn = s.qn();
  l.nt = scored_nt(s.D, qn);
  const int nc = 8 * l.nt;
  l.n_hsub = (qn + nc - 1) / nc;
  l.qns = (qn + 1) / 2 * 2;
  const int64_t units = static_cast<int64_t>(s.batch) * s.n_kv_heads * l.n_hsub;
  const int64_t tiles = units * ((s.rows() + kTileRows - 1) / kTileRows);
  const int warps = scored_warps(elt, s.D, l.nt);
  // few tiles spread over as many SMs as there are workers
  l.grid = static_cast<int>(std::min<int64_t>(num_sms, (tiles + kMinTiles - 1) / kMinTiles));
  l.workers = l.grid * warps;
  const size_t recs = 2 * static_cast<size_t>(l.workers) * nc;
  l.rec_o = 0;
  l.rec_ml = up256(recs * s.D * 4);
  l.units = l.rec_ml + up256(recs * 8);
  l.lse = l.units + up256(static_cast<size_t>(units) * 16);
  l.logits = l.lse + (scored ? up256(static_cast<size_t>(s.batch) * s.n_tok * s.n_q_heads * 4) : 0);
  l.total = l.logits +
            (scored ? up256(static_cast<size_t>(s.batch) * s.n_kv_heads * s.rows() * l.qns * 4) : 0);
  return l;
}

// What the size query answers: one size for either kind of cache.
size_t workspace_needed(const ScoredShape& s, bool scored, int num_sms) {
  return std::max(layout(s, 1, scored, num_sms).total, layout(s, 2, scored, num_sms).total);
}

using EncodeTiledFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                   const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                   CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn encode_tiled_fn() {
  static std::once_flag once;
  static EncodeTiledFn fn = nullptr;
  std::call_once(once, [] {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q) ==
            cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<EncodeTiledFn>(f);
  });
  return fn;
}

// The pool as [num_blocks * n_kv_heads * block_size rows, D] in boxes of 16
// rows by 128 bytes (64 bytes where a row is that short), swizzled by as much.
kvc_status pool_map(const void* cache, int64_t pool_rows, int D, int elt, CUtensorMap* map) {
  EncodeTiledFn encode = encode_tiled_fn();
  if (encode == nullptr) return fail(KVC_ERR_CUDA, "cuTensorMapEncodeTiled is unavailable");
  const int row_bytes = D * elt, box_bytes = std::min(128, row_bytes);
  // 16-bit elements are only moved: one element type serves bf16 and f16
  const CUtensorMapDataType dt = elt == 1 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_UINT16;
  const cuuint64_t dims[2] = {static_cast<cuuint64_t>(D), static_cast<cuuint64_t>(pool_rows)};
  const cuuint64_t strides[1] = {static_cast<cuuint64_t>(row_bytes)};
  const cuuint32_t box[2] = {static_cast<cuuint32_t>(box_bytes / elt), kTileRows};
  const cuuint32_t es[2] = {1, 1};
  CUresult r = encode(map, dt, 2, const_cast<void*>(cache), dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
                      box_bytes == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
                      CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) return fail(KVC_ERR_CUDA, "tensor map for the cache: CUresult %d", static_cast<int>(r));
  return KVC_OK;
}

// Cache element of a call: a 16-bit type, or one-byte codes.
enum class Cache { kBf16, kF16, kE4m3, kInt8 };

kvc_status decode(Cache cache, const ScoredShape& s, const void* q, kvc_dtype q_dtype, const void* k_cache,
                  const void* v_cache, const float* k_scale, const float* v_scale, const int32_t* block_tables,
                  const int32_t* context_lens, float scale, int64_t num_blocks, void* out, kvc_dtype out_dtype,
                  float* scores, void* workspace, size_t workspace_bytes, cudaStream_t stream) {
  kvc_status st = check_shape(s);
  if (st != KVC_OK) return st;
  if (!dtype_ok(out_dtype)) return fail(KVC_ERR_INVALID_ARG, "unknown out_dtype %d", static_cast<int>(out_dtype));
  if (num_blocks < 1) return fail(KVC_ERR_INVALID_ARG, "num_blocks must be >= 1");
  if (num_blocks > ((1ll << 31) - 1) / s.block_size / s.n_kv_heads)
    return fail(KVC_ERR_UNSUPPORTED, "num_blocks x n_kv_heads x block_size must be below 2^31");
  if (q == nullptr || k_cache == nullptr || v_cache == nullptr || block_tables == nullptr ||
      context_lens == nullptr || out == nullptr)
    return fail(KVC_ERR_INVALID_ARG, "NULL pointer");
  if (!aligned16(q) || !aligned16(k_cache) || !aligned16(v_cache))
    return fail(KVC_ERR_INVALID_ARG, "q, k_cache and v_cache must be 16-byte aligned");
  DeviceInfo* dev = nullptr;
  if ((st = current_device(&dev)) != KVC_OK) return st;
  const int elt = cache == Cache::kBf16 || cache == Cache::kF16 ? 2 : 1;
  const ScoredLayout l = layout(s, elt, scores != nullptr, dev->num_sms);
  const size_t needed = workspace_needed(s, scores != nullptr, dev->num_sms);
  if (workspace == nullptr || workspace_bytes < needed)
    return fail(KVC_ERR_WORKSPACE, "workspace of %zu bytes, %zu needed", workspace == nullptr ? 0 : workspace_bytes,
                needed);
  if ((reinterpret_cast<uintptr_t>(workspace) & 255u) != 0)
    return fail(KVC_ERR_INVALID_ARG, "workspace must be 256-byte aligned");
  CUtensorMap tk, tv;
  const int64_t pool_rows = num_blocks * s.n_kv_heads * s.block_size;
  if ((st = pool_map(k_cache, pool_rows, s.D, elt, &tk)) != KVC_OK) return st;
  if ((st = pool_map(v_cache, pool_rows, s.D, elt, &tv)) != KVC_OK) return st;

  char* ws = static_cast<char*>(workspace);
  ScoredParams p{};
  p.q = q;
  p.v_cache = v_cache;
  p.block_tables = block_tables;
  p.context_lens = context_lens;
  p.k_scale = k_scale;
  p.v_scale = v_scale;
  p.out = out;
  p.scores = scores;
  p.rec_o = reinterpret_cast<float*>(ws + l.rec_o);
  p.rec_ml = reinterpret_cast<float*>(ws + l.rec_ml);
  p.units = reinterpret_cast<int4*>(ws + l.units);
  p.lse = reinterpret_cast<float*>(ws + l.lse);
  p.logits = reinterpret_cast<float*>(ws + l.logits);
  p.err = dev->error_word;
  p.num_blocks = num_blocks;
  p.batch = s.batch;
  p.n_q_heads = s.n_q_heads;
  p.n_kv_heads = s.n_kv_heads;
  p.group = s.group();
  p.n_tok = s.n_tok;
  p.qn = s.qn();
  p.qns = l.qns;
  p.n_hsub = l.n_hsub;
  p.block_size = s.block_size;
  p.max_blocks = s.max_blocks;
  p.rows = static_cast<int>(s.rows());
  p.out_dtype = out_dtype;
  p.q_f16 = q_dtype == KVC_F16 ? 1 : 0;
  p.qscale = scale * 1.4426950408889634f;  // log2(e): softmax is evaluated with exp2
  p.wait_polls = static_cast<unsigned int>(option(KVC_OPT_WAIT_POLLS));
  const int64_t cap = option(KVC_OPT_MAX_CTAS), forced = option(KVC_OPT_BLOCKS_PER_CTA);
  const int grid = static_cast<int>(cap > 0 ? std::min<int64_t>(cap, l.grid) : l.grid);
  p.workers = grid * scored_warps(elt, s.D, l.nt);
  // the work split's option counts cache blocks per worker, here a warp
  p.min_tiles = forced > 0 ? static_cast<int>(std::min<int64_t>(forced, 1 << 20)) * (s.block_size / kTileRows)
                           : kMinTiles;
  switch (cache) {
    case Cache::kBf16: st = scored_launch<__nv_bfloat16>(p, s.D, l.nt, grid, tk, tv, stream); break;
    case Cache::kF16: st = scored_launch<__half>(p, s.D, l.nt, grid, tk, tv, stream); break;
    case Cache::kE4m3: st = scored_launch<fp8e4m3>(p, s.D, l.nt, grid, tk, tv, stream); break;
    case Cache::kInt8: st = scored_launch<s8q>(p, s.D, l.nt, grid, tk, tv, stream); break;
  }
  if (st != KVC_OK) return st;
  return finish_call(stream);
}

}  // namespace
}  // namespace kvc

extern "C" {

kvc_status kvc_decode_scored_workspace_size(int batch, int n_tokens, int n_q_heads, int n_kv_heads, int head_dim,
                                            int block_size, int max_blocks_per_seq, int scored, size_t* bytes) {
  using namespace kvc;
  clear_error();
  if (bytes == nullptr) return fail(KVC_ERR_INVALID_ARG, "bytes is NULL");
  const ScoredShape s{batch, n_tokens, n_q_heads, n_kv_heads, head_dim, block_size, max_blocks_per_seq};
  kvc_status st = check_shape(s);
  if (st != KVC_OK) return st;
  DeviceInfo* dev = nullptr;
  if ((st = current_device(&dev)) != KVC_OK) return st;
  *bytes = workspace_needed(s, scored != 0, dev->num_sms);
  return KVC_OK;
}

kvc_status kvc_decode_attention_scored(const void* q, const void* k_cache, const void* v_cache,
                                       const int32_t* block_tables, int max_blocks_per_seq,
                                       const int32_t* context_lens, int batch, int n_tokens, float scale,
                                       int n_q_heads, int n_kv_heads, int head_dim, int block_size,
                                       int64_t num_blocks, kvc_dtype dtype, void* out, kvc_dtype out_dtype,
                                       float* scores, void* workspace, size_t workspace_bytes, kvc_stream stream) {
  using namespace kvc;
  clear_error();
  if (!dtype_ok(dtype)) return fail(KVC_ERR_INVALID_ARG, "unknown dtype %d", static_cast<int>(dtype));
  if (dtype == KVC_F32) return fail(KVC_ERR_UNSUPPORTED, "caches of 16-bit elements only (F16, BF16)");
  if (scores == nullptr) return fail(KVC_ERR_INVALID_ARG, "scores is NULL");
  const ScoredShape s{batch, n_tokens, n_q_heads, n_kv_heads, head_dim, block_size, max_blocks_per_seq};
  return decode(dtype == KVC_BF16 ? Cache::kBf16 : Cache::kF16, s, q, dtype, k_cache, v_cache, nullptr, nullptr,
                block_tables, context_lens, scale, num_blocks, out, out_dtype, scores, workspace, workspace_bytes,
                static_cast<cudaStream_t>(stream));
}

kvc_status kvc_decode_attention_block8(const void* q, const void* k_cache, const void* v_cache, const float* k_scale,
                                       const float* v_scale, kvc_code code, const int32_t* block_tables,
                                       int max_blocks_per_seq, const int32_t* context_lens, int batch, int n_tokens,
                                       float scale, int n_q_heads, int n_kv_heads, int head_dim, int block_size,
                                       int64_t num_blocks, kvc_dtype q_dtype, void* out, kvc_dtype out_dtype,
                                       float* scores, void* workspace, size_t workspace_bytes, kvc_stream stream) {
  using namespace kvc;
  clear_error();
  if (code != KVC_E4M3 && code != KVC_INT8)
    return fail(KVC_ERR_INVALID_ARG, "unknown code format %d", static_cast<int>(code));
  if (!dtype_ok(q_dtype)) return fail(KVC_ERR_INVALID_ARG, "unknown q_dtype %d", static_cast<int>(q_dtype));
  if (q_dtype == KVC_F32) return fail(KVC_ERR_UNSUPPORTED, "queries of 16-bit elements only (F16, BF16)");
  if (k_scale == nullptr || v_scale == nullptr) return fail(KVC_ERR_INVALID_ARG, "k_scale / v_scale is NULL");
  const ScoredShape s{batch, n_tokens, n_q_heads, n_kv_heads, head_dim, block_size, max_blocks_per_seq};
  return decode(code == KVC_E4M3 ? Cache::kE4m3 : Cache::kInt8, s, q, q_dtype, k_cache, v_cache, k_scale, v_scale,
                block_tables, context_lens, scale, num_blocks, out, out_dtype, scores, workspace, workspace_bytes,
                static_cast<cudaStream_t>(stream));
}

}  // extern "C"
