// Parameters of the weight-accumulating decode (kvc_decode_attention_scored)
// and of the decode over block-scaled one-byte caches
// (kvc_decode_attention_block8), shared by the host planner and the kernels.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <cstddef>
#include <cstdint>

#include "kvc_internal.h"

namespace kvc {

struct ScoredParams {
  const void* q;                // [batch, n_tok, n_q_heads, D]
  const int32_t* block_tables;  // [batch, max_blocks]
  const int32_t* context_lens;  // [batch]
  const void* v_cache;
  const float* k_scale;         // one-byte caches: [num_blocks, n_kv_heads]
  const float* v_scale;
  void* out;      // [batch, n_tok, n_q_heads, D]
  float* scores;  // [batch, n_kv_heads, rows]; NULL: weights are not accumulated
  // workspace
  float* rec_o;   // [2 * workers, 8 * NT, D] unnormalised partial outputs, see scored_decode_kernel
  float* rec_ml;  // [2 * workers, 8 * NT, 2] (maximum in log2 units, sum of weights)
  int4* units;    // [batch * n_kv_heads * n_hsub] where a unit's records are, see kUnit*
  float* lse;     // [batch * n_tok * n_q_heads] log2 of the softmax denominator, units of one worker (scores only)
  float* logits;  // [batch * n_kv_heads, rows, qns] scaled scores in log2 units (scores only)
  unsigned int* err;
  int64_t num_blocks;
  int batch, n_q_heads, n_kv_heads;
  int group;   // n_q_heads / n_kv_heads
  int n_tok;   // new query tokens per sequence
  int qn;      // queries of a kv head: n_tok * group
  int qns;     // qn rounded up to an even number
  int n_hsub;  // column groups of 8 * NT queries that make up qn
  int block_size, max_blocks;
  int rows;    // max_blocks * block_size
  int out_dtype;
  int q_f16;      // one-byte caches: queries are f16 (else bf16)
  int workers;    // warps that share the work
  int min_tiles;  // tiles a worker takes at least
  float qscale;   // scale * log2(e)
  unsigned int wait_polls;
};

// ScoredParams::units entries: x = the first worker that holds tiles of the
// unit, or one of kUnit*; y = the last one; z = 1 if that one's part ends before
// its range does (a record of its own); w = workers per CTA.
constexpr int kUnitWhole = -1;  // one worker had the whole unit and wrote its output
constexpr int kUnitEmpty = -2;  // the sequence's length is invalid: outputs are zeros

constexpr int kTileRows = 16;
constexpr int kScoredMaxBatch = 4096;
constexpr int kScoredMaxTokens = 256;
constexpr int kScoredMaxQueries = 4096;  // n_tok * group: their denominators sit in shared memory

// Compile-time geometry for a cache element of ELT bytes, head size D and NT
// groups of 8 queries per warp.
template <int ELT, int D, int NT>
struct ScoredGeo {
  static constexpr int kRowBytes = D * ELT;
  static constexpr int kBoxBytes = kRowBytes < 128 ? kRowBytes : 128;  // swizzled span
  static constexpr int kHalves = kRowBytes / kBoxBytes;
  static constexpr int kTileBytes = kTileRows * kRowBytes;
  // A stage holds the K and the V tiles of kStageTiles tiles: 8 KB, or 16 KB
  // where one tile pair is that large.
  static constexpr int kStageTiles = 2 * kTileBytes >= 8192 ? 1 : 8192 / (2 * kTileBytes);
  static constexpr int kStageBytes = 2 * kStageTiles * kTileBytes;
  // Warps and stages fill 192 KB. One-byte tiles carry twice the products per
  // byte: more warps, as far as their registers allow, hide the products'
  // latency better than more stages do (e4m3, batch 32 x U[512, 4096]: 36.9 us
  // with 12 warps of 2 stages, 39.9 us with 8 of 3, 43.0 us with 16 of 3
  // half-size stages, where registers spill).
  static constexpr int kWarps = kStageBytes > 8192 ? 4 : (ELT == 1 && D <= 128 && NT == 1) ? 12 : 8;
  static constexpr int kStages = kWarps == 12 ? 2 : 3;
  static constexpr int kThreads = kWarps * 32;
  static constexpr size_t kRingBytes = static_cast<size_t>(kWarps) * kStages * kStageBytes;
};

// Shared memory: [ring, 1024-byte aligned][full barriers][scales of the
// stages' tiles][prefix sums of the sequences' tiles].
template <int ELT, int D, int NT>
__host__ __device__ constexpr size_t scored_smem_bytes(int batch) {
  using G = ScoredGeo<ELT, D, NT>;
  return 1024 + G::kRingBytes + G::kWarps * G::kStages * 8 + G::kWarps * G::kStages * G::kStageTiles * 2 * 4 +
         (static_cast<size_t>(batch) + 1 + 32) * 4;
}

// Groups of 8 queries that a warp carries at once.
inline int scored_nt(int D, int qn) { return D <= 128 && qn > 8 ? 2 : 1; }
// Warps per CTA of the kernel for this element size, head size and nt: what the
// host sizes records and counts workers by (checked against ScoredGeo where the
// kernel is launched).
constexpr int scored_warps(int elt, int D, int nt) {
  return elt == 2 && D == 256 ? 4 : (elt == 1 && D <= 128 && nt == 1) ? 12 : 8;
}

// Launches the decode and its finishing kernel. CT: __nv_bfloat16, __half,
// fp8e4m3 or s8q.
template <typename CT>
kvc_status scored_launch(const ScoredParams& p, int D, int nt, int grid, const CUtensorMap& tk, const CUtensorMap& tv,
                         cudaStream_t stream);

}  // namespace kvc
