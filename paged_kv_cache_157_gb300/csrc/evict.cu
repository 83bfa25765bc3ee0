// Eviction by accumulated attention weight: per sequence and kv head the rows
// worth keeping are chosen (select) and moved, in their order, into the blocks
// of a new table (move).
//
// Of n rows m = min(n, budget) stay: the newest min(recent, m), and of the
// others those with the largest scores, ties to the lower row. The order of
// the rows stays, so windows and causal masks keep their meaning.
//
// select: one cluster of CTAs per (sequence, kv head). The scores become
// unsigned keys of the same order; counting passes over digits of 11 bits (8
// in a cluster) find the key T of the last row that stays and how many rows
// with that key stay (they end early when all that match so far stay); a prefix
// sum over the rows writes the kept rows in order.
// A CTA holds its share of the keys in registers, so a score is read once
// (shares beyond 8192 rows are read again each pass). Bound by the chain of
// passes and barriers (11 us for 256 rows of 4096 scores, 15 us for 8 rows of
// 65537); a cluster splits a long row over up to 8 SMs.
//
// move: one warp per 32 kept rows (one block of the new table for one-byte
// codes). Lanes look up the rows' addresses together, then move 16-byte chunks
// with several loads in flight. Bound by HBM: every kept row is read and
// written once (32 x 8 heads x 1024 bf16 rows of 128: 268 MB in 41 to 48 us,
// 5.6 to 6.5 TB/s).
#include <algorithm>

#include <cooperative_groups.h>

#include "code8.cuh"

namespace kvc {

namespace {

namespace cg = cooperative_groups;

struct EvictParams {
  const float* scores;          // [batch, n_heads, rows]
  const int32_t* tables;        // [batch, max_blocks]
  const int32_t* lens;          // [batch]
  const int32_t* new_tables;    // [batch, new_max_blocks]
  int32_t* kept;                // [batch, n_heads, budget]
  int32_t* new_lens;            // [batch]
  float* new_scores;            // [batch, n_heads, new_rows]
  unsigned char* pool[2];       // K, V
  float* scale[2];              // one-byte caches: [num_blocks, n_heads]
  int64_t num_blocks;
  int batch, n_heads, block_size, max_blocks, new_max_blocks;
  int rows, new_rows;           // max_blocks * block_size, new_max_blocks * block_size
  int budget, recent;
  int row_chunks, row_shift;    // 16-byte chunks of a cached row, log2 of it if it is a power of two
  unsigned int* err;
};

__device__ __forceinline__ int rows_of(const EvictParams& p, int b, bool* bad = nullptr) {
  const int n = __ldg(p.lens + b);
  const bool wrong = n < 0 || n > p.rows;
  if (bad != nullptr) *bad = wrong;
  return wrong ? 0 : n;
}

// Unsigned key of the same order as the score; NaN below everything, -0 as 0.
__device__ __forceinline__ uint32_t key_of(float x) {
  if (x != x) return 0u;
  const uint32_t u = __float_as_uint(x + 0.f);  // -0 + 0 = 0
  return (u & 0x80000000u) ? ~u : u | 0x80000000u;
}

constexpr int kSelectThreads = 512;
constexpr int kSelectWarps = kSelectThreads / 32;
constexpr int kKeys = 16;                            // keys a thread holds
constexpr int kSpan = kKeys * kSelectThreads;        // keys a CTA holds
constexpr int kBins = 2048;
constexpr int kMaxCluster = 8;

// Inclusive prefix sum over the lanes.
__device__ __forceinline__ uint32_t warp_scan(uint32_t v, int lane) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t u = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += u;
  }
  return v;
}

__global__ void __launch_bounds__(kSelectThreads, 2) select_kernel(const EvictParams p) {
  constexpr uint32_t full = 0xffffffffu;
  cg::cluster_group cluster = cg::this_cluster();
  const int C = static_cast<int>(cluster.num_blocks()), cr = static_cast<int>(cluster.block_rank());
  __shared__ __align__(16) uint32_t s_hist[3 * kBins];  // a pass's counts behind the last one's
  __shared__ uint32_t s_warp[kSelectWarps];
  __shared__ uint32_t s_found[3];                   // digit, rows above it and with it in this pass
  __shared__ uint32_t s_total[2];                   // this CTA's rows above T, and at T
  __shared__ uint32_t s_cnt[kKeys][kSelectWarps];   // rows above T (low half) and at T of a warp's 32 keys
  __shared__ uint32_t s_row[kKeys];
  const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  auto sync_all = [&]() {
    if (C == 1) __syncthreads(); else cluster.sync();
  };
  const uint32_t unit32 = blockIdx.x / C;
  const int64_t unit = unit32;
  const int b = static_cast<int>(unit32 / p.n_heads);
  bool bad;
  const int n = rows_of(p, b, &bad);
  const int m = min(n, p.budget), recent = min(p.recent, m);
  const int cand = n - recent;  // rows that compete for k places
  const int k = m - recent;
  int32_t* kept = p.kept + unit * p.budget;
  const float* scores = p.scores + unit * p.rows;
  const int gt = cr * kSelectThreads + tid, gn = C * kSelectThreads;
  if (gt == 0) {
    if (bad) set_flag(p.err, KVC_FLAG_BAD_LEN);
    if (unit32 % p.n_heads == 0) p.new_lens[b] = m;
  }
  for (int i = gt; i < recent; i += gn) kept[k + i] = cand + i;
  for (int i = m + gt; i < p.budget; i += gn) kept[i] = -1;
  if (k == cand || k == 0) {  // all of them, or none (the same in every CTA of the cluster)
    for (int i = gt; i < k; i += gn) kept[i] = i;
    return;
  }

  // this CTA's rows: a stretch of the candidates, in spans of kSpan keys; the
  // keys of the only span stay in registers, several are read again each pass
  const int per = (cand + C - 1) / C;
  // (never empty: a CTA beyond the candidates takes none of the last row)
  const int lo = min(cand - 1, cr * per), cnt = min(cand - lo, cr * per < cand ? per : 0);
  const int spans = max(1, (cnt + kSpan - 1) / kSpan);
  uint32_t key[kKeys];  // of row lo + span * kSpan + j * kSelectThreads + tid
  auto load = [&](int span) {
    float x[kKeys];  // all loads first (of the last row where there is none): no branch between them
#pragma unroll
    for (int j = 0; j < kKeys; ++j)
      x[j] = __ldg(scores + lo + min(span * kSpan + j * kSelectThreads + tid, max(cnt, 1) - 1));
#pragma unroll
    for (int j = 0; j < kKeys; ++j) key[j] = key_of(x[j]);
  };
  auto valid = [&](int span, int j) { return span * kSpan + j * kSelectThreads + tid < cnt; };
  load(0);
  for (int i = tid; i < (C == 1 ? 3 * kBins : 4 * 256); i += kSelectThreads) s_hist[i] = 0;
  if (tid < 2) s_total[tid] = 0;
  __syncthreads();

  // digits of 11, 11 and 10 bits, or of 8 in a cluster, whose CTAs read each
  // other's counts: 2048 bins of 8 CTAs took 4500 cycles a pass, mostly that
  const int width = C == 1 ? 11 : 8, passes = C == 1 ? 3 : 4;
  uint32_t prefix = 0, need = static_cast<uint32_t>(k);  // T's leading bits, places left among rows that match them
  uint32_t at_t = 0;                                     // rows that match them
  int shift = 32;
  for (int pass = 0; pass < passes; ++pass) {
    const int bits = min(width, shift);
    shift -= bits;
    uint32_t* hist = s_hist + (pass << width);
    for (int span = 0; span < spans; ++span) {
      if (spans > 1) load(span);
#pragma unroll
      for (int j = 0; j < kKeys; ++j) {
        if (span * kSpan + j * kSelectThreads >= cnt) break;  // short rows: nothing to do for any thread
        if (valid(span, j) && (pass == 0 || (key[j] >> (shift + bits)) == prefix))
          atomicAdd(&hist[(key[j] >> shift) & ((1u << bits) - 1u)], 1u);
      }
    }
    sync_all();
    // every CTA adds up the cluster's counts: thread t the digits of its four
    // bins from the top, so that a prefix sum over the threads counts the rows
    // with a larger digit
    const int bin = (1 << width) - 4 - 4 * tid;
    uint4 c = make_uint4(0u, 0u, 0u, 0u);
    if (bin >= 0) {
      c = *reinterpret_cast<const uint4*>(&hist[bin]);
      if (C > 1) {
        uint4 x[kMaxCluster];  // all reads in flight together
#pragma unroll
        for (int r = 0; r < kMaxCluster; ++r)
          if (r < C && r != cr) x[r] = *reinterpret_cast<const uint4*>(cluster.map_shared_rank(&hist[bin], r));
#pragma unroll
        for (int r = 0; r < kMaxCluster; ++r) {
          if (r < C && r != cr) {
            c.x += x[r].x;
            c.y += x[r].y;
            c.z += x[r].z;
            c.w += x[r].w;
          }
        }
      }
    }
    const uint32_t sum = c.x + c.y + c.z + c.w, v = warp_scan(sum, lane);
    if (lane == 31) s_warp[w] = v;
    __syncthreads();
    const uint32_t ws = warp_scan(lane < kSelectWarps ? s_warp[lane] : 0u, lane);
    const uint32_t before = __shfl_sync(full, ws, (w + 31) & 31);
    uint32_t above = v - sum + (w > 0 ? before : 0u);  // rows above this thread's bins
    if (above < need && above + sum >= need) {
      const uint32_t cs[4] = {c.w, c.z, c.y, c.x};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (above < need && above + cs[i] >= need) {
          s_found[0] = static_cast<uint32_t>(bin + 3 - i);
          s_found[1] = above;
          s_found[2] = cs[i];
        }
        above += cs[i];
      }
    }
    __syncthreads();
    prefix = (prefix << bits) | s_found[0];
    need -= s_found[1];
    at_t = s_found[2];
    if (at_t == need) break;  // all that match stay, whatever their lower digits (the same in every CTA)
  }

  // prefix is the key T, or the leading bits of the keys at it that all stay
  // (mostly: then they count as above T); else the `need` lowest rows at T stay.
  // What the cluster's earlier CTAs hold comes first.
  const bool ties = at_t != need;
  auto is_more = [&](int span, int j) {
    return valid(span, j) && (ties ? key[j] > prefix : (key[j] >> shift) >= prefix);
  };
  auto is_same = [&](int span, int j) { return valid(span, j) && key[j] == prefix; };
  uint32_t before_more = 0, before_same = 0;
  if (C > 1) {
    uint32_t more = 0, same = 0;
    for (int span = 0; span < spans; ++span) {
      if (spans > 1) load(span);
#pragma unroll
      for (int j = 0; j < kKeys; ++j) {
        if (span * kSpan + j * kSelectThreads >= cnt) break;
        more += __popc(__ballot_sync(full, is_more(span, j)));
        if (ties) same += __popc(__ballot_sync(full, is_same(span, j)));
      }
    }
    if (lane == 0) {
      atomicAdd(&s_total[0], more);
      atomicAdd(&s_total[1], same);
    }
    cluster.sync();
#pragma unroll
    for (int r = 0; r < kMaxCluster - 1; ++r) {
      if (r < cr) {
        before_more += *cluster.map_shared_rank(&s_total[0], r);
        before_same += *cluster.map_shared_rank(&s_total[1], r);
      }
    }
  }
  const uint32_t below = (1u << lane) - 1u;
  for (int span = 0; span < spans; ++span) {
    if (spans > 1) {
      load(span);
      __syncthreads();  // the last span's counts have been read
    }
#pragma unroll
    for (int j = 0; j < kKeys; ++j) {
      uint32_t x = 0;
      if (span * kSpan + j * kSelectThreads < cnt) {
        x = __popc(__ballot_sync(full, is_more(span, j)));
        if (ties) x |= __popc(__ballot_sync(full, is_same(span, j))) << 16;
      }
      if (lane == 0) s_cnt[j][w] = x;
    }
    __syncthreads();
    {  // prefix sums of both halves at once: a span has fewer than 2^16 keys
      static_assert(kKeys == kSelectWarps, "one warp per row of counts");
      const uint32_t x = lane < kSelectWarps ? s_cnt[w][lane] : 0u, v = warp_scan(x, lane);
      if (lane < kSelectWarps) s_cnt[w][lane] = v - x;
      if (lane == 31) s_row[w] = v;
    }
    __syncthreads();
#pragma unroll
    for (int j = 0; j < kKeys; ++j) {
      if (span * kSpan + j * kSelectThreads >= cnt) break;
      const uint32_t x = s_cnt[j][w], total = s_row[j];
      const int row = lo + span * kSpan + j * kSelectThreads + tid;
      const bool m1 = is_more(span, j);
      const uint32_t more = before_more + (x & 0xffffu) + __popc(__ballot_sync(full, m1) & below);
      if (!ties) {
        if (m1) kept[more] = row;
      } else {
        const bool s1 = is_same(span, j);
        const uint32_t same = before_same + (x >> 16) + __popc(__ballot_sync(full, s1) & below);
        if (m1 || (s1 && same < need)) kept[more + min(same, need)] = row;
      }
      before_more += total & 0xffffu;
      before_same += total >> 16;
    }
  }
  if (C > 1) cluster.sync();  // no CTA ends while another reads its totals
}

// ---------------------------------------------------------------------- move

constexpr int kMoveWarps = 8;
constexpr int kMoveUnroll = 4;

// Physical row (block * n_heads + head) * block_size + row % block_size, -1
// for a block outside the pool (flagged).
__device__ __forceinline__ int64_t pool_row(const EvictParams& p, const int32_t* table, int row, int h) {
  const int blk = row / p.block_size;
  const int phys = __ldg(table + blk);
  if (phys < 0 || phys >= p.num_blocks) {
    set_flag(p.err, KVC_FLAG_BAD_BLOCK);
    return -1;
  }
  return (static_cast<int64_t>(phys) * p.n_heads + h) * p.block_size + (row - blk * p.block_size);
}

// Q8 0: rows of row_chunks 16-byte chunks are copied, 32 rows per warp. Q8 1
// (e4m3), 2 (int8): a warp fills one block of the new table; its scale is the
// largest of its rows' old scales, and rows from blocks with a smaller scale
// are rounded again.
// POW2: row_chunks is a power of two.
template <int Q8, bool POW2>
__global__ void __launch_bounds__(32 * kMoveWarps) move_kernel(const EvictParams p) {
  constexpr uint32_t full = 0xffffffffu;
  asm volatile("griddepcontrol.wait;" ::: "memory");  // launched while select runs
  const int lane = threadIdx.x & 31;
  const int group = Q8 == 0 ? 32 : p.block_size;  // rows per warp
  const int groups = (p.budget + group - 1) / group;
  const uint32_t wi = blockIdx.x * kMoveWarps + (threadIdx.x >> 5);  // below 2^31: checked on the host
  const uint32_t unit32 = wi / groups;
  const int64_t unit = unit32;
  const int b = static_cast<int>(unit32 / p.n_heads), h = static_cast<int>(unit32 % p.n_heads);
  if (b >= p.batch) return;
  const int j0 = static_cast<int>(wi % groups) * group;
  const int m = min(rows_of(p, b), p.budget);
  const int j1 = min(m, j0 + group);
  if (j0 >= j1) return;
  const int32_t* kept = p.kept + unit * p.budget;
  const int32_t* table = p.tables + static_cast<int64_t>(b) * p.max_blocks;
  const int32_t* new_table = p.new_tables + static_cast<int64_t>(b) * p.new_max_blocks;
  float to[2] = {0.f, 0.f};  // the new block's scales
  if constexpr (Q8 != 0) {
    for (int j = j0 + lane; j < j1; j += 32) {
      const int blk = kept[j] / p.block_size;
      const int phys = __ldg(table + blk);
      if (phys >= 0 && phys < p.num_blocks) {
        const int64_t at = static_cast<int64_t>(phys) * p.n_heads + h;
        to[0] = fmaxf(to[0], p.scale[0][at]);
        to[1] = fmaxf(to[1], p.scale[1][at]);
      }
    }
    to[0] = warp_max(to[0]);
    to[1] = warp_max(to[1]);
  }
  for (int jb = j0; jb < j1; jb += 32) {
    const int j = jb + lane;
    int64_t src = -1, dst = -1;
    float f[2] = {1.f, 1.f};
    if (j < j1) {
      const int row = kept[j];
      p.new_scores[unit * p.new_rows + j] = __ldg(p.scores + unit * p.rows + row);
      src = pool_row(p, table, row, h);
      dst = pool_row(p, new_table, j, h);
      if constexpr (Q8 != 0) {
        if (src >= 0) {
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const float s = p.scale[i][src / p.block_size];
            f[i] = to[i] > 0.f ? __fdiv_rn(s, to[i]) : 0.f;
          }
        }
        if (j == j0 && dst >= 0) {
          p.scale[0][dst / p.block_size] = to[0];
          p.scale[1][dst / p.block_size] = to[1];
        }
      }
    }
    const int chunks = min(32, j1 - jb) * p.row_chunks;
    for (int c0 = lane; c0 - lane < chunks; c0 += 32 * kMoveUnroll) {
      uint4 u[2][kMoveUnroll];
      int64_t d[kMoveUnroll];
      float fr[2][kMoveUnroll];
#pragma unroll
      for (int i = 0; i < kMoveUnroll; ++i) {
        const int c = c0 + 32 * i;
        const int r = POW2 ? min(c >> p.row_shift, 31) : min(c / p.row_chunks, 31);
        const int part = POW2 ? c & (p.row_chunks - 1) : c - r * p.row_chunks;
        const int64_t s = __shfl_sync(full, src, r);
        d[i] = __shfl_sync(full, dst, r);
        if constexpr (Q8 != 0) {
          fr[0][i] = __shfl_sync(full, f[0], r);
          fr[1][i] = __shfl_sync(full, f[1], r);
        }
        if (c >= chunks || s < 0) d[i] = -1;
        if (d[i] >= 0) {
          d[i] = (POW2 ? d[i] << p.row_shift : d[i] * p.row_chunks) + part;
          const int64_t from = (POW2 ? s << p.row_shift : s * p.row_chunks) + part;
          u[0][i] = __ldcs(reinterpret_cast<const uint4*>(p.pool[0]) + from);
          u[1][i] = __ldcs(reinterpret_cast<const uint4*>(p.pool[1]) + from);
        }
      }
#pragma unroll
      for (int i = 0; i < kMoveUnroll; ++i) {
        if (d[i] < 0) continue;
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          uint4 x = u[t][i];
          if constexpr (Q8 != 0) {
            if (fr[t][i] != 1.f) x = rescale16<Q8 == 2>(x, fr[t][i]);
          }
          reinterpret_cast<uint4*>(p.pool[t])[d[i]] = x;
        }
      }
    }
  }
}

// ---------------------------------------------------------------------- host

// row_bytes: bytes of a cached row; code -1: 16- or 32-bit elements, moved as they are.
kvc_status evict(const float* scores, void* k_cache, void* v_cache, float* k_scale, float* v_scale, int code,
                 const int32_t* tables, int max_blocks, const int32_t* lens, int batch, int budget, int recent,
                 const int32_t* new_tables, int new_max_blocks, int64_t num_blocks, int block_size, int n_heads,
                 int64_t row_bytes, int32_t* kept, int32_t* new_lens, float* new_scores, cudaStream_t stream) {
  if (batch < 1 || n_heads < 1 || block_size < 1 || num_blocks < 1 || max_blocks < 1 || new_max_blocks < 1 ||
      row_bytes < 1)
    return fail(KVC_ERR_INVALID_ARG, "batch, heads, head_dim, block_size and block counts must be >= 1");
  if (budget < 1 || recent < 0 || recent > budget)
    return fail(KVC_ERR_INVALID_ARG, "budget must be >= 1 and recent within 0 .. budget (got %d, %d)", budget, recent);
  const int64_t rows = static_cast<int64_t>(max_blocks) * block_size;
  const int64_t new_rows = static_cast<int64_t>(new_max_blocks) * block_size;
  if (budget > new_rows)
    return fail(KVC_ERR_INVALID_ARG, "budget %d does not fit the new tables' %lld rows", budget,
                static_cast<long long>(new_rows));
  if (row_bytes % 16 != 0)
    return fail(KVC_ERR_UNSUPPORTED, "head_dim x element size must be a multiple of 16 bytes");
  if (row_bytes > (1 << 20)) return fail(KVC_ERR_UNSUPPORTED, "head_dim x element size above 1 MB");
  if (rows > (1ll << 30) || new_rows > (1ll << 30))
    return fail(KVC_ERR_UNSUPPORTED, "max_blocks_per_seq x block_size too large");
  const int64_t units = static_cast<int64_t>(batch) * n_heads;
  const int group = code < 0 ? 32 : block_size;
  const int64_t warps = units * ((budget + group - 1) / group);
  if (units * 8 >= (1ll << 31) || warps >= (1ll << 31) - kMoveWarps)
    return fail(KVC_ERR_UNSUPPORTED, "batch x heads x budget too large");
  if (scores == nullptr || k_cache == nullptr || v_cache == nullptr || tables == nullptr || lens == nullptr ||
      new_tables == nullptr || kept == nullptr || new_lens == nullptr || new_scores == nullptr)
    return fail(KVC_ERR_INVALID_ARG, "NULL pointer");
  if (code >= 0 && (k_scale == nullptr || v_scale == nullptr))
    return fail(KVC_ERR_INVALID_ARG, "k_scale / v_scale is NULL");
  if (!aligned16(k_cache) || !aligned16(v_cache))
    return fail(KVC_ERR_INVALID_ARG, "the caches must be 16-byte aligned");
  if (new_scores == scores || new_lens == lens || new_tables == tables)
    return fail(KVC_ERR_INVALID_ARG, "new_scores, new_lens and new_tables must not be the old ones");
  DeviceInfo* dev = nullptr;
  kvc_status st = current_device(&dev);
  if (st != KVC_OK) return st;
  EvictParams p{};
  p.scores = scores;
  p.tables = tables;
  p.lens = lens;
  p.new_tables = new_tables;
  p.kept = kept;
  p.new_lens = new_lens;
  p.new_scores = new_scores;
  p.pool[0] = static_cast<unsigned char*>(k_cache);
  p.pool[1] = static_cast<unsigned char*>(v_cache);
  p.scale[0] = k_scale;
  p.scale[1] = v_scale;
  p.num_blocks = num_blocks;
  p.batch = batch;
  p.n_heads = n_heads;
  p.block_size = block_size;
  p.max_blocks = max_blocks;
  p.new_max_blocks = new_max_blocks;
  p.rows = static_cast<int>(rows);
  p.new_rows = static_cast<int>(new_rows);
  p.budget = budget;
  p.recent = recent;
  p.row_chunks = static_cast<int>(row_bytes / 16);
  while ((1 << p.row_shift) < p.row_chunks) ++p.row_shift;
  p.err = dev->error_word;

  // CTAs per row of scores: as many as the table's rows fill with 4096 each, up to 8, while the GPU has SMs for them
  int C = 1;
  while (C < kMaxCluster && C * 4096LL < rows && units * C * 2 <= dev->num_sms) C *= 2;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = C;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(units * C));
  cfg.blockDim = dim3(kSelectThreads);
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cudaError_t e = cudaLaunchKernelEx(&cfg, select_kernel, p);
  if (e != cudaSuccess) return cuda_fail(e, "cudaLaunchKernelEx(evict select)");
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.gridDim = dim3(static_cast<unsigned>((warps + kMoveWarps - 1) / kMoveWarps));
  cfg.blockDim = dim3(32 * kMoveWarps);
  const bool pow2 = (1 << p.row_shift) == p.row_chunks;
  auto* move = code < 0              ? (pow2 ? move_kernel<0, true> : move_kernel<0, false>)
               : code == KVC_E4M3 ? (pow2 ? move_kernel<1, true> : move_kernel<1, false>)
                                  : (pow2 ? move_kernel<2, true> : move_kernel<2, false>);
  e = cudaLaunchKernelEx(&cfg, move, p);
  if (e != cudaSuccess) return cuda_fail(e, "cudaLaunchKernelEx(evict move)");
  return finish_call(stream);
}

}  // namespace
}  // namespace kvc

extern "C" {

kvc_status kvc_evict_rows(const float* scores, void* k_cache, void* v_cache, const int32_t* block_tables,
                          int max_blocks_per_seq, const int32_t* context_lens, int batch, int budget, int recent,
                          const int32_t* new_block_tables, int new_max_blocks_per_seq, int64_t num_blocks,
                          int block_size, int n_kv_heads, int head_dim, kvc_dtype dtype, int32_t* kept,
                          int32_t* new_lens, float* new_scores, kvc_stream stream) {
  using namespace kvc;
  clear_error();
  if (!dtype_ok(dtype)) return fail(KVC_ERR_INVALID_ARG, "unknown dtype %d", static_cast<int>(dtype));
  return evict(scores, k_cache, v_cache, nullptr, nullptr, -1, block_tables, max_blocks_per_seq, context_lens, batch,
               budget, recent, new_block_tables, new_max_blocks_per_seq, num_blocks, block_size, n_kv_heads,
               static_cast<int64_t>(head_dim) * static_cast<int64_t>(dtype_size(dtype)), kept, new_lens, new_scores,
               static_cast<cudaStream_t>(stream));
}

kvc_status kvc_evict_rows_block8(const float* scores, void* k_cache, void* v_cache, float* k_scale, float* v_scale,
                                 kvc_code code, const int32_t* block_tables, int max_blocks_per_seq,
                                 const int32_t* context_lens, int batch, int budget, int recent,
                                 const int32_t* new_block_tables, int new_max_blocks_per_seq, int64_t num_blocks,
                                 int block_size, int n_kv_heads, int head_dim, int32_t* kept, int32_t* new_lens,
                                 float* new_scores, kvc_stream stream) {
  using namespace kvc;
  clear_error();
  if (code != KVC_E4M3 && code != KVC_INT8)
    return fail(KVC_ERR_INVALID_ARG, "unknown code format %d", static_cast<int>(code));
  return evict(scores, k_cache, v_cache, k_scale, v_scale, code, block_tables, max_blocks_per_seq, context_lens, batch,
               budget, recent, new_block_tables, new_max_blocks_per_seq, num_blocks, block_size, n_kv_heads, head_dim,
               kept, new_lens, new_scores, static_cast<cudaStream_t>(stream));
}

}  // extern "C"
