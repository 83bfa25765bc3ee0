// Prompt attention over a paged 16-bit cache (kvc_prompt_attention): a ragged
// batch of new tokens, each attending its sequence's cached rows up to its own,
// optionally only a window of them and the sequence's first rows.
//
// Mathematics. The token at position pos sees row r if r <= pos and (r > pos -
// window or r < sinks): o = sum_r p_r v_r / sum_r p_r, p_r = 2^(x_r - m), x_r =
// scale * log2(e) * q . k_r, in one pass over the rows with a running
// reference m and sum. The reference lies kBelow under the largest score when
// it moves, and moves only when a score exceeds it by kAbove: exact in exact
// arithmetic for any m, and O is rarely rescaled.
//
// What bounds it: the tensor core, and the units' ends. 128 x 128 x 128 takes it 512
// cycles, so a KV tile of both halves 2048; measured are about 2600, 1.44 us: the softmax of
// one half, from S to the first part of P, takes longer than the other half's
// products (its exponentials alone are 512 cycles, 8 per cycle and scheduler). A unit
// takes 6 us besides: its queries' copy, the first tile's second run, the outputs of both
// halves with nothing for the tensor core. (Fitted to 32 query, 8 kv heads, D 128, bf16:
// 8192 tokens 359 us, 1.53 PFLOP/s; 16384 tokens 1335 us, 1.65.)
//
// A work unit is 2 x 128 query rows of one kv head: the `group` query heads of
// each token are rows of their own (row = token * group + head), so that a kv
// head's rows are read once for its whole group and a tile's causal edge spans few
// tokens. Both products run on tcgen05.mma, 128 x 128 x D each:
//   S = Q K^T       Q and K from shared memory, S in TMEM
//   O += P V        P from TMEM (where S was, 16 bits), V read MN-major
// The two halves of a unit take turns: while one's softmax runs on its eight
// warps (two threads per row, no shuffles), the tensor core has the other's
// products. One warp copies pages by TMA (boxes of gcd(block_size, 128) rows) into
// a ring of K and V tiles and hands out the units, one thread of another issues the
// products. (Two threads per row with 32 scores at a time in registers: 1.46
// PFLOP/s, one thread with all 128, which spills, 1.08. P is handed over in two
// parts, so that its second half overlaps the first one's product.)
//
// P in 16 bits: its rounding (2^-8 of a weight in bf16, 2^-11 in f16) is of the
// size of the output's own, and a second product for the rest would cost half
// as much again. f16 weights use f16's whole range (see PromptMargin).
//
// Work split. Calls with no more units than SMs, none of them long, have no plan: each
// CTA finds its unit (a few short turns 18 -> 13.5 us). Else a planning kernel lists
// the units' tiles (sequence, token range), sorted by cost, and they are dealt out in
// turn, the largest first. Where that leaves the longest CTA more than kSplitGain KV
// tiles behind the mean, the KV tiles of all units are laid end to end instead and cut
// into equal ranges, one per CTA; the parts of a unit leave records that a merge
// kernel joins (120 units of 70 to 235 KV tiles: 175 us, 16 of them the merge). The plan
// adds up what each CTA would get: with 160 units of 236 tiles, the longest has 471 and
// the mean is 253 (1280 tokens over 30,000 rows: 689 us whole, 430 split).
//
// Rows that nobody in a unit sees are neither looked up nor read (TMA fills
// zeros), those beside visible ones are cleared in shared memory.
//
// Infinities and NaN in V: 0 x infinity is NaN, so they reach every row of a unit
// through the second product, and a weight that is 0 loses them. A unit (or part of
// one) with an output that is not finite is done again when the CTA's others are done: on the
// way, what is not finite in its V tiles is replaced by 0 and written down, dim by dim, for
// the rows that all tokens of the unit see together and row by row for the others;
// each output then is the finite sum, or what its token sees of those. (One infinity in the
// first of 2048 rows: 146 us against 46.) The code for it is apart: in the loops that every call
// runs, it cost 3 to 8 % through the registers alone.
//
// Sources: the chunk mask of "单请求 KV Cache" (query row i of a chunk sees
// columns up to past_len + i) and the block table of "KV Cache（键值缓存）" section
// 2.3; Window Attention of "KV-Cache——为什么AI回复越来越快" section 08.
#include <cuda.h>

#include <algorithm>
#include <atomic>
#include <cmath>
#include <mutex>
#include <numeric>

#include "kvc_internal.h"
#include "packed.cuh"
#include "umma.cuh"
#include "umma_wide.cuh"

namespace kvc {

namespace {

using namespace umma;

constexpr int kPromptMaxBatch = 4096;
constexpr int kM = 128;            // query rows of a half (M of the products)
constexpr int kRows = 128;         // cached rows of a tile
constexpr int kSoftWarps = 16;      // softmax warps: [half][column group][TMEM quarter]
constexpr int kCols = kRows / 2;    // columns of S that a softmax thread has
constexpr int kPromptThreads = (kSoftWarps + 4) * 32;  // one warpgroup more: copies, products, two idle warps
constexpr int kMinTiles = 4;       // KV tiles of a range at least, where units are split
// Units are split where that makes the longest CTA's work shorter by more than
// these KV tiles: what the records and their merge cost (about 15 us).
constexpr int kSplitGain = 10;
constexpr float kLowest = -3.40282347e38f;  // where a reference begins: no score that is a number lies below
constexpr int kBadRing = 8;        // tiles whose bad blocks are remembered: more than the ring holds

struct PromptShape {
  int batch;
  int64_t num_tokens;
  int n_q_heads, n_kv_heads, D, block_size, max_blocks;
  int group() const { return n_q_heads / n_kv_heads; }
  int tokens() const { return kM / group(); }  // of a half
  int64_t tiles() const { return num_tokens / (2 * tokens()) + batch; }  // at most
};

// A token range of one sequence: at most 2 * tokens() new tokens.
struct Tile {
  int first, pos;            // its first row of q and that token's position
  unsigned short seq, count;
  int cost;                  // KV tiles that it sees (in a Part: its place among PromptParams::odd)
};

// How units are handed out: one per CTA without a plan; planned, whole; planned,
// split where that pays.
enum { kPlanNone = 0, kPlanWhole = 1, kPlanSplit = 2 };

struct PromptParams {
  const void* q;  // [num_tokens, n_q_heads, D]
  void* out;
  const int32_t* block_tables;
  const int32_t* query_starts;  // [batch + 1]
  const int32_t* context_lens;
  // workspace
  int* head;     // number of tiles, their total cost, whether units are split
  Tile* tiles;
  int* before;   // KV tiles of the tiles before each (where units are split)
  float* rec_o;  // [2 * CTAs, 2 * kM, D] unnormalised partial outputs
  float* rec_ml; // [2 * CTAs, 2 * kM, 2] (reference, sum of weights)
  struct OddUnit* odd;  // [units, then records] those to be done again: lists, one per CTA
  unsigned int* err;
  int64_t num_blocks;
  int n_kv_heads, block_size, window, sinks;
  int batch, num_tokens, n_q_heads, group, max_blocks, rows, tokens, max_tiles;
  int mode, grid;  // mode: kPlan*
  int box, box_log2;  // rows of a TMA box: gcd(block_size, 128)
  int pool_rows;  // rows of the pool: one past the last, TMA fills zeros
  float qscale;   // |scale| * log2(e), not 0
  int negative;   // scale < 0
};

// Where a query's reference m (log2 units) lies: kBelow under the largest score
// when it moves, and it moves when a score exceeds it by kAbove. f16 ends at
// 2^-24, and rows beside an attention sink have weights of that size: its
// largest weights are 2^7 to 2^15, so that weights down to 2^-21 of the largest
// keep their 11 bits. (Room for 8 binary places before O is rescaled: with 4, 432 us
// for 8192 tokens against 382.)
template <bool BF>
struct PromptMargin {
  static constexpr float kBelow = BF ? 0.f : 7.f;
  static constexpr float kAbove = BF ? 8.f : 15.f;
};

// ------------------------------------------------------------------- plan

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

// The KV tiles that tokens at positions [pos, pos + count) see: `front` ones of
// the sinks, then those from `start` on; tile i of them is i < front ? i : i -
// front + start.
struct Seen {
  int front, start, total;
};
__host__ __device__ __forceinline__ Seen seen_tiles(int pos, int count, int window, int sinks) {
  const int low = pos >= window ? pos - window + 1 : 0;  // first row of the first token's window
  Seen s;
  s.start = low / kRows;
  const int need = sinks < low ? sinks : low;  // sinks before the window
  s.front = (need + kRows - 1) / kRows;
  if (s.front > s.start) s.front = s.start;
  s.total = s.front + (pos + count - 1) / kRows - s.start + 1;
  return s;
}

constexpr int kPlanThreads = 1024;
constexpr int kBuckets = 1024;
constexpr int kSplitTiles = kPromptMaxBatch + 1024;  // of calls whose units may be split, at most

// Exclusive prefix sum over the CTA; *total: the sum. Two barriers.
__device__ __forceinline__ int block_scan(int v, int* s_warp, int* total) {
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  int x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  if (lane == 31) s_warp[w] = x;
  __syncthreads();
  int before = 0, sum = 0;
  for (int i = 0; i < kPlanThreads / 32; ++i) {
    const int y = s_warp[i];
    if (i < w) before += y;
    sum += y;
  }
  *total = sum;
  __syncthreads();
  return before + x - v;
}

__global__ void __launch_bounds__(kPlanThreads, 1) prompt_plan_kernel(const PromptParams p, int elem_bytes, int D) {
  __shared__ int s_first[kPromptMaxBatch + 1];  // tiles of the sequences before
  __shared__ int s_warp[kPlanThreads / 32], s_hist[kBuckets], s_load[kBuckets], s_cost[kSplitTiles];
  const int tid = threadIdx.x, B = p.batch, per_tile = 2 * p.tokens;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int per = (B + kPlanThreads - 1) / kPlanThreads;
  const int b0 = min(B, tid * per), b1 = min(B, b0 + per);
  int local = 0, most = 0;
  bool invalid = false;
  for (int b = b0; b < b1; ++b) {
    const Span s = span_of(p, b, true);
    if (s.count > 0 && s.rows == 0) {
      invalid = true;
      continue;
    }
    local += (s.count + per_tile - 1) / per_tile;
    if (s.count > 0) most = max(most, seen_tiles(s.rows - 1, 1, p.window, p.sinks).total + 1);
  }
  int n = 0;
  int run = block_scan(local, s_warp, &n);
  for (int b = b0; b < b1; ++b) {
    s_first[b] = run;
    const Span s = span_of(p, b, false);
    if (s.count > 0 && s.rows > 0) run += (s.count + per_tile - 1) / per_tile;
  }
  // (the prefix sums are read behind the next barrier)
  if (__syncthreads_or(invalid)) {
    for (int b = 0; b < B; ++b) {
      const Span s = span_of(p, b, false);
      if (s.count == 0 || s.rows > 0) continue;
      const int64_t row_words = static_cast<int64_t>(p.n_q_heads) * D * elem_bytes / 16;
      uint4* to = static_cast<uint4*>(p.out) + s.first * row_words;
      for (int64_t i = tid; i < s.count * row_words; i += kPlanThreads) to[i] = make_uint4(0u, 0u, 0u, 0u);
    }
  }
  if (n > p.max_tiles) {  // starts that overlap
    if (tid == 0) set_flag(p.err, KVC_FLAG_BAD_LEN);
    n = p.max_tiles;
  }
  auto tile_of = [&](int i) {
    int a = 0, b = B - 1;  // the last sequence whose first tile is <= i
    while (a < b) {
      const int mid = (a + b + 1) >> 1;
      if (s_first[mid] <= i) a = mid; else b = mid - 1;
    }
    const Span s = span_of(p, a, false);
    Tile t;
    const int t0 = (i - s_first[a]) * per_tile;
    t.seq = static_cast<unsigned short>(a);
    t.first = s.first + t0;
    t.count = static_cast<unsigned short>(min(per_tile, s.count - t0));
    t.pos = s.rows - s.count + t0;
    t.cost = seen_tiles(t.pos, t.count, p.window, p.sinks).total;
    return t;
  };
  most = max(__reduce_max_sync(0xffffffffu, most), 1);
  if ((tid & 31) == 0) s_warp[tid >> 5] = most;
  s_hist[tid] = s_load[tid] = 0;
  __syncthreads();
  for (int i = 0; i < kPlanThreads / 32; ++i) most = max(most, s_warp[i]);
  __syncthreads();
  int total = 0;
  bool split = false;
  Tile mine{};  // (of most calls all that there are: found once)
  if (tid < n) mine = tile_of(tid);
  auto tile = [&](int i) { return i == tid ? mine : tile_of(i); };
  // sorted by cost, in up to 1024 classes
  int shift = 0;
  while ((most >> shift) >= kBuckets) ++shift;
  auto bucket = [&](int cost) { return min(kBuckets - 1, max(0, (most >> shift) - (cost >> shift))); };
  for (int i0 = 0; i0 < n; i0 += kPlanThreads) {
    const int cost = i0 + tid < n ? tile(i0 + tid).cost : 0;
    if (i0 + tid < n) atomicAdd(&s_hist[bucket(cost)], 1);
    if (p.mode == kPlanSplit) {  // few tiles: their prefix sums
      int sum = 0;
      const int before = block_scan(cost, s_warp, &sum);
      if (i0 + tid < n) p.before[i0 + tid] = total + before;
      total += sum;
    }
  }
  // Does splitting pay? What the longest CTA has of whole units against the mean
  const int units = n * p.n_kv_heads, mean = total * p.n_kv_heads / p.grid;
  const bool one_each = units <= p.grid;
  if (p.mode == kPlanSplit && one_each) split = most - mean > kSplitGain;
  if (!split) {
    __syncthreads();
    int sum = 0;
    s_hist[tid] = block_scan(s_hist[tid], s_warp, &sum);
    __syncthreads();
    for (int i = tid; i < n; i += kPlanThreads) {
      const Tile t = tile(i);
      const int at = atomicAdd(&s_hist[bucket(t.cost)], 1);  // the order among equals is free
      p.tiles[at] = t;
      if (p.mode == kPlanSplit) s_cost[at] = t.cost >> shift << shift;  // (so that it is here, too)
    }
    if (p.mode == kPlanSplit && !one_each) {
      __syncthreads();
      for (int j = tid; j < units; j += kPlanThreads) {
        const int r = j / p.grid, c = j - r * p.grid;  // as Walk::unit deals them out
        atomicAdd(&s_load[(r & 1) ? p.grid - 1 - c : c], s_cost[j / p.n_kv_heads]);
      }
      __syncthreads();
      int longest = 0;
      for (int c = tid & 31; c < p.grid; c += 32) longest = max(longest, s_load[c]);
      split = __reduce_max_sync(0xffffffffu, longest) - mean > kSplitGain;
    }
  }
  if (split) {  // in order
    __syncthreads();
    for (int i = tid; i < n; i += kPlanThreads) p.tiles[i] = tile(i);
  }
  if (tid == 0) {
    p.head[0] = n;
    p.head[1] = total;
    p.head[2] = split ? 1 : 0;
  }
}
static_assert(kBuckets == kPlanThreads, "one class per thread, and one counter per CTA");

// The equal ranges of split units: range x is [start(x), start(x + 1)) of N positions.
struct Ranges {
  int N, W;  // N < 2^31: checked on the host
  __device__ __forceinline__ Ranges(int n_tiles, int total, int heads, int grid) {
    N = total * heads;
    W = min(grid, max(n_tiles * heads, N / kMinTiles + 1));
    W = min(W, N);
  }
  __device__ __forceinline__ int start(int x) const { return static_cast<int>(static_cast<int64_t>(x) * N / W); }
  __device__ __forceinline__ int holder(int pos) const {
    return static_cast<int>((static_cast<int64_t>(pos + 1) * W - 1) / N);
  }
};

// A unit (tile, kv head) or the part of it in this CTA's range: KV tiles [i0, i1).
struct Part {
  Tile t;
  int kvh, i0, i1;
  int rec;  // -1: the whole unit
};
// One with an output that was not finite, and the place of the CTA's next one, -1: none.
struct OddUnit {
  Part u;
  int next;
  int pad[3];
};
static_assert(sizeof(Tile) == 16 && sizeof(Part) == 32 && sizeof(OddUnit) == 48, "copied as 16-byte words");

struct OddList {
  int at;
  __device__ __forceinline__ bool next(const PromptParams& p, Part& u) {
    if (at < 0) return false;
    const OddUnit e = p.odd[at];  // (written by this CTA)
    u = e.u;
    at = e.next;
    return true;
  }
};

// The CTA's units. One warp walks (all lanes with the same values) and tells the others.
struct Walk {
  int n, at, hi, lo;  // whole units: `at` the next round; split ones: the next position of [lo, hi)
  int i, kvh, split;  // split ones: the next unit
  Tile ahead;         // of the next unit: loaded while this one is worked on
  __device__ __forceinline__ static Tile load(const PromptParams& p, int i) {
    union {
      int4 v;
      Tile t;
    } u;
    u.v = __ldcg(reinterpret_cast<const int4*>(p.tiles + i));  // (L2: the plan may have run beside this kernel's start)
    return u.t;
  }
  // Unit of round r, dealt out there and back, so that nobody always gets the larger one.
  __device__ __forceinline__ static int unit(const PromptParams& p, int r) {
    const int c = static_cast<int>(blockIdx.x);
    return r * p.grid + ((r & 1) ? p.grid - 1 - c : c);
  }
  __device__ __forceinline__ Walk(const PromptParams& p) {
    at = lo = hi = i = kvh = split = 0;
    const int H = p.n_kv_heads, lane = threadIdx.x & 31;
    if (p.mode == kPlanNone) {
      // the CTA's only unit: tiles of the sequences added up, 32 sequences at a time
      n = 0;
      const int want = static_cast<int>(blockIdx.x) / H, per = 2 * p.tokens;
      for (int b0 = 0; b0 < p.batch; b0 += 32) {
        Span s{0, 0, 0};
        if (b0 + lane < p.batch) s = span_of(p, b0 + lane, false);
        const int mine = s.rows > 0 ? (s.count + per - 1) / per : 0;
        int x = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int y = __shfl_up_sync(0xffffffffu, x, o);
          if (lane >= o) x += y;
        }
        const uint32_t has = __ballot_sync(0xffffffffu, n + x > want);
        if (has != 0) {
          const int src = __ffs(has) - 1;
          const int t0 = (want - n - __shfl_sync(0xffffffffu, x - mine, src)) * per;
          const int first = __shfl_sync(0xffffffffu, s.first, src), count = __shfl_sync(0xffffffffu, s.count, src);
          const int rows = __shfl_sync(0xffffffffu, s.rows, src);
          ahead.seq = static_cast<unsigned short>(b0 + src);
          ahead.first = first + t0;
          ahead.count = static_cast<unsigned short>(min(per, count - t0));
          ahead.pos = rows - count + t0;
          ahead.cost = seen_tiles(ahead.pos, ahead.count, p.window, p.sinks).total;
          n = want + 1;
          break;
        }
        n += __shfl_sync(0xffffffffu, x, 31);
      }
      return;
    }
    n = __ldcg(p.head);
    split = __ldcg(p.head + 2);
    if (n == 0) return;
    if (!split) {
      if (unit(p, 0) < n * H) ahead = load(p, unit(p, 0) / H);
      return;
    }
    const Ranges r(n, __ldcg(p.head + 1), H, p.grid);
    if (static_cast<int>(blockIdx.x) >= r.W) return;
    lo = at = r.start(blockIdx.x);
    hi = r.start(blockIdx.x + 1);
    int b = n - 1;  // i: the last tile that begins at or before the position
    while (i < b) {
      const int mid = (i + b + 1) >> 1;
      if (H * __ldcg(p.before + mid) <= at) i = mid; else b = mid - 1;
    }
    ahead = load(p, i);
    kvh = (at - H * __ldcg(p.before + i)) / ahead.cost;
    lo -= H * __ldcg(p.before + i) + kvh * ahead.cost;  // from the first unit's begin on
    hi -= at - lo;
    at = lo;
  }
  __device__ __forceinline__ bool next(const PromptParams& p, Part& u) {
    const int H = p.n_kv_heads;
    if (!split) {
      const int j = unit(p, at);
      if (j >= n * H) return false;
      u = {ahead, j % H, 0, ahead.cost, -1};
      u.t.cost = j;
      ++at;
      const int k = unit(p, at);
      if (p.mode != kPlanNone && k < n * H) ahead = load(p, k / H);
      return true;
    }
    if (at >= hi) return false;
    const bool begins = at == lo;
    u.t = ahead;
    u.kvh = kvh;
    u.i0 = begins ? lo : 0;
    u.i1 = min(u.t.cost, u.i0 + (hi - at));
    u.rec = u.i0 == 0 && u.i1 == u.t.cost ? -1 : 2 * static_cast<int>(blockIdx.x) + (begins ? 0 : 1);
    u.t.cost = u.rec < 0 ? i * H + kvh : p.max_tiles * H + u.rec;
    at += u.i1 - u.i0;
    if (++kvh == H) {
      kvh = 0;
      if (++i < n) ahead = load(p, i);
    }
    return true;
  }
};

// ------------------------------------------------------------ main kernel

template <int D>
struct PromptGeo {
  static constexpr int kHalves = D / 64;                  // 128-byte wide parts of a row
  static constexpr uint32_t kPart = kRows * 128;          // one part of a tile
  static constexpr uint32_t kTile = kHalves * kPart;      // a K or V tile, or a half's queries
  // Queries lie part by part; K and V tiles in groups of 8 rows, [group][part][8
  // rows][128 bytes], so that one copy brings all parts of a page: of 16-row
  // pages a tile needs 8 copies, and issuing twice as many cost 20 % (16384 rows).
  static constexpr uint32_t kRowGroup = kHalves * 1024;
  static constexpr int kSlots = D == 128 ? 4 : 8;         // K and V tiles in the ring (a fifth brings nothing)
  static constexpr uint32_t kOffRing = 2 * kTile;         // behind both halves' queries
  static constexpr uint32_t kOffStage = kOffRing + kSlots * kTile;  // 2 KB per softmax warp: outputs on their way
  static constexpr uint32_t kOffBar = kOffStage + kSoftWarps * 2048;
  enum {
    QFULL = 0, QEMPTY, FULL0, EMPTY0 = FULL0 + kSlots, SFULL0 = EMPTY0 + kSlots, PFULL0 = SFULL0 + 2,
    OFULL0 = PFULL0 + 4, OEMPTY0 = OFULL0 + 2, UFULL0 = OEMPTY0 + 2, UEMPTY0 = UFULL0 + 2, FINAL = UEMPTY0 + 2,
    ODDFULL, COUNT
  };
  // a second set for the units done again: the first one's phases need not be known then
  static constexpr uint32_t kOffMisc = kOffBar + 2 * COUNT * 8;  // TMEM address, abort flag, odd units, bad blocks
  static constexpr uint32_t kOffPart = kOffMisc + 20 + kBadRing * 4;  // what the threads of a row tell each other
  static constexpr uint32_t kOffFail = kOffPart + kSoftWarps * 32 * 4;
  static constexpr uint32_t kOffUnit = (kOffFail + kSoftWarps * 4 + 15) / 16 * 16;  // two units: this and the next
  static constexpr uint32_t kBytes = kOffUnit + 2 * sizeof(Part);
  static_assert(kBytes <= 227 * 1024, "shared memory of a CTA");
  // While a unit is done again, where outputs are staged: an OddDims of each (row of a tile,
  // column group) for the rows that every token sees, then of each (row that some see,
  // column group): at most 255 behind the first token's and 255 that leave the window.
  static constexpr uint32_t kOffOddRows = kOffStage + kRows * 2 * 16;
  static_assert(kOffOddRows + 2 * (2 * kM - 1) * 2 * 16 <= kOffBar, "records of what is not finite");
  // TMEM columns: S (P over it) of both halves, O of both
  static constexpr uint32_t kColO = 256;
  static constexpr uint32_t kTmemCols = 512;
};

__device__ __forceinline__ void tma_load_4d(uint32_t dst, const CUtensorMap* map, int w, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %2, %2, %3}], "
      "[%4];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(0), "r"(w), "r"(bar)
      : "memory");
}

__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap* map, int x, int y, int z, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], "
      "[%5];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(bar)
      : "memory");
}

// D += A . B with A read from TMEM.
__device__ __forceinline__ void mma_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc,
                                       uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}

__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

template <bool BF>
__device__ __forceinline__ uint32_t pack16(float lo, float hi) {
  uint32_t r;
  if constexpr (BF)
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  else
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// True in one thread of the warp. The compiler knows that it is one, which
// `lane == 0` does not tell it: operands of tcgen05.mma need no loop over the
// threads then.
__device__ __forceinline__ bool elect_one() {
  uint32_t one;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(one));
  return one != 0;
}

// The n lowest bits of 64.
__device__ __forceinline__ uint64_t bits_below(int n) { return n <= 0 ? 0ull : n >= 64 ? ~0ull : (1ull << n) - 1; }

// Barrier of the two warps that share query rows; pair_or: the OR of a
// predicate over their 64 threads.
__device__ __forceinline__ void pair_sync(int id) { asm volatile("bar.sync %0, 64;" ::"r"(id) : "memory"); }
__device__ __forceinline__ bool pair_or(int id, bool pred) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.u32 p, %2, 0;\n\t"
      "bar.red.or.pred q, %1, 64, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"(id), "r"(pred ? 1u : 0u)
      : "memory");
  return r != 0;
}

// What is not finite among values of a column group's dims (bits): x, y +infinity, z, w
// -infinity, NaN both.
using OddDims = uint4;

// Replaces what is not finite in 16 bytes of V by 0 and notes it: dim0 the first element's.
template <bool BF>
__device__ __forceinline__ void take_odd(unsigned char* at, int dim0, OddDims& odd) {
  constexpr uint32_t EXP = BF ? 0x7f80u : 0x7c00u;
  uint32_t x[4];
  *reinterpret_cast<uint4*>(x) = *reinterpret_cast<const uint4*>(at);
  uint32_t plus = 0, minus = 0;
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    const uint32_t h = (x[k >> 1] >> (16 * (k & 1))) & 0xffffu;
    if ((h & EXP) != EXP) continue;
    const bool nan = (h & (0x7fffu & ~EXP)) != 0;
    if (nan || h < 0x8000u) plus |= 1u << k;
    if (nan || h >= 0x8000u) minus |= 1u << k;
    x[k >> 1] &= k & 1 ? 0x0000ffffu : 0xffff0000u;
  }
  if ((plus | minus) == 0) return;
  *reinterpret_cast<uint4*>(at) = *reinterpret_cast<const uint4*>(x);
  (dim0 < 32 ? odd.x : odd.y) |= plus << (dim0 & 31);
  (dim0 < 32 ? odd.z : odd.w) |= minus << (dim0 & 31);
}

// x, or what its dim has of infinities and NaN.
__device__ __forceinline__ float odd_or(float x, uint32_t plus, uint32_t minus, int bit) {
  const uint32_t b = 1u << bit;
  if (((plus | minus) & b) == 0) return x;
  const float inf = __builtin_huge_valf();
  return (plus & b) == 0 ? -inf : (minus & b) == 0 ? inf : __int_as_float(0x7fffffff);
}

// The roles of a CTA's warps for all of its units (AGAIN: for those that are to be done
// again). Ends with a CTA barrier.
template <typename CT, int D, bool AGAIN>
__device__ __forceinline__ void prompt_roles(const CUtensorMap& tm_q, const CUtensorMap& tm_k, const CUtensorMap& tm_v,
                                             const PromptParams& p, unsigned char* sm, uint32_t tmem) {
  using G = PromptGeo<D>;
  constexpr bool BF = std::is_same<CT, __nv_bfloat16>::value;
  constexpr uint32_t full = 0xffffffffu;
  const uint32_t base = smem_addr(sm);
  volatile int* s_abort = reinterpret_cast<volatile int*>(sm + G::kOffMisc + 4);
  // the list of odd units' first; whether the units of s_unit are on it
  volatile int* s_odd = reinterpret_cast<volatile int*>(sm + G::kOffMisc + 8);
  volatile uint32_t* s_bad = reinterpret_cast<volatile uint32_t*>(sm + G::kOffMisc + 20);
  auto bar = [&](int i) -> uint32_t {
    return base + G::kOffBar + 8u * static_cast<uint32_t>(i + (AGAIN ? G::COUNT : 0));
  };
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int bs = p.block_size, window = p.window, sinks = p.sinks;
  Part* s_unit = reinterpret_cast<Part*>(sm + G::kOffUnit);

  if (warp == kSoftWarps) {
    // ------------------------------------------------------------ producer
    // Lane i has box i of every tile: its table entry is read before the slot is
    // free. One barrier per K or V tile.
    uint32_t kk = 0, gt = 0, un = 0, nq = 0;  // tiles copied, KV tiles, units told, units' queries copied
    uint32_t issued[G::kSlots] = {};
    const int boxes = kRows / p.box;
    bool ok = true;
    auto walk = [&] {
      if constexpr (AGAIN) return OddList{*s_odd};
      else return Walk(p);
    }();
    for (; ok; ++un) {
      Part u;
      const bool have = walk.next(p, u);
      if (!have) u.t.count = 0;  // the end
      bool got = true;
      // A unit done again has the CTA to itself: its records lie where outputs are staged
      constexpr uint32_t kBefore = AGAIN ? 1 : 2;
      if (lane == 0 && un >= kBefore)
        got = wait_phase(bar(G::UEMPTY0 + ((un - kBefore) & 1)), ((un - kBefore) >> 1) & 1u, s_abort, p.err);
      if (!__shfl_sync(full, got ? 1 : 0, 0)) break;
      if (lane == 0) {
        s_unit[un & 1] = u;
        s_odd[1 + (un & 1)] = 0;
        arrive(bar(G::UFULL0 + (un & 1)));
      }
      __syncwarp();
      if (!have) break;
      const int last = u.t.pos + u.t.count - 1;
      const int low = u.t.pos >= window ? u.t.pos - window + 1 : 0;
      const Seen seen = seen_tiles(u.t.pos, u.t.count, window, sinks);
      const bool two = u.t.count > p.tokens;
      const int32_t* table = p.block_tables + static_cast<int64_t>(u.t.seq) * p.max_blocks;
      // ---- queries
      if (lane == 0 && un > 0) got = wait_phase(bar(G::QEMPTY), (un - 1) & 1u, s_abort, p.err);
      if (!__shfl_sync(full, got ? 1 : 0, 0)) break;
      if (lane == 0) {
        const uint32_t bytes = static_cast<uint32_t>(p.tokens * p.group) * 128u * G::kHalves;
        arrive_expect(bar(G::QFULL), two ? 2 * bytes : bytes);
        for (int h = 0; h < (two ? 2 : 1); ++h)
          for (int x = 0; x < G::kHalves; ++x)
            tma_load_3d(base + h * G::kTile + x * G::kPart, &tm_q, 64 * x, u.kvh * p.group,
                        u.t.first + h * p.tokens, bar(G::QFULL));
      }
      __syncwarp();
      ++nq;
      // ---- rows
      auto wanted = [&](int i) {
        const int kt = i < seen.front ? i : i - seen.front + seen.start;
        const int r0 = kt * kRows + lane * p.box;
        return lane < boxes && r0 <= last && (r0 + p.box > low || r0 < sinks) ? r0 : -1;
      };
      int r0 = wanted(u.i0);
      int phys = r0 >= 0 ? __ldg(table + r0 / bs) : -1;
      for (int i = u.i0; i < u.i1; ++i, ++gt) {
        const bool want = r0 >= 0;
        const bool there = phys >= 0 && phys < p.num_blocks;
        const uint32_t bad = __ballot_sync(full, want && !there);
        const int y = (there ? (phys * p.n_kv_heads + u.kvh) * bs + r0 % bs : p.pool_rows) >> 3;
        if (i + 1 < u.i1) {  // the next tile's entry, while this one waits for its slots
          r0 = wanted(i + 1);
          phys = r0 >= 0 ? __ldg(table + r0 / bs) : -1;
        }
#pragma unroll
        for (int kv = 0; kv < 2; ++kv, ++kk) {
          const uint32_t slot = kk % G::kSlots;
          got = true;
          if (lane == 0 && kk >= G::kSlots)
            got = wait_phase(bar(G::EMPTY0 + slot), (kk / G::kSlots - 1) & 1u, s_abort, p.err);
          if (!__shfl_sync(full, got ? 1 : 0, 0)) {
            ok = false;
            break;
          }
          if (lane == 0) {
            if (kv == 0) {
              s_bad[gt % kBadRing] = bad;
              if (bad != 0) set_flag(p.err, KVC_FLAG_BAD_BLOCK);
            }
            arrive_expect(bar(G::FULL0 + slot), G::kTile);
          }
          __syncwarp();
          if (lane < boxes) {
            const uint32_t dst =
                base + G::kOffRing + slot * G::kTile + static_cast<uint32_t>(lane * p.box) * (G::kRowGroup / 8);
            tma_load_4d(dst, kv == 0 ? &tm_k : &tm_v, y, bar(G::FULL0 + slot));
          }
          ++issued[slot];
        }
        if (!ok) break;
      }
    }
    if (*s_abort && lane == 0) {
      // Copies still in flight must land before this shared memory goes away.
      for (int s = 0; s < G::kSlots; ++s) {
        if (issued[s] == 0) continue;
        const uint64_t t0 = globaltimer_ns();
        while (!try_wait(bar(G::FULL0 + s), (issued[s] - 1) & 1u) && globaltimer_ns() - t0 < kWaitNs) {
        }
      }
      if (nq > 0) {
        const uint64_t t0 = globaltimer_ns();
        while (!try_wait(bar(G::QFULL), (nq - 1) & 1u) && globaltimer_ns() - t0 < kWaitNs) {
        }
      }
    }
  } else if (warp == kSoftWarps + 1) {
    // ---------------------------------------------------------- MMA issuer
    // Order per KV tile j: PV of half 0 (j), S of half 0 (j + 1), PV of half 1
    // (j), S of half 1 (j + 1). P lies where S was: S (j + 1) follows PV (j).
    if (elect_one()) {
      const uint32_t id_s = instr_desc(kM, kRows, 0, 0, BF);
      const uint32_t id_pv = instr_desc(kM, D, 0, 1, BF);
      uint32_t gt = 0, un = 0;        // KV tiles begun, units begun
      uint32_t np[2] = {0, 0}, nu[2] = {0, 0};  // per half: tiles whose P was used, units
      bool ok = true;
      // S of half h with KV tile g (of the CTA's count)
      auto issue_s = [&](int h, uint32_t g) {
        const uint32_t slot = (2 * g) % G::kSlots;
        const uint64_t a = smem_desc(base + h * G::kTile, 16, 1024, 2);
        const uint64_t b = smem_desc(base + G::kOffRing + slot * G::kTile, 16, G::kRowGroup, 2);
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks)
          mma(tmem + h * kRows, a + (((ks >> 2) * G::kPart + (ks & 3) * 32) >> 4),
              b + (((ks >> 2) * 1024 + (ks & 3) * 32) >> 4), id_s, ks == 0 ? 0u : 1u);
        commit(bar(G::SFULL0 + h));
      };
      auto full_slot = [&](uint32_t k) {
        return wait_phase(bar(G::FULL0 + k % G::kSlots), (k / G::kSlots) & 1u, s_abort, p.err);
      };
      for (; ok && !*s_abort; ++un) {
        if (!wait_phase(bar(G::UFULL0 + (un & 1)), (un >> 1) & 1u, s_abort, p.err)) break;
        const Part u = s_unit[un & 1];
        arrive(bar(G::UEMPTY0 + (un & 1)));
        if (u.t.count == 0) break;
        const int halves = u.t.count > p.tokens ? 2 : 1;
        const int J = u.i1 - u.i0;
        if (!wait_phase(bar(G::QFULL), un & 1u, s_abort, p.err)) break;
        if (!full_slot(2 * gt)) break;
        fence_after();
        for (int h = 0; h < halves; ++h) issue_s(h, gt);
        commit(bar(G::EMPTY0 + (2 * gt) % G::kSlots));
        if (J == 1) commit(bar(G::QEMPTY));
        for (int j = 0; j < J && ok; ++j, ++gt) {
          const bool more = j + 1 < J;
          if (!full_slot(2 * gt + 1)) { ok = false; break; }
          const uint32_t vslot = (2 * gt + 1) % G::kSlots;
          const uint64_t v = smem_desc(base + G::kOffRing + vslot * G::kTile, 1024, G::kRowGroup, 2);
          for (int h = 0; h < halves; ++h) {
            if (!wait_phase(bar(G::PFULL0 + 2 * h), np[h] & 1u, s_abort, p.err)) { ok = false; break; }
            // O of the unit before has been read
            if (j == 0 && nu[h] > 0 && !wait_phase(bar(G::OEMPTY0 + h), (nu[h] - 1) & 1u, s_abort, p.err)) {
              ok = false;
              break;
            }
            // P comes in two parts, 32 columns of each column group at a time
#pragma unroll
            for (int part = 0; part < 2; ++part) {
              if (part == 1) {
                if (!wait_phase(bar(G::PFULL0 + 2 * h + 1), np[h] & 1u, s_abort, p.err)) { ok = false; break; }
              }
              fence_after();
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                const int ks = (k >> 1) * 4 + part * 2 + (k & 1);
                mma_ts(tmem + G::kColO + h * D, tmem + h * kRows + ks * 8, v + ((ks * 2 * G::kRowGroup) >> 4), id_pv,
                       j == 0 && part == 0 && k == 0 ? 0u : 1u);
              }
            }
            if (!ok) break;
            ++np[h];
            if (!more) commit(bar(G::OFULL0 + h));
            if (h == halves - 1) commit(bar(G::EMPTY0 + vslot));
            if (more) {
              if (h == 0) {
                if (!full_slot(2 * gt + 2)) { ok = false; break; }
                fence_after();
              }
              issue_s(h, gt + 1);
              if (h == halves - 1) {
                commit(bar(G::EMPTY0 + (2 * gt + 2) % G::kSlots));
                if (j + 2 == J) commit(bar(G::QEMPTY));
              }
            }
          }
        }
        for (int h = 0; h < halves; ++h) ++nu[h];
      }
      // all products are done before TMEM is freed
      commit(bar(G::FINAL));
      const uint64_t t0 = globaltimer_ns();
      while (!try_wait(bar(G::FINAL), 0) && globaltimer_ns() - t0 < kWaitNs) {
      }
    }
  } else if (warp >= kSoftWarps) {
    // Without a plan: flags of invalid sequences, and their zeros.
    if (!AGAIN && p.mode == kPlanNone) {
      for (int b = static_cast<int>(blockIdx.x) * 2 + warp - kSoftWarps - 2; b < p.batch; b += 2 * gridDim.x) {
        const Span s = span_of(p, b, lane == 0);
        if (s.count == 0 || s.rows > 0) continue;
        const int64_t words = static_cast<int64_t>(p.n_q_heads) * D * 2 / 16;
        uint4* to = static_cast<uint4*>(p.out) + s.first * words;
        for (int64_t i = lane; i < s.count * words; i += 32) to[i] = make_uint4(0u, 0u, 0u, 0u);
      }
    }
  } else {
    // --------------------------------------------------- softmax, epilogue
    // Two threads per query row (TMEM lane) of half hf: column group cg has
    // columns 64 cg .. of S and half the columns of O. The two warps of a row
    // meet at a barrier per tile, which also says whether the reference has to
    // move (or one of them gave up).
    const int hf = warp >> 3, cg = (warp >> 2) & 1;
    const int r = (warp & 3) * 32 + lane;
    const uint32_t lane_addr = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);
    const uint32_t col_s = lane_addr + hf * kRows + cg * kCols;       // S
    const uint32_t col_p = lane_addr + hf * kRows + cg * (kCols / 2);  // P
    constexpr int OC = D / 2;
    const uint32_t col_o = lane_addr + G::kColO + hf * D + cg * OC;
    float* s_part = reinterpret_cast<float*>(sm + G::kOffPart);
    volatile int* s_fail = reinterpret_cast<volatile int*>(sm + G::kOffFail);
    const int mine = warp * 32 + lane, other = mine ^ 128;  // the row's other thread
    const int pair = 1 + hf * 4 + (warp & 3);                // barrier of the two warps
    const int tk = r / p.group;  // token of the half
    // (done again, weights of bf16 stay at or below 1: its values end where fp32 does)
    constexpr float BELOW = PromptMargin<BF>::kBelow, ABOVE = AGAIN && BF ? 0.f : PromptMargin<BF>::kAbove;
    const float qs = p.qscale;
    // a warp goes on or gives up as one
    auto wait_warp = [&](uint32_t b, uint32_t parity) {
      return __all_sync(full, wait_phase_suspend(b, parity, s_abort, p.err));
    };
    // The row's other thread's x; ok: of both warps.
    auto exchange = [&](float x, bool& ok) {
      s_part[mine] = x;
      if (lane == 0) s_fail[warp] = ok ? 0 : 1;
      pair_sync(pair);
      const float y = s_part[other];
      ok = ok && s_fail[warp ^ 4] == 0;
      pair_sync(pair);
      return y;
    };
    uint32_t gt = 0, n = 0, nu = 0;  // the CTA's KV tiles; tiles and units of this half
    bool ok = true;
    for (uint32_t un = 0;; ++un) {
      // both warps of a row go on or give up: neither may wait at their barrier alone
      if (pair_or(pair, !wait_warp(bar(G::UFULL0 + (un & 1)), (un >> 1) & 1u))) break;
      const Part& u = s_unit[un & 1];
      if (u.t.count == 0) break;
      if (hf * p.tokens >= u.t.count) {  // the half has no token
        gt += u.i1 - u.i0;
        __syncwarp();
        if (lane == 0) arrive(bar(G::UEMPTY0 + (un & 1)));
        continue;
      }
      const int first = u.t.pos + hf * p.tokens;  // positions of the half
      const int last = min(u.t.pos + u.t.count, first + p.tokens) - 1;
      const bool valid = tk < p.tokens && first + tk <= last;
      const int pos = min(first + tk, last);
      // Tiles [f0, f1) lie in every row's window and behind no row: not masked
      int f0, f1;
      {
        const Seen seen = seen_tiles(u.t.pos, u.t.count, window, sinks);
        const int open = last >= window ? (last - window) / kRows + 1 : 0;
        f0 = seen.front + max(0, open - seen.start);
        f1 = AGAIN ? 0 : seen.front + (first + 1) / kRows - seen.start;
      }
      // What is not finite: at [row of a tile] in the rows that every token of the unit sees;
      // of the others at [row behind the first token's own], then [row leaving the window].
      OddDims* odd_all = reinterpret_cast<OddDims*>(sm + G::kOffStage) + cg;
      OddDims* odd_row = reinterpret_cast<OddDims*>(sm + G::kOffOddRows) + cg;
      if (AGAIN && hf == 0) odd_all[2 * r] = make_uint4(0u, 0u, 0u, 0u);
      float m = kLowest, l = 0.f;  // finite: a row may meet only hidden columns
      const int i0 = u.i0, i1 = u.i1;
      for (int i = i0; i < i1; ++i, ++gt, ++n) {
        ok = wait_warp(bar(G::SFULL0 + hf), n & 1u);
        fence_after();
        const uint32_t bad = s_bad[gt % kBadRing];
        float s[32];
        uint32_t w[16], see[2] = {0xffffffffu, 0xffffffffu};  // see: which columns are visible
        float2 sum[2];
        auto load = [&](int part) {
          tmem_ld32(col_s + 32 * part, s);
          if (p.negative) {
#pragma unroll
            for (int c = 0; c < 32; ++c) s[c] = -s[c];
          }
          if (see[part] != 0xffffffffu) {
#pragma unroll
            for (int c = 0; c < 32; ++c)
              if ((see[part] & (1u << c)) == 0) s[c] = -__builtin_huge_valf();
          }
        };
        auto largest = [&]() {
          float mx[2] = {max3(s[0], s[1], s[2]), max3(s[3], s[4], s[5])};
#pragma unroll
          for (int c = 6; c < 30; c += 4) {
            mx[0] = max3(mx[0], s[c], s[c + 1]);
            mx[1] = max3(mx[1], s[c + 2], s[c + 3]);
          }
          return max3(fmaxf(mx[0], mx[1]), s[30], s[31]);
        };
        auto weigh = [&]() {
          const float2 q2 = make_float2(qs, qs), m2 = make_float2(-m, -m);
#pragma unroll
          for (int k = 0; k < 16; ++k) {
            const float2 a = make_float2(s[2 * k], s[2 * k + 1]);
            const float2 x = AGAIN ? fadd2(make_float2(__fmul_rn(a.x, qs), __fmul_rn(a.y, qs)), m2) : ffma2(a, q2, m2);
            const float2 e = make_float2(fast_exp2(x.x), fast_exp2(x.y));
            sum[k & 1] = fadd2(sum[k & 1], e);
            w[k] = pack16<BF>(e.x, e.y);
          }
        };
        if (i < f0 || i >= f1 || bad != 0) {
          const Seen seen = seen_tiles(u.t.pos, u.t.count, window, sinks);
          const int r0 = (i < seen.front ? i : i - seen.front + seen.start) * kRows;
          const int c0 = r0 + cg * kCols;  // row of the first column
          uint64_t bits = bits_below(pos - c0 + 1) & (~bits_below(pos - window - c0 + 1) | bits_below(sinks - c0));
          for (int b = 0; bad != 0 && b < kRows >> p.box_log2; ++b)
            if ((bad >> b) & 1u)
              bits &= ~(bits_below(((b + 1) << p.box_log2) - cg * kCols) & ~bits_below((b << p.box_log2) - cg * kCols));
          see[0] = static_cast<uint32_t>(bits);
          see[1] = static_cast<uint32_t>(bits >> 32);
          // V rows that nobody in the unit sees may hold anything, and 0 x NaN is
          // NaN: half 0 clears them (its products come first).
          const int end = u.t.pos + u.t.count - 1;
          const int low = u.t.pos >= window ? u.t.pos - window + 1 : 0;
          if (hf == 0 && (AGAIN || r0 + kRows - 1 > end || (r0 < low && r0 + kRows > sinks))) {
            const uint32_t k = 2 * gt + 1, slot = k % G::kSlots;
            ok = ok && wait_warp(bar(G::FULL0 + slot), (k / G::kSlots) & 1u);
            const int row = r0 + r;
            unsigned char* v = sm + G::kOffRing + slot * G::kTile + (r >> 3) * G::kRowGroup + (r & 7) * 128;
            constexpr int CH = G::kHalves * 4;  // 16-byte chunks of a thread
            if (ok && (row > end || (row < low && row >= sinks))) {
#pragma unroll
              for (int c = 0; c < CH; ++c) {
                const int ch = cg * CH + c;
                *reinterpret_cast<uint4*>(v + (ch >> 3) * 1024 + 16 * (ch & 7)) = make_uint4(0u, 0u, 0u, 0u);
              }
            } else if (AGAIN && ok) {
              OddDims odd = make_uint4(0u, 0u, 0u, 0u);
#pragma unroll 1
              for (int c = 0; c < CH; ++c) {  // (the swizzle: chunk c of row r lies at c ^ (r & 7))
                const int ch = cg * CH + c;
                take_odd<BF>(v + (ch >> 3) * 1024 + 16 * ((ch & 7) ^ (r & 7)), 8 * c, odd);
              }
              if (row > u.t.pos) {
                odd_row[2 * (row - u.t.pos - 1)] = odd;
              } else if (row <= end - window && row >= sinks) {
                odd_row[2 * (2 * kM - 1 + row - low)] = odd;
              } else {
                OddDims& all = odd_all[2 * r];
                all = make_uint4(all.x | odd.x, all.y | odd.y, all.z | odd.z, all.w | odd.w);
              }
            }
            fence_proxy_async_smem();
            if constexpr (AGAIN) __syncwarp();
          }
        }
        // Once; again where the reference had to move. The first half of the
        // weights does not wait for the second half's scores and the vote, and no
        // scores need be kept: S is still in TMEM. (64 scores at once spill.)
#pragma unroll 1
        for (;;) {
          load(0);
          float top = largest();
          sum[0] = sum[1] = make_float2(0.f, 0.f);
          weigh();
          load(1);
          top = fmaxf(top, largest()) * qs;
          fence_before();  // both warps have read S before either writes P
          if (!pair_or(pair, !ok || (valid && top > m + ABOVE))) break;
          top = fmaxf(top, exchange(top, ok));
          if (!ok) break;
          const float to = fmaxf(m, top - BELOW);
          const float f = fast_exp2(m - to);
          l *= f;
          m = to;
          if (i > i0) {  // PV of the tile before is done: S came behind it
#pragma unroll 1
            for (int c = 0; c < OC; c += 16) {
              float o[16];
              tmem_ld16(col_o + c, o);
#pragma unroll
              for (int k = 0; k < 16; ++k) o[k] *= f;
              tmem_st16_async(col_o + c, reinterpret_cast<const uint32_t*>(o));
            }
          }
        }
        if (!ok) break;
        fence_after();
        tmem_st16_async(col_p, w);
        tmem_wait_st();
        fence_before();
        __syncwarp();
        if (lane == 0) arrive(bar(G::PFULL0 + 2 * hf));
        weigh();
        tmem_st16_async(col_p + 16, w);
        sum[0] = fadd2(sum[0], sum[1]);
        l += sum[0].x + sum[0].y;
        tmem_wait_st();
        fence_before();
        __syncwarp();
        if (lane == 0) arrive(bar(G::PFULL0 + 2 * hf + 1));
      }
      // ---- epilogue
      if (!ok) break;  // both warps of a row
      if (AGAIN && hf == 0) {
        __syncwarp();
        if (lane == 0) arrive(bar(G::ODDFULL));
      }
      ok = wait_warp(bar(G::OFULL0 + hf), nu & 1u) && (!AGAIN || wait_warp(bar(G::ODDFULL), un & 1u));
      l += exchange(l, ok);
      if (!ok) break;
      ++nu;
      fence_after();
      const int head = u.kvh * p.group + r - tk * p.group;
      const int row = u.t.first + hf * p.tokens + tk;
      const int rec = u.rec;
      const float inv = rec >= 0 ? 1.f : l == 0.f ? 0.f : 1.f / l;
      // Threads have rows, and a row's pieces lie far from the next row's: they go
      // through shared memory, so that four lanes write 64 bytes of a row (one
      // 16-byte piece per lane and row cost 8 times the cycles in the load-store unit).
      unsigned char* to = nullptr;
      if (valid)
        to = rec < 0 ? static_cast<unsigned char*>(p.out) +
                           ((static_cast<int64_t>(row) * p.n_q_heads + head) * D + cg * OC) * 2
                     : reinterpret_cast<unsigned char*>(
                           p.rec_o + ((static_cast<int64_t>(rec) * 2 + hf) * kM + r) * D + cg * OC);
      unsigned char* stage = sm + G::kOffStage + warp * 2048;
      auto put = [&](const uint32_t* x, int off) {  // 64 bytes of every row
#pragma unroll
        for (int k = 0; k < 4; ++k)
          *reinterpret_cast<uint4*>(stage + lane * 64 + ((k ^ ((lane >> 1) & 3)) << 4)) =
              make_uint4(x[4 * k], x[4 * k + 1], x[4 * k + 2], x[4 * k + 3]);
        __syncwarp();
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int src = 8 * k + (lane >> 2);
          unsigned char* at = reinterpret_cast<unsigned char*>(
              __shfl_sync(full, reinterpret_cast<unsigned long long>(to), src));
          const uint4 v = *reinterpret_cast<const uint4*>(stage + src * 64 + (((lane & 3) ^ ((src >> 1) & 3)) << 4));
          if (at != nullptr) *reinterpret_cast<uint4*>(at + off + 16 * (lane & 3)) = v;
        }
        __syncwarp();
      };
      if constexpr (!AGAIN) {
        float zero = 0.f;  // NaN if an output is not finite
#pragma unroll 1
        for (int c = 0; c < OC; c += 32) {
          float o[32];
          tmem_ld32(col_o + c, o);
#pragma unroll
          for (int k = 0; k < 32; ++k) o[k] *= inv;
          if (rec >= 0) {
#pragma unroll
            for (int k = 0; k < 32; ++k) zero = fmaf(o[k], 0.f, zero);
            put(reinterpret_cast<const uint32_t*>(o), 4 * c);
            put(reinterpret_cast<const uint32_t*>(o) + 16, 4 * c + 64);
          } else {
            uint32_t w[16];
#pragma unroll
            for (int k = 0; k < 16; ++k) {
              zero = fmaf(o[2 * k], 0.f, fmaf(o[2 * k + 1], 0.f, zero));
              w[k] = pack16<BF>(o[2 * k], o[2 * k + 1]);
            }
            put(w, 2 * c);
          }
        }
        // Where a visible score is NaN the sum is, and so are all outputs of the row: nothing to
        // find out. A sum of 0 or infinity: the reference is the rounded product of a score, the
        // weights' exponents are not, and for scores beyond 2^30 the difference alone leaves
        // fp32's exponents. Done again, those are differences of rounded products.
        // The unit's first warp that meets one puts it on the list.
        if (__any_sync(full, valid && ((zero != 0.f && l == l) || (l == 0.f && m > kLowest))) && lane == 0 &&
            atomicExch(const_cast<int*>(s_odd) + 1 + (un & 1), 1) == 0) {
          OddUnit& e = p.odd[u.t.cost];
          e.u = u;
          e.next = atomicExch(const_cast<int*>(s_odd), u.t.cost);
        }
      } else {
        OddDims odd = make_uint4(0u, 0u, 0u, 0u);
        auto add = [&](const OddDims& x) {
          odd.x |= x.x;
          odd.y |= x.y;
          odd.z |= x.z;
          odd.w |= x.w;
        };
        for (int i = 0; i < kRows; ++i) add(odd_all[2 * i]);
        // of the others those that this token sees, in this part's tiles
        const Seen seen = seen_tiles(u.t.pos, u.t.count, window, sinks);
        const int low = u.t.pos >= window ? u.t.pos - window + 1 : 0, end = u.t.pos + u.t.count - 1;
        const int r0 = (i0 - seen.front + seen.start) * kRows, r1 = (i1 - seen.front + seen.start) * kRows;
        for (int x = max(u.t.pos + 1, r0); x <= min(pos, r1 - 1); ++x)
          if (x > pos - window || x < sinks) add(odd_row[2 * (x - u.t.pos - 1)]);
        for (int x = max(max(low, pos - window + 1), max(sinks, r0)); x <= min(min(end - window, u.t.pos), r1 - 1); ++x)
          add(odd_row[2 * (2 * kM - 1 + x - low)]);
        if (l != l) odd = make_uint4(0u, 0u, 0u, 0u);  // NaN throughout
        __syncwarp();
#pragma unroll 1
        for (int c = 0; c < OC; c += 16) {
          float o[16];
          tmem_ld16(col_o + c, o);
          const uint32_t plus = (c < 32 ? odd.x : odd.y) >> (c & 31), minus = (c < 32 ? odd.z : odd.w) >> (c & 31);
#pragma unroll
          for (int k = 0; k < 16; ++k) o[k] = odd_or(o[k] * inv, plus, minus, k);
          if (to != nullptr && rec >= 0) {
#pragma unroll
            for (int k = 0; k < 4; ++k)
              reinterpret_cast<float4*>(to)[c / 4 + k] = make_float4(o[4 * k], o[4 * k + 1], o[4 * k + 2], o[4 * k + 3]);
          } else if (to != nullptr) {
            uint32_t w[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) w[k] = pack16<BF>(o[2 * k], o[2 * k + 1]);
            reinterpret_cast<uint4*>(to)[c / 8] = make_uint4(w[0], w[1], w[2], w[3]);
            reinterpret_cast<uint4*>(to)[c / 8 + 1] = make_uint4(w[4], w[5], w[6], w[7]);
          }
          __syncwarp();
        }
      }
      fence_before();
      __syncwarp();
      if (lane == 0) arrive(bar(G::OEMPTY0 + hf));
      if (rec >= 0 && valid && cg == 0)
        *reinterpret_cast<float2*>(p.rec_ml + ((static_cast<int64_t>(rec) * 2 + hf) * kM + r) * 2) = make_float2(m, l);
      __syncwarp();
      if (lane == 0) arrive(bar(G::UEMPTY0 + (un & 1)));
    }
  }

  fence_before();
  __syncthreads();
  fence_after();
}

// (out of line: its registers are its own)
template <typename CT, int D>
__device__ __noinline__ void prompt_roles_again(const CUtensorMap& tm_q, const CUtensorMap& tm_k,
                                                const CUtensorMap& tm_v, const PromptParams& p, unsigned char* sm,
                                                uint32_t tmem) {
  prompt_roles<CT, D, true>(tm_q, tm_k, tm_v, p, sm, tmem);
}

template <typename CT, int D>
__global__ void __launch_bounds__(kPromptThreads, 1)
    prompt_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                  const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ PromptParams p) {
  using G = PromptGeo<D>;
  extern __shared__ __align__(1024) unsigned char sm[];  // the swizzle counts from multiples of 1024
  const uint32_t base = smem_addr(sm);
  volatile uint32_t* s_tmem = reinterpret_cast<volatile uint32_t*>(sm + G::kOffMisc);
  volatile int* s_abort = reinterpret_cast<volatile int*>(sm + G::kOffMisc + 4);
  volatile int* s_odd = reinterpret_cast<volatile int*>(sm + G::kOffMisc + 8);
  const int tid = threadIdx.x, warp = tid >> 5;

  if ((base & 1023u) != 0) {  // the alignment above was not kept
    set_flag(p.err, KVC_FLAG_TIMEOUT);
    return;
  }
  if (tid < 2 * G::COUNT) {
    const int i = tid % G::COUNT;
    uint32_t from = 1;
    if ((i >= G::PFULL0 && i < G::OFULL0) || (i >= G::OEMPTY0 && i < G::UFULL0) || i == G::ODDFULL)
      from = kSoftWarps / 2;
    if (i >= G::UEMPTY0 && i < G::FINAL) from = kSoftWarps + 1;
    mbar_init(reinterpret_cast<uint64_t*>(sm + G::kOffBar) + tid, from);
    fence_barrier_init();
  }
  if (tid == 0) {
    *s_abort = 0;
    *s_odd = -1;
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&tm_q)) : "memory");
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&tm_k)) : "memory");
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&tm_v)) : "memory");
  }
  // Query rows that no token has (128 is no multiple of the group) stay zeros.
  if (p.tokens * p.group < kM) {
    for (uint32_t i = tid; i < 2 * G::kTile / 16; i += kPromptThreads)
      *reinterpret_cast<uint4*>(sm + 16 * i) = make_uint4(0u, 0u, 0u, 0u);
    fence_proxy_async_smem();
  }
  if (warp == kSoftWarps + 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(base + G::kOffMisc),
                 "r"(G::kTmemCols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  fence_before();
  __syncthreads();
  fence_after();
  const uint32_t tmem = *s_tmem;
  prompt_roles<CT, D, false>(tm_q, tm_k, tm_v, p, sm, tmem);
  if (*s_odd >= 0 && *s_abort == 0) prompt_roles_again<CT, D>(tm_q, tm_k, tm_v, p, sm, tmem);
  if (warp == kSoftWarps + 1)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(G::kTmemCols) : "memory");
}

// ------------------------------------------------------------------ merge

// Joins the records of units that several ranges share: o = sum_x 2^(m_x - M)
// O_x / sum_x 2^(m_x - M) l_x, M the largest m so far; an infinity or NaN of a record stays
// as it is, whatever its factor. A warp has four rows at a time,
// lanes over the dims, the loads of two records of each in flight: bound by a chain of
// three loads (tile, its prefix sum, records) per unit.
constexpr int kMergeRows = 32;  // rows of a unit per CTA
constexpr int kMergeWarpRows = kMergeRows / 8;

template <typename CT, int D>
__global__ void __launch_bounds__(256) prompt_merge_kernel(const PromptParams p) {
  constexpr int N = D / 32, K = kMergeWarpRows;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int H = p.n_kv_heads, n = __ldcg(p.head);
  if (__ldcg(p.head + 2) == 0) return;  // no unit was split
  const Ranges r(n, __ldcg(p.head + 1), H, p.grid);
  const int lane = threadIdx.x & 31;
  auto finite = [](float x) { return fabsf(x) < __builtin_huge_valf(); };
  constexpr int CH = 2 * kM / kMergeRows;  // CTAs' shares of a unit
  for (int64_t w = blockIdx.x; w < static_cast<int64_t>(n) * H * CH; w += gridDim.x) {
    const int unit = static_cast<int>(w / CH), i = unit / H, kvh = unit - i * H;
    const Tile t = Walk::load(p, i);
    const int u0 = H * __ldcg(p.before + i) + kvh * t.cost;
    const int a = r.holder(u0), b = r.holder(u0 + t.cost - 1);
    if (a == b) continue;
    // a range's first part is its record 0: all parts of the unit but the first one's,
    // unless that begins its range too
    const int second = u0 > r.start(a) ? 1 : 0;
    const int row0 = static_cast<int>(w % CH) * kMergeRows + (threadIdx.x >> 5) * K;  // half and row
    int tok[K], head[K];
    float M[K], L[K], o[K][N];
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int hf = (row0 + k) / kM, at = (row0 + k) % kM, tk = at / p.group;
      tok[k] = tk < p.tokens && hf * p.tokens + tk < t.count ? hf * p.tokens + tk : -1;
      head[k] = kvh * p.group + at - tk * p.group;
      M[k] = kLowest;
      L[k] = 0.f;
#pragma unroll
      for (int c = 0; c < N; ++c) o[k][c] = 0.f;
    }
    for (int x0 = a; x0 <= b; x0 += 2) {
      float2 ml[2][K];
      float y[2][K][N];
#pragma unroll
      for (int d = 0; d < 2; ++d) {
        const int x = min(x0 + d, b);
        const int64_t rec = (2ll * x + (x == a ? second : 0)) * 2 * kM + row0;
#pragma unroll
        for (int k = 0; k < K; ++k) {
          if (tok[k] < 0) continue;
          ml[d][k] = __ldcg(reinterpret_cast<const float2*>(p.rec_ml + (rec + k) * 2));
          const float* from = p.rec_o + (rec + k) * D + lane * N;
          if constexpr (N == 4) {
            const float4 v = __ldcg(reinterpret_cast<const float4*>(from));
            y[d][k][0] = v.x;
            y[d][k][1] = v.y;
            y[d][k][2] = v.z;
            y[d][k][3] = v.w;
          } else {
            const float2 v = __ldcg(reinterpret_cast<const float2*>(from));
            y[d][k][0] = v.x;
            y[d][k][1] = v.y;
          }
        }
      }
#pragma unroll
      for (int d = 0; d < 2; ++d) {
        if (x0 + d > b) break;
#pragma unroll
        for (int k = 0; k < K; ++k) {
          if (tok[k] < 0) continue;
          const float to = fmaxf(M[k], ml[d][k].x);
          const float f = fast_exp2(M[k] - to), g = fast_exp2(ml[d][k].x - to);
          M[k] = to;
          L[k] = fmaf(g, ml[d][k].y, L[k] * f);
#pragma unroll
          for (int c = 0; c < N; ++c)
            o[k][c] = fmaf(finite(y[d][k][c]) ? g : 1.f, y[d][k][c], finite(o[k][c]) ? o[k][c] * f : o[k][c]);
        }
      }
    }
#pragma unroll
    for (int k = 0; k < K; ++k) {
      if (tok[k] < 0) continue;
      const float inv = L[k] == 0.f ? 0.f : 1.f / L[k];
#pragma unroll
      for (int c = 0; c < N; ++c) o[k][c] *= finite(o[k][c]) || inv != inv ? inv : 1.f;
      store_out_vec<N>(p.out, (static_cast<int64_t>(t.first + tok[k]) * p.n_q_heads + head[k]) * D + lane * N, o[k],
                       std::is_same<CT, __half>::value ? KVC_F16 : KVC_BF16);
    }
  }
}

// ------------------------------------------------------------------- host

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
  // the kernels' sums of KV tiles are 32-bit
  const int64_t rows = static_cast<int64_t>(s.max_blocks) * s.block_size;
  if (s.tiles() >= (1ll << 31) / s.n_kv_heads / (rows / kRows + 2))
    return fail(KVC_ERR_UNSUPPORTED, "num_tokens x max_blocks_per_seq x block_size too large");
  return KVC_OK;
}

// Workspace: [head][tiles][their prefix sums][records' outputs][records'
// references and sums][odd units], each 256-byte aligned; records and prefix sums only where
// units may be split, in this call or in one of fewer tokens: the size for the largest
// call serves all smaller ones.
struct PromptLayout {
  size_t tiles, before, rec_o, rec_ml, odd, total;
  int mode;
};

// Units per SM from which none is split: dealt out by size they end together.
constexpr int kWholeUnits = 4;
// Sequences that a call without a plan looks through.
constexpr int kUnplannedBatch = 256;

inline size_t up256(size_t x) { return (x + 255) / 256 * 256; }

PromptLayout layout(const PromptShape& s, int num_sms) {
  PromptLayout l;
  const int64_t units = (s.num_tokens + 2 * s.tokens() - 1) / (2 * s.tokens()) * s.n_kv_heads;  // at least
  const int64_t most = static_cast<int64_t>(s.max_blocks) * s.block_size / kRows + 2;           // KV tiles of a unit
  l.mode = kPlanWhole;
  if (units < static_cast<int64_t>(kWholeUnits) * num_sms && most > kSplitGain && s.tiles() <= kSplitTiles &&
      num_sms <= kBuckets)
    l.mode = kPlanSplit;
  else if (s.tiles() * s.n_kv_heads <= num_sms && s.batch <= kUnplannedBatch)
    l.mode = kPlanNone;
  l.tiles = 256;
  l.before = l.tiles + up256(static_cast<size_t>(s.tiles()) * sizeof(Tile));
  l.rec_o = l.before + up256(most > kSplitGain ? static_cast<size_t>(s.tiles()) * 4 : 0);
  const size_t recs = most > kSplitGain ? 2 * static_cast<size_t>(num_sms) * 2 * kM : 0;
  l.rec_ml = l.rec_o + up256(recs * s.D * 4);
  l.odd = l.rec_ml + up256(recs * 8);
  l.total = l.odd + up256((static_cast<size_t>(s.tiles()) * s.n_kv_heads + 2 * num_sms) * sizeof(OddUnit));
  return l;
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

// A map of 16-bit elements with 128-byte swizzled boxes, 64 elements wide. (The
// elements are only moved: one type serves bf16 and f16.)
kvc_status make_map(const void* base, int rank, const cuuint64_t* dims, const cuuint64_t* strides,
                    const cuuint32_t* box, CUtensorMap* map) {
  EncodeTiledFn encode = encode_tiled_fn();
  if (encode == nullptr) return fail(KVC_ERR_CUDA, "cuTensorMapEncodeTiled is unavailable");
  const cuuint32_t es[4] = {1, 1, 1, 1};
  const CUresult r = encode(map, CU_TENSOR_MAP_DATA_TYPE_UINT16, rank, const_cast<void*>(base), dims, strides, box, es,
                            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) return fail(KVC_ERR_CUDA, "tensor map: CUresult %d", static_cast<int>(r));
  return KVC_OK;
}

template <typename CT, int D>
kvc_status launch(const PromptParams& p, const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv,
                  cudaStream_t stream) {
  auto* kernel = prompt_kernel<CT, D>;
  // The opt-in to large shared memory holds per device: made at the first call on each.
  static std::atomic<uint64_t> opted{0};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return cuda_fail(e, "cudaGetDevice");
  const uint64_t bit = dev < 64 ? 1ull << dev : 0;
  if ((opted.load() & bit) == 0) {
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             static_cast<int>(PromptGeo<D>::kBytes));
    if (e != cudaSuccess) return cuda_fail(e, "cudaFuncSetAttribute(prompt)");
    opted.fetch_or(bit);
  }
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (p.mode != kPlanNone) {
    cfg.gridDim = dim3(1);
    cfg.blockDim = dim3(kPlanThreads);
    e = cudaLaunchKernelEx(&cfg, prompt_plan_kernel, p, static_cast<int>(sizeof(CT)), D);
    if (e != cudaSuccess) return cuda_fail(e, "cudaLaunchKernelEx(prompt plan)");
  }
  cfg.gridDim = dim3(static_cast<unsigned>(p.grid));
  cfg.blockDim = dim3(kPromptThreads);
  cfg.dynamicSmemBytes = PromptGeo<D>::kBytes;
  e = cudaLaunchKernelEx(&cfg, kernel, tq, tk, tv, p);
  if (e != cudaSuccess) return cuda_fail(e, "cudaLaunchKernelEx(prompt)");
  if (p.mode == kPlanSplit) {
    const int64_t shares = static_cast<int64_t>(p.max_tiles) * p.n_kv_heads * (2 * kM / kMergeRows);
    cfg.gridDim = dim3(static_cast<unsigned>(std::min<int64_t>(shares, 8 * p.grid)));  // what the GPU holds at once
    cfg.blockDim = dim3(256);
    cfg.dynamicSmemBytes = 0;
    e = cudaLaunchKernelEx(&cfg, prompt_merge_kernel<CT, D>, p);
    if (e != cudaSuccess) return cuda_fail(e, "cudaLaunchKernelEx(prompt merge)");
  }
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
  *bytes = layout({batch, num_tokens, n_q_heads, n_kv_heads, head_dim, block_size, max_blocks_per_seq},
                  dev->num_sms).total;
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
  const PromptShape shape{batch, num_tokens, n_q_heads, n_kv_heads, head_dim, block_size, max_blocks_per_seq};
  kvc_status st = check_shape(shape);
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
  const PromptLayout l = layout(shape, dev->num_sms);
  const size_t needed = l.total;
  if (workspace == nullptr || workspace_bytes < needed)
    return fail(KVC_ERR_WORKSPACE, "workspace of %zu bytes, %zu needed", workspace == nullptr ? 0 : workspace_bytes,
                needed);
  if ((reinterpret_cast<uintptr_t>(workspace) & 255u) != 0)
    return fail(KVC_ERR_INVALID_ARG, "workspace must be 256-byte aligned");
  char* ws = static_cast<char*>(workspace);
  PromptParams p{};
  // positions are below 2^30: larger windows are all rows, and differences of them stay in 32 bits
  p.window = std::min(window, 1 << 30);
  p.sinks = std::min(sinks, 1 << 30);
  p.num_blocks = num_blocks;
  p.n_kv_heads = n_kv_heads;
  p.block_size = block_size;
  p.q = q;
  p.out = out;
  p.block_tables = block_tables;
  p.query_starts = query_starts;
  p.context_lens = context_lens;
  p.head = reinterpret_cast<int*>(ws);
  p.tiles = reinterpret_cast<Tile*>(ws + l.tiles);
  p.before = reinterpret_cast<int*>(ws + l.before);
  p.rec_o = reinterpret_cast<float*>(ws + l.rec_o);
  p.rec_ml = reinterpret_cast<float*>(ws + l.rec_ml);
  p.odd = reinterpret_cast<OddUnit*>(ws + l.odd);
  p.err = dev->error_word;
  p.batch = batch;
  p.num_tokens = static_cast<int>(num_tokens);
  p.n_q_heads = n_q_heads;
  p.group = shape.group();
  p.max_blocks = max_blocks_per_seq;
  p.rows = max_blocks_per_seq * block_size;
  p.tokens = shape.tokens();
  p.max_tiles = static_cast<int>(shape.tiles());
  p.mode = l.mode;
  const int64_t cap = option(KVC_OPT_MAX_CTAS);
  p.grid = static_cast<int>(cap > 0 ? std::min<int64_t>(cap, dev->num_sms) : dev->num_sms);
  if (p.mode == kPlanNone) {
    if (p.max_tiles * n_kv_heads <= p.grid)
      p.grid = p.max_tiles * n_kv_heads;
    else
      p.mode = kPlanWhole;
  }
  p.box = std::gcd(block_size, kRows);
  while ((1 << p.box_log2) < p.box) ++p.box_log2;
  p.pool_rows = static_cast<int>(num_blocks * n_kv_heads * block_size);
  // hidden scores are -infinity, which a factor of 0 would turn into NaN
  p.qscale = std::max(std::fabs(scale * 1.4426950408889634f), 1e-35f);
  p.negative = scale < 0.f ? 1 : 0;
  CUtensorMap tq, tk, tv;
  const cuuint64_t d = static_cast<cuuint64_t>(head_dim);
  {
    const cuuint64_t dims[3] = {d, static_cast<cuuint64_t>(n_q_heads), static_cast<cuuint64_t>(num_tokens)};
    const cuuint64_t strides[2] = {d * 2, d * 2 * n_q_heads};
    const cuuint32_t box[3] = {64, static_cast<cuuint32_t>(p.group), static_cast<cuuint32_t>(p.tokens)};
    if ((st = make_map(q, 3, dims, strides, box, &tq)) != KVC_OK) return st;
  }
  {
    // [8-row group][part][row of the group][64 elements]
    const cuuint64_t dims[4] = {64, 8, d / 64, static_cast<cuuint64_t>(p.pool_rows / 8)};
    const cuuint64_t strides[3] = {d * 2, 128, d * 16};
    const cuuint32_t box[4] = {64, 8, static_cast<cuuint32_t>(head_dim / 64), static_cast<cuuint32_t>(p.box / 8)};
    if ((st = make_map(k_cache, 4, dims, strides, box, &tk)) != KVC_OK) return st;
    if ((st = make_map(v_cache, 4, dims, strides, box, &tv)) != KVC_OK) return st;
  }
  cudaStream_t cs = static_cast<cudaStream_t>(stream);
  if (dtype == KVC_F16)
    st = head_dim == 64 ? launch<__half, 64>(p, tq, tk, tv, cs) : launch<__half, 128>(p, tq, tk, tv, cs);
  else
    st = head_dim == 64 ? launch<__nv_bfloat16, 64>(p, tq, tk, tv, cs) : launch<__nv_bfloat16, 128>(p, tq, tk, tv, cs);
  if (st != KVC_OK) return st;
  return finish_call(cs);
}

}  // extern "C"
