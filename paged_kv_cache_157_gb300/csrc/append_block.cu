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
// A CTA finds the runs that begin in a stretch of tokens and takes them one by
// one for some of the heads, a short run by one warp, a long one by all. A
// run's rows are read once, in 16-byte loads that are all in flight together,
// and stay in registers between the maximum and the codes (runs beyond 16 KB
// are read again, out of L2). Bound, for prompts, by the load, barrier and store
// phases of four CTAs per SM rather than by HBM; for a decode step, whose tokens
// get a warp each, by the chain slots -> rows and scale -> codes of dependent
// accesses. Measured (8 heads, D 128, bf16): a prompt of 16384 tokens 29.4 us
// (3.4 TB/s of its 101 MB, 36 % issue), a step of 64 tokens 6.3 us.
#include <algorithm>
#include <type_traits>

#include "code8.cuh"

namespace kvc {

namespace {

// Largest |x| of m and the values of one 16-byte chunk of T; NaN if any is.
template <typename T>
__device__ __forceinline__ float chunk_max(float m, const uint4& u) {
#pragma unroll
  for (int i = 0; i < 16 / static_cast<int>(sizeof(T)) / 2; ++i) {
    const float2 x = Elem<T>::pair(u, i);
    asm("max.NaN.abs.f32 %0, %0, %1, %2;" : "+f"(m) : "f"(x.x), "f"(x.y));
  }
  return m;
}

// Largest finite |x| among the values of one 16-byte chunk of T.
template <typename T>
__device__ __forceinline__ float finite_max(const uint4& u) {
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
  int stretch;     // tokens a CTA looks at at a time
  unsigned items;  // stretches x heads x 2
  int scouts;      // CTAs behind the others that look for blocks with more than one run
  unsigned parts;  // of a window's blocks, by hash: a table each
  unsigned tasks;  // windows x parts
  uint64_t block_inv;  // ceil(2^64 / block_size)
  unsigned int* err;
};

// Block of a slot, -1 if the token is not written.
__device__ __forceinline__ int64_t block_of(int64_t slot, const AppendBlockParams& p) {
  if (slot < 0 || slot >= p.num_slots) return -1;
  return ((slot | p.block_size) >> 32) == 0 ? static_cast<uint32_t>(slot) / static_cast<uint32_t>(p.block_size)
                                            : slot / p.block_size;
}

constexpr int kAppendWarps = 4;
constexpr int kAppendThreads = 32 * kAppendWarps;
// windows of 32 tokens that a CTA looks at: its stretch (at most 4) and what its last run may reach
constexpr int kWindows = 8;
constexpr int kInFlight = 8;      // 16-byte chunks a lane holds
constexpr int kAppendCtasPerSm = 4;

// Two runs of one block would race for its codes and scale, so a slot mapping
// that has them is flagged. A few CTAs look for them beside the others: the
// blocks that begin runs go into a hash table in shared memory, and one that is
// there already has two. A table takes a part of the blocks of a window of
// tokens (five eighths of its size if every token were a run), a CTA one or
// more of them. Windows overlap by half. Their length, and with it the times a
// token is looked at, grows with the heads, as the others' time does, so that the
// check ends before they do (16384 tokens, 8 heads: 29.1 us without it, 29.4 with).
constexpr int kTableBits = 10;
constexpr int kTokensPerPart = 5 << (kTableBits - 3);
constexpr int kMinParts = 4;  // of a window, if the call has that many tokens
constexpr int kLookAt = 8;  // tokens per lane in flight; a warp's are in one piece

// (four CTAs stay within 32 KB: what they spill lives in the rest of the L1)
union AppendShared {
  struct {
    int64_t slot[1 + 32 * kWindows];  // of the token before the stretch, and of the windows' tokens
    int64_t block[kAppendThreads];
    int first[kAppendThreads], end[kAppendThreads];  // the runs: first token, and the one behind
    uint32_t ends[kWindows];                         // bit masks: a token that is not written, or begins a run
    int count[kAppendWarps];                         // per window
    uint32_t red[2 * kAppendWarps];
  } runs;
  struct {
    uint4 table[(1 << kTableBits) / 4];
    uint16_t queue[kAppendWarps][32 * kLookAt];
  } check;
};

__device__ __noinline__ void find_split_blocks(const AppendBlockParams& p, unsigned scout, AppendShared& sh) {
  constexpr uint32_t full = 0xffffffffu, size = 1u << kTableBits;
  uint4* s_table4 = sh.check.table;
  uint32_t* s_table = reinterpret_cast<uint32_t*>(s_table4);
  const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
  uint16_t* queue = sh.check.queue[w];
  bool found = false;
  for (unsigned task = scout; task < p.tasks; task += p.scouts) {
    const unsigned window = task / p.parts, part = task - window * p.parts;
    const int64_t begin = window * (static_cast<int64_t>(p.parts) * (kTokensPerPart / 2));
    const int64_t end = min(p.num_tokens, begin + static_cast<int64_t>(p.parts) * kTokensPerPart);
    __syncthreads();  // the last table is done with
#pragma unroll
    for (uint32_t i = 0; i < size / 4; i += kAppendThreads) s_table4[i + tid] = make_uint4(0u, 0u, 0u, 0u);
    __syncthreads();
#pragma unroll 1
    for (int64_t t0 = begin + w * (32 * kLookAt); t0 < end; t0 += kAppendThreads * kLookAt) {
      const int64_t left = end - t0 - lane;
      const int64_t* at = p.slots + t0 + lane;
      int64_t slot[kLookAt];
      int64_t last = lane == 31 && t0 > begin ? __ldg(p.slots + t0 - 1) : -1;  // of the token before lane 0's
#pragma unroll
      for (int i = 0; i < kLookAt; ++i) slot[i] = 32 * i < left ? __ldg(at + 32 * i) : -1;
      // a token one row behind the one before begins a run only at a block's start, a multiple of 16
      int n = 0;
#pragma unroll
      for (int i = 0; i < kLookAt; ++i) {
        const int64_t prev = __shfl_sync(full, lane == 31 ? last : slot[i], (lane + 31) & 31);
        last = slot[i];
        const bool may = slot[i] >= 0 && slot[i] < p.num_slots && (slot[i] != prev + 1 || (slot[i] & 15) == 0);
        const uint32_t m = __ballot_sync(full, may);
        if (may) queue[n + __popc(m & ((1u << lane) - 1u))] = static_cast<uint16_t>(32 * i + lane);
        n += __popc(m);
      }
      __syncwarp();
      for (int q = lane; q < n; q += 32) {
        const int64_t t = t0 + queue[q], sl = __ldg(p.slots + t), prev = t > begin ? __ldg(p.slots + t - 1) : -1;
        // block (exact for slots below 2^57) and its first slot; multiplicative
        // hashing: the top bits choose the part, others the place
        const uint64_t blk = __umul64hi(static_cast<uint64_t>(sl), p.block_inv);
        const int64_t first = static_cast<int64_t>(blk) * p.block_size;
        if (prev >= first && prev - first < p.block_size) continue;
        const uint64_t hash = blk * 0x9E3779B97F4A7C15ull;
        if (__umulhi(static_cast<uint32_t>(hash >> 32), p.parts) != part) continue;
        const uint32_t entry = static_cast<uint32_t>(blk) + 1;  // (no memory holds 2^32 blocks)
        uint32_t place = static_cast<uint32_t>(hash >> 20) % size;
        for (uint32_t k = 0; k < size; ++k, place = (place + 1) % size) {
          const uint32_t there = atomicCAS(&s_table[place], 0u, entry);
          found |= there == entry;
          if (there == 0 || there == entry) break;
        }
      }
      __syncwarp();
    }
  }
  if (found) set_flag(p.err, KVC_FLAG_BAD_SLOT);
}

// A run: `rows` tokens from the one x and slots point at.
struct Run {
  const uint4* x;        // head h of the run's first token
  const int64_t* slots;  // of the run's first token
  int64_t first_slot;    // of the block
  float* scale;
  unsigned char* dst;    // the block's codes of head h
  int rows;
  int first;             // its lowest row in the block
};

// One run by a group of NW warps (thread g of it); token_chunks: 16-byte
// chunks from a token to the next. ASC: the tokens fill ascending rows, from
// run.first on; otherwise each token's slot is looked up.
template <typename T, bool INT8, int D, int NW, bool ASC>
__device__ __noinline__ void append_run(const Run run, uint32_t token_chunks, int g, uint32_t* s_red) {
  constexpr int VEC = 16 / sizeof(T);  // values per 16-byte chunk
  constexpr int CPR = D / VEC;         // chunks per row
  constexpr int STEP = 32 * NW;
  constexpr int RPS = STEP >= CPR ? STEP / CPR : 1;  // rows per step (a row may take two steps)
  constexpr int SPR = STEP >= CPR ? 1 : CPR / STEP;  // steps per row
  const int lane = g & 31;
  // the lane's chunk of step i: row (i / SPR) * RPS + r0 of the run, chunk c0 + (i % SPR) * STEP of it
  const int r0 = g / CPR, c0 = g % CPR;
  const int steps = (run.rows + RPS - 1) / RPS * SPR;
  auto row_of = [&](int i) { return (i / SPR) * RPS + r0; };
  // rows past the end: the last one, whose values count already
  const uint4* x0 = run.x + c0;
  auto chunk_of = [&](int i) {
    const int r = min(row_of(i), run.rows - 1);
    // ascending rows: at most a block of them, 32-bit offsets
    if constexpr (ASC) return x0 + (static_cast<uint32_t>(r) * token_chunks + (i % SPR) * STEP);
    return x0 + (static_cast<int64_t>(r) * token_chunks + (i % SPR) * STEP);
  };
  auto block_row = [&](int i) {
    return ASC ? run.first + row_of(i) : static_cast<int>(__ldg(run.slots + row_of(i)) - run.first_slot);
  };
  const float held = *run.scale;
  uint4 u[kInFlight];
  auto load = [&](int i0) {
#pragma unroll
    for (int j = 0; j < kInFlight; ++j)
      if (j == 0 || i0 + j < steps) u[j] = *chunk_of(i0 + j);
  };
  float m = 0.f;
  for (int i0 = 0; i0 < steps; i0 += kInFlight) {
    load(i0);
#pragma unroll
    for (int j = 0; j < kInFlight; ++j)
      if (j == 0 || i0 + j < steps) m = chunk_max<T>(m, u[j]);
  }
  // as integers the magnitudes keep their order, with infinity and NaN on top
  uint32_t mb = __reduce_max_sync(0xffffffffu, __float_as_uint(m) & 0x7fffffffu);
  if constexpr (NW > 1) {  // (also: every warp has read the old scale)
    if (lane == 0) s_red[g >> 5] = mb;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < NW; ++i) mb = max(mb, s_red[i]);
    __syncthreads();  // s_red may be used again
  }
  const bool odd = mb >= 0x7f800000u;  // the run has a value that is not finite (the same in every thread)
  m = __uint_as_float(mb);
  if (odd) {
    m = 0.f;
#pragma unroll 1
    for (int i = 0; i < steps; ++i) m = fmaxf(m, finite_max<T>(*chunk_of(i)));
    m = warp_max(m);
    if constexpr (NW > 1) {
      if (lane == 0) s_red[g >> 5] = __float_as_uint(m);
      __syncthreads();
#pragma unroll
      for (int i = 0; i < NW; ++i) m = fmaxf(m, __uint_as_float(s_red[i]));
      __syncthreads();
    }
  }
  const float old = run.first == 0 ? 0.f : held;
  float s = fmaxf(old, m * Code8<INT8>::kInvMax);
  if (!(s >= kTinyScale)) s = 0.f;
  const float inv = s > 0.f ? __fdiv_rn(1.0f, s) : 0.f;
  if (run.first > 0 && s != old) {
    const float f = s > 0.f ? __fdiv_rn(old, s) : 0.f;
    uint4* rows16 = reinterpret_cast<uint4*>(run.dst);
#pragma unroll 1
    for (int i = g; i < run.first * (D / 16); i += STEP) rows16[i] = rescale16<INT8>(rows16[i], f);
  }
  // Codes of a chunk to its row of the block. Products and codes are rounded
  // separately: no fused multiply-add.
  unsigned char* dst0 = run.dst + c0 * VEC;
  auto put = [&](int i, const uint4& x, const auto& in_range) {
    unsigned char* to = dst0 + static_cast<uint32_t>(block_row(i) * D + (i % SPR) * STEP * VEC);
    uint32_t code[VEC / 4];
#pragma unroll
    for (int k = 0; k < VEC / 4; ++k) {
      float2 a = Elem<T>::pair(x, 2 * k), b = Elem<T>::pair(x, 2 * k + 1);
      a = make_float2(__fmul_rn(a.x, inv), __fmul_rn(a.y, inv));
      b = make_float2(__fmul_rn(b.x, inv), __fmul_rn(b.y, inv));
      if constexpr (std::decay_t<decltype(in_range)>::value)
        code[k] = encode4_in_range<INT8>(a, b);
      else
        code[k] = s > 0.f ? encode4<INT8>(a.x, a.y, b.x, b.y) : 0u;
    }
    if constexpr (VEC == 8)
      *reinterpret_cast<uint2*>(to) = make_uint2(code[0], code[1]);
    else
      *reinterpret_cast<uint32_t*>(to) = code[0];
  };
  if (odd || s == 0.f) {
    // values that are not finite saturate; with scale 0 every finite entry counts as 0
#pragma unroll 1
    for (int i = 0; i < steps; ++i)
      if (row_of(i) < run.rows) put(i, *chunk_of(i), std::false_type{});
  } else {
    // with finite values and s >= A / Q, |x / s| rounds to at most Q
    for (int i0 = 0; i0 < steps; i0 += kInFlight) {
      if (steps > kInFlight) load(i0);
#pragma unroll
      for (int j = 0; j < kInFlight; ++j)
        if (row_of(i0 + j) < run.rows) put(i0 + j, u[j], std::true_type{});
    }
  }
  if (g == 0) *run.scale = s;
}

// Work: items (stretch, head, K or V), stretch-major; every CTA takes an equal
// range of them, so that it finds a stretch's runs once for several heads (a
// CTA per item spent 15 of 36 us of a 16384-token prompt on finding them).
template <typename T, bool INT8, int D>
__global__ void __launch_bounds__(kAppendThreads, kAppendCtasPerSm)
    append_block_kernel(const __grid_constant__ AppendBlockParams p) {
  constexpr int CPR = D * static_cast<int>(sizeof(T)) / 16;
  constexpr uint32_t full = 0xffffffffu;
  __shared__ AppendShared sh;
  uint32_t* s_red = sh.runs.red;
  int64_t* s_slot = sh.runs.slot;
  uint32_t* s_ends = sh.runs.ends;
  int *s_first = sh.runs.first, *s_end = sh.runs.end, *s_runs = sh.runs.count;
  int64_t* s_block = sh.runs.block;
  // a decode launched behind this kernel may set itself up meanwhile; it waits
  // for this grid to end before it reads any cached row
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const unsigned cta = blockIdx.x, ctas = gridDim.x - p.scouts;
  if (cta >= ctas) {
    find_split_blocks(p, cta - ctas, sh);
    return;
  }
  const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
  const int bs = p.block_size;
  const int per_stretch = 2 * p.n_heads;
  const uint32_t token_chunks = static_cast<uint32_t>(p.n_heads) * CPR;
  unsigned item = static_cast<unsigned>(static_cast<uint64_t>(p.items) * cta / ctas);
  const unsigned item_end = static_cast<unsigned>(static_cast<uint64_t>(p.items) * (cta + 1) / ctas);
#pragma unroll 1
  while (item < item_end) {
    const unsigned st = item / per_stretch;
    const int r0 = static_cast<int>(item - st * per_stretch);
    const int r1 = min(per_stretch, r0 + static_cast<int>(item_end - item));  // (head, K or V) of this stretch
    item += r1 - r0;
    const int64_t t0 = static_cast<int64_t>(st) * p.stretch, left = p.num_tokens - t0;
    const int len = left < p.stretch ? static_cast<int>(left) : p.stretch;
    const int windows = (len + 31) / 32, seen = windows + (bs + 31) / 32;  // with runs of this stretch, and looked at
    __syncthreads();  // the last stretch's tables have been read
#pragma unroll
    for (int i = 0; i < 32 * kWindows; i += kAppendThreads) {
      int64_t slot = -1;
      if (i + tid < 32 * seen && i + tid < left) slot = __ldg(p.slots + t0 + i + tid);
      s_slot[1 + i + tid] = slot;
      if (i + tid < len && slot >= p.num_slots) set_flag(p.err, KVC_FLAG_BAD_SLOT);
    }
    if (tid == 0) s_slot[0] = t0 > 0 ? __ldg(p.slots + t0 - 1) : -1;
    __syncthreads();
    // a run begins at a token that is written and does not share its block
    // with the one before, and ends at the next token that begins one or is not written
    uint32_t leads = 0;
    int64_t blk = -1;
#pragma unroll
    for (int i = kWindows - kAppendWarps; i >= 0; i -= kAppendWarps) {  // this warp's windows, the stretch's last
      const int64_t slot = s_slot[1 + 32 * (i + w) + lane], prev = s_slot[32 * (i + w) + lane];
      blk = block_of(slot, p);
      const bool ends = blk < 0 || !(prev >= blk * bs && prev < blk * bs + bs);
      const uint32_t be = __ballot_sync(full, ends);
      leads = __ballot_sync(full, ends && blk >= 0 && 32 * w + lane < len);
      if (lane == 0) s_ends[i + w] = be;
    }
    if (lane == 0) s_runs[w] = __popc(leads);
    __syncthreads();
    int n = 0, runs = 0;  // runs before this warp's, and all
#pragma unroll
    for (int i = 0; i < kAppendWarps; ++i) {
      if (i < w) n += s_runs[i];
      runs += s_runs[i];
    }
    if ((leads >> lane) & 1u) {
      int end = 32 * kWindows;
      uint32_t x = s_ends[w] & ~((2u << lane) - 1u);
      for (int j = w;;) {
        if (x != 0) {
          end = 32 * j + __ffs(x) - 1;
          break;
        }
        if (++j == kWindows) break;
        x = s_ends[j];
      }
      n += __popc(leads & ((1u << lane) - 1u));
      s_first[n] = 32 * w + lane;
      s_end[n] = end;
      s_block[n] = blk;
    }
    __syncthreads();
    int nth = 0;
#pragma unroll 1
    for (int i = 0; i < runs; ++i) {
      Run run;
      const int a = s_first[i];
      const int64_t b = s_block[i];
      int end = s_end[i];
      run.first_slot = b * bs;
      if (end >= 32 * seen && end < left) {  // longer than a block: a slot is named more than once
        for (int64_t e = t0 + 32 * seen;; e += 32) {
          const int64_t sl = e + lane < p.num_tokens ? __ldg(p.slots + e + lane) : -1;
          const uint32_t out = __ballot_sync(full, !(sl >= run.first_slot && sl < run.first_slot + bs));
          end = static_cast<int>(e - t0) + (out != 0 ? __ffs(out) - 1 : 32);
          if (out != 0) break;
        }
      }
      run.rows = end - a;
      run.slots = p.slots + t0 + a;
      // its lowest row, and whether the rows ascend by one: the same in every thread
      int first = bs;
      bool asc = true;
      for (int t = lane; t < run.rows; t += 32) {
        const int64_t sl = a + t < 32 * seen ? s_slot[1 + a + t] : __ldg(run.slots + t);
        first = min(first, static_cast<int>(sl - run.first_slot));
        asc = asc && sl - s_slot[1 + a] == t;
      }
      run.first = __reduce_min_sync(full, first);
      asc = __all_sync(full, asc);
      const bool all = run.rows * CPR > 32 * kInFlight;  // all warps take it together
#pragma unroll 1
      for (int r = r0; r < r1; ++r) {
        if (!all && nth++ % kAppendWarps != w) continue;
        const int h = r >> 1;
        const bool v = r & 1;
        const int64_t head = b * p.n_heads + h;
        run.x = static_cast<const uint4*>(v ? p.v : p.k) + ((t0 + a) * p.n_heads + h) * CPR;
        run.scale = (v ? p.v_scale : p.k_scale) + head;
        run.dst = (v ? p.v_codes : p.k_codes) + head * bs * D;
        if (all && asc)
          append_run<T, INT8, D, kAppendWarps, true>(run, token_chunks, tid, s_red);
        else if (all)
          append_run<T, INT8, D, kAppendWarps, false>(run, token_chunks, tid, s_red);
        else if (asc)
          append_run<T, INT8, D, 1, true>(run, token_chunks, lane, s_red);
        else
          append_run<T, INT8, D, 1, false>(run, token_chunks, lane, s_red);
      }
    }
  }
}

template <typename T, bool INT8>
void launch(const AppendBlockParams& p, int D, int64_t grid, cudaStream_t s) {
  const dim3 g(static_cast<unsigned>(grid)), b(kAppendThreads);
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
  const int64_t resident = static_cast<int64_t>(kAppendCtasPerSm) * dev->num_sms;
  const int64_t parts = std::min<int64_t>((num_tokens + kTokensPerPart - 1) / kTokensPerPart,
                                          std::max(kMinParts, std::min(n_kv_heads, 64)));
  const int64_t step = parts * (kTokensPerPart / 2), beyond = std::max<int64_t>(0, num_tokens - 2 * step);
  const int64_t tasks = (1 + (beyond + step - 1) / step) * parts;
  if (tasks >= (1ll << 31)) return fail(KVC_ERR_UNSUPPORTED, "num_tokens too large");
  p.parts = static_cast<unsigned>(parts);
  p.tasks = static_cast<unsigned>(tasks);
  p.block_inv = ~0ull / static_cast<unsigned>(block_size) + 1;
  // Stretches of a block for prompts, so that a stretch has one run. With few
  // tokens, shorter ones: the CTAs are to fill the GPU, none with a second item
  // (a chunk of 2232 tokens: 9 us, 12 where ten CTAs have one), with a run for
  // each of a CTA's warps if every token is one (a decode step).
  // (the check's share of a long call is 4 % of the work with one head, 2 % with eight)
  const int64_t ctas = resident - std::min(tasks, std::max<int64_t>(1, resident / (16 + 2 * std::min(n_kv_heads, 8))));
  const int64_t heads2 = 2ll * n_kv_heads, fit = std::max<int64_t>(1, ctas / heads2);  // stretches at a time
  p.stretch = static_cast<int>(
      std::min<int64_t>(block_size, std::max<int64_t>(kAppendWarps, (num_tokens + fit - 1) / fit)));
  const int64_t items = (num_tokens + p.stretch - 1) / p.stretch * heads2;
  if (items >= (1ll << 31)) return fail(KVC_ERR_UNSUPPORTED, "num_tokens x n_kv_heads too large");
  p.items = static_cast<unsigned>(items);
  // the check gets what the items leave free: as many CTAs as take no more items each
  const int64_t each = (items + ctas - 1) / ctas, busy = (items + each - 1) / each;
  p.scouts = static_cast<int>(std::min(tasks, resident - busy));
  const int64_t grid = busy + p.scouts;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  switch (dtype) {
    case KVC_F32: launch<float>(p, head_dim, code, grid, s); break;
    case KVC_F16: launch<__half>(p, head_dim, code, grid, s); break;
    case KVC_BF16: launch<__nv_bfloat16>(p, head_dim, code, grid, s); break;
  }
  return finish_call(s);
}
