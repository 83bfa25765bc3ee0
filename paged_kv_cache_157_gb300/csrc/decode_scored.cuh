// Paged decode attention that also adds up the attention weight each cached
// row receives, over 16-bit caches and over one-byte caches with one scale per
// (block, kv head).
//
// Mathematics. Query v of a kv head (v = t * group + j: new token t, query
// head j of the group) attends rows r <= n - n_tok + t:
//   x_vr = scale * q_v . k_r,  p_vr = exp(x_vr) / sum_r exp(x_vr),
//   o_v = sum_r p_vr v_r,      score_r += sum_v p_vr
// with k_r = code * k_scale[block], v_r = code * v_scale[block] for one-byte
// caches. One pass over the rows with the running maximum and sum of the
// softmax; the weights of a row are only known once the denominator is, so the
// pass leaves the scaled scores x (fp32) in the workspace, and the finishing
// kernel, which merges the partial outputs anyway, turns them into weights and
// adds them up. That moves 8 bytes per query and row, mostly through L2; forming
// the scores again from K would read D elements per row instead: more for up to
// 31 queries (16-bit, D 128) or 15 (one byte), less beyond, but with the first
// product done twice. exp2 and log2 are the hardware's (2^-22).
//
// What bounds it, for up to about 16 queries per kv head: HBM in large 16-bit
// batches; every cached row is read once, by TMA, into a ring in shared memory.
// Measured (32 query, 8 kv heads, D 128), decode and finish: bf16, batch 32 x
// 4096 rows 98.8 us (about 90 us of them the decode, 6 TB/s); e4m3 blocks, batch 32 x
// U[512, 4096] 35.9 us, of which about 13 us are start, the SMs' different ends
// and the finish, at 7.0 TB/s for what a larger batch adds (DRAM 53 % busy over
// the whole decode); int8 likewise 40.8 us. More queries are bound by the
// products: 32 tokens, 128 queries per kv head over 2 x 4000 rows 38 us (bf16),
// 40 us (f16), 86 us (e4m3), 60 us (int8); 256 tokens over 4000 rows 209 us (f16).
//
// Work split. The 16-row tiles of all (sequence, kv head, column group) units
// are laid end to end and cut into equal ranges, one per WARP. A warp is a
// worker of its own: it issues its copies, waits for them and runs the
// products, with no barrier between warps, so a unit may have any number of
// kv heads, any length and any group, and eight or twelve workers per SM keep
// 128 to 192 KB of copies in flight. Neighbouring workers sit in one CTA: what
// its warps hold at the ends of their ranges is merged in shared memory, so a
// unit has about one record (maximum, sum, output) per CTA it spans.
//
// Products on m16n8k16 MMAs, rows (or dims) x queries:
//   S^T [16 rows x 8 queries] = K [16 x D] . Q^T,
//   O^T [D x 8 queries] += V^T [D x 16 rows] . P^T
// fp32 accumulation. The weights enter as 16-bit parts: two f16 parts (22 bits,
// see Margin) or, for bf16 caches, three bf16 parts (24 bits), because fp32 outputs
// are to be as good as an fp32 softmax; in large batches the extra products are
// mostly hidden behind HBM. One-byte codes are exact f16 values and are converted
// in registers; queries become f16 after a scaling by a power of two, per query.
#pragma once

#include <algorithm>
#include <atomic>
#include <type_traits>

#include "decode_gqa_mma.cuh"
#include "decode_scored.h"

namespace kvc {

namespace scored {

// Byte offset of 16-byte chunk q of row r in a box of kBoxBytes-wide rows as
// TMA leaves it: 128-byte swizzle (q ^ (r & 7)), or 64-byte swizzle
// (q ^ ((r >> 1) & 3)).
template <int BOXB>
__device__ __forceinline__ uint32_t chunk_at(int r, int q) {
  if constexpr (BOXB == 128) return static_cast<uint32_t>(r * 128 + ((q ^ (r & 7)) << 4));
  return static_cast<uint32_t>(r * 64 + ((q ^ ((r >> 1) & 3)) << 4));
}

__device__ __forceinline__ uint2 lds64(uint32_t addr) {
  uint2 v;
  asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(addr));
  return v;
}

__device__ __forceinline__ void cp_async4(uint32_t dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ float fast_log2(float x) {
  float y;
  asm("lg2.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Where a query's reference m (log2 units) lies: kBelow under the largest score
// when it moves, and it moves when a score exceeds it by kAbove.
//
// A weight 2^(x - m) enters the second product in 16-bit parts. Three bf16 parts
// hold any fp32 weight in 24 bits: the reference is the maximum, and weights
// reach 2^8. f16 ends at 2^-24, and rows beside an attention sink have weights
// of that size. So f16 parts use the whole range (largest weight 2^11 to 2^15),
// and the second part is the rest times 2^11 (kRestScale; at most 2^14), in a
// product of its own that is scaled back: 22 bits down to 2^-25 of the largest
// weight, and off by at most 2^-47 of the largest one below.
template <bool BF>
struct Margin {
  static constexpr float kBelow = BF ? 0.f : 11.f;
  static constexpr float kAbove = BF ? 8.f : 15.f;
};
constexpr float kRestScale = 2048.f;

// State of a segment (one unit's tiles in one worker's range). Lane 4g + c
// holds queries 2c and 2c + 1 of every group of 8 (index e & 1).
template <int D, int NT, bool ONE>
struct State {
  uint32_t q[NT][D / 16][2];  // Q^T B fragments
  float o[NT][D / 16][4];     // O^T C fragments
  float m[NT][2];             // reference maxima (log2 units), equal over g
  float l[NT][2];             // this lane's sums of weights
  float mo[ONE ? NT : 1][2];  // one-byte caches: the outputs' reference, max of x + log2(v_scale)
  float fq[ONE ? NT : 1][2];  // one-byte caches: qscale / the query's power of two
  int dt[NT][2];              // newest rows the query may not see: n_tok - 1 - t
};

// Sets x to -inf where the row is not visible. rem: the sequence's rows from
// the tile's first on.
template <int D, int NT, bool ONE>
__device__ __forceinline__ void mask_edge(float (&x)[NT][4], const State<D, NT, ONE>& st, int rem, int g) {
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    const int v0 = rem - st.dt[n][0], v1 = rem - st.dt[n][1];
    if (g >= v0) x[n][0] = kNegInf;
    if (g >= v1) x[n][1] = kNegInf;
    if (g + 8 >= v0) x[n][2] = kNegInf;
    if (g + 8 >= v1) x[n][3] = kNegInf;
  }
}

// Moves the references up (all lanes of the warp together) and rescales sums
// and outputs. lvs: log2 of the tile's V scale (one-byte caches).
template <int D, int NT, bool ONE, bool BF>
__device__ __forceinline__ void raise_references(const float (&x)[NT][4], State<D, NT, ONE>& st, float lvs) {
  constexpr float BELOW = Margin<BF>::kBelow;
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    float t[2] = {fmaxf(x[n][0], x[n][2]), fmaxf(x[n][1], x[n][3])};
#pragma unroll
    for (int e = 0; e < 2; ++e) {
#pragma unroll
      for (int msk = 4; msk < 32; msk <<= 1) t[e] = fmaxf(t[e], __shfl_xor_sync(0xffffffffu, t[e], msk));
    }
    float a[2];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const float m = fmaxf(st.m[n][e], t[e] - BELOW);
      a[e] = fast_exp2(st.m[n][e] - m);
      st.l[n][e] *= a[e];
      st.m[n][e] = m;
      if constexpr (ONE) {
        const float mo = fmaxf(st.mo[n][e], t[e] + lvs - BELOW);
        a[e] = fast_exp2(st.mo[n][e] - mo);
        st.mo[n][e] = mo;
      }
    }
#pragma unroll
    for (int i = 0; i < D / 16; ++i) {
      st.o[n][i][0] *= a[0];
      st.o[n][i][1] *= a[1];
      st.o[n][i][2] *= a[0];
      st.o[n][i][3] *= a[1];
    }
  }
}

// The weights' B fragments: parts of the 16-bit type, transposed from the C
// fragment [rows][queries] to [rows = k][queries = n]. bf16: their sum is the
// weight; f16: the first plus the second / kRestScale.
template <bool BF, int NT, int NP>
__device__ __forceinline__ void weight_parts(const float (&w)[NT][4], uint32_t (&b)[NT][NP][2]) {
  using namespace wmma16;
  constexpr float SCALE = BF ? 1.f : kRestScale;
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    float r0 = w[n][0], r1 = w[n][1], r2 = w[n][2], r3 = w[n][3];
#pragma unroll
    for (int k = 0; k < NP; ++k) {
      const uint32_t h01 = pack2<BF>(r0, r1), h23 = pack2<BF>(r2, r3);
      b[n][k][0] = movm_t(h01);
      b[n][k][1] = movm_t(h23);
      if (k + 1 < NP) {
        const float2 f01 = unpack2<BF>(h01), f23 = unpack2<BF>(h23);
        r0 = (r0 - f01.x) * SCALE;
        r1 = (r1 - f01.y) * SCALE;
        r2 = (r2 - f23.x) * SCALE;
        r3 = (r3 - f23.y) * SCALE;
      }
    }
  }
}

// o += a . (the weights' parts) for one output tile.
template <bool BF, int NP>
__device__ __forceinline__ void add_products(float (&o)[4], const uint32_t (&a)[4], const uint32_t (&b)[NP][2]) {
  using namespace wmma16;
  if constexpr (BF) {
#pragma unroll
    for (int j = 0; j < NP; ++j) mma<true>(o, a, b[j][0], b[j][1]);
  } else {
    static_assert(NP == 2, "a weight and its scaled rest");
    float rest[4] = {0.f, 0.f, 0.f, 0.f};
    mma<false>(rest, a, b[1][0], b[1][1]);
    mma<false>(o, a, b[0][0], b[0][1]);
#pragma unroll
    for (int e = 0; e < 4; ++e) o[e] = fmaf(rest[e], 1.f / kRestScale, o[e]);
  }
}

// Leaves a tile's scaled scores to the finishing kernel, two queries at a time.
// The column that pads an odd number of queries gets weight 0 whatever its
// product was (0 x infinity is NaN).
template <int NT>
__device__ __forceinline__ void store_scores(const float (&x)[NT][4], float* lg, int qns, int col0, int qn, int rem,
                                             int lane) {
  const int g = lane >> 2, c = lane & 3;
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    const int col = col0 + 8 * n + 2 * c;
    if (col < qn) {
      const bool pad = col + 1 == qn;
      float* at = lg + static_cast<int64_t>(g) * qns + col;
      if (g < rem) *reinterpret_cast<float2*>(at) = make_float2(x[n][0], pad ? kNegInf : x[n][1]);
      if (g + 8 < rem) *reinterpret_cast<float2*>(at + 8 * qns) = make_float2(x[n][2], pad ? kNegInf : x[n][3]);
    }
  }
}

// Clears the V rows at and behind rem (< 16) of a tile: they may hold anything,
// and 0 x NaN is NaN. The fence orders these writes before the copy that
// next fills the stage.
template <int BOXB, int HALVES>
__device__ __forceinline__ void clear_rows(uint32_t v, int rem, int lane) {
  constexpr int CH = BOXB / 16;
#pragma unroll 1
  for (int i = rem * CH + lane; i < kTileRows * CH; i += 32) {
#pragma unroll
    for (int h = 0; h < HALVES; ++h)
      asm volatile("st.shared.v4.u32 [%0], {%1, %1, %1, %1};" ::"r"(v + h * (kTileRows * BOXB) + i * 16), "r"(0u)
                   : "memory");
  }
  fence_proxy_async_smem();
  __syncwarp();
}

// Rows [r0, r1) of a tile's V, which some of the new tokens see and others do
// not: an infinity or NaN there would reach the latter too (0 x NaN), so it
// becomes 0 (give_odd_values gives it to the others). True if there was one.
// FIELD: the elements' exponents (e4m3: all but the sign), LOW: their lowest
// bits; a full field carries into its element's sign.
template <int BOXB, int HALVES, uint32_t FIELD, uint32_t LOW>
__device__ __forceinline__ bool clean_rows(uint32_t v, int r0, int r1, int lane) {
  constexpr int CH = BOXB / 16;
  constexpr uint32_t SIGN = FIELD + LOW, ELEM = SIGN == 0x80808080u ? 0xffu : 0xffffu;
  bool any = false;
#pragma unroll 2
  for (int i = r0 * CH + lane; i < r1 * CH; i += 32) {
#pragma unroll
    for (int h = 0; h < HALVES; ++h) {
      const uint32_t at = v + h * (kTileRows * BOXB) + i * 16;
      const uint4 u = wmma16::lds128(at);
      auto odd = [](uint32_t x) { return (((x & FIELD) + LOW) & SIGN) / (ELEM / 2 + 1) * ELEM; };
      const uint32_t a = odd(u.x), b = odd(u.y), c = odd(u.z), d = odd(u.w);
      if ((a | b | c | d) == 0) continue;
      any = true;
      asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(u.x & ~a), "r"(u.y & ~b), "r"(u.z & ~c),
                   "r"(u.w & ~d)
                   : "memory");
    }
  }
  any = __any_sync(0xffffffffu, any);
  if (any) {
    fence_proxy_async_smem();
    __syncwarp();
  }
  return any;
}

// Running softmax over one tile: x becomes the weights relative to the
// references (of the outputs), sums take the weights relative to m.
template <int D, int NT, bool ONE, bool BF>
__device__ __forceinline__ void softmax_step(float (&x)[NT][4], State<D, NT, ONE>& st, float lvs) {
  constexpr float ABOVE = Margin<BF>::kAbove;
  bool need = false;
#pragma unroll
  for (int n = 0; n < NT; ++n) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      need |= x[n][e] > st.m[n][e & 1] + ABOVE;
      if constexpr (ONE) need |= x[n][e] + lvs > st.mo[n][e & 1] + ABOVE;
    }
  }
  if (__any_sync(0xffffffffu, need)) raise_references<D, NT, ONE, BF>(x, st, lvs);
#pragma unroll
  for (int n = 0; n < NT; ++n) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float p = fast_exp2(x[n][e] - st.m[n][e & 1]);
      st.l[n][e & 1] += p;
      // one-byte caches: p * v_scale / 2^(mo - m), from its own exponent so
      // that neither factor can leave the range of fp32
      x[n][e] = ONE ? fast_exp2(x[n][e] + lvs - st.mo[ONE ? n : 0][e & 1]) : p;
    }
  }
}

// One 16-row tile of a 16-bit cache. k, v: the tile's boxes; rem: the
// sequence's rows from the tile's first on; edge: some query does not see all
// 16. (One body for both: small calls run every line once, and what they wait
// for then is instructions.)
template <bool BF, int D, int NT>
__device__ __forceinline__ void tile16(uint32_t k, uint32_t v, int rem, bool edge, float qscale, float* lg, int qns,
                                       int col0, int qn, State<D, NT, false>& st, int lane) {
  using namespace wmma16;
  constexpr int NP = BF ? 3 : 2;
  constexpr int CH = NT == 1 ? 4 : 2;  // independent accumulator chains
  constexpr uint32_t BOX = kTileRows * 128;
  const int g = lane >> 2, c = lane & 3;
  const int sw = lane & 7, s2 = sw >> 1;
  float x[NT][4];
  {
    float sc[NT][CH][4];
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int j = 0; j < CH; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) sc[n][j][e] = 0.f;
    // lane l addresses row (l & 7) + 8 ((l >> 3) & 1), dims chunk 2 ks + (l >> 4)
    const uint32_t row = k + static_cast<uint32_t>(((lane & 7) + ((lane >> 3) & 1) * 8) * 128) +
                         static_cast<uint32_t>((((lane >> 4) ^ sw) & 1) << 4);
#pragma unroll
    for (int ks = 0; ks < D / 16; ++ks) {
      uint32_t a[4];
      ldsm_x4(row + (ks >> 2) * BOX + static_cast<uint32_t>(((ks & 3) ^ s2) << 5), a);
#pragma unroll
      for (int n = 0; n < NT; ++n) mma<BF>(sc[n][ks % CH], a, st.q[n][ks][0], st.q[n][ks][1]);
    }
#pragma unroll
    for (int n = 0; n < NT; ++n) {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        float s = sc[n][0][e] + sc[n][1][e];
        if constexpr (CH == 4) s += sc[n][2][e] + sc[n][3][e];
        x[n][e] = s * qscale;
      }
    }
  }
  if (edge) {
    mask_edge<D, NT, false>(x, st, rem, g);
    if (rem < kTileRows) clear_rows<128, D / 64>(v, rem, lane);
  }
  if (lg != nullptr) store_scores<NT>(x, lg, qns, col0, qn, rem, lane);
  softmax_step<D, NT, false, BF>(x, st, 0.f);
  uint32_t b[NT][NP][2];
  weight_parts<BF, NT, NP>(x, b);
  // lane l addresses row (l & 7) + 8 (l >> 4), dims chunk 2 i + ((l >> 3) & 1)
  const uint32_t row = v + static_cast<uint32_t>(((lane & 7) + (lane >> 4) * 8) * 128) +
                       static_cast<uint32_t>(((((lane >> 3) & 1) ^ sw) & 1) << 4);
#pragma unroll
  for (int i = 0; i < D / 16; ++i) {
    uint32_t a[4];
    ldsm_x4_t(row + (i >> 2) * BOX + static_cast<uint32_t>(((i & 3) ^ s2) << 5), a);
#pragma unroll
    for (int n = 0; n < NT; ++n) add_products<BF, NP>(st.o[n][i], a, b[n]);
  }
}

// One 16-row tile of a one-byte cache (Q8 1: e4m3, 2: int8) whose block has
// the scales ks and vs.
//
// The order of the dims inside a product is free, so a lane takes whole
// 16-byte chunks: for S, lane 4g + c takes dims [D/4 of each 128] of rows g and
// g + 8 (k-step s uses 4 bytes: the MMA's k-columns 2c, 2c + 1, 2c + 8, 2c + 9);
// for PV, dims 16g .. 16g + 15 of every 128 (8g .. 8g + 7 of 64) of rows
// 2c, 2c + 1, 2c + 8, 2c + 9, and a byte permute pairs two rows of one dim. Output
// tile i of a span then holds its dims 16g + 2i and 16g + 2i + 1 (8g + 2i).
template <int Q8, int D, int NT>
__device__ __forceinline__ void tile8(uint32_t k, uint32_t v, int rem, bool edge, float ks, float vs, float* lg,
                                      int qns, int col0, int qn, State<D, NT, true>& st, int lane) {
  using namespace wmma16;
  constexpr int NP = 2;
  constexpr int CH = NT == 1 ? 4 : 2;
  constexpr int BOXB = D < 128 ? D : 128;
  constexpr int SPANS = D / BOXB;
  constexpr int KS = BOXB / 16;  // k-steps (and output tiles) per span
  constexpr uint32_t BOX = kTileRows * BOXB;
  const int g = lane >> 2, c = lane & 3;
  float x[NT][4];
  {
    float sc[NT][CH][4];
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int j = 0; j < CH; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) sc[n][j][e] = 0.f;
#pragma unroll
    for (int sp = 0; sp < SPANS; ++sp) {
      uint32_t kw[2][KS];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
#pragma unroll
        for (int j = 0; j < KS / 4; ++j) {
          const uint4 u = lds128(k + sp * BOX + chunk_at<BOXB>(g + 8 * h, (KS / 4) * c + j));
          kw[h][4 * j] = u.x;
          kw[h][4 * j + 1] = u.y;
          kw[h][4 * j + 2] = u.z;
          kw[h][4 * j + 3] = u.w;
        }
      }
#pragma unroll
      for (int s = 0; s < KS; ++s) {
        uint32_t a[4];
        codes_to_f16x2<Q8>(kw[0][s], a[0], a[2]);
        codes_to_f16x2<Q8>(kw[1][s], a[1], a[3]);
#pragma unroll
        for (int n = 0; n < NT; ++n) mma<false>(sc[n][s % CH], a, st.q[n][sp * KS + s][0], st.q[n][sp * KS + s][1]);
      }
    }
#pragma unroll
    for (int n = 0; n < NT; ++n) {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        float s = sc[n][0][e] + sc[n][1][e];
        if constexpr (CH == 4) s += sc[n][2][e] + sc[n][3][e];
        x[n][e] = s * (st.fq[n][e & 1] * ks);
      }
    }
  }
  if (edge) {
    mask_edge<D, NT, true>(x, st, rem, g);
    if (rem < kTileRows) clear_rows<BOXB, SPANS>(v, rem, lane);
  }
  if (lg != nullptr) store_scores<NT>(x, lg, qns, col0, qn, rem, lane);
  softmax_step<D, NT, true, false>(x, st, fast_log2(vs));
  uint32_t b[NT][NP][2];
  weight_parts<false, NT, NP>(x, b);
#pragma unroll
  for (int sp = 0; sp < SPANS; ++sp) {
    uint32_t vw[4][KS / 2];  // rows 2c, 2c + 1, 2c + 8, 2c + 9
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int r = 2 * c + (j & 1) + 8 * (j >> 1);
      if constexpr (BOXB == 128) {
        const uint4 u = lds128(v + sp * BOX + chunk_at<BOXB>(r, g));
        vw[j][0] = u.x;
        vw[j][1] = u.y;
        vw[j][2] = u.z;
        vw[j][3] = u.w;
      } else {
        const uint2 u = lds64(v + chunk_at<BOXB>(r, g >> 1) + 8 * (g & 1));
        vw[j][0] = u.x;
        vw[j][1] = u.y;
      }
    }
#pragma unroll
    for (int i = 0; i < KS; ++i) {
      // bytes 2 (i & 1) and + 1 of word i >> 1 of two rows, interleaved
      const uint32_t sel = (i & 1) ? 0x7362u : 0x5140u;
      uint32_t a[4];
      codes_to_f16x2<Q8>(__byte_perm(vw[0][i >> 1], vw[1][i >> 1], sel), a[0], a[1]);
      codes_to_f16x2<Q8>(__byte_perm(vw[2][i >> 1], vw[3][i >> 1], sel), a[2], a[3]);
#pragma unroll
      for (int n = 0; n < NT; ++n) add_products<false, NP>(st.o[n][sp * KS + i], a, b[n]);
    }
  }
}

// The MMA column (query) g of column group n: its row of q and whether it exists.
__device__ __forceinline__ int64_t query_row(const ScoredParams& p, int seq, int kvh, int v) {
  const int t = v / p.group;
  return (static_cast<int64_t>(seq) * p.n_tok + t) * p.n_q_heads + kvh * p.group + (v - t * p.group);
}

// Rows of a sequence that are cached, 0 if its length is invalid.
__device__ __forceinline__ int valid_rows(const ScoredParams& p, int b) {
  const int n = __ldg(p.context_lens + b);
  return (n < p.n_tok || n > p.rows) ? 0 : n;
}

__device__ __forceinline__ int tiles_of(int rows) { return (rows + kTileRows - 1) / kTileRows; }

// Exclusive prefix sums of the sequences' tiles into s_scan[0 .. batch]; the
// whole CTA takes part. s_scan has batch + 33 entries.
__device__ inline void scan_tiles(const ScoredParams& p, int* s_scan) {
  const int tid = threadIdx.x, nt = blockDim.x, lane = tid & 31, wid = tid >> 5, B = p.batch;
  const int per = (B + nt - 1) / nt;
  const int b0 = min(B, tid * per), b1 = min(B, b0 + per);
  int local = 0;
  for (int b = b0; b < b1; ++b) local += tiles_of(valid_rows(p, b));
  int v = local;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int u = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += u;
  }
  int* wsum = s_scan + B + 1;
  if (lane == 31) wsum[wid] = v;
  __syncthreads();
  int run = v - local;
  for (int i = 0; i < wid; ++i) run += wsum[i];
  for (int b = b0; b < b1; ++b) {
    s_scan[b] = run;
    run += tiles_of(valid_rows(p, b));
    if (b == B - 1) s_scan[B] = run;
  }
  __syncthreads();
}

// n / d for d >= 1 from m = magic(d): exact while n * d < 2^32.
__device__ __forceinline__ uint32_t magic(uint32_t d) { return d == 1 ? 0u : 0xffffffffu / d + 1u; }
__device__ __forceinline__ int divided(int n, uint32_t m) {
  return m == 0u ? n : static_cast<int>(__umulhi(static_cast<uint32_t>(n), m));
}

// Tiles of the work: positions [0, N) in equal ranges, the first `rest` of
// them one longer. All positions are below 2^31 (checked on the host).
struct Split {
  int per, rest;
  __device__ __forceinline__ int start(int wk) const { return wk * per + min(wk, rest); }
  __device__ __forceinline__ int holder(int pos) const {
    const int longer = rest * (per + 1);
    return pos < longer ? pos / (per + 1) : rest + (pos - longer) / per;
  }
};

// A (sequence, kv head, column group) and its tiles [u0, u0 + tiles).
struct Unit {
  int u0, seq, kvh, hsub, tiles;
};

// Rows and tiles of the sequences and where their units lie. Up to 32
// sequences sit in the lanes of every warp (no barrier, no search); more in
// shared memory, as prefix sums.
struct Batch {
  int rows, tiles, before;  // of sequence `lane`; before: tiles of the sequences before it
  int total;
  const int* s_scan;  // NULL: in the lanes
  __device__ __forceinline__ Unit locate(int pos, const ScoredParams& p) const {
    const int HN = p.n_kv_heads * p.n_hsub;
    Unit u;
    int first;
    if (s_scan == nullptr) {
      // the last sequence whose first tile is <= pos (skips empty ones)
      const bool below = static_cast<int>(threadIdx.x & 31) < p.batch && HN * before <= pos;
      u.seq = 31 - __clz(__ballot_sync(0xffffffffu, below));
      u.tiles = __shfl_sync(0xffffffffu, tiles, u.seq);
      first = HN * __shfl_sync(0xffffffffu, before, u.seq);
    } else {
      int a = 0, hi = p.batch - 1;
      while (a < hi) {
        const int mid = (a + hi + 1) >> 1;
        if (HN * s_scan[mid] <= pos) a = mid; else hi = mid - 1;
      }
      u.seq = a;
      u.tiles = s_scan[a + 1] - s_scan[a];
      first = HN * s_scan[a];
    }
    const int idx = static_cast<int>(static_cast<uint32_t>(pos - first) / static_cast<uint32_t>(u.tiles));
    u.kvh = p.n_hsub == 1 ? idx : idx / p.n_hsub;
    u.hsub = idx - u.kvh * p.n_hsub;
    u.u0 = first + idx * u.tiles;
    return u;
  }
  __device__ __forceinline__ int rows_of(int seq, const ScoredParams& p) const {
    return s_scan == nullptr ? __shfl_sync(0xffffffffu, rows, seq) : valid_rows(p, seq);
  }
};

// Dim of o[.][i][0 and 1] in the lanes with lane / 4 = g; that of [2 and 3] is
// 8 behind it (16-bit caches) or 1 (one-byte caches).
template <int D, bool ONE>
__device__ __forceinline__ int out_dim(int i, int g) {
  constexpr int BOXB = D < 128 ? D : 128;
  constexpr int KS = BOXB / 16;
  return ONE ? (i / KS) * BOXB + (BOXB / 8) * g + 2 * (i % KS) : 16 * i + g;
}

// An infinity or NaN in V becomes the output of the queries that see its row,
// as sum_r p_r v_r has it (p_r > 0), but the products cannot give that: a
// weight's parts may be 0 or negative, and 0 x infinity is NaN. So where a
// segment met one, its rows [r0, r1) are searched once more and what is found
// (the sum of all: infinities of both signs make NaN) replaces the outputs of
// the queries `cols` (bits), written before: part [8 NT, D], or p.out if NULL.
// Rare, and out of the main loop's registers.
template <typename CT, int D>
__device__ __noinline__ void give_odd_values(const ScoredParams& p, int seq, int kvh, int col0, uint32_t cols,
                                             int n_rows, int r0, int r1, float* part) {
  constexpr int PER = D / 32;  // dims per lane: lane, lane + 32, ..
  const int lane = threadIdx.x & 31;
  auto search = [&](int from, int to, float (&z)[PER]) {
#pragma unroll 1
    for (int r = from; r < to; ++r) {
      const int b = r / p.block_size;
      const int phys = __ldg(p.block_tables + static_cast<int64_t>(seq) * p.max_blocks + b);
      if (phys < 0 || phys >= p.num_blocks) continue;
      const int64_t at = (static_cast<int64_t>(phys) * p.n_kv_heads + kvh) * p.block_size + (r - b * p.block_size);
      const CT* row = static_cast<const CT*>(p.v_cache) + at * D + lane;
#pragma unroll
      for (int i = 0; i < PER; ++i) {
        float y = 0.f;
        if constexpr (sizeof(CT) == 1) {  // e4m3 has a NaN and no infinity
          if ((__ldg(reinterpret_cast<const unsigned char*>(row + 32 * i)) & 0x7f) == 0x7f)
            y = __int_as_float(0x7fffffff);
        } else {
          y = wmma16::unpack2<std::is_same<CT, __nv_bfloat16>::value>(
                  __ldg(reinterpret_cast<const unsigned short*>(row + 32 * i))).x;
        }
        if (!(fabsf(y) < __builtin_huge_valf())) z[i] += y;
      }
    }
  };
  const int shared_rows = n_rows - p.n_tok + 1;  // rows that all tokens see
  float all[PER];
#pragma unroll
  for (int i = 0; i < PER; ++i) all[i] = 0.f;
  search(r0, min(r1, shared_rows), all);
#pragma unroll 1
  for (; cols != 0; cols &= cols - 1) {
    const int col = __ffs(cols) - 1, v = col0 + col, t = v / p.group;
    float z[PER];
#pragma unroll
    for (int i = 0; i < PER; ++i) z[i] = all[i];
    search(max(r0, shared_rows), min(r1, shared_rows + t), z);
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      if (z[i] == 0.f) continue;
      if (part != nullptr)
        part[col * D + lane + 32 * i] = z[i];
      else
        store_out(p.out, query_row(p, seq, kvh, v) * D + lane + 32 * i, z[i], p.out_dtype);
    }
  }
}

// The weight of a record relative to the largest one. Not below the smallest
// normal number, which changes no finite sum and keeps an infinity.
__device__ __forceinline__ float record_weight(float m, float largest) {
  return fmaxf(fast_exp2(m - largest), 1.17549435e-38f);
}

}  // namespace scored

// SHUT: rows of the last tokens are searched for infinities and NaN, which
// earlier tokens do not see (several new tokens; other calls are spared the code).
template <typename CT, int D, int NT, bool SHUT>
__global__ void __launch_bounds__(ScoredGeo<sizeof(CT), D, NT>::kThreads, 1)
    scored_decode_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                         const __grid_constant__ ScoredParams p) {
  using namespace scored;
  constexpr bool ONE = sizeof(CT) == 1;
  constexpr bool BF = std::is_same<CT, __nv_bfloat16>::value;
  constexpr int Q8 = std::is_same<CT, fp8e4m3>::value ? 1 : 2;
  using G = ScoredGeo<sizeof(CT), D, NT>;
  constexpr int TS = G::kStageTiles, S = G::kStages, W = G::kWarps, NC = 8 * NT;
  constexpr uint32_t full = 0xffffffffu;
  static_assert(static_cast<size_t>(S) * G::kStageBytes >= (D + 2) * NC * 4, "a warp's part fits its ring");
  __shared__ int s_held[W];
  extern __shared__ unsigned char smem_raw[];
  const uint32_t raw = smem_addr(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  unsigned char* smem = smem_raw + (base - raw);
  const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + G::kRingBytes) + w * S;
  float* s_scale = reinterpret_cast<float*>(smem + G::kRingBytes + W * S * 8) + w * S * TS * 2;
  int* s_scan = reinterpret_cast<int*>(smem + G::kRingBytes + W * S * 8 + W * S * TS * 2 * 4);
  const uint32_t ring = base + static_cast<uint32_t>(w * S * G::kStageBytes);

  if (lane < S) mbar_init(bars + lane, 1);
  fence_barrier_init();
  if (tid == 0) {
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&tm_k)) : "memory");
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&tm_v)) : "memory");
  }
  __syncwarp();
  // The kernel may start while the stream's previous one runs; nothing of the
  // caller's is read or written before that one has ended.
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  // Small calls spend their time in this prologue (11000 cycles before it was
  // cut down): no barrier for up to 32 sequences, 32-bit positions, one copy of
  // each piece of code.
  Batch bt;
  if (p.batch <= 32) {
    bt.s_scan = nullptr;
    bt.rows = lane < p.batch ? valid_rows(p, lane) : 0;
    bt.tiles = tiles_of(bt.rows);
    int v = bt.tiles;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int x = __shfl_up_sync(full, v, o);
      if (lane >= o) v += x;
    }
    bt.before = v - bt.tiles;
    bt.total = __shfl_sync(full, v, 31);
  } else {
    scan_tiles(p, s_scan);  // ends with a CTA barrier
    bt.s_scan = s_scan;
    bt.rows = bt.tiles = bt.before = 0;
    bt.total = s_scan[p.batch];
  }

  // Sequences of invalid length: flagged, their units marked for zero outputs.
  const int HN = p.n_kv_heads * p.n_hsub;
  for (int b = blockIdx.x * blockDim.x + tid; b < p.batch; b += gridDim.x * blockDim.x) {
    if (valid_rows(p, b) == 0) {
      set_flag(p.err, KVC_FLAG_BAD_LEN);
      for (int i = 0; i < HN; ++i) p.units[static_cast<int64_t>(b) * HN + i] = make_int4(kUnitEmpty, 0, 0, 0);
    }
  }

  const int N = HN * bt.total;
  if (N == 0) return;
  const int We = min(static_cast<int>((static_cast<uint32_t>(N) + p.min_tiles - 1) / p.min_tiles), p.workers);
  // K workers per CTA, so that few workers spread over all SMs
  const int K = static_cast<int>((We + gridDim.x - 1) / gridDim.x);
  const int wk = static_cast<int>(blockIdx.x) * K + w;
  const bool works = w < K && wk < We;
  // Merging the CTA's parts costs every CTA a barrier and about 2 us at its
  // end; it pays where a query would otherwise have many records to merge
  // (e4m3, one sequence of 131071 rows: 77 -> 69 us; batch 32 x U[512, 4096],
  // seven records each: 37 -> 39 us).
  const bool merge = K > 1 && We > 16 * p.batch * HN;
  if (!works && !merge) return;
  Split sp;
  sp.per = N / We;
  sp.rest = N - sp.per * We;
  const int lo = works ? sp.start(wk) : 0, hi = works ? sp.start(wk + 1) : 0;
  const uint32_t tpb = p.block_size / kTileRows;  // tiles per cache block
  const uint32_t m_tpb = magic(tpb), m_group = magic(p.group);
  const uint64_t pol = policy_evict_first();

  // ---- copies: the next tiles of the range into the next stage
  int ipos = lo, iend = lo;
  int ij = 0, iseq = 0, ikvh = 0, wb = 0, tw = -1;
  uint32_t islot = 0, ivalid = 0;  // ivalid: bit slot * TS + t: the tile's block is inside the pool
  int issued = 0;
  auto issue = [&]() {
    if (ipos < hi) {
      if (ipos >= iend) {
        const Unit u = bt.locate(ipos, p);
        iseq = u.seq;
        ikvh = u.kvh;
        ij = ipos - u.u0;
        iend = min(u.u0 + u.tiles, hi);
        wb = -64;  // no entries yet
      }
      const int cnt = min(iend - ipos, TS);
      const int b_last = divided(ij + cnt - 1, m_tpb);
      if (b_last >= wb + 32) {  // lane i holds the table's entry wb + i
        wb = divided(ij, m_tpb);
        tw = wb + lane < p.max_blocks ? __ldg(p.block_tables + static_cast<int64_t>(iseq) * p.max_blocks + wb + lane)
                                      : -1;
      }
      // lane i copies box i: [tile][K or V][half]
      constexpr int PER = 2 * G::kHalves;
      const int t = lane / PER < cnt ? lane / PER : 0;
      const int jt = ij + t, blk = divided(jt, m_tpb);
      const int phys = __shfl_sync(full, tw, blk - wb);
      const bool ok = phys >= 0 && phys < p.num_blocks;
      uint32_t mask = 0;
#pragma unroll
      for (int i = 0; i < TS; ++i)
        if (i < cnt) mask |= (__shfl_sync(full, ok ? 1u : 0u, i * PER)) << i;
      ivalid = (ivalid & ~(((1u << TS) - 1u) << (islot * TS))) | (mask << (islot * TS));
      uint64_t* bar = bars + islot;
      if (lane == 0) {
        if (mask == 0)
          mbar_arrive(bar);
        else
          mbar_arrive_expect_tx(bar, __popc(mask) * 2 * G::kTileBytes);
        if (__popc(mask) != cnt) set_flag(p.err, KVC_FLAG_BAD_BLOCK);
      }
      __syncwarp();
      if (lane < PER * cnt && ok) {
        const int kv = (lane % PER) / G::kHalves, half = lane % G::kHalves;
        const int y = (phys * p.n_kv_heads + ikvh) * p.block_size + (jt - blk * static_cast<int>(tpb)) * kTileRows;
        const uint32_t dst = ring + islot * G::kStageBytes + (t * 2 + kv) * G::kTileBytes +
                             half * (kTileRows * G::kBoxBytes);
        wmma16::tma2d(dst, kv == 0 ? &tm_k : &tm_v, half * (G::kBoxBytes / static_cast<int>(sizeof(CT))), y,
                      smem_addr(bar), pol);
      }
      if constexpr (ONE) {
        // lane i copies scale i: [tile][K or V]
        const int t2 = (lane >> 1) < cnt ? lane >> 1 : 0;
        const int phys2 = __shfl_sync(full, tw, divided(ij + t2, m_tpb) - wb);
        if (lane < 2 * cnt && phys2 >= 0 && phys2 < p.num_blocks)
          cp_async4(smem_addr(s_scale + (islot * TS + t2) * 2 + (lane & 1)),
                    ((lane & 1) ? p.v_scale : p.k_scale) + static_cast<int64_t>(phys2) * p.n_kv_heads + ikvh);
      }
      ipos += cnt;
      ij += cnt;
      ++issued;
      islot = islot + 1 == S ? 0 : islot + 1;
    }
    if constexpr (ONE) cp_async_commit();  // one group per call, whether or not it copied
  };

  // ---- products, stage by stage; a segment is one unit's tiles in the range
  uint32_t slot = 0, ph = 0;
  int used = 0, ahead = 0;  // stages released; issue() calls ahead of the next one to use
  bool ok = true;
  int held = -1;  // the unit of the part at the range's end
  const int lanes_g = lane >> 2, c = lane & 3;
  State<D, NT, ONE> st;
  Unit u{};
  int end = lo, n_rows = 0, col0 = 0, j = 0;
  int shared_rows = 0;  // rows that all tokens see
  bool odd = false;     // this segment met an infinity or NaN in V
  float* lg0 = nullptr;
#pragma unroll 1
  for (int pos = lo; pos < hi;) {
#pragma unroll 1
    for (; ahead < S; ++ahead) issue();
    if (pos == end) {  // a new segment
      u = bt.locate(pos, p);
      end = min(u.u0 + u.tiles, hi);
      n_rows = bt.rows_of(u.seq, p);
      shared_rows = n_rows - p.n_tok + 1;
      col0 = u.hsub * NC;
      j = pos - u.u0;
      lg0 = p.scores == nullptr
                ? nullptr
                : p.logits + (static_cast<int64_t>(u.seq) * p.n_kv_heads + u.kvh) * p.rows * p.qns;
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        // ---- Q^T fragments of query g (columns past the last query: zeros)
        const int v = col0 + 8 * n + lanes_g;
        const bool have = v < p.qn;
        const int tq = divided(v, m_group);
        const int64_t qrow =
            (static_cast<int64_t>(u.seq) * p.n_tok + tq) * p.n_q_heads + u.kvh * p.group + v - tq * p.group;
        const unsigned short* qr = static_cast<const unsigned short*>(p.q) + (have ? qrow * D : 0);
        if constexpr (!ONE) {
#pragma unroll
          for (int ks = 0; ks < D / 16; ++ks) {
#pragma unroll
            for (int h = 0; h < 2; ++h)
              st.q[n][ks][h] = have ? __ldg(reinterpret_cast<const uint32_t*>(qr + 16 * ks + 8 * h + 2 * c)) : 0u;
          }
        } else {
          // dims of lane c, k-step s of a span: 4 s .. 4 s + 3 of its part; scaled
          // by 2^t so that the query's largest entry lies in [2^14, 2^15): entries
          // down to 2^-31 (bf16; f16: 2^-28) of it are exact in f16, smaller ones are
          // off by at most 2^-39 of it
          constexpr int BOXB = D < 128 ? D : 128;
          constexpr int KS = BOXB / 16;
          float y[D / 16][4];
          float amax = 0.f;
#pragma unroll
          for (int s = 0; s < D / 16; ++s) {
            const int d = (s / KS) * BOXB + (BOXB / 4) * c + 4 * (s % KS);
            uint2 u2 = make_uint2(0u, 0u);
            if (have) u2 = __ldg(reinterpret_cast<const uint2*>(qr + d));
            float2 a, b;
            if (p.q_f16) {
              a = wmma16::unpack2<false>(u2.x);
              b = wmma16::unpack2<false>(u2.y);
            } else {
              a = wmma16::unpack2<true>(u2.x);
              b = wmma16::unpack2<true>(u2.y);
            }
            y[s][0] = a.x;
            y[s][1] = a.y;
            y[s][2] = b.x;
            y[s][3] = b.y;
#pragma unroll
            for (int e = 0; e < 4; ++e) amax = fmaxf(amax, fabsf(y[s][e]));
          }
          amax = fmaxf(amax, __shfl_xor_sync(full, amax, 1));
          amax = fmaxf(amax, __shfl_xor_sync(full, amax, 2));
          const int field = min(253, max(1, 268 - static_cast<int>((__float_as_uint(amax) >> 23) & 0xffu)));
          const float up = __uint_as_float(static_cast<uint32_t>(field) << 23);
          const float down = p.qscale * __uint_as_float(static_cast<uint32_t>(254 - field) << 23);
#pragma unroll
          for (int s = 0; s < D / 16; ++s) {
            st.q[n][s][0] = wmma16::pack2<false>(y[s][0] * up, y[s][1] * up);
            st.q[n][s][1] = wmma16::pack2<false>(y[s][2] * up, y[s][3] * up);
          }
          st.fq[n][0] = __shfl_sync(full, down, 8 * c);      // of query 2c, held by the lanes with g = 2c
          st.fq[n][1] = __shfl_sync(full, down, 8 * c + 4);  // of query 2c + 1
        }
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          st.m[n][e] = -1e30f;  // finite: a query that meets only masked rows keeps weight 0
          st.l[n][e] = 0.f;
          if constexpr (ONE) st.mo[n][e] = -1e30f;
          const int t = divided(col0 + 8 * n + 2 * c + e, m_group);
          st.dt[n][e] = t < p.n_tok ? p.n_tok - 1 - t : 0;
        }
#pragma unroll
        for (int i = 0; i < D / 16; ++i) {
#pragma unroll
          for (int e = 0; e < 4; ++e) st.o[n][i][e] = 0.f;
        }
      }
    }
    const int cnt = min(end - pos, TS);
    ok = mbar_wait_data(bars + slot, ph, p.wait_polls);
    ok = __all_sync(full, ok);
    if (!ok) break;
    if constexpr (ONE) {
      cp_async_wait<S - 1>();
      __syncwarp();
    }
    if constexpr (SHUT) {
      if ((j + cnt) * kTileRows > shared_rows) {
        constexpr uint32_t FIELD = ONE ? 0x7f7f7f7fu : BF ? 0x7f807f80u : 0x7c007c00u;
        constexpr uint32_t LOW = ONE ? 0x01010101u : BF ? 0x00800080u : 0x04000400u;
#pragma unroll 1
        for (int t = 0; t < cnt; ++t) {
          const int r0 = (j + t) * kTileRows;
          if ((ivalid >> (slot * TS + t)) & 1u)
            odd |= clean_rows<G::kBoxBytes, G::kHalves, FIELD, LOW>(
                ring + slot * G::kStageBytes + (2 * t + 1) * G::kTileBytes, max(shared_rows - r0, 0),
                min(n_rows - r0, kTileRows), lane);
        }
      }
    }
#pragma unroll 1
    for (int t = 0; t < cnt; ++t) {
      const int r0 = (j + t) * kTileRows;
      const int rem = n_rows - r0;
      float* lg = lg0 == nullptr ? nullptr : lg0 + static_cast<int64_t>(r0) * p.qns;
      const uint32_t kt = ring + slot * G::kStageBytes + t * 2 * G::kTileBytes, vt = kt + G::kTileBytes;
      if ((ivalid >> (slot * TS + t)) & 1u) {
        const bool edge = rem < kTileRows + p.n_tok - 1;
        if constexpr (ONE) {
          const float* sc = s_scale + (slot * TS + t) * 2;
          tile8<Q8, D, NT>(kt, vt, rem, edge, sc[0], sc[1], lg, p.qns, col0, p.qn, st, lane);
        } else {
          tile16<BF, D, NT>(kt, vt, rem, edge, p.qscale, lg, p.qns, col0, p.qn, st, lane);
        }
      } else if (lg != nullptr) {  // a block outside the pool: its rows get no weight
        const int cols = min(NC, p.qns - col0);
        for (int i = lane; i < min(rem, kTileRows) * cols; i += 32)
          lg[static_cast<int64_t>(i / cols) * p.qns + col0 + i % cols] = kNegInf;
      }
    }
    __syncwarp();  // every lane has read the stage
    slot = slot + 1 == S ? 0 : slot + 1;
    if (slot == 0) ph ^= 1u;
    ++used;
    --ahead;
    pos += cnt;
    j += cnt;
    if (pos < end) continue;

    // ---- close the segment. A whole unit: its outputs. A part that ends
    // inside the range (the unit began in an earlier worker's): record 2 wk.
    // The part at the range's end: merged with its neighbours' below.
    const int begin = max(u.u0, lo);
    const int64_t unit = (static_cast<int64_t>(u.seq) * p.n_kv_heads + u.kvh) * p.n_hsub + u.hsub;
    const bool whole = begin == u.u0 && pos == u.u0 + u.tiles;
    if (lane == 0 && begin == u.u0) {
      int4 info = make_int4(kUnitWhole, 0, 0, 0);
      if (!whole) {
        const int last = u.u0 + u.tiles;  // behind its last tile
        const int c1 = sp.holder(last - 1);
        info = make_int4(wk, c1, last < sp.start(c1 + 1) ? 1 : 0, merge ? K : 1);
      }
      p.units[unit] = info;
    }
    // The part at the range's end goes to this warp's ring (all its copies have
    // landed) if it is to be merged.
    const bool last_part = !whole && pos == hi, keep = last_part && merge;
    float* so = reinterpret_cast<float*>(smem + static_cast<size_t>(w) * S * G::kStageBytes);
    const int64_t rec = 2ll * wk + (last_part ? 1 : 0);
    if (keep) __syncwarp();
    auto dim = [&](int i) { return out_dim<D, ONE>(i, lanes_g); };
    constexpr int SECOND = ONE ? 1 : 8;
#pragma unroll
    for (int n = 0; n < NT; ++n) {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float l = st.l[n][e];
#pragma unroll
        for (int msk = 4; msk < 32; msk <<= 1) l += __shfl_xor_sync(full, l, msk);
        const int col = 8 * n + 2 * c + e, v = col0 + col;
        if (v >= p.qn) continue;
        float f = 1.f;
        if constexpr (ONE) f = fast_exp2(st.mo[n][e] - st.m[n][e]);
        if (!whole) {
          float* ro = keep ? so + col * D : p.rec_o + (rec * NC + col) * D;
          float* ml = keep ? so + NC * D + 2 * col : p.rec_ml + (rec * NC + col) * 2;
#pragma unroll
          for (int i = 0; i < D / 16; ++i) {
            ro[dim(i)] = st.o[n][i][e] * f;
            ro[dim(i) + SECOND] = st.o[n][i][e + 2] * f;
          }
          if (lanes_g == 0) *reinterpret_cast<float2*>(ml) = make_float2(st.m[n][e], l);
          continue;
        }
        const int64_t row = query_row(p, u.seq, u.kvh, v);
        const float inv = l == 0.f ? 0.f : f / l;
        if (p.out_dtype == KVC_F32) {
          float* to = static_cast<float*>(p.out) + row * D;
#pragma unroll
          for (int i = 0; i < D / 16; ++i) {
            to[dim(i)] = st.o[n][i][e] * inv;
            to[dim(i) + SECOND] = st.o[n][i][e + 2] * inv;
          }
        } else {
          unsigned short* to = static_cast<unsigned short*>(p.out) + row * D;
          const bool f16 = p.out_dtype == KVC_F16;
#pragma unroll
          for (int i = 0; i < D / 16; ++i) {
            const float a = st.o[n][i][e] * inv, b = st.o[n][i][e + 2] * inv;
            const uint32_t x = f16 ? wmma16::pack2<false>(a, b) : wmma16::pack2<true>(a, b);
            to[dim(i)] = static_cast<unsigned short>(x);
            to[dim(i) + SECOND] = static_cast<unsigned short>(x >> 16);
          }
        }
        if (p.scores != nullptr && lanes_g == 0) p.lse[row] = st.m[n][e] + fast_log2(l);
      }
    }
    if constexpr (!ONE || SHUT) {
      if constexpr (!ONE) {
        float zero = 0.f;  // NaN if an output is not finite
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int i = 0; i < D / 16; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) zero = fmaf(st.o[n][i][e], 0.f, zero);
        odd |= __any_sync(full, zero != 0.f);
      }
      if (odd) {
        // queries without weight here, or whose weights are not finite, keep what the products gave
        uint32_t cols = 0;
#pragma unroll
        for (int n = 0; n < NT; ++n) {
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float l = st.l[n][e];
#pragma unroll
            for (int msk = 4; msk < 32; msk <<= 1) l += __shfl_xor_sync(full, l, msk);
            const uint32_t has = __ballot_sync(full, l > 0.f && l < __builtin_huge_valf() &&
                                                         col0 + 8 * n + 2 * c + e < p.qn);
#pragma unroll
            for (int k = 0; k < 4; ++k) cols |= ((has >> k) & 1u) << (8 * n + 2 * k + e);
          }
        }
        __syncwarp();  // the segment's outputs have been written
        if (cols != 0)
          give_odd_values<CT, D>(p, u.seq, u.kvh, col0, cols, n_rows, (begin - u.u0) * kTileRows,
                                 min(n_rows, (pos - u.u0) * kTileRows),
                                 whole ? nullptr : keep ? so : p.rec_o + rec * NC * D);
        odd = false;
      }
    }
    if (keep) held = static_cast<int>(unit);
  }
  if (!ok) {
    // Gave up: report it and wait (bounded) for this warp's own copies still in
    // flight, so that shared memory is not reused under them.
    if (lane == 0) set_flag(p.err, KVC_FLAG_TIMEOUT);
    for (; used < issued; ++used) {
      (void)mbar_wait_bounded(bars + slot, ph);
      slot = slot + 1 == S ? 0 : slot + 1;
      if (slot == 0) ph ^= 1u;
    }
  }
  if constexpr (ONE) cp_async_wait<0>();

  // ---- merge the parts at the ends of the CTA's ranges: neighbouring warps
  // that hold the same unit leave one record, 2 (first warp's worker) + 1
  if (!merge) return;  // the same in every warp of the grid
  if (lane == 0) s_held[w] = held;
  __syncthreads();
  for (int a = 0; a < K;) {
    const int unit = s_held[a];
    int b = a + 1;
    while (b < K && s_held[b] == unit) ++b;
    if (unit >= 0) {
      const int64_t rec = 2 * (static_cast<int64_t>(blockIdx.x) * K + a) + 1;
      const int cols = min(NC, p.qn - (unit % p.n_hsub) * NC);
      auto part = [&](int i) {
        return reinterpret_cast<const float*>(smem + static_cast<size_t>(i) * S * G::kStageBytes);
      };
      for (int i = tid; i < cols * (D / 4); i += G::kThreads) {
        const int col = i / (D / 4), d = 4 * (i % (D / 4));
        float m = kNegInf;
        for (int x = a; x < b; ++x) m = fmaxf(m, part(x)[NC * D + 2 * col]);
        float l = 0.f;
        float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int x = a; x < b; ++x) {
          const float f = record_weight(part(x)[NC * D + 2 * col], m);
          const float4 y = *reinterpret_cast<const float4*>(part(x) + col * D + d);
          l += f * part(x)[NC * D + 2 * col + 1];
          o.x += f * y.x;
          o.y += f * y.y;
          o.z += f * y.z;
          o.w += f * y.w;
        }
        *reinterpret_cast<float4*>(p.rec_o + (rec * NC + col) * D + d) = o;
        if (d == 0) *reinterpret_cast<float2*>(p.rec_ml + (rec * NC + col) * 2) = make_float2(m, l);
      }
    }
    a = b;
  }
}

// ------------------------------------------------------------------ finish
//
// One grid column (blockIdx.x) per unit of (sequence, kv head). The first
// out_ctas CTAs of a column share the unit's queries: o_v = sum_r 2^(m_r - M)
// O_r / sum_r 2^(m_r - M) l_r over the records r of v, one warp per query while
// a warp's lanes hold its records, the whole CTA beyond. The others share its
// rows: score += sum_v 2^(x - lse_v), lanes over the queries of a row, in a
// fixed order. Every step loads what it needs at once: bound by the scores' and
// logits' bytes (which mostly sit in L2), for small calls by the chain unit ->
// maxima -> outputs, or logits, of three loads: 5 us for a few short sequences,
// about 8 us behind the decode for 32 x 4096 rows of 4 queries (25 MB; 13 us alone).
constexpr int kFinishThreads = 256;
constexpr int kFinishWarps = kFinishThreads / 32;
// cached rows a CTA takes at least: about 4 KB of scores, 16 KB of wide rows
__host__ __device__ inline int finish_rows(int qns) { return qns <= 8 ? 256 : qns <= 32 ? 128 : 64; }
constexpr int kFewRecords = 16;
constexpr int kFinishCtas = 4 * 152;  // what the GPU holds at once, about

// Records of a query's unit: one per CTA from CTA `cta` on, left by the first
// of its workers that held the unit's end of range, then perhaps the last worker's own.
struct RecList {
  int first, cta, K, merged, n, last;
};
__device__ __forceinline__ RecList record_list(const int4 u, int workers) {
  RecList r;
  r.n = 0;
  // entries outside the workspace (left by a call that gave up) are not followed
  if (u.x < 0 || u.y < u.x || u.y >= workers || u.w < 1 || u.w > 32) return r;
  r.first = u.x;
  r.last = u.y;
  r.K = u.w;
  r.cta = u.x / u.w;
  const int end = u.y / u.w;
  r.merged = end - r.cta + 1;
  // the last worker's part is a record of its own: none from its CTA if it comes first there
  if (u.z != 0 && max(u.x, end * u.w) == u.y) --r.merged;
  r.n = r.merged + (u.z != 0 ? 1 : 0);
  return r;
}
__device__ __forceinline__ int64_t record_slot(const RecList& r, int i) {
  return i < r.merged ? 2ll * max(r.first, (r.cta + i) * r.K) + 1 : 2ll * r.last;
}

// V consecutive floats (V 2, 4 or 8; aligned to 8 or 16 bytes).
template <int V>
__device__ __forceinline__ void load_floats(const float* p, float (&x)[V]) {
  if constexpr (V == 2) {
    const float2 t = __ldcg(reinterpret_cast<const float2*>(p));
    x[0] = t.x;
    x[1] = t.y;
  } else {
#pragma unroll
    for (int i = 0; i < V; i += 4) {
      const float4 t = __ldcg(reinterpret_cast<const float4*>(p + i));
      x[i] = t.x;
      x[i + 1] = t.y;
      x[i + 2] = t.z;
      x[i + 3] = t.w;
    }
  }
}

// log2 of a softmax denominator as the rows use it: without any weight (an
// empty sum) it is +inf, so that 2^(x - lse) is 0.
__device__ __forceinline__ float row_lse(float m, float l) {
  const float lse = m + scored::fast_log2(l);
  return lse == kNegInf ? -kNegInf : lse;
}

// Adds the weights of the rows [r0, r1) of one (sequence, kv head) to their
// scores. SUB lanes share a row, W (2 or 4) of its queries at a time; ONCE: that
// covers all of them. e: the queries' log2 denominators, +inf past the last.
template <int W, int SUB, bool ONCE>
__device__ __forceinline__ void add_weights(const float* lg, float* sc, const float* e, int r0, int r1, int n_old,
                                            int qns) {
  constexpr int U = 4;                       // rows in flight per lane
  constexpr int PER = kFinishThreads / SUB;  // rows per pass
  const int sl = threadIdx.x % SUB, tr = threadIdx.x / SUB;
  float ee[W];
  bool ready = false;  // e is complete
  for (int rb = r0 + tr; rb - tr < r1; rb += PER * U) {
    float s[U], old[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      s[u] = 0.f;
      old[u] = rb + u * PER < r1 && rb + u * PER < n_old && sl == 0 ? sc[rb + u * PER] : 0.f;
    }
    for (int k = W * sl; ONCE || k - W * sl < qns; k += W * SUB) {
      float x[U][W];
#pragma unroll
      for (int u = 0; u < U; ++u) {
#pragma unroll
        for (int i = 0; i < W; ++i) x[u][i] = 0.f;
        if (rb + u * PER < r1 && k < qns) {
          const float* at = lg + static_cast<int64_t>(rb + u * PER) * qns + k;
          if constexpr (W == 4) {
            const float4 t = __ldcg(reinterpret_cast<const float4*>(at));
            x[u][0] = t.x;
            x[u][1] = t.y;
            x[u][2] = t.z;
            x[u][3] = t.w;
          } else {
            const float2 t = __ldcg(reinterpret_cast<const float2*>(at));
            x[u][0] = t.x;
            x[u][1] = t.y;
          }
        }
      }
      if (!ONCE || !ready) {
        if (!ready) __syncthreads();
        ready = true;
#pragma unroll
        for (int i = 0; i < W; ++i) ee[i] = k < qns ? e[k + i] : -kNegInf;
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
#pragma unroll
        for (int i = 0; i < W; ++i) s[u] += fast_exp2(x[u][i] - ee[i]);
      }
      if constexpr (ONCE) break;
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
#pragma unroll
      for (int o = SUB / 2; o > 0; o /= 2) s[u] += __shfl_xor_sync(0xffffffffu, s[u], o);
      // the call's own rows are new: their weight starts here (old is 0)
      if (rb + u * PER < r1 && sl == 0) sc[rb + u * PER] = old[u] + s[u];
    }
  }
}

template <int W>
__device__ __forceinline__ void add_weights(const float* lg, float* sc, const float* e, int r0, int r1, int n_old,
                                            int qns) {
  const int vecs = qns / W;
  if (vecs <= 1) add_weights<W, 1, true>(lg, sc, e, r0, r1, n_old, qns);
  else if (vecs <= 2) add_weights<W, 2, true>(lg, sc, e, r0, r1, n_old, qns);
  else if (vecs <= 4) add_weights<W, 4, true>(lg, sc, e, r0, r1, n_old, qns);
  else if (vecs <= 8) add_weights<W, 8, true>(lg, sc, e, r0, r1, n_old, qns);
  else if (vecs <= 32) add_weights<W, 32, true>(lg, sc, e, r0, r1, n_old, qns);
  else add_weights<W, 32, false>(lg, sc, e, r0, r1, n_old, qns);
}

// SCORED: with rows to score; then four CTAs per SM hide the loads (64 registers:
// 32-token window 40.5 -> 37.1 us), without them the outputs' loads want the registers (decode of
// e4m3 blocks, batch 32: 34.8 us against 36.1).
template <int D, bool SCORED>
__global__ void __launch_bounds__(kFinishThreads, SCORED ? 4 : 2)
    scored_finish_kernel(const ScoredParams p, int nc_log2, int out_ctas) {
  using namespace scored;
  const int NC = 1 << nc_log2;  // queries of a column group
  constexpr int V = D / 32;  // output dims per lane
  constexpr int U = D > 128 ? 4 : 8;  // records' outputs in flight per warp
  constexpr uint32_t full = 0xffffffffu;
  extern __shared__ float s_dyn[];  // [max(qns, records of a unit)]
  __shared__ float s_red[2][kFinishWarps], s_o[kFinishWarps][D];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
  const int64_t pair = blockIdx.x;
  const int seq = static_cast<int>(blockIdx.x / static_cast<unsigned>(p.n_kv_heads));
  const int kvh = static_cast<int>(blockIdx.x) - seq * p.n_kv_heads;
  const int4* units = p.units + pair * p.n_hsub;
  auto store = [&](int v, const float (&o)[V], float inv) {
    float val[V];
#pragma unroll
    for (int i = 0; i < V; ++i) val[i] = o[i] * inv;
    store_out_vec<V>(p.out, query_row(p, seq, kvh, v) * D + V * lane, val, p.out_dtype);
  };

  // ---- outputs, one warp per query
  if (static_cast<int>(blockIdx.y) < out_ctas) {
    for (int v = blockIdx.y * kFinishWarps + w; v < p.qn; v += out_ctas * kFinishWarps) {
      const int4 u = __ldcg(units + (v >> nc_log2));
      const int col = (v & (NC - 1));
      float o[V];
#pragma unroll
      for (int i = 0; i < V; ++i) o[i] = 0.f;
      if (u.x == kUnitEmpty) {
        store(v, o, 0.f);
        continue;
      }
      const RecList r = record_list(u, p.workers);
      if (r.n == 0 || r.n > 32) continue;
      float m = kNegInf, l = 0.f;
      if (lane < r.n) {
        const float2 ml = __ldcg(reinterpret_cast<const float2*>(p.rec_ml + (record_slot(r, lane) * NC + col) * 2));
        m = ml.x;
        l = ml.y;
      }
      const float M = warp_max(m);
      const float f = lane < r.n ? record_weight(m, M) : 0.f;
      const float L = warp_sum(f * l);
      for (int i0 = 0; i0 < r.n; i0 += U) {
        float x[U][V];
#pragma unroll
        for (int i = 0; i < U; ++i)
          if (i0 + i < r.n) load_floats<V>(p.rec_o + (record_slot(r, i0 + i) * NC + col) * D + V * lane, x[i]);
#pragma unroll
        for (int i = 0; i < U; ++i) {
          const float fi = __shfl_sync(full, f, min(i0 + i, 31));
          if (i0 + i < r.n) {
#pragma unroll
            for (int k = 0; k < V; ++k) o[k] += fi * x[i][k];
          }
        }
      }
      store(v, o, L == 0.f ? 0.f : 1.0f / L);
    }
    // ---- outputs of units with many records, the whole CTA per query
    for (int v = blockIdx.y; v < p.qn; v += out_ctas) {
      const RecList r = record_list(__ldcg(units + (v >> nc_log2)), p.workers);
      if (r.n <= 32) continue;
      const int col = (v & (NC - 1));
      float m = kNegInf;
      __syncthreads();  // the previous query's shared values have been read
      for (int i = tid; i < r.n; i += kFinishThreads) {
        const float mi = __ldcg(p.rec_ml + (record_slot(r, i) * NC + col) * 2);
        s_dyn[i] = mi;
        m = fmaxf(m, mi);
      }
      m = warp_max(m);
      if (lane == 0) s_red[0][w] = m;
      __syncthreads();
      m = s_red[0][0];
      for (int i = 1; i < kFinishWarps; ++i) m = fmaxf(m, s_red[0][i]);
      float l = 0.f;
      for (int i = tid; i < r.n; i += kFinishThreads) {
        const float f = record_weight(s_dyn[i], m);
        l += f * __ldcg(p.rec_ml + (record_slot(r, i) * NC + col) * 2 + 1);
        s_dyn[i] = f;
      }
      l = warp_sum(l);
      if (lane == 0) s_red[1][w] = l;
      __syncthreads();
      float o[V];
#pragma unroll
      for (int k = 0; k < V; ++k) o[k] = 0.f;
      for (int i0 = w; i0 < r.n; i0 += kFinishWarps * U) {
        float x[U][V];
#pragma unroll
        for (int i = 0; i < U; ++i) {
          const int j = i0 + i * kFinishWarps;
          if (j < r.n) load_floats<V>(p.rec_o + (record_slot(r, j) * NC + col) * D + V * lane, x[i]);
        }
#pragma unroll
        for (int i = 0; i < U; ++i) {
          const int j = i0 + i * kFinishWarps;
          if (j < r.n) {
            const float f = s_dyn[j];
#pragma unroll
            for (int k = 0; k < V; ++k) o[k] += f * x[i][k];
          }
        }
      }
#pragma unroll
      for (int k = 0; k < V; ++k) s_o[w][V * lane + k] = o[k];
      __syncthreads();
      if (w == 0) {
        float L = 0.f;
#pragma unroll
        for (int k = 0; k < V; ++k) o[k] = 0.f;
        for (int i = 0; i < kFinishWarps; ++i) {
          L += s_red[1][i];
#pragma unroll
          for (int k = 0; k < V; ++k) o[k] += s_o[i][V * lane + k];
        }
        store(v, o, L == 0.f ? 0.f : 1.0f / L);
      }
    }
    return;
  }
  if constexpr (!SCORED) return;

  // ---- rows
  const int n = valid_rows(p, seq);
  const int row_ctas = gridDim.y - out_ctas, y = blockIdx.y - out_ctas;
  const int stretch = max(finish_rows(p.qns), ((n + row_ctas - 1) / row_ctas + 31) / 32 * 32);
  const int64_t first = static_cast<int64_t>(y) * stretch;
  if (first >= n) return;
  const int r0 = static_cast<int>(first), r1 = min(n, r0 + stretch);

  // ---- log2 of the queries' softmax denominators: a thread per query with
  // few records, a warp per query with many
  bool many = false;
  for (int v = tid; v < p.qn; v += kFinishThreads) {
    const int4 u = __ldcg(units + (v >> nc_log2));
    if (u.x == kUnitWhole) {
      s_dyn[v] = row_lse(__ldcg(p.lse + query_row(p, seq, kvh, v)), 1.f);
      continue;
    }
    const RecList r = record_list(u, p.workers);
    if (r.n > kFewRecords) {
      many = true;
      continue;
    }
    float m = kNegInf, l = 0.f;
    for (int i0 = 0; i0 < r.n; i0 += 4) {
      float2 ml[4];
      float M = m;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        ml[i] = make_float2(kNegInf, 0.f);
        if (i0 + i < r.n)
          ml[i] = __ldcg(reinterpret_cast<const float2*>(p.rec_ml) + record_slot(r, i0 + i) * NC + (v & (NC - 1)));
        M = fmaxf(M, ml[i].x);
      }
      l *= fast_exp2(m - M);
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (i0 + i < r.n) l += ml[i].y * fast_exp2(ml[i].x - M);
      m = M;
    }
    s_dyn[v] = row_lse(m, l);
  }
  if (__syncthreads_or(many)) {
    for (int v = w; v < p.qn; v += kFinishWarps) {
      const RecList r = record_list(__ldcg(units + (v >> nc_log2)), p.workers);
      if (r.n <= kFewRecords) continue;
      float m = kNegInf, l = 0.f;
      for (int i = lane; i < r.n; i += 32) {
        const float2 ml = __ldcg(reinterpret_cast<const float2*>(p.rec_ml) + record_slot(r, i) * NC + (v & (NC - 1)));
        const float M = fmaxf(m, ml.x);
        l = l * fast_exp2(m - M) + ml.y * fast_exp2(ml.x - M);
        m = M;
      }
      const float M = warp_max(m);
      const float L = warp_sum(m == kNegInf ? 0.f : l * fast_exp2(m - M));
      if (lane == 0) s_dyn[v] = row_lse(M, L);
    }
  }
  if (tid == 0 && p.qns > p.qn) s_dyn[p.qn] = -kNegInf;
  // (add_weights waits for the CTA's denominators when it has its first scores)

  const float* lg = p.logits + pair * p.rows * p.qns;
  float* sc = p.scores + pair * p.rows;
  if (p.qns % 4 == 0)
    add_weights<4>(lg, sc, s_dyn, r0, r1, n - p.n_tok, p.qns);
  else
    add_weights<2>(lg, sc, s_dyn, r0, r1, n - p.n_tok, p.qns);
}

// ------------------------------------------------------------------ launch

namespace scored {

template <typename CT, int D, int NT, bool SHUT>
kvc_status run_decode(const ScoredParams& p, int grid, const CUtensorMap& tk, const CUtensorMap& tv,
                      cudaLaunchAttribute* attr, cudaStream_t stream) {
  static_assert(scored_warps(sizeof(CT), D, NT) == ScoredGeo<sizeof(CT), D, NT>::kWarps,
                "the host counts a CTA's workers as the kernel does");
  auto* k = scored_decode_kernel<CT, D, NT, SHUT>;
  // The opt-in to large shared memory holds per device: made at the first call on each.
  static std::atomic<uint64_t> opted{0};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return cuda_fail(e, "cudaGetDevice");
  const uint64_t bit = dev < 64 ? 1ull << dev : 0;
  if ((opted.load() & bit) == 0) {
    e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             static_cast<int>(scored_smem_bytes<sizeof(CT), D, NT>(kScoredMaxBatch)));
    if (e != cudaSuccess) return cuda_fail(e, "cudaFuncSetAttribute(scored decode)");
    opted.fetch_or(bit);
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(ScoredGeo<sizeof(CT), D, NT>::kThreads);
  cfg.dynamicSmemBytes = scored_smem_bytes<sizeof(CT), D, NT>(p.batch);
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, k, tk, tv, p);
  return e == cudaSuccess ? KVC_OK : cuda_fail(e, "cudaLaunchKernelEx(scored decode)");
}

template <typename CT, int D, int NT>
kvc_status run(const ScoredParams& p, int grid, const CUtensorMap& tk, const CUtensorMap& tv, cudaStream_t stream) {
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  constexpr bool FINITE = std::is_same<CT, s8q>::value;  // every int8 code is
  const kvc_status st = FINITE || p.n_tok == 1 ? run_decode<CT, D, NT, false>(p, grid, tk, tv, attr, stream)
                                               : run_decode<CT, D, NT, !FINITE>(p, grid, tk, tv, attr, stream);
  if (st != KVC_OK) return st;
  // CTAs per (sequence, kv head): one wave of them on the GPU, no more than
  // there is work for. For the outputs a warp per query or a few of them in
  // turn, or up to a CTA per query where few units share all workers and a
  // query may have more than 32 records; the rest for the rows.
  const int64_t pairs = static_cast<int64_t>(p.batch) * p.n_kv_heads;
  const int64_t want = std::max<int64_t>(1, kFinishCtas / pairs);
  int64_t out_ctas = (p.qn + kFinishWarps - 1) / kFinishWarps;
  if (pairs * 32 < p.workers)
    out_ctas = std::max(out_ctas, std::min<int64_t>(want, p.qn));
  else if (p.scores != nullptr)
    out_ctas = std::max<int64_t>(1, std::min(out_ctas, want / 4));
  int64_t row_ctas = 0;
  if (p.scores != nullptr)
    row_ctas = std::max<int64_t>(1, std::min<int64_t>(want - std::min(want / 4, out_ctas),
                                                      (p.rows + finish_rows(p.qns) - 1) / finish_rows(p.qns)));
  cudaLaunchConfig_t fin = {};
  fin.gridDim = dim3(static_cast<unsigned>(pairs), static_cast<unsigned>(out_ctas + row_ctas));
  fin.blockDim = dim3(kFinishThreads);
  fin.dynamicSmemBytes = static_cast<size_t>(std::max(p.qns, p.workers + 1)) * 4;
  fin.stream = stream;
  fin.attrs = attr;
  fin.numAttrs = 1;
  auto* finish = p.scores != nullptr ? scored_finish_kernel<D, true> : scored_finish_kernel<D, false>;
  const cudaError_t e = cudaLaunchKernelEx(&fin, finish, p, NT == 1 ? 3 : 4, static_cast<int>(out_ctas));
  if (e != cudaSuccess) return cuda_fail(e, "cudaLaunchKernelEx(scored finish)");
  return KVC_OK;
}

}  // namespace scored

template <typename CT>
kvc_status scored_launch(const ScoredParams& p, int D, int nt, int grid, const CUtensorMap& tk, const CUtensorMap& tv,
                         cudaStream_t stream) {
  if (D == 64 && nt == 1) return scored::run<CT, 64, 1>(p, grid, tk, tv, stream);
  if (D == 64) return scored::run<CT, 64, 2>(p, grid, tk, tv, stream);
  if (D == 128 && nt == 1) return scored::run<CT, 128, 1>(p, grid, tk, tv, stream);
  if (D == 128) return scored::run<CT, 128, 2>(p, grid, tk, tv, stream);
  return scored::run<CT, 256, 1>(p, grid, tk, tv, stream);
}

}  // namespace kvc
