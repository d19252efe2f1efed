// tree_attn.cuh — attention of drafted token trees over the per-head pools, on the tensor
// cores.
//
//   x[r, t] = scale q[r] . k_t,   o[r] = sum_t exp2(x[r, t] - m[r]) v_t / sum_t exp2(x[r, t] - m[r])
//
// r: a (query, head) row of one kv head; t: the tokens t < len - n_q, and the drafted tokens
// (the last n_q) that the query's mask row names.  A token's key and value are read once for
// all rows of its kv head: with R rows it costs 4 R D operations and the stored bytes (4 D in
// bf16), so HBM bounds up to about R = 250 rows, the tensor cores beyond.
//
// Layout.  The rows are the MMA's M (a tile of 128), 64 tokens a tile its N:
//   S [128 x 64] = Q [128 x D] K^T          Q and K in shared memory, K-major
//   O [128 x D] += P [128 x 64] V           P over S in tensor memory (bf16), V MN-major
// A thread of a softmax warpgroup owns a row: no reduction leaves the thread.  Two warpgroups
// share the work by mode:
//   kPair   more than 128 rows: a tile of rows each, all key tiles
//   kTurns  up to 128 rows: the same rows, key tiles in turns, an O each, added at the end
//   kSolo   head_dim 256 (whose O fills half of tensor memory): one of them takes all
// S is double-buffered per warpgroup, so that the next product runs under the softmax.  The
// reference m moves only when a logit (in log2 units) passes it by more than 8: O is then rescaled.
//
// bf16 keys and values go from the pool to swizzled operand tiles by 16-byte asynchronous
// copies, which fill tokens that nobody sees (past the length, unused drafts) with zeros: a
// stale NaN reaches neither product.  Packed ones are expanded to fp16 operands by twelve warps, a
// tile's keys and its values each under the power of two that puts the largest near 2^13.  The
// keys' power goes back into the logits.  The values' e goes into the probabilities' exponent,
//   P[t] = exp2(x[t] - m + c),   c = max(e - u, -64),
// so that O needs nothing: u (`up`), an integer, is O's power of two beside 2^m and follows x + e - m as m follows
// x.  The sum is of the x alone: it takes a tile's P times 2^-c.  (A P that the 64 raises is below
// 2^-56 all the same and 0 in fp16, while its share of the sum stays what it is.)  A reference from 2^22 on comes
// off first, which is exact where x is near it; below, c - m is.  Any magnitudes fit; within a tile,
// what is 2^-27 of the largest and less (or 2^-114) loses bits.  (Powers by token took 48 loads a row and tile in the softmax:
// three times its time.)
//
// Every kv head has a column of CTAs, one CTA a SM.  The key tiles of a head's units (sequence, 128 or
// 256 rows) are laid end to end and split evenly in cost over its column, so that the columns pass
// the same tokens at about the same time: a packed head's row of a token is often less than a
// line, which the other heads share (8 x 16384 tokens in K4/V4: 477 MB read from DRAM with one
// column for all heads, 204 MB, what is stored, with one each).  A unit inside one CTA's share is
// written directly; a split one leaves FP32 records that a second kernel merges in order.
//
// P has 16 bits (as its product wants both operands of one type, bf16 or fp16), the sums it is divided by 32: with
// the output's own rounding the results are off by 0.0023 (bf16) and 0.0019 to 0.0021 (packed) of their size, where
// the rounding of the output alone is 0.0017.
//
// Measured on one GB300, with the merge, in a stream of calls: 16 trees of 64 drafts behind 16384 tokens
// (bf16, 16 of 8 heads of 128) 183 to 189 us, 5.7 to 5.9 TB/s: HBM.  16 trees of 13, 32 of 8 heads of 64, behind 2048,
// 4096, 8192 tokens: 25.0, 37.6, 61.5 us: 5.6 TB/s from length to length, and 14 us for what does not hang on it: the
// start (walk, block rows, queries), the last tiles, the records and their merge.  8 trees of 24 behind 2048, 8192, 16384
// in K4/V4: 30.2, 65.1, 108.6 us, 0.8 us a tile and CTA: the hand-over of tiles and the feeders' loads and expansion
// (16384: 85 us without either of the latter, 75 without both).  1 tree of 8 behind 1000: 11.7 us, latency.
// More than 128 rows: 4 trees behind 16384, 100 drafts of 2 heads 69 us, 64 drafts of 4 heads 71, of 8 heads (two
// units) 125, where the bytes take 40 and the operations 28, 35 and 71.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "drafts.cuh"
#include "tcgen05.cuh"

namespace pkv {
namespace tree {

enum Mode { kTurns = 0, kPair = 1, kSolo = 2 };

constexpr int kTile = 64;               // tokens a tile
constexpr int kRows = 128;              // rows a tile of rows
// Warps 0..7: softmax; 8: the products with the keys; 9: those with the values; 10 (packed): where
// the tiles lie (scout); the last ones: keys and values (feeders).
constexpr int kSoftmaxThreads = 256;
constexpr float kSlack = 8.0f;          // log2 of how far a logit may pass the reference
constexpr float kNoMax = -3.402823466e38f;  // the reference before any visible token: no logit is below it
constexpr float kExact = 4194304.0f;    // 2^22: whole numbers up to twice that are exact in fp32, with c's 2^8 among them
constexpr float kLeast = -64.0f;        // packed: no probability is lifted by less (2^(kSlack - 64) is 0 in fp16)
constexpr int kSmemLimit = 232448;      // 227 KB opt-in shared memory per block
constexpr int kAtRing = 8;              // packed: tiles that the scout runs ahead
constexpr int kPowRing = 12;            // packed: tiles whose powers are held

// Packed: the six warpgroups share the launch's registers, 2 x 112 + 40 + 3 x 72 = 6 x 80 (the
// launcher checks that the kernel was built with 80).  Their paths do not rejoin: each ends in a
// return.  (120 and 64 for softmax and feeders, or 128 and 56, are no faster.)
constexpr int kLaunchRegs = 80;

// Cost of a unit's start in the split over the CTAs, in quarter tiles: its queries are loaded
// and its output or record written.  (4, 7, 10 tiles: 4 x 16384, 64 drafts 58.1, 56.1, 56.6 us;
// the same with heads of 64 38.1, 37.1, 37.9; K8/V8 8 x 16384, 24 drafts 75.1, 74.4, 74.0.)
constexpr int kSegCost = 28;
constexpr int kCost = 4;

template <int D, int MODE, int KB, int VB>
struct Plan {
  static constexpr bool PACKED = KB < 16;
  // Packed: three warpgroups of feeders (warp 11 fills the MMA warps'), in teams that take tiles in
  // turns, so that one team's loads and waits lie under the others' work.  A warp then has (KB +
  // VB) / 2 pieces of a tile in registers (D = 256, one team: a third less), eight at most.  Two
  // teams instead of one took 8 x 16384 tokens in K4/V4 from 188 to 155 us; three warpgroups
  // instead of two from 123 to 108, 16 x 6000 in K8/V8 with heads of 64 from 79 to 72.
  static constexpr int kWarps = PACKED ? 12 : 2;  // (bf16: 12 warps in all, 168 registers a thread)
  static constexpr int kFeeders = kWarps * 32;
  static constexpr int kTeams = !PACKED || D == 256 ? 1 : 384 / D;
  static constexpr int kTeam = kFeeders / kTeams;  // threads that bring a tile
  static constexpr int kFeeder0 = PACKED ? 384 : 320;  // the first feeder thread
  static constexpr int kThreads = kFeeder0 + kFeeders;
  static constexpr int kTileRows = MODE == kPair ? 2 * kRows : kRows;  // rows a unit
  static constexpr int kQBytes = kTileRows * D * 2;
  static constexpr int kSlot = kTile * D * 2;
  static constexpr int kK = D == 256 ? 2 : D == 64 ? 8 : PACKED ? 4 : 5;
  static constexpr int kV = D == 256 ? 2 : D == 128 ? 4 : 8;
  static constexpr int kSmall = 12 * 1024;
  static constexpr int kSmem = 1024 + kQBytes + (kK + kV) * kSlot + kSmall;
  static_assert(kSmem <= kSmemLimit, "shared memory");
  // A tile's powers are overwritten kPowRing tiles later: its keys' slot was freed then by the S of
  // the tile kPowRing - kK later, which waited for the values of the tile four before it at least.
  static_assert(!PACKED || kK + 4 <= kPowRing, "powers are read until the softmax is done");
  // A slot's barrier is waited on by parity: a team that comes to tile t knows by its last one, t -
  // kTeams, that the slot's use before the last, t - 2 kK, is over, so that the parity is not stale.
  static_assert(kTeams <= kK && kTeams <= kV && kTeams <= kAtRing, "a team a ring ahead");
};

struct Params {
  TreeAttnArgs a;
  int G;         // query heads a kv head
  int rows;      // n_q * G
  int tile_rows; // rows a unit
  int n_rt;      // units a (sequence, kv head)
  int rec_rows;  // rows a record
  int cols;      // columns of CTAs: a kv head's each, or one for all (fewer CTAs than heads)
  int col_ctas;  // CTAs a column
  int words;     // mask words a query
  int group_log; // packed: log2 of the values a group
  int2* meta;    // [B * hkv * n_rt]: first CTA of a split unit (-1: written directly), last CTA
  float2* ml;    // [2 * grid][rec_rows]: reference and sum of a record's rows
  float* acc;    // [2 * grid][D / 4][rec_rows][4], over the sums: lanes, which own rows, store and load whole lines
};

__device__ __forceinline__ int32_t length(const Params& P, int b) {
  bool bad;
  return draft_ctx(P.a.ctx[b], (int64_t)P.a.max_blocks * kBlockTokens, P.a.n_q, &bad);
}

// A CTA's share of its column's tiles: a unit of n tiles costs kCost n + kSegCost, its tile k sits
// at kSegCost + kCost k from its start, and the column's CTA g holds the positions [g V, (g + 1) V).
// V is at least kCost, so the CTAs that hold a unit's tiles are consecutive.
struct Segment {
  int b, len, x;    // sequence, its length, unit within it: kv head * n_rt + group of rows
  int k0, k1, n;    // this CTA's tiles of it, and all of them
};

struct Walk {
  int b, x;
  int x0;          // the column's first unit of a sequence
  int64_t at;      // position of sequence b's first unit
  int64_t lo, hi;  // positions of this CTA

  // Warp-uniform values, known as such: copies and MMAs are issued with what follows from them.
  __device__ __forceinline__ bool next(const Params& P, Segment& s) {
    const int upb = P.a.lv.hkv / P.cols * P.n_rt;
    while (b < P.a.B) {
      const int len = uniform(length(P, b));
      const int n = (len + kTile - 1) / kTile;
      const int64_t cost = n > 0 ? (int64_t)kCost * n + kSegCost : 0;
      const int64_t first = at + x * cost + kSegCost;  // position of the unit's first tile
      if (n > 0 && first >= hi) return false;
      s.b = b, s.len = len, s.n = n, s.x = x0 + x;
      if (n == 0 || ++x == upb) {
        at += upb * cost;
        x = 0;
        ++b;
      }
      if (n == 0) continue;
      const int64_t f = first >= lo ? 0 : (lo - first + kCost - 1) / kCost;
      const int64_t e = (hi - first + kCost - 1) / kCost;
      s.k0 = uniform((int)(f < n ? f : n));
      s.k1 = uniform((int)(e < n ? e : n));
      if (s.k1 > s.k0) return true;
    }
    return false;
  }
};

// One warp: the CTA's positions and where its walk starts.
__device__ __forceinline__ Walk start_walk(const Params& P) {
  constexpr int kHeld = 128;  // sequences whose lengths are read once
  const int lane = threadIdx.x & 31;
  const int64_t upb = (int64_t)(P.a.lv.hkv / P.cols) * P.n_rt;
  const int col = (int)blockIdx.x / P.col_ctas, g = (int)blockIdx.x % P.col_ctas;
  auto cost = [&](int b) -> int64_t {
    if (b >= P.a.B) return 0;
    const int n = (length(P, b) + kTile - 1) / kTile;
    return n > 0 ? upb * ((int64_t)kCost * n + kSegCost) : 0;
  };
  int64_t held[kHeld / 32], total = 0;
#pragma unroll
  for (int c = 0; c < kHeld / 32; ++c) {
    held[c] = 32 * c < P.a.B ? cost(32 * c + lane) : 0;
    total += held[c];
  }
  for (int b = kHeld + lane; b < P.a.B; b += 32) total += cost(b);
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) total += __shfl_xor_sync(0xffffffffu, total, off);
  Walk w;
  const int64_t v = (total + P.col_ctas - 1) / P.col_ctas;
  const int64_t V = v > kCost ? v : kCost;
  w.lo = g * V;
  w.hi = w.lo + V;
  w.b = P.a.B;
  w.x = 0;
  w.x0 = (int)(col * upb);
  w.at = total;
  int64_t carry = 0;
  // the first sequence that ends past the CTA's first position
  auto found = [&](int base, int64_t c) {
    int64_t inc = c;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int64_t y = __shfl_up_sync(0xffffffffu, inc, off);
      if (lane >= off) inc += y;
    }
    const unsigned hit = __ballot_sync(0xffffffffu, c > 0 && carry + inc > w.lo);
    if (hit) {
      const int l = __ffs(hit) - 1;
      const int64_t mine = __shfl_sync(0xffffffffu, c, l);
      w.b = base + l;
      w.at = carry + __shfl_sync(0xffffffffu, inc - c, l);
      w.x = w.lo > w.at ? (int)((w.lo - w.at) / (mine / upb)) : 0;
      return true;
    }
    carry += __shfl_sync(0xffffffffu, inc, 31);
    return false;
  };
#pragma unroll
  for (int c = 0; c < kHeld / 32; ++c)
    if (32 * c < P.a.B && found(32 * c, held[c])) return w;
  for (int base = kHeld; base < P.a.B; base += 32)
    if (found(base, cost(base + lane))) return w;
  return w;
}

// Packed: where a tile lies, as the scout finds it.
struct __align__(16) Place {
  const uint8_t *slab0, *slab1;  // its blocks' slabs
  uint32_t row0, row1;           // the kv head's first row in each; row0 = kNoTile: no tile is left
  uint32_t live0, live1;         // tokens that are read
};
constexpr uint32_t kNoTile = 0xffffffffu;

// Shared-memory state besides the operands.
struct Small {
  uint64_t k_full[8], k_empty[8], v_full[8], v_empty[8];  // by slot
  uint64_t s_full[2][2], p_full[2][2];                    // by warpgroup and buffer
  uint64_t pv_done[2][2], q_full, q_empty, drain[2], done;
  uint64_t at_full[kAtRing], at_empty[kAtRing];           // packed: by tile
  Walk walk;
  uint32_t tmem;
  int dead;                    // a wait gave up: every role runs on without waiting or issuing
  float m[2][kRows], up[2][kRows], l[2][kRows];  // the warpgroups' references, O's powers and sums of shared rows
  // Packed: log2 of the power of two that a row's query was divided by, for every other segment: a
  // warpgroup may load the next segment's queries before the other has read this one's powers.
  int q_pow[2][2 * kRows];
  // Packed, by tile: log2 of the powers of two that its keys and its values were divided by.
  alignas(8) int2 pow[kPowRing];
  Place at[kAtRing];           // packed
  float2 widest[6][2][12];      // by team, parity of its tile and warp: largest key and value
};

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool ok, uint64_t policy) {
  asm volatile("cp.async.cg.shared.global.L2::cache_hint [%0], [%1], 16, %2, %3;" ::"r"(dst), "l"(src), "r"(ok ? 16 : 0),
               "l"(policy)
               : "memory");
}
// This thread's copies so far count as one arrival once they have landed.
__device__ __forceinline__ void cp_async_arrive(uint64_t* bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}

__device__ __forceinline__ uint64_t pair2(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ void split2(uint64_t r, float& a, float& b) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(r));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

// Bits of the tokens j0 .. j0 + 31 (counted from the first drafted one): before it all are
// set, from n_q on none.  word(w): the w-th word of a mask, 0 <= w < words.
template <typename F>
__device__ __forceinline__ uint32_t bits_at(int j0, int n_q, int words, F&& word) {
  if (j0 >= n_q) return 0u;
  if (j0 + 31 < 0) return 0xffffffffu;
  const int w = j0 >> 5, s = j0 & 31;
  const uint32_t a = w < 0 ? 0xffffffffu : word(w), b = w + 1 < words ? word(w + 1) : 0u;
  uint32_t r = __funnelshift_r(a, b, s);
  if (j0 + 32 > n_q) r &= (1u << (n_q - j0)) - 1u;
  return r;
}

// A feeder warp's view of a segment: the blocks of its next tiles, and which of their tokens
// some query sees (the others' slots may hold anything).
struct Feed {
  const uint8_t* base;  // lane l: block 2 ub + l: keys of its slab (null outside the pool)
  int r;                // its row in the slab
  uint32_t named;       // lane w: OR over the queries of mask word w

  __device__ __forceinline__ void see(const Params& P, const Segment& s) {
    const int lane = threadIdx.x & 31;
    named = 0;
    if (s.k1 * kTile <= s.len - P.a.n_q) return;  // no drafted token here
    const uint32_t* mask = P.a.mask + s.b * P.a.mask_stride;
    for (int w = 0; w < P.words; ++w) {
      uint32_t v = 0;
      for (int i = lane; i < P.a.n_q; i += 32) v |= mask[(int64_t)i * P.words + w];
      v = __reduce_or_sync(0xffffffffu, v);
      if (lane == w) named = v;
    }
  }
  // blocks of the tiles from ub on (16 of them)
  __device__ __forceinline__ void look_up(const Params& P, const Segment& s, int ub) {
    const int j = 2 * ub + (int)(threadIdx.x & 31);
    base = nullptr;
    r = 0;
    if (j < 2 * s.k1 && j * kBlockTokens < s.len) {
      const int32_t row = P.a.bt[(int64_t)s.b * P.a.max_blocks + j];
      if (draft_row_ok(P.a.lv, row)) {
        const int32_t slab = row / P.a.lv.slab_blocks;
        r = row - slab * P.a.lv.slab_blocks;
        base = P.a.lv.tab.base[(size_t)slab * P.a.lv.tab.stride];
      } else {
        atomicOr(P.a.lv.err, ERR_ROW);
      }
    }
  }
  // the 64 tokens of tile u that are read
  __device__ __forceinline__ uint2 tokens(const Params& P, const Segment& s, int u) const {
    if ((u + 1) * kTile <= s.len - P.a.n_q) return make_uint2(0xffffffffu, 0xffffffffu);
    const int j0 = u * kTile - (s.len - P.a.n_q);
    auto word = [&](int w) { return __shfl_sync(0xffffffffu, named, w); };
    const uint32_t lo = bits_at(j0, P.a.n_q, P.words, word);
    return make_uint2(lo, bits_at(j0 + 32, P.a.n_q, P.words, word));
  }
};

// Offset of 16-byte piece c (of the row's D / 8) of row r in an operand of rows of 64 values
// under the 128-byte swizzle; col: bytes of one 64-value column (all rows).
__device__ __forceinline__ uint32_t swizzled(int r, int c, uint32_t col) {
  return (uint32_t)(c >> 3) * col + (uint32_t)r * 128 + (uint32_t)(((c & 7) ^ (r & 7)) << 4);
}

// log2 of the power of two that puts mx near 2^13
__device__ __forceinline__ int power_of(float mx) {
  return max(-100, min(120, (int)(__float_as_uint(mx) >> 23) - 127 - 13));
}

// 4-bit codes are expanded two at a time, i and i + 4 of each eight values: an operand row holds
// them in the order 0 4 1 5 2 6 3 7.  A warp's row of fp16 values (E a lane) into that order:
template <int E>
__device__ __forceinline__ void octets(uint32_t (&w)[E / 2]) {
  const int lane = threadIdx.x & 31;
  auto lows = [](uint32_t a, uint32_t b) { return __byte_perm(a, b, 0x5410); };
  auto highs = [](uint32_t a, uint32_t b) { return __byte_perm(a, b, 0x7632); };
  if constexpr (E == 2) {
    const int j = lane & 3, from = (lane & ~3) + (j >> 1);
    const uint32_t a = __shfl_sync(0xffffffffu, w[0], from), b = __shfl_sync(0xffffffffu, w[0], from + 2);
    w[0] = j & 1 ? highs(a, b) : lows(a, b);
  } else if constexpr (E == 4) {
    const bool odd = lane & 1;
    const uint32_t got = __shfl_xor_sync(0xffffffffu, odd ? w[0] : w[1], 1);
    const uint32_t a = odd ? got : w[0], b = odd ? w[1] : got;
    w[0] = lows(a, b);
    w[1] = highs(a, b);
  } else {
    const uint32_t a = w[0], b = w[1], c = w[2], d = w[3];
    w[0] = lows(a, c), w[1] = highs(a, c), w[2] = lows(b, d), w[3] = highs(b, d);
  }
}
// Where column c of an operand made from BITS-bit codes lies among its values, and the inverse.
__host__ __device__ constexpr int octet_column(int c) { return (c & ~7) | (c & 3) << 1 | (c & 4) >> 2; }

// Queries of a unit's rows into shared memory, a row a warp at a time; packed: into the keys'
// basis, under a power of two in fp16.
template <int D, int KB>
__device__ __forceinline__ void load_queries(const Params& P, const Segment& s, uint8_t* qs, int* q_pow, int row0, int nrow) {
  constexpr int E = D / 32;
  constexpr bool PACKED = KB < 16;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int kvh = s.x / P.n_rt;
  float sign[E];
  if constexpr (PACKED) {
#pragma unroll
    for (int e = 0; e < E; ++e) sign[e] = P.a.signs[lane * E + e] * (D == 64 ? 0.125f : D == 128 ? 0.08838834764831845f : 0.0625f);
  }
  constexpr int U = D == 256 || PACKED ? 8 : 16;  // rows in flight
  for (int rb = warp; rb < nrow; rb += 8 * U) {
    uint32_t w[U][E / 2];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int r = row0 + min(rb + 8 * u, nrow - 1);
      const int i = r / P.G, g = r - i * P.G;
      const uint16_t* src = P.a.q + (((int64_t)s.b * P.a.n_q + i) * P.a.Hq + kvh * P.G + g) * D + lane * E;
      if constexpr (E == 2)
        w[u][0] = *reinterpret_cast<const uint32_t*>(src);
      else if constexpr (E == 4) {
        const uint2 v = *reinterpret_cast<const uint2*>(src);
        w[u][0] = v.x, w[u][1] = v.y;
      } else {
        const uint4 v = *reinterpret_cast<const uint4*>(src);
        w[u][0] = v.x, w[u][1] = v.y, w[u][2] = v.z, w[u][3] = v.w;
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int r = rb + 8 * u;
      if (r >= nrow) break;
      if constexpr (PACKED) {
        float x[E];
#pragma unroll
        for (int e = 0; e < E; e += 2) {
          bf16x2_to_f32(w[u][e / 2], x[e], x[e + 1]);
          x[e] *= sign[e], x[e + 1] *= sign[e + 1];
        }
#pragma unroll
        for (int hs = 1; hs < E; hs <<= 1)
#pragma unroll
          for (int e = 0; e < E; ++e)
            if ((e & hs) == 0) {
              const float a = x[e], b = x[e + hs];
              x[e] = a + b;
              x[e + hs] = a - b;
            }
#pragma unroll
        for (int m = 1; m < 32; m <<= 1)
#pragma unroll
          for (int e = 0; e < E; ++e) {
            const float other = __shfl_xor_sync(0xffffffffu, x[e], m);
            x[e] = lane & m ? other - x[e] : x[e] + other;
          }
        float mx = 0.f;
#pragma unroll
        for (int e = 0; e < E; ++e) mx = fmaxf(mx, fabsf(x[e]));
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, off));
        const int ex = power_of(mx);
        const float f = pow2(-ex);
#pragma unroll
        for (int e = 0; e < E; e += 2) w[u][e / 2] = fp16x2(x[e] * f, x[e + 1] * f);
        if (lane == 0) q_pow[r] = ex;
        if constexpr (KB == 4) octets<E>(w[u]);
      }
      const int byte = lane * E * 2, tile = r / kRows, rr = r % kRows;
      uint8_t* dst = qs + tile * (kRows * D * 2) + swizzled(rr, byte / 16, kRows * 128) + byte % 16;
      if constexpr (E == 2)
        *reinterpret_cast<uint32_t*>(dst) = w[u][0];
      else if constexpr (E == 4)
        *reinterpret_cast<uint2*>(dst) = make_uint2(w[u][0], w[u][1]);
      else
        *reinterpret_cast<uint4*>(dst) = make_uint4(w[u][0], w[u][1], w[u][2], w[u][3]);
    }
  }
}

// A packed tile's pieces (16 bytes of codes with their group's scale and offset) of one kind,
// in units of 32: `kTokens` tokens by D values.  The lanes are laid out so that eight of them
// write operand pieces to eight different bank groups.
template <int D, int BITS>
struct Pieces {
  static constexpr int kUnits = D * BITS / 64;      // units a tile
  static constexpr int kCol = BITS == 4 ? 2 : 4;    // pieces of 64 values
  static constexpr int kTokens = 32 / (kCol * (D / 64));
  int token, value;          // this lane's token of the unit, its piece's first value
  uint32_t code_at, meta_at;      // their bytes in a slab, from the unit's first token on
  uint32_t code_row, meta_row;    // bytes from head to head
  uint32_t code_step, meta_step;  // bytes from token to token
  // `code_off`, `meta_off`: where the kind's two tensors lie in a slab (below 2^32 bytes)
  __device__ __forceinline__ Pieces(int hkv, int row_bytes, int meta_bytes, uint32_t code_off, uint32_t meta_off, int group_log) {
    const int lane = threadIdx.x & 31;
    token = lane / kCol % kTokens;
    value = lane / (kCol * kTokens) * 64 + lane % kCol * (64 / kCol);
    code_row = (uint32_t)row_bytes;
    meta_row = (uint32_t)meta_bytes;
    code_step = (uint32_t)(hkv * row_bytes);
    meta_step = (uint32_t)(hkv * meta_bytes);
    code_at = code_off + (uint32_t)token * code_step + (uint32_t)(value * BITS / 8);
    meta_at = meta_off + (uint32_t)token * meta_step + (uint32_t)(value >> group_log) * 8u;
  }
  // unit g of a tile, one of whose blocks it lies in: `row` is that block's first row of the head
  __device__ __forceinline__ void load(const uint8_t* slab, uint32_t row, int g, uint32_t live, uint4& c, float2& m) const {
    const uint32_t t0 = (uint32_t)(g * kTokens) & 31u;
    c = make_uint4(0, 0, 0, 0);
    m = make_float2(0.f, 0.f);
    if (live >> (t0 + token) & 1u) {
      c = *reinterpret_cast<const uint4*>(slab + (row * code_row + t0 * code_step + code_at));
      m = *reinterpret_cast<const float2*>(slab + (row * meta_row + t0 * meta_step + meta_at));
    }
  }
  // the largest magnitude of a piece
  __device__ __forceinline__ static float widest(const float2& m) {
    return fmaxf(fabsf(m.y), fabsf(fmaf(m.x, (float)((1 << BITS) - 1), m.y)));
  }
};

__device__ __forceinline__ __half2 half2_of(uint32_t w) { return *reinterpret_cast<const __half2*>(&w); }
__device__ __forceinline__ uint32_t bits_of(__half2 h) { return *reinterpret_cast<const uint32_t*>(&h); }

// Codes of a piece as operand pieces in fp16: s c + o, s and o rounded to fp16, one rounding
// for the rest.  `s` comes as 2^BITS s, about the group's range, which stays a normal fp16 as long as that does
// (s itself is 2^BITS smaller: it would lose bits that much earlier), and c as c / 2^BITS: a code under a
// fitting exponent is 4 + c / 256, 64 + c / 16 or, four bits up, 4 + c / 16, exactly.
template <int BITS>
__device__ __forceinline__ void expand(const uint4& code, float s, float o, uint8_t* slot, int token, int value) {
  const uint32_t w[4] = {code.x, code.y, code.z, code.w};
  const __half2 ss = __float2half2_rn(s), oo = __float2half2_rn(o);
  const __half2 k64 = half2_of(0x54005400u), k4 = half2_of(0x44004400u);
  constexpr int N = BITS == 4 ? 4 : 2;  // operand pieces of eight values
#pragma unroll
  for (int q = 0; q < N; ++q) {
    uint32_t out[4];
    if constexpr (BITS == 4) {
      // pairs (0, 4), (1, 5), (2, 6), (3, 7)
      const uint32_t lo = w[q], hi = w[q] >> 8;
      out[0] = bits_of(__hfma2(__hsub2(half2_of((lo & 0x000f000fu) | 0x54005400u), k64), ss, oo));
      out[1] = bits_of(__hfma2(__hsub2(half2_of((lo & 0x00f000f0u) | 0x44004400u), k4), ss, oo));
      out[2] = bits_of(__hfma2(__hsub2(half2_of((hi & 0x000f000fu) | 0x54005400u), k64), ss, oo));
      out[3] = bits_of(__hfma2(__hsub2(half2_of((hi & 0x00f000f0u) | 0x44004400u), k4), ss, oo));
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        out[i] = bits_of(__hfma2(
            __hsub2(half2_of(__byte_perm(w[2 * q + (i >> 1)], 0x44444444u, i & 1 ? 0x4342 : 0x4140)), k4), ss, oo));
    }
    *reinterpret_cast<uint4*>(slot + swizzled(token, value / 8 + q, kTile * 128)) = make_uint4(out[0], out[1], out[2], out[3]);
  }
}

template <int D, int MODE, int KB, int VB>
__global__ void __launch_bounds__(Plan<D, MODE, KB, VB>::kThreads, 1) tree_attn_kernel(const __grid_constant__ Params P) {
  using L = Plan<D, MODE, KB, VB>;
  constexpr bool PACKED = L::PACKED;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
  uint8_t* qs = smem;
  uint8_t* ks = qs + L::kQBytes;
  uint8_t* vs = ks + L::kK * L::kSlot;
  Small& sm = *reinterpret_cast<Small*>(vs + L::kV * L::kSlot);
  static_assert(sizeof(Small) <= L::kSmall, "small state");
  const int warp = uniform((int)(threadIdx.x >> 5)), lane = threadIdx.x & 31;
  volatile int* dead = &sm.dead;
  int32_t* err = P.a.lv.err;

  if (threadIdx.x == 0) {
    for (int i = 0; i < 8; ++i) {
      mbar_init(&sm.k_full[i], L::kTeam);
      mbar_init(&sm.v_full[i], L::kTeam);
      mbar_init(&sm.k_empty[i], 1);
      mbar_init(&sm.v_empty[i], 1);
    }
    for (int t = 0; t < 2; ++t) {
      for (int i = 0; i < 2; ++i)
        mbar_init(&sm.s_full[t][i], 1), mbar_init(&sm.p_full[t][i], 128), mbar_init(&sm.pv_done[t][i], 1);
      mbar_init(&sm.drain[t], 1);
    }
    mbar_init(&sm.q_full, kSoftmaxThreads);
    mbar_init(&sm.q_empty, 1);
    for (int i = 0; i < kAtRing; ++i) mbar_init(&sm.at_full[i], 1), mbar_init(&sm.at_empty[i], L::kTeam / 32);
    mbar_init(&sm.done, kSoftmaxThreads);
    sm.dead = 0;
    fence_mbar_init();
  }
  if (warp == 8) tc_alloc(&sm.tmem, 512);
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (warp == 0) {
    const Walk w = start_walk(P);
    if (lane == 0) sm.walk = w;
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = uniform(sm.tmem);
  auto tm_s = [&](int t, int buf) { return tmem + (t * 2 + buf) * kTile; };
  auto tm_o = [&](int t) { return tmem + 256 + t * D; };
  Walk walk = {uniform(sm.walk.b), uniform(sm.walk.x), uniform(sm.walk.x0), uniform(sm.walk.at), uniform(sm.walk.lo), uniform(sm.walk.hi)};
  Segment seg;
  // Which warpgroups work on tile `it` (counted over the CTA's segments) of a unit with nrow rows
  auto works = [&](int t, int it, int nrow) {
    return MODE == kTurns ? (it & 1) == t : MODE == kPair ? t == 0 || nrow > kRows : t == 0;
  };

  if (warp < 8) {
    // ---------------------------------------------------------------- softmax
    if constexpr (PACKED) asm volatile("setmaxnreg.inc.sync.aligned.u32 112;");
    const int t = warp >> 2;
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    const int tr = (warp & 3) * 32 + lane;  // row of the tile
    int it0 = 0, n_seg = 0;
    int jobs = 0, others = 0;               // tiles that this warpgroup and the other took, over all segments
    while (walk.next(P, seg)) {
      const int row0 = seg.x % P.n_rt * L::kTileRows, nrow = min(L::kTileRows, P.rows - row0);
      const int kvh = seg.x / P.n_rt;
      if (n_seg > 0) wait_or_die(&sm.q_empty, (n_seg - 1) & 1, dead, err);
      int* q_pow = sm.q_pow[n_seg & 1];  // (read for the last time before the barrier of the segment in between)
      load_queries<D, KB>(P, seg, qs, q_pow, row0, nrow);
      fence_async_shared();
      mbar_arrive(&sm.q_full);
      __syncwarp();
      named_barrier_sync(1, kSoftmaxThreads);  // q_pow is written; where both O are read by both, that is done
      ++n_seg;
      const int rr = MODE == kPair ? t * kRows + tr : tr;  // row of the unit
      const bool mine = rr < nrow;
      const bool idle = (MODE == kPair ? t * kRows : 0) + (warp & 3) * 32 >= nrow;  // a warp without rows
      const int r = row0 + (mine ? rr : 0);
      const int qp = PACKED && mine ? q_pow[rr] : 0;
      float m = kNoMax, up = 0.f;  // O is in units of 2^(m + up)
      float slack = kSlack;  // (packed: none for a reference from kExact on)
      uint64_t l = 0;  // two partial sums, in units of 2^m
      const int before = jobs;
      int it = it0;
      for (int u = seg.k0; u < seg.k1; ++u, ++it) {
        if (!works(t, it, nrow)) continue;
        const int job = jobs++, buf = job & 1;
        wait_or_die(&sm.s_full[t][buf], (job >> 1) & 1, dead, err);
        if (!idle) {
          tc_fence_after();
          // Logits are in units of scale (times the row's and the tile's powers).
          float sc = P.a.scale_log2, lift = 0.f;
          if constexpr (PACKED) {
            // (by halves: no product of two of the three leaves fp32's range unless all three do)
            const int2 f = sm.pow[it % kPowRing];
            const int e = f.x + qp, half = e >> 1;
            sc = sc * pow2(half) * pow2(e - half), lift = (float)f.y;
          }
          const uint64_t sc2 = pair2(sc, sc);
          // 32 tokens at a time: 64 logits would not fit the registers beside the rest.
#pragma unroll 1
          for (int q = 0; q < 2; ++q) {
            float x[32];
            {
              uint32_t a[32];
              tc_ld_rows<32>(tm_s(t, buf) + 32 * q + lanes, a);
              tc_wait_ld();
#pragma unroll
              for (int c = 0; c < 32; ++c) x[c] = __uint_as_float(a[c]);
            }
#pragma unroll
            for (int c = 0; c < 32; c += 2) split2(mul2(pair2(x[c], x[c + 1]), sc2), x[c], x[c + 1]);
            const int j0 = u * kTile + 32 * q - (seg.len - P.a.n_q);
            if (j0 + 32 > 0) {
              const uint32_t* mask = P.a.mask + seg.b * P.a.mask_stride + (int64_t)(r / P.G) * P.words;
              const uint32_t bits = bits_at(j0, P.a.n_q, P.words, [&](int w) { return mask[w]; });
#pragma unroll
              for (int c = 0; c < 32; ++c)
                if (!(bits >> c & 1u)) x[c] = -INFINITY;
            }
            float mx[4] = {x[0], x[1], x[2], x[3]};
#pragma unroll
            for (int c = 4; c + 4 < 32; c += 8)
#pragma unroll
              for (int e = 0; e < 4; ++e) mx[e] = max3(mx[e], x[c + e], x[c + 4 + e]);
#pragma unroll
            for (int e = 0; e < 4; ++e) mx[e] = fmaxf(mx[e], x[28 + e]);
            // rows past the unit's hold anything: they must not move the references of this warp's others
            const float top = mine ? fmaxf(max3(mx[0], mx[1], mx[2]), mx[3]) : -INFINITY;
            float from = m;
            if (__any_sync(0xffffffffu, top - m > slack || (PACKED && top - m + lift - up > kSlack))) {
              const float mn = fmaxf(m, rintf(top)), fell = m - mn;
              float f = ex2(fell);
              l = mul2(l, pair2(f, f));
              if constexpr (PACKED) {
                const float was = up + fell;
                up = fmaxf(was, rintf(top - mn + lift));
                f = ex2(was - up);
              }
              from = m = mn;
              if constexpr (PACKED) {
                // A reference that c - m would round comes off first (and from now on in every half).
                const bool far = fabsf(m) >= kExact && m != kNoMax;
                slack = far ? -INFINITY : kSlack;
                from = far ? 0.f : m;
#pragma unroll
                for (int i = 0; i < 32; i += 2) split2(add2(pair2(x[i], x[i + 1]), pair2(from - m, from - m)), x[i], x[i + 1]);
              }
              if (job > before) {
                wait_or_die(&sm.pv_done[t][(job - 1) & 1], ((job - 1) >> 1) & 1, dead, err);
                tc_fence_after();
#pragma unroll 1
                for (int k = 0; k < D / 32; ++k) {
                  uint32_t o[32];
                  tc_ld_rows<32>(tm_o(t) + 32 * k + lanes, o);
                  tc_wait_ld();
#pragma unroll
                  for (int c = 0; c < 32; ++c) o[c] = __float_as_uint(__uint_as_float(o[c]) * f);
                  tc_st_rows<32>(tm_o(t) + 32 * k + lanes, o);
                }
                tc_wait_st();  // the tile's other half may load these columns again
              }
              if (q > 0) {
                // the tile's first half is written: f is a power of two, which P takes exactly
                uint32_t w[16];
                tc_wait_st();
                tc_ld_rows<16>(tm_s(t, buf) + lanes, w);
                tc_wait_ld();
#pragma unroll
                for (int c = 0; c < 16; ++c) {
                  if constexpr (PACKED) {
                    const float2 v = __half22float2(half2_of(w[c]));
                    w[c] = fp16x2(v.x * f, v.y * f);
                  } else {
                    float v0, v1;
                    bf16x2_to_f32(w[c], v0, v1);
                    w[c] = bf2(v0 * f, v1 * f);
                  }
                }
                tc_st_rows<16>(tm_s(t, buf) + lanes, w);
              }
            }
            __syncwarp();
            const float c = PACKED ? fmaxf(lift - up, kLeast) : 0.f;
            const uint64_t mm = pair2(c - from, c - from);
            uint64_t sum = 0, other = 0;
            uint32_t w[16];
#pragma unroll
            for (int i = 0; i < 16; i += 2) {
              float e0, e1, e2, e3;
              split2(add2(pair2(x[2 * i], x[2 * i + 1]), mm), e0, e1);
              split2(add2(pair2(x[2 * i + 2], x[2 * i + 3]), mm), e2, e3);
              e0 = ex2(e0), e1 = ex2(e1), e2 = ex2(e2), e3 = ex2(e3);
              sum = add2(sum, pair2(e0, e1));
              other = add2(other, pair2(e2, e3));
              w[i] = PACKED ? fp16x2(e0, e1) : bf2(e0, e1);
              w[i + 1] = PACKED ? fp16x2(e2, e3) : bf2(e2, e3);
            }
            sum = add2(sum, other);
            if constexpr (PACKED) {
              const float back = ex2(-c);
              l = fma2(sum, pair2(back, back), l);
            } else {
              l = add2(l, sum);
            }
            tc_st_rows<16>(tm_s(t, buf) + 16 * q + lanes, w);
          }
          tc_wait_st();
          tc_fence_before();
        }
        mbar_arrive(&sm.p_full[t][buf]);
      }
      // Tiles that each warpgroup took of this segment.
      const int n = seg.k1 - seg.k0;
      auto taken = [&](int k) {
        return MODE == kTurns ? (n + (((it0 & 1) == k) ? 1 : 0)) / 2 : works(k, 0, nrow) ? n : 0;
      };
      const int took0 = taken(0), took1 = taken(1);
      others += t ? took0 : took1;
      it0 += n;
      // Output of the segment: O / sum, or that in a record with the reference and the sum, to be merged.
      const bool whole = seg.k0 == 0 && seg.k1 == seg.n;
      const int64_t slot = 2 * (int64_t)blockIdx.x + (seg.k0 > 0 ? 0 : 1);
      if (threadIdx.x == 0) {
        int2* meta = P.meta + (int64_t)seg.b * P.a.lv.hkv * P.n_rt + seg.x;
        if (seg.k0 == 0) meta->x = whole ? -1 : (int)blockIdx.x;
        if (seg.k1 == seg.n) meta->y = (int)blockIdx.x;
      }
      float l0, l1;
      split2(l, l0, l1);
      float sum = l0 + l1, f[2] = {1.f, 0.f};
      // kTurns, kSolo: each warpgroup takes half of the columns of both O.
      const bool shared_rows = MODE != kPair;
      if (shared_rows) {
        sm.m[t][tr] = m;
        sm.l[t][tr] = sum;
        if constexpr (PACKED) sm.up[t][tr] = up;
        __syncwarp();
        named_barrier_sync(1, kSoftmaxThreads);
        const float m0 = sm.m[0][tr], m1 = sm.m[1][tr];
        m = fmaxf(m0, m1);
        f[0] = ex2(m0 - m), f[1] = ex2(m1 - m);
        sum = f[0] * sm.l[0][tr] + f[1] * sm.l[1][tr];
        if constexpr (PACKED) {
          const float u0 = sm.up[0][tr] + (m0 - m), u1 = sm.up[1][tr] + (m1 - m);
          up = fmaxf(u0, u1);
          f[0] = ex2(u0 - up), f[1] = ex2(u1 - up);
        }
      }
      const int64_t rec = slot * P.rec_rows + rr;
      if (!whole && mine && (!shared_rows || t == 0)) P.ml[rec] = make_float2(m, sum);
      // the last product of this warpgroup's O, and of the other's where both are read
      auto settled = [&](int k, int last) { wait_or_die(&sm.pv_done[k][last & 1], (last >> 1) & 1, dead, err); };
      if ((t ? took1 : took0) > 0) settled(t, jobs - 1);
      if (shared_rows && (t ? took0 : took1) > 0) settled(t ^ 1, others - 1);
      tc_fence_after();
      if (!idle) {
        const float inv = sum > 0.f ? (PACKED ? ex2(up) : 1.f) / sum : 0.f;
        f[0] *= inv, f[1] *= inv;
        const int i = r / P.G, g = r - i * P.G;
        uint16_t* out = P.a.out + (((int64_t)seg.b * P.a.n_q + i) * P.a.Hq + kvh * P.G + g) * D;
        float4* acc = reinterpret_cast<float4*>(P.acc) + slot * (D / 4) * P.rec_rows + rr;
        const int c0 = shared_rows ? t * (D / 64) : 0, c1 = shared_rows ? c0 + D / 64 : D / 32;
#pragma unroll 1
        for (int q = c0; q < c1; ++q) {
          float o[32];
          uint32_t a[32];
          // The tensor-memory loads want the whole warp at once, which has just stored by rows.
          __syncwarp();
          if (shared_rows && took0 == 0) {
#pragma unroll
            for (int c = 0; c < 32; ++c) o[c] = 0.f;
          } else {
            tc_ld_rows<32>(tm_o(shared_rows ? 0 : t) + 32 * q + lanes, a);
            tc_wait_ld();
#pragma unroll
            for (int c = 0; c < 32; ++c) o[c] = __uint_as_float(a[c]) * f[0];
          }
          if (MODE == kTurns && took1 > 0) {
            tc_ld_rows<32>(tm_o(1) + 32 * q + lanes, a);
            tc_wait_ld();
#pragma unroll
            for (int c = 0; c < 32; ++c) o[c] = fmaf(__uint_as_float(a[c]), f[1], o[c]);
          }
          if constexpr (VB == 4) {
            float y[32];
#pragma unroll
            for (int c = 0; c < 32; ++c) y[c] = o[octet_column(c)];
#pragma unroll
            for (int c = 0; c < 32; ++c) o[c] = y[c];
          }
          if (mine && whole) {
#pragma unroll
            for (int c = 0; c < 4; ++c)
              reinterpret_cast<uint4*>(out + 32 * q)[c] =
                  make_uint4(bf2(o[8 * c], o[8 * c + 1]), bf2(o[8 * c + 2], o[8 * c + 3]), bf2(o[8 * c + 4], o[8 * c + 5]),
                             bf2(o[8 * c + 6], o[8 * c + 7]));
          } else if (mine) {
#pragma unroll
            for (int c = 0; c < 8; ++c)
              acc[(int64_t)(8 * q + c) * P.rec_rows] = make_float4(o[4 * c], o[4 * c + 1], o[4 * c + 2], o[4 * c + 3]);
          }
        }
      }
      __syncwarp();
      tc_fence_before();
    }
    mbar_arrive(&sm.done);
    return;
  }
  if (warp < L::kFeeder0 / 32) {
    // -------------------------------------------------------------------- MMAs
    if constexpr (PACKED) asm volatile("setmaxnreg.dec.sync.aligned.u32 40;");
    if constexpr (PACKED) {
      if (warp == 10) {
        // The tiles' places, kAtRing tiles ahead of the feeders.
        Feed feed, next;  // 16 tiles each
        int it = 0;
        auto put = [&](const Place& p) {
          const int slot = it % kAtRing;
          if (it >= kAtRing) wait_or_die(&sm.at_empty[slot], (it / kAtRing - 1) & 1, dead, err);
          if (lane == 0) {
            sm.at[slot] = p;
            mbar_arrive(&sm.at_full[slot]);
          }
          __syncwarp();
          ++it;
        };
        while (walk.next(P, seg)) {
          const int kvh = seg.x / P.n_rt;
          feed.see(P, seg);
          next.look_up(P, seg, seg.k0);
          for (int u = seg.k0; u < seg.k1; ++u) {
            const int i = (u - seg.k0) & 15;
            if (i == 0) {
              feed.base = next.base, feed.r = next.r;
              next.look_up(P, seg, u + 16);
            }
            const uint2 live = feed.tokens(P, seg, u);
            Place p;
            p.slab0 = lane_ptr(feed.base, 2 * i);
            p.slab1 = lane_ptr(feed.base, 2 * i + 1);
            p.row0 = (uint32_t)(__shfl_sync(0xffffffffu, feed.r, 2 * i) * kBlockTokens * P.a.lv.hkv + kvh);
            p.row1 = (uint32_t)(__shfl_sync(0xffffffffu, feed.r, 2 * i + 1) * kBlockTokens * P.a.lv.hkv + kvh);
            p.live0 = live.x;
            p.live1 = live.y;
            put(p);
          }
        }
        // one end for each team
        for (int k = 0; k < L::kTeams; ++k) put(Place{nullptr, nullptr, kNoTile, 0u, 0u, 0u});
        return;
      }
    }
    if (warp > 9) return;
    bool alive = true;
    auto ready = [&](uint64_t* bar, uint32_t parity) { alive = alive && warp_wait(bar, parity, dead, err); };
    if (warp == 8) {
      // -------------------------------------------------------------- S = Q K^T
      constexpr uint32_t id_s = tc_idesc(kRows, kTile, false, false, PACKED);
      const uint64_t d_q = tc_desc(smem_u32(qs), 16, 1024), d_k = tc_desc(smem_u32(ks), 16, 1024);
      int it = 0, n_seg = 0, jobs[2] = {0, 0};
      uint32_t slot = 0, round = 0;
      while (alive && walk.next(P, seg)) {
        const int nrow = uniform(min(L::kTileRows, P.rows - seg.x % P.n_rt * L::kTileRows));
        const int n = uniform(seg.k1 - seg.k0);
        ready(&sm.q_full, n_seg++ & 1);
        for (int i = 0; alive && i < n; ++i, ++it) {
          ready(&sm.k_full[slot], round & 1);
          fence_async_shared();  // the copies' writes, seen through the barrier, before the product's reads
#pragma unroll
          for (int t = 0; t < 2; ++t) {
            if (!works(t, it, nrow)) continue;
            const int buf = jobs[t] & 1;
            // the P that lay here has met its values
            if (jobs[t] >= 2) ready(&sm.pv_done[t][buf], ((jobs[t] >> 1) - 1) & 1);
            tc_fence_after();
            if (alive && elect_one()) {
              const uint64_t q = d_q + ((MODE == kPair ? t * (kRows * D * 2) : 0) >> 4), k = d_k + ((slot * L::kSlot) >> 4);
#pragma unroll
              for (int c = 0; c < D / 16; ++c)
                tc_mma(tm_s(t, buf), q + (((c >> 2) * (kRows * 128) + (c & 3) * 32) >> 4),
                       k + (((c >> 2) * (kTile * 128) + (c & 3) * 32) >> 4), id_s, c > 0);
              tc_commit(&sm.s_full[t][buf]);
            }
            ++jobs[t];
          }
          if (alive && elect_one()) {
            tc_commit(&sm.k_empty[slot]);
            if (i == n - 1) tc_commit(&sm.q_empty);
          }
          if (++slot == L::kK) slot = 0, ++round;
        }
      }
      __syncwarp();
      if (elect_one()) tc_commit(&sm.drain[0]);
      // every MMA has completed, and the softmax warps have read their last column
      mbar_wait_bounded(&sm.drain[0], 0, err);
      __syncwarp();
      mbar_wait_bounded(&sm.drain[1], 0, err);
      __syncwarp();
      mbar_wait_bounded(&sm.done, 0, err);
      tc_fence_after();
      __syncwarp();
      tc_dealloc(tmem, 512);
      return;
    }
    // ---------------------------------------------------------------- O += P V
    constexpr uint32_t id_o = tc_idesc(kRows, D, false, true, PACKED);
    const uint64_t d_v = tc_desc(smem_u32(vs), kTile * 128, 1024);
    int it = 0, jobs[2] = {0, 0};
    uint32_t slot = 0, round = 0;
    while (alive && walk.next(P, seg)) {
      const int nrow = uniform(min(L::kTileRows, P.rows - seg.x % P.n_rt * L::kTileRows));
      const int n = uniform(seg.k1 - seg.k0), first[2] = {jobs[0], jobs[1]};
      for (int i = 0; alive && i < n; ++i, ++it) {
        ready(&sm.v_full[slot], round & 1);
        fence_async_shared();
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          if (!works(t, it, nrow)) continue;
          const int buf = jobs[t] & 1;
          ready(&sm.p_full[t][buf], (jobs[t] >> 1) & 1);
          tc_fence_after();
          if (alive && elect_one()) {
            const uint64_t v = d_v + ((slot * L::kSlot) >> 4);
#pragma unroll
            for (int c = 0; c < kTile / 16; ++c)
              tc_mma_ts(tm_o(t), tm_s(t, buf) + 8 * c, v + ((c * 2048) >> 4), id_o, jobs[t] > first[t] || c > 0);
            tc_commit(&sm.pv_done[t][buf]);
          }
          ++jobs[t];
        }
        if (alive && elect_one()) tc_commit(&sm.v_empty[slot]);
        if (++slot == L::kV) slot = 0, ++round;
      }
    }
    __syncwarp();
    if (elect_one()) tc_commit(&sm.drain[1]);
    return;
  }
  if constexpr (!PACKED) {
    // ------------------------------------------------------------------ copies
    constexpr int CPT = D / 8;                  // 16-byte pieces of a token's row
    constexpr int TPP = L::kFeeders / CPT;      // tokens a pass
    const int tid = threadIdx.x - L::kFeeder0;
    const int c = tid % CPT, tk = tid / CPT;
    const uint64_t policy = P.n_rt == 1 ? l2_policy_evict_first() : l2_policy_evict_normal();
    const int64_t v_off = (int64_t)P.a.lv.slab_blocks * kBlockTokens * P.a.lv.hkv * (D * 2);  // a slab's values follow its keys
    const int64_t token = (int64_t)P.a.lv.hkv * (D * 2);
    uint32_t kslot = 0, kround = 0, vslot = 0, vround = 0;
    Feed feed;
    while (walk.next(P, seg)) {
      const int kvh = seg.x / P.n_rt;
      feed.see(P, seg);
      for (int ub = seg.k0; ub < seg.k1; ub += 16) {
        feed.look_up(P, seg, ub);
        const int ue = min(ub + 16, seg.k1);
        for (int u = ub; u < ue; ++u) {
          const uint2 live = feed.tokens(P, seg, u);
          const uint8_t* blk[2];
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            blk[k] = lane_ptr(feed.base, 2 * (u - ub) + k);
            const int row = __shfl_sync(0xffffffffu, feed.r, 2 * (u - ub) + k);
            if (blk[k]) blk[k] += (int64_t)row * kBlockTokens * token + (int64_t)kvh * (D * 2) + c * 16;
          }
          auto copy = [&](uint8_t* dst, int64_t off, uint64_t* full) {
#pragma unroll
            for (int p = 0; p < kTile / TPP; ++p) {
              const int tok = p * TPP + tk;
              const uint8_t* from = blk[p * TPP / 32];
              const bool ok = from && ((p * TPP < 32 ? live.x : live.y) >> (tok & 31) & 1u);
              cp_async16(smem_u32(dst) + swizzled(tok, c, kTile * 128),
                         ok ? from + off + (tok & 31) * token : reinterpret_cast<const uint8_t*>(P.a.q), ok, policy);
            }
            cp_async_arrive(full);
          };
          if (kround > 0) wait_or_die(&sm.k_empty[kslot], (kround - 1) & 1, dead, err);
          copy(ks + kslot * L::kSlot, 0, &sm.k_full[kslot]);
          if (++kslot == L::kK) kslot = 0, ++kround;
          if (vround > 0) wait_or_die(&sm.v_empty[vslot], (vround - 1) & 1, dead, err);
          copy(vs + vslot * L::kSlot, v_off, &sm.v_full[vslot]);
          if (++vslot == L::kV) vslot = 0, ++vround;
        }
      }
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
  } else {
    // --------------------------------------------------------------- expansion
    asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
    const LayerView& lv = P.a.lv;
    const uint32_t slab_rows = (uint32_t)(lv.slab_blocks * kBlockTokens * lv.hkv);
    const uint32_t v_off = slab_rows * lv.row_bytes[0], km_off = v_off + slab_rows * lv.row_bytes[1],
                   vm_off = km_off + slab_rows * lv.row_bytes[2];
    using KP = Pieces<D, KB>;
    using VP = Pieces<D, VB>;
    const KP kp(lv.hkv, lv.row_bytes[0], lv.row_bytes[2], 0, km_off, P.group_log);
    const VP vp(lv.hkv, lv.row_bytes[1], lv.row_bytes[2], v_off, vm_off, P.group_log);
    // Unit j of the keys goes to warp j % W of the team, the values' units to the warps from there on.
    constexpr int W = L::kWarps / L::kTeams, KN = (KP::kUnits + W - 1) / W, VN = (VP::kUnits + W - 1) / W;
    const int w = warp - L::kFeeder0 / 32, team = w / W;
    const int kw = w % W, vw = (kw - KP::kUnits % W + W) % W;
    Place at;
    // The place of tile `it`; false: none is left.
    auto next_place = [&](int it) {
      wait_or_die(&sm.at_full[it % kAtRing], (it / kAtRing) & 1, dead, err);
      at = sm.at[it % kAtRing];
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm.at_empty[it % kAtRing]);
      if (!at.slab0) at.live0 = 0;
      if (!at.slab1) at.live1 = 0;
      return at.row0 != kNoTile && !__any_sync(0xffffffffu, *dead);
    };
    // (Loaded ahead, in registers, the pieces' arrival was waited for all the same: by the loads from
    // shared memory that came in between.  More teams cover it.)
    uint4 kc[KN], vc[VN];
    float2 km[KN], vm[VN];
    auto load_key = [&](int j) {
      const int g = kw + W * j;
      if (KP::kUnits % W && g >= KP::kUnits) return;
      const bool k = g * KP::kTokens >= 32;
      kp.load(k ? at.slab1 : at.slab0, k ? at.row1 : at.row0, g, k ? at.live1 : at.live0, kc[j], km[j]);
    };
    auto load_value = [&](int j) {
      const int g = vw + W * j;
      if (VP::kUnits % W && g >= VP::kUnits) return;
      const bool k = g * VP::kTokens >= 32;
      vp.load(k ? at.slab1 : at.slab0, k ? at.row1 : at.row0, g, k ? at.live1 : at.live0, vc[j], vm[j]);
    };
    for (int it = team; next_place(it); it += L::kTeams) {
      const int kslot = it % L::kK, vslot = it % L::kV;
#pragma unroll
      for (int j = 0; j < KN; ++j) load_key(j);
#pragma unroll
      for (int j = 0; j < VN; ++j) load_value(j);
      if (it >= L::kK) wait_or_die(&sm.k_empty[kslot], (it / L::kK - 1) & 1, dead, err);
      // The tile's largest key and value: of the warp's pieces, then over the team's warps.
      float kmax = 0.f, vmax = 0.f;
#pragma unroll
      for (int j = 0; j < KN; ++j)
        if (KP::kUnits % W == 0 || kw + W * j < KP::kUnits) kmax = fmaxf(kmax, KP::widest(km[j]));
#pragma unroll
      for (int j = 0; j < VN; ++j)
        if (VP::kUnits % W == 0 || vw + W * j < VP::kUnits) vmax = fmaxf(vmax, VP::widest(vm[j]));
#pragma unroll
      for (int off = 16; off > 0; off >>= 1) {
        kmax = fmaxf(kmax, __shfl_xor_sync(0xffffffffu, kmax, off));
        vmax = fmaxf(vmax, __shfl_xor_sync(0xffffffffu, vmax, off));
      }
      float2* all = sm.widest[team][it / L::kTeams & 1];
      if (lane == 0) all[kw] = make_float2(kmax, vmax);
      __syncwarp();
      named_barrier_sync(2 + team, 32 * W);
#pragma unroll
      for (int i = 0; i < W; ++i) kmax = fmaxf(kmax, all[i].x), vmax = fmaxf(vmax, all[i].y);
      const int kx = power_of(kmax), vx = power_of(vmax);
      const float kf = pow2(-kx), vf = pow2(-vx), ks2 = pow2(KB - kx), vs2 = pow2(VB - vx);
      if (kw == 0 && lane == 0) sm.pow[it % kPowRing] = make_int2(kx, vx);
#pragma unroll
      for (int j = 0; j < KN; ++j) {
        const int g = kw + W * j;
        if (KP::kUnits % W && g >= KP::kUnits) continue;
        expand<KB>(kc[j], km[j].x * ks2, km[j].y * kf, ks + kslot * L::kSlot, g * KP::kTokens + kp.token, kp.value);
      }
      // (the warps that issue the products order these writes before the products' reads)
      mbar_arrive(&sm.k_full[kslot]);
      if (it >= L::kV) wait_or_die(&sm.v_empty[vslot], (it / L::kV - 1) & 1, dead, err);
#pragma unroll
      for (int j = 0; j < VN; ++j) {
        const int g = vw + W * j;
        if (VP::kUnits % W && g >= VP::kUnits) continue;
        expand<VB>(vc[j], vm[j].x * vs2, vm[j].y * vf, vs + vslot * L::kSlot, g * VP::kTokens + vp.token, vp.value);
      }
      mbar_arrive(&sm.v_full[vslot]);
    }
  }
}

template <int D, int MODE, int KB, int VB>
cudaError_t launch(const Params& P) {
  using L = Plan<D, MODE, KB, VB>;
  if constexpr (L::PACKED) {
    static const bool regs_ok = [] {
      cudaFuncAttributes f;
      return cudaFuncGetAttributes(&f, tree_attn_kernel<D, MODE, KB, VB>) == cudaSuccess && f.numRegs == kLaunchRegs;
    }();
    if (!regs_ok) return cudaErrorInvalidDeviceFunction;
  }
  static std::atomic<uint64_t> raised{0};  // devices whose shared-memory limit is set
  return tc_launch(tree_attn_kernel<D, MODE, KB, VB>, dim3((unsigned)(P.cols * P.col_ctas)), L::kThreads, (size_t)L::kSmem, P.a.stream, P,
                   P.a.device, &raised);
}

// KB, VB: bits a key and a value (16: bf16).
template <int KB, int VB>
cudaError_t launch_mode(const Params& P, int mode) {
  if (P.a.D == 256) return launch<256, kSolo, KB, VB>(P);
  if (P.a.D == 128) return mode == kPair ? launch<128, kPair, KB, VB>(P) : launch<128, kTurns, KB, VB>(P);
  return mode == kPair ? launch<64, kPair, KB, VB>(P) : launch<64, kTurns, KB, VB>(P);
}

}  // namespace tree

// The attention kernel by format, defined in tree_*.cu.
cudaError_t launch_tree_bf16(const tree::Params& P, int mode);
cudaError_t launch_tree_k4v4(const tree::Params& P, int mode);
cudaError_t launch_tree_k8v4(const tree::Params& P, int mode);
cudaError_t launch_tree_k8v8(const tree::Params& P, int mode);

}  // namespace pkv
