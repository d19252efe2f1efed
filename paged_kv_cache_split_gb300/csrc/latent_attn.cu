// latent_attn.cu — absorbed attention over a latent pool, on the tensor cores.
//
//   x[t, n] = scale (ql[n] . c_t + qr[n] . r_t)        n: a row (query, head) of a sequence
//   o[n]    = sum_t exp2(x[t, n] - m[n]) c_t / sum_t exp2(x[t, n] - m[n])
//
// Every token's row of R + 64 values is read once and used twice, as a key by all rows
// and as a value (its first R).  With H rows a token costs 2 H (2R + 64) operations and
// 2 (R + 64) bytes: at H = 128 both sides of the roofline take about as long, below that
// HBM bounds.
//
// Layout.  Both products have the tokens, or the latent's dims, as the MMA's M and the
// rows as its N, so the head count sets N (16, 32 or 64 rows a tile; more rows take more
// tiles) and small head counts waste nothing:
//   S^T [64 tokens x N] = K [64 x (R + 64)] Q^T      K as it lies in shared memory
//   O^T [R x N]        += V^T [R x 64] P^T [64 x N]  the same bytes, read MN-major
// O^T stays in tensor memory (R / 128 blocks of N columns), S^T is double-buffered there.
//
// A CTA runs one warp that issues copies, one that issues MMAs and four for the softmax.
// Cache rows arrive by TMA, 32 tokens x 256 values a copy, into a ring of 32 KB slots
// (64 tokens x 256 latent values) and one of 8 KB slots (64 tokens' position keys); the
// next tile's S^T product runs while the softmax works on this one, and a slot is refilled
// as soon as its blocks of O^T have been added to.  The softmax reference m moves only when
// a logit passes it by more than 2^8 (all rescaling of O^T is skipped otherwise): p is
// then at most 2^8 and loses nothing in bf16, and the sums are FP32.
//
// Tiles of every sequence are laid end to end and split evenly over groups of CTAs (one
// CTA per row tile in a group).  A sequence inside one CTA's share is written directly; a
// split one leaves FP32 records that a second kernel merges in order.
//
// Measured (one GB300, both kernels, in a captured graph): 16 x 16384 tokens, 32 heads 59.5 us,
// 5.10 TB/s (the card copies at 6.79; DRAM reads equal the rows' bytes); 64 sequences of up
// to 8192, 16 heads 55 us, 4.93 TB/s; 16 x 8192 with 16 / 32 / 64 / 128 heads 34 / 36 / 42 /
// 67 us; 1 x 1000, 16 heads 8.9 us.  Up to 32 rows a CTA streams at 6 TB/s x 1/152 and the
// rest is the start (5 us: lengths, block table, slab address, first rows) and the end
// (records, merge: 6 us).  With 64 rows a tile the ring holds two tiles only and a copy's
// latency shows (1.7 us a tile); 128 heads also read every row twice, the second time from L2.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "latent.cuh"
#include "tcgen05.cuh"

namespace pkv {
namespace {

constexpr int kTile = 64;             // tokens a tile
constexpr int kSoftmaxThreads = 128;  // warps 0..3
constexpr int kThreads = 192;         // + warp 4: copies, warp 5: MMAs
constexpr int kChunkBytes = kTile * 128;               // 64 tokens x 64 values
constexpr int kQuadBytes = kLatentQuad * kChunkBytes;  // 64 tokens x 256 values: [8 x 8 tokens][4][8][128 bytes]
constexpr int kAtom = 1024;                            // eight tokens of a column: the swizzle's atom
constexpr float kSlack = 8.0f;        // log2 of how far a logit may pass the reference
constexpr float kNoMax = -3.402823466e38f;  // the reference before any visible token: no logit is below it
constexpr int kSmemLimit = 232448;    // 227 KB opt-in shared memory per block
constexpr int kSmall = 3 * 1024;      // alignment (1024), barriers and per-row values
constexpr int kInFlight = 8;          // more tiles than the rings hold

// Cost of a sequence's start in quarter tiles, in the split over the CTAs: its queries are
// loaded and its output or record written.
constexpr int kSegCost = 8;
constexpr int kCost = 4;

// Ring sizes: the next tile's S^T product needs its whole tile while this tile's latent
// slots are still held, so two tiles at least; what is left of shared memory goes to more.
template <int R, int N>
struct Plan {
  static constexpr int kQuads = R / 256;  // latent slots a tile
  static constexpr int kQBytes = N * (R + kRope) * 2;
  static constexpr int kPBytes = N * 128;
  static constexpr int kRoom = kSmemLimit - kSmall - kQBytes - kPBytes;
  static constexpr int kTileBytes = kQuads * kQuadBytes + kChunkBytes;
  static constexpr int kRopeSlots =
      kRoom / kTileBytes + (kRoom % kTileBytes >= kQuadBytes + kChunkBytes ? 1 : 0);
  static constexpr int kQuadSlots = (kRoom - kRopeSlots * kChunkBytes) / kQuadBytes;
  static constexpr int kSmem = kSmall + kQBytes + kPBytes + kQuadSlots * kQuadBytes + kRopeSlots * kChunkBytes;
  static constexpr int kTmemUsed = (2 + R / 128) * N;  // two S^T buffers, O^T
  static constexpr int kTmem = kTmemUsed <= 64 ? 64 : kTmemUsed <= 128 ? 128 : kTmemUsed <= 256 ? 256 : 512;
  static_assert(kQuadSlots >= 2 * kQuads && kRopeSlots >= 2, "two tiles have to fit");
  static_assert(kRopeSlots < kInFlight && kQuadSlots < kInFlight * kQuads, "tiles in flight");
  static_assert(kSmem <= kSmemLimit && kTmemUsed <= 512, "shared memory or TMEM");
};

struct Params {
  LatentAttnArgs a;
  CUtensorMap ql_map, qr_map;  // the queries' rows, in boxes of 64 values x N rows
  int rows;     // n_q * Hq: rows of a sequence
  int n_rt;     // row tiles of a sequence
  int groups;   // CTAs along the token axis (each with n_rt row tiles)
  int2* meta;   // [B][n_rt]: first record slot of a split sequence (-1: written directly), last group
  float2* ml;   // [2 * grid][N]: reference and sum of a record's rows
  float* acc;   // [2 * grid][N][R]
};

// Tokens that the last (most) of tile rt's rows sees, 0 for an unused or bad sequence.
template <int N>
__device__ __forceinline__ int32_t visible(const Params& P, int b, int rt, int32_t* len) {
  bool bad;
  const int32_t L =
      latent_ctx(P.a.ctx[b], (int64_t)P.a.max_blocks * kBlockTokens, P.a.n_q, &bad);
  *len = L;
  if (L == 0) return 0;
  const int last = min(P.rows, (rt + 1) * N) - 1;
  return L - P.a.n_q + last / P.a.Hq + 1;
}

// A CTA's share of the tiles.  Tile k of sequence b, the u-th of all, sits at position
// kCost u + kSegCost (b + 1); group g holds the positions [g V, (g + 1) V).  V is at least
// kCost, so the groups that hold a sequence's tiles are consecutive.
struct Segment {
  int b, len, vis;   // sequence, its length, tokens the last row sees
  int k0, k1, n;     // this CTA's tiles of it, and all of them
};

// The walk's values are warp-uniform and known as such: what the copies and MMAs are issued
// with follows from them.
struct Walk {
  int b;
  int64_t up;      // tiles before sequence b
  int64_t lo, hi;  // positions of this CTA

  template <int N>
  __device__ __forceinline__ bool next(const Params& P, int rt, Segment& s) {
    while (b < P.a.B) {
      const int64_t base = kCost * up + (int64_t)kSegCost * (b + 1);
      if (base >= hi) return false;
      s.b = b;
      s.vis = uniform(visible<N>(P, b, rt, &s.len));
      s.len = uniform(s.len);
      s.n = (s.vis + kTile - 1) / kTile;
      const int64_t f = base >= lo ? 0 : (lo - base + kCost - 1) / kCost;
      const int64_t e = (hi - base + kCost - 1) / kCost;
      s.k0 = (int)(f < s.n ? f : s.n);
      s.k1 = (int)(e < s.n ? e : s.n);
      up += s.n;
      ++b;
      if (s.k1 > s.k0) return true;
    }
    return false;
  }
};

// One warp: the CTA's positions and the sequence its walk starts at.  The lengths of the
// first kHeld sequences are read once.
template <int N>
__device__ __forceinline__ Walk start_walk(const Params& P, int rt, int group) {
  constexpr int kHeld = 128;
  const int lane = threadIdx.x & 31;
  auto tiles = [&](int b) -> int32_t {
    int32_t len;
    return b < P.a.B ? (visible<N>(P, b, rt, &len) + kTile - 1) / kTile : 0;
  };
  int32_t held[kHeld / 32];
  int64_t total = 0;
#pragma unroll
  for (int c = 0; c < kHeld / 32; ++c) {
    held[c] = 32 * c < P.a.B ? tiles(32 * c + lane) : 0;
    total += held[c];
  }
  for (int b = kHeld + lane; b < P.a.B; b += 32) total += tiles(b);
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) total += __shfl_xor_sync(0xffffffffu, total, off);
  Walk w;
  const int64_t v = (kCost * total + (int64_t)kSegCost * P.a.B + P.groups - 1) / P.groups;
  const int64_t V = v > kCost ? v : kCost;
  w.lo = group * V;
  w.hi = w.lo + V;
  w.b = P.a.B;
  w.up = total;
  int64_t carry = 0;
  // the first sequence whose last tile reaches the CTA's first position
  auto found = [&](int base, int32_t n) {
    int32_t inc = n;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int32_t y = __shfl_up_sync(0xffffffffu, inc, off);
      if (lane >= off) inc += y;
    }
    const int b = base + lane;
    const unsigned hit = __ballot_sync(
        0xffffffffu, b < P.a.B && kCost * (carry + inc - 1) + (int64_t)kSegCost * (b + 1) >= w.lo);
    if (hit) {
      const int l = __ffs(hit) - 1;
      w.b = base + l;
      w.up = carry + __shfl_sync(0xffffffffu, inc - n, l);
      return true;
    }
    carry += __shfl_sync(0xffffffffu, inc, 31);
    return false;
  };
#pragma unroll
  for (int c = 0; c < kHeld / 32; ++c)
    if (32 * c < P.a.B && found(32 * c, held[c])) return w;
  for (int base = kHeld; base < P.a.B; base += 32)
    if (found(base, tiles(base + lane))) return w;
  return w;
}

// Shared-memory state besides the operands.
template <int R, int N>
struct Small {
  using L = Plan<R, N>;
  uint64_t full[kInFlight];  // by tile: its position keys and all of its latent slots
  uint64_t quad_empty[L::kQuadSlots], rope_empty[L::kRopeSlots];
  uint64_t s_full[2], p_full, pv_done, q_full, q_empty, drain;
  Walk walk;
  uint32_t tmem;
  int dead;          // a wait gave up: every role runs on without waiting or issuing
  int vis[N];        // tokens each row sees
  float fac[N];      // per row: rescale factor, or 1 / sum
  float part[4][N];  // per warp: maxima, or sums
};

__device__ __forceinline__ bool softmax_any(bool p) {
  uint32_t r;
  asm volatile(
      "{ .reg .pred p, q; setp.ne.u32 p, %1, 0; barrier.cta.red.or.pred q, 1, 128, p; selp.u32 %0, 1, 0, q; }"
      : "=r"(r)
      : "r"((uint32_t)p)
      : "memory");
  return r != 0;
}

template <int R, int N>
__global__ void __launch_bounds__(kThreads, 1) latent_attn_kernel(const __grid_constant__ Params P) {
  using L = Plan<R, N>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
  uint8_t* quads = smem;
  uint8_t* ropes = quads + L::kQuadSlots * kQuadBytes;
  uint8_t* qs = ropes + L::kRopeSlots * kChunkBytes;
  uint8_t* ps = qs + L::kQBytes;
  Small<R, N>& sm = *reinterpret_cast<Small<R, N>*>(ps + L::kPBytes);
  static_assert(sizeof(Small<R, N>) <= kSmall - 1024, "small state");

  const int warp = uniform((int)(threadIdx.x >> 5)), lane = threadIdx.x & 31;
  const int rt = blockIdx.x % P.n_rt, group = blockIdx.x / P.n_rt;
  volatile int* dead = &sm.dead;
  int32_t* err = P.a.lv.err;

  if (threadIdx.x == 0) {
    for (int i = 0; i < kInFlight; ++i) mbar_init(&sm.full[i], 1);
    for (int i = 0; i < L::kQuadSlots; ++i) mbar_init(&sm.quad_empty[i], 1);
    for (int i = 0; i < L::kRopeSlots; ++i) mbar_init(&sm.rope_empty[i], 1);
    for (int i = 0; i < 2; ++i) mbar_init(&sm.s_full[i], 1);
    mbar_init(&sm.p_full, kSoftmaxThreads);
    mbar_init(&sm.pv_done, 1);
    mbar_init(&sm.q_full, 1);
    mbar_init(&sm.q_empty, 1);
    mbar_init(&sm.drain, 1);
    sm.dead = 0;
    fence_mbar_init();
  }
  if (warp == 5) tc_alloc(&sm.tmem, L::kTmem);
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (warp == 0) {
    const Walk w = start_walk<N>(P, rt, group);
    if (lane == 0) sm.walk = w;
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = uniform(sm.tmem);
  const uint32_t tm_s = tmem, tm_o = tmem + 2 * N;
  Walk walk = {uniform(sm.walk.b), uniform(sm.walk.up), uniform(sm.walk.lo), uniform(sm.walk.hi)};
  Segment seg;

  if (warp < 4) {
    // ---------------------------------------------------------------- softmax
    const int tid = threadIdx.x;
    const int c2 = 2 * (lane & 3), tq = lane >> 2;
    const uint32_t lanes = (uint32_t)(warp * 32) << 16;
    float m[N / 4], l[N / 4];
    int it = 0;
    while (walk.next<N>(P, rt, seg)) {
      const int row0 = rt * N, nrow = min(N, P.rows - row0);
      const int64_t qrow = (int64_t)seg.b * P.rows + row0;
      if (tid < N) {
        const int r = min(row0 + tid, P.rows - 1);
        sm.vis[tid] = seg.len - P.a.n_q + r / P.a.Hq + 1;
      }
      const int vis_first = seg.len - P.a.n_q + row0 / P.a.Hq + 1;
      softmax_any(false);  // sm.vis is ready
      // A tile's rows past the sequence's are other sequences' queries: with a reference that
      // no logit passes they never move the others' (their own columns hold anything).
#pragma unroll
      for (int k = 0; k < N / 4; ++k) m[k] = 8 * (k >> 1) + c2 + (k & 1) < nrow ? kNoMax : INFINITY, l[k] = 0.f;

      for (int u = seg.k0; u < seg.k1; ++u, ++it) {
        const int buf = it & 1;
        wait_or_die(&sm.s_full[buf], (it >> 1) & 1, dead, err);
        tc_fence_after();
        float x[N / 2];
        {
          uint32_t r[N / 2];
          tc_ld_frag16<N>(tm_s + buf * N + lanes, r);
          tc_wait_ld();
#pragma unroll
          for (int k = 0; k < N / 2; ++k) x[k] = __uint_as_float(r[k]) * P.a.scale_log2;
        }
        if ((u + 1) * kTile > vis_first) {
          const int t0 = u * kTile + 16 * warp + tq;
#pragma unroll
          for (int j = 0; j < N / 8; ++j)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const int v = sm.vis[8 * j + c2 + e];
              if (t0 >= v) x[4 * j + e] = -INFINITY;
              if (t0 + 8 >= v) x[4 * j + 2 + e] = -INFINITY;
            }
        }
        float over = -INFINITY;
#pragma unroll
        for (int j = 0; j < N / 8; ++j)
#pragma unroll
          for (int e = 0; e < 2; ++e)
            over = fmaxf(over, fmaxf(x[4 * j + e], x[4 * j + 2 + e]) - m[2 * j + e]);
        const bool raise = softmax_any(over > kSlack);
        if (it > 0) {
          wait_or_die(&sm.pv_done, (it - 1) & 1, dead, err);
          tc_fence_after();
        }
        if (raise) {
          float cm[N / 4];
#pragma unroll
          for (int k = 0; k < N / 4; ++k) {
            cm[k] = fmaxf(x[4 * (k >> 1) + (k & 1)], x[4 * (k >> 1) + 2 + (k & 1)]);
#pragma unroll
            for (int off = 4; off < 32; off <<= 1) cm[k] = fmaxf(cm[k], __shfl_xor_sync(0xffffffffu, cm[k], off));
            if (lane < 4) sm.part[warp][8 * (k >> 1) + c2 + (k & 1)] = cm[k];
          }
          softmax_any(false);
#pragma unroll
          for (int k = 0; k < N / 4; ++k) {
            const int col = 8 * (k >> 1) + c2 + (k & 1);
            const float mn = fmaxf(fmaxf(fmaxf(sm.part[0][col], sm.part[1][col]), fmaxf(sm.part[2][col], sm.part[3][col])), m[k]);
            const float f = ex2(m[k] - mn);
            m[k] = mn;
            l[k] *= f;
            if (warp == 0 && lane < 4) sm.fac[col] = f;
          }
          softmax_any(false);
          if (u > seg.k0) {
#pragma unroll 1
            for (int mb = 0; mb < R / 128; ++mb)
#pragma unroll 1
              for (int q = 0; q < N; q += 16) {
                uint32_t o[16];
                const uint32_t at = tm_o + mb * N + q + lanes;
                tc_ld_rows<16>(at, o);
                tc_wait_ld();
#pragma unroll
                for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * sm.fac[q + i]);
                tc_st_rows<16>(at, o);
              }
            tc_wait_st();
          }
        }
#pragma unroll
        for (int j = 0; j < N / 8; ++j)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int k = 2 * j + e;
            x[4 * j + e] = ex2(x[4 * j + e] - m[k]);
            x[4 * j + 2 + e] = ex2(x[4 * j + 2 + e] - m[k]);
            l[k] += x[4 * j + e] + x[4 * j + 2 + e];
          }
        // P [N rows][64 tokens]: fragments (8 tokens x 8 rows) stored transposed.
        const int i8 = lane & 7, quad = lane >> 3;
#pragma unroll
        for (int j = 0; j < N / 8; j += 2) {
          const int r = 8 * (j + (quad >> 1)) + i8, chunk = 2 * warp + (quad & 1);
          const uint32_t dst = smem_u32(ps) + r * 128 + ((chunk ^ (r & 7)) << 4);
          asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(dst),
                       "r"(bf2(x[4 * j], x[4 * j + 1])), "r"(bf2(x[4 * j + 2], x[4 * j + 3])),
                       "r"(bf2(x[4 * j + 4], x[4 * j + 5])), "r"(bf2(x[4 * j + 6], x[4 * j + 7]))
                       : "memory");
        }
        // Slots past the last visible token hold anything (0 x NaN is NaN): their values
        // become zero; their keys only reached logits that were masked.
        const int valid = seg.vis - u * kTile;
        if (valid < kTile) {
          constexpr int per = R / 8;  // 16-byte pieces of a token's latent
          for (int i = tid; i < (kTile - valid) * per; i += kSoftmaxThreads) {
            const int t = valid + i / per, w = i % per;
            const int slot = (int)(((unsigned)it * L::kQuads + w / (8 * kLatentQuad)) % L::kQuadSlots);
            const int col = (w >> 3) % kLatentQuad;
            *reinterpret_cast<uint4*>(quads + slot * kQuadBytes + ((t >> 3) * kLatentQuad + col) * kAtom +
                                      (t & 7) * 128 + (w & 7) * 16) = make_uint4(0, 0, 0, 0);
          }
        }
        fence_async_shared();
        tc_fence_before();
        mbar_arrive(&sm.p_full);
      }
      // Output of the segment: O^T / sum, or a record (reference, sum, O^T) to be merged.
      softmax_any(false);  // a warp may still be rescaling O^T by sm.fac, raised in the last tile
#pragma unroll
      for (int k = 0; k < N / 4; ++k) {
#pragma unroll
        for (int off = 4; off < 32; off <<= 1) l[k] += __shfl_xor_sync(0xffffffffu, l[k], off);
        if (lane < 4) sm.part[warp][8 * (k >> 1) + c2 + (k & 1)] = l[k];
        if (warp == 0 && lane < 4) sm.fac[8 * (k >> 1) + c2 + (k & 1)] = m[k];
      }
      softmax_any(false);
      const bool whole = seg.k0 == 0 && seg.k1 == seg.n;
      // record slot: the CTA's first or its last segment (any between is whole)
      const bool first_seg = seg.k0 > 0 || it == seg.k1 - seg.k0;
      const size_t slot = 2 * (size_t)blockIdx.x + (first_seg ? 0 : 1);
      if (tid == 0) {
        int2* meta = P.meta + (size_t)seg.b * P.n_rt + rt;
        if (seg.k0 == 0) meta->x = whole ? -1 : (int)slot;
        if (seg.k1 == seg.n) meta->y = group;
      }
      if (tid < N) {
        const float s = sm.part[0][tid] + sm.part[1][tid] + sm.part[2][tid] + sm.part[3][tid];
        if (whole)
          sm.fac[tid] = 1.f / s;
        else
          P.ml[slot * N + tid] = make_float2(sm.fac[tid], s);
      }
      softmax_any(false);
      wait_or_die(&sm.pv_done, (it - 1) & 1, dead, err);
      tc_fence_after();
#pragma unroll 1
      for (int mb = 0; mb < R / 128; ++mb)
#pragma unroll 1
        for (int q = 0; q < nrow; q += 16) {
          uint32_t o[16];
          tc_ld_rows<16>(tm_o + mb * N + q + lanes, o);
          tc_wait_ld();
          const int d = mb * 128 + tid;
          if (whole) {
            uint16_t* out = P.a.out + (qrow + q) * R + d;
#pragma unroll
            for (int i = 0; i < 16; ++i)
              if (q + i < nrow)
                out[(int64_t)i * R] = __bfloat16_as_ushort(__float2bfloat16_rn(__uint_as_float(o[i]) * sm.fac[q + i]));
          } else {
            float* out = P.acc + (slot * N + q) * R + d;
#pragma unroll
            for (int i = 0; i < 16; ++i)
              if (q + i < nrow) out[i * R] = __uint_as_float(o[i]);
          }
        }
      tc_fence_before();
      softmax_any(false);  // sm.fac, sm.part and sm.vis are free again
    }
  } else if (warp == 4) {
    // ------------------------------------------------------------------ copies
    const uint64_t keep = l2_policy_evict_normal();
    const uint64_t policy = P.n_rt == 1 ? l2_policy_evict_first() : keep;
    uint32_t qs_ = 0, qround = 0, rs_ = 0, rround = 0;  // next slot and round of each ring
    int n_tile = 0, n_seg = 0;                          // started so far
    bool alive = true;
    // The row tile's queries (rows past the sequence's are other rows, or zero: unused).
    auto copy_queries = [&](int qrow) {
      if (n_seg > 0) alive = warp_wait(&sm.q_empty, (n_seg - 1) & 1, dead, err);
      if (!alive) return;
      if (elect_one()) {
        mbar_arrive_expect_tx(&sm.q_full, L::kQBytes);
#pragma unroll 1
        for (int c = 0; c < R / 64; ++c) tma_load_2d(qs + c * N * 128, &P.ql_map, 64 * c, qrow, &sm.q_full, keep);
        tma_load_2d(qs + (R / 64) * N * 128, &P.qr_map, 0, qrow, &sm.q_full, keep);
      }
      ++n_seg;
    };
    while (alive && walk.next<N>(P, rt, seg)) {
      const int nblk = (seg.vis + kBlockTokens - 1) / kBlockTokens;
      const int k0 = uniform(seg.k0), k1 = uniform(seg.k1);
      const int qrow = uniform(seg.b * P.rows + rt * N);
      if (n_seg == 0) copy_queries(qrow);
      for (int ub = k0; alive && ub < k1; ub += 16) {
        // lane l looks up block 2 ub + l of the sequence
        const int j = 2 * ub + lane;
        const uint8_t* map = nullptr;
        int y0 = 0;
        if (j < nblk && j < 2 * k1) {
          const int32_t row = P.a.bt[(int64_t)seg.b * P.a.max_blocks + j];
          if (latent_row_ok(P.a.lv, row)) {
            const int32_t slab = row / P.a.lv.slab_blocks;
            y0 = (row - slab * P.a.lv.slab_blocks) * (kBlockTokens / 8);
            map = P.a.lv.tab.base[(size_t)slab * P.a.lv.tab.stride] + P.a.lv.map_delta;
            latent_maps_acquire(map);
          } else {
            atomicOr(err, ERR_ROW);
          }
        }
        __syncwarp();  // the issuing lane's copies come after the lookups' acquires
        const int ue = min(ub + 16, k1);
        for (int u = ub; u < ue; ++u) {
          const int i = 2 * (u - ub);
          const uint8_t *m0 = lane_ptr(map, i), *m1 = lane_ptr(map, i + 1);
          const int ya = __shfl_sync(0xffffffffu, y0, i), yb = __shfl_sync(0xffffffffu, y0, i + 1);
          const uint32_t bytes = ((m0 != nullptr) + (m1 != nullptr)) * kBlockTokens * (R + kRope) * 2;
          uint64_t* full = &sm.full[n_tile % kInFlight];
          if (rround > 0) alive = warp_wait(&sm.rope_empty[rs_], (rround - 1) & 1, dead, err);
          if (!alive) break;
          if (elect_one()) {
            uint8_t* dst = ropes + rs_ * kChunkBytes;
            mbar_arrive_expect_tx(full, bytes);
            if (m0) latent_copy_column(dst, m0, R / 64, ya, full, policy);
            if (m1) latent_copy_column(dst + kChunkBytes / 2, m1, R / 64, yb, full, policy);
          }
          ++n_tile;
          if (++rs_ == L::kRopeSlots) rs_ = 0, ++rround;
#pragma unroll 1
          for (int p = 0; p < L::kQuads; ++p) {
            if (qround > 0) alive = warp_wait(&sm.quad_empty[qs_], (qround - 1) & 1, dead, err);
            if (!alive) break;
            if (elect_one()) {
              uint8_t* dst = quads + qs_ * kQuadBytes;
              if (m0) latent_copy_quad(dst, m0, kLatentQuad * p, ya, full, policy);
              if (m1) latent_copy_quad(dst + kQuadBytes / 2, m1, kLatentQuad * p, yb, full, policy);
            }
            if (++qs_ == L::kQuadSlots) qs_ = 0, ++qround;
          }
          if (!alive) break;
          // a later segment's queries wait for the products of the one before: after its
          // first tile, which needs no wait
          if (u == k0 && n_tile > 1) copy_queries(qrow);
          if (!alive) break;
        }
      }
    }
    // No copy may be in flight when the CTA ends.  (A role that gave up in the middle of a
    // tile leaves its barrier short of bytes: that wait runs into its limit.)
    for (int i = max(0, n_tile - kInFlight); i < n_tile; ++i)
      mbar_wait_bounded(&sm.full[i % kInFlight], (i / kInFlight) & 1, err);
    if (n_seg > 0) mbar_wait_bounded(&sm.q_full, (n_seg - 1) & 1, err);
  } else {
    // -------------------------------------------------------------------- MMAs
    constexpr uint32_t id_s = tc_idesc(64, N, false, false);
    constexpr uint32_t id_o = tc_idesc(128, N, true, false);
    const uint64_t d_rope = tc_desc(smem_u32(ropes), 16, kAtom), d_quad = tc_desc(smem_u32(quads), 16, kLatentQuad * kAtom);
    const uint64_t d_q = tc_desc(smem_u32(qs), 16, kAtom), d_p = tc_desc(smem_u32(ps), 16, kAtom);
    const uint64_t d_v = tc_desc(smem_u32(quads), kAtom, kLatentQuad * kAtom);
    int it = 0, n_seg = 0;
    uint32_t ks = 0, vs = 0, rs_ = 0;  // slots of the next tile's K, V and position keys
    bool alive = true, pending_first = false;
    // O^T (+)= V^T P^T of tile i
    auto add_values = [&](int i, bool first) {
      alive = alive && warp_wait(&sm.p_full, i & 1, dead, err);
      if (!alive) return;
      tc_fence_after();
      if (elect_one()) {
#pragma unroll
        for (int p = 0; p < L::kQuads; ++p) {
          const uint32_t slot = vs + p < L::kQuadSlots ? vs + p : vs + p - L::kQuadSlots;
          const uint64_t a = d_v + ((slot * kQuadBytes) >> 4);
#pragma unroll
          for (int h = 0; h < 2; ++h)  // 128 latent values at a time
#pragma unroll
            for (int k = 0; k < 4; ++k)  // 16 tokens
              tc_mma(tm_o + (2 * p + h) * N, a + ((h * 2 * kAtom + k * 2 * kLatentQuad * kAtom) >> 4),
                     d_p + (k * 32 >> 4), id_o, !(first && k == 0));
          tc_commit(&sm.quad_empty[slot]);
        }
        tc_commit(&sm.pv_done);
      }
      vs = vs + L::kQuads < L::kQuadSlots ? vs + L::kQuads : vs + L::kQuads - L::kQuadSlots;
    };
    // The next tile's S^T is issued before this tile's values where its rows have arrived: it
    // runs under the softmax.  Where they have not, the values go first, so that their
    // slots are refilled while the rows are on the way.  The S^T buffer is free either way:
    // the softmax of the tile two before handed its P over, and its values were issued.
    while (alive && walk.next<N>(P, rt, seg)) {
      const int k0 = uniform(seg.k0), k1 = uniform(seg.k1);
      for (int u = k0; alive && u < k1; ++u, ++it) {
        const bool first = u == k0;
        const int buf = it & 1;
        uint64_t* full = &sm.full[it % kInFlight];
        const uint32_t par = (it / kInFlight) & 1;
        const bool late = it > 0 && !__all_sync(0xffffffffu, mbar_test_wait(full, par));
        if (late) add_values(it - 1, pending_first);
        if (first) alive = alive && warp_wait(&sm.q_full, n_seg++ & 1, dead, err);
        alive = alive && warp_wait(full, par, dead, err);
        if (!alive) break;
        tc_fence_after();
        if (elect_one()) {
          const uint64_t ar = d_rope + ((rs_ * kChunkBytes) >> 4);
#pragma unroll
          for (int k = 0; k < 4; ++k)
            tc_mma(tm_s + buf * N, ar + (k * 32 >> 4), d_q + (((R / 64) * N * 128 + k * 32) >> 4), id_s, k > 0);
          tc_commit(&sm.rope_empty[rs_]);
#pragma unroll
          for (int p = 0; p < L::kQuads; ++p) {
            const uint32_t slot = ks + p < L::kQuadSlots ? ks + p : ks + p - L::kQuadSlots;
            const uint64_t a = d_quad + ((slot * kQuadBytes) >> 4), q = d_q + ((kLatentQuad * p * N * 128) >> 4);
#pragma unroll
            for (int k = 0; k < 4 * kLatentQuad; ++k)
              tc_mma(tm_s + buf * N, a + (((k >> 2) * kAtom + (k & 3) * 32) >> 4),
                     q + (((k >> 2) * N * 128 + (k & 3) * 32) >> 4), id_s, true);
          }
          tc_commit(&sm.s_full[buf]);
          if (u == k1 - 1) tc_commit(&sm.q_empty);
        }
        if (++rs_ == L::kRopeSlots) rs_ = 0;
        ks = ks + L::kQuads < L::kQuadSlots ? ks + L::kQuads : ks + L::kQuads - L::kQuadSlots;
        if (it > 0 && !late) add_values(it - 1, pending_first);
        pending_first = first;
      }
    }
    if (it > 0 && alive) add_values(it - 1, pending_first);
    __syncwarp();
    if (elect_one()) tc_commit(&sm.drain);  // every MMA has completed before the CTA ends
    mbar_wait_bounded(&sm.drain, 0, err);
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 5) tc_dealloc(tmem, L::kTmem);
}

// Merge of the records of split sequences: one CTA per row, its warps taking the records
// in turn, then the warps' sums in order.  Also the zero rows of unused or bad sequences.
template <int R, int N>
__global__ void __launch_bounds__(128) latent_combine_kernel(const __grid_constant__ Params P) {
  constexpr int V = R / 128;  // float4 per lane
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int64_t row = blockIdx.x;
  const int b = (int)(row / P.rows), r = (int)(row % P.rows);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rt = r / N, rr = r % N;
  const int2 meta = P.meta[(size_t)b * P.n_rt + rt];  // (garbage where L is 0)
  bool bad;
  const int32_t L = latent_ctx(P.a.ctx[b], (int64_t)P.a.max_blocks * kBlockTokens, P.a.n_q, &bad);
  uint16_t* out = P.a.out + row * R;
  if (L == 0) {
    if (bad && r == 0 && threadIdx.x == 0) atomicOr(P.a.lv.err, ERR_CTX);
    for (int i = threadIdx.x; i < R / 8; i += 128) reinterpret_cast<uint4*>(out)[i] = make_uint4(0, 0, 0, 0);
    return;
  }
  if (meta.x < 0) return;
  // records: the first in slot meta.x, then slot 0 of every later group's CTA
  const int g0 = (meta.x >> 1) / P.n_rt, n = meta.y - g0 + 1;
  auto slot_of = [&](int i) -> size_t {
    return i == 0 ? (size_t)meta.x : 2 * ((size_t)(g0 + i) * P.n_rt + rt);
  };
  // the first records are asked for together with every record's reference
  constexpr int U = 4;  // records in flight per warp
  float4 v[U][V];
  float2 ml[U];
  auto load = [&](int i0) {
#pragma unroll
    for (int k = 0; k < U; ++k) {
      const int i = i0 + 4 * k;
      if (i < n) {
        const size_t at = slot_of(i) * N + rr;
        ml[k] = P.ml[at];
#pragma unroll
        for (int e = 0; e < V; ++e) v[k][e] = reinterpret_cast<const float4*>(P.acc + at * R)[lane + 32 * e];
      }
    }
  };
  load(warp);
  float M = kNoMax;
  for (int i = lane; i < n; i += 32) M = fmaxf(M, P.ml[slot_of(i) * N + rr].x);
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, off));
  float s = 0.f;
  float4 acc[V] = {};
  for (int i0 = warp; i0 < n; i0 += 4 * U) {
    if (i0 != warp) load(i0);
#pragma unroll
    for (int k = 0; k < U; ++k)
      if (i0 + 4 * k < n) {
        const float w = ex2(ml[k].x - M);
        s += w * ml[k].y;
#pragma unroll
        for (int e = 0; e < V; ++e) {
          acc[e].x += w * v[k][e].x;
          acc[e].y += w * v[k][e].y;
          acc[e].z += w * v[k][e].z;
          acc[e].w += w * v[k][e].w;
        }
      }
  }
  __shared__ float4 sh[4][32 * V];
  __shared__ float shs[4];
#pragma unroll
  for (int e = 0; e < V; ++e) sh[warp][lane + 32 * e] = acc[e];
  if (lane == 0) shs[warp] = s;
  __syncthreads();
  if (threadIdx.x < 32 * V) {
    const float inv = 1.f / (shs[0] + shs[1] + shs[2] + shs[3]);
    const float4 a = sh[0][threadIdx.x], c = sh[1][threadIdx.x], d = sh[2][threadIdx.x], e = sh[3][threadIdx.x];
    const uint2 o = make_uint2(bf2((a.x + c.x + d.x + e.x) * inv, (a.y + c.y + d.y + e.y) * inv),
                               bf2((a.z + c.z + d.z + e.z) * inv, (a.w + c.w + d.w + e.w) * inv));
    reinterpret_cast<uint2*>(out)[threadIdx.x] = o;
  }
}

// Rows a tile: the smallest of 16, 32 and 64 that holds all of a sequence's.
struct Geometry {
  int rows, N, n_rt, groups;
  size_t meta, ml, total;  // workspace offsets
};

Geometry geometry(int R, int B, int n_q, int Hq, int ctas) {
  Geometry g;
  g.rows = n_q * Hq;
  g.N = g.rows <= 16 ? 16 : g.rows <= 32 ? 32 : 64;
  g.n_rt = (g.rows + g.N - 1) / g.N;
  g.groups = ctas / g.n_rt > 1 ? ctas / g.n_rt : 1;
  auto up = [](size_t x) { return (x + 255) / 256 * 256; };
  // a single group walks every sequence whole: no records
  const size_t slots = g.groups > 1 ? 2 * (size_t)g.groups * g.n_rt : 0;
  g.meta = up(sizeof(int2) * (size_t)B * g.n_rt);
  g.ml = g.meta + up(sizeof(float2) * slots * g.N);
  g.total = g.ml + sizeof(float) * slots * g.N * R;
  return g;
}

template <int R, int N>
cudaError_t launch_rn(const Params& P) {
  static std::atomic<uint64_t> raised{0};  // devices whose shared-memory limit is set
  const cudaError_t e = tc_launch(latent_attn_kernel<R, N>, dim3((unsigned)(P.groups * P.n_rt)), kThreads,
                                  (size_t)Plan<R, N>::kSmem, P.a.stream, P, P.a.device, &raised);
  if (e != cudaSuccess) return e;
  return tc_launch(latent_combine_kernel<R, N>, dim3((unsigned)((int64_t)P.a.B * P.rows)), 128, (size_t)0, P.a.stream, P,
                   P.a.device, &raised);
}

}  // namespace

size_t latent_attn_workspace(int R, int B, int n_q, int Hq, int ctas) {
  return geometry(R, B, n_q, Hq, ctas).total;
}

cudaError_t launch_latent_attn(const LatentAttnArgs& a) {
  const Geometry g = geometry(a.R, a.B, a.n_q, a.Hq, a.ctas);
  Params P;
  P.a = a;
  P.rows = g.rows;
  P.n_rt = g.n_rt;
  P.groups = g.groups;
  P.meta = reinterpret_cast<int2*>(a.ws);
  P.ml = reinterpret_cast<float2*>((uint8_t*)a.ws + g.meta);
  P.acc = reinterpret_cast<float*>((uint8_t*)a.ws + g.ml);
  const uint64_t rows = (uint64_t)a.B * g.rows;
  const uint64_t ld[2] = {(uint64_t)a.R, rows}, rd[2] = {kRope, rows};
  const uint64_t ls[1] = {(uint64_t)a.ql_stride * 2}, rs[1] = {(uint64_t)a.qr_stride * 2};
  const uint32_t box[2] = {64, (uint32_t)g.N};
  if (!encode_bf16_map(&P.ql_map, a.ql, 2, ld, ls, box) || !encode_bf16_map(&P.qr_map, a.qr, 2, rd, rs, box))
    return cudaErrorInvalidValue;
  if (a.R == 512) {
    if (g.N == 16) return launch_rn<512, 16>(P);
    if (g.N == 32) return launch_rn<512, 32>(P);
    return launch_rn<512, 64>(P);
  }
  if (g.N == 16) return launch_rn<256, 16>(P);
  if (g.N == 32) return launch_rn<256, 32>(P);
  return launch_rn<256, 64>(P);
}

}  // namespace pkv
