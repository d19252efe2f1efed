// latent_prefill.cu — expanded attention over a latent pool, on the tensor cores: an
// expansion of the latent rows to per-head keys and values, then causal attention.
//
//   k[t, h] = (Wk[h] c_t, r_t),  v[t, h] = Wv[h] c_t
//   o[i, h] = sum_t exp2(x - m) v[t, h] / sum_t exp2(x - m),  x = scale q[i, h] . k[t, h]
//
// Both kernels are bound by the tensor cores: the expansion takes 512 R operations per
// token and head, the attention 640 per (query, key, head).
//
// Measured (one GB300, both kernels, in a captured graph): a prompt of 8192 with 16 heads
// 273 us, 1383 TFLOP/s (cuBLAS reaches 1888 in a burst); of 4096 with 32 heads 165 us; 1000
// new tokens behind four contexts of up to 4096, 16 heads 108 us; 100 tokens, 4 heads 16.5 us.  The attention runs
// its tensor cores 63 to 65% of the time: a step of two tiles takes 3590 cycles of 2560, S with
// both operands in shared memory (128 bytes a cycle, its whole bandwidth) 88 cycles an MMA
// instead of 64.  The expansion, 37 us of the 273, runs them 43 to 46%: three stages in the ring
// do not cover the copies' latency (2400 cycles under load), its start and end take 10 us.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cmath>

#include "latent.cuh"
#include "tcgen05.cuh"

namespace pkv {
namespace {

constexpr int DH = kLatentHead;
constexpr int kTile = 128;               // tokens (keys) a tile, queries a tile
constexpr int kSlot = kTile * 128;       // 128 rows x 64 values: one swizzled box column
constexpr int kBlockBytes = kBlockTokens * 128;  // one column of a block
constexpr int kAtom = 1024;              // eight tokens of a column: the swizzle's atom
constexpr int kSmall = 3 * 1024;         // alignment (1024) and barriers
constexpr float kSlack = 8.0f;           // log2 of how far a logit may pass the reference
constexpr float kNoMax = -3.402823466e38f;  // no logit is below it
constexpr int kMaxExp = 110;             // value tiles' exponents lie within +-kMaxExp
// The lowest power a tile's P is given, relative to the largest tile's.  At P <= 2^(7 + 8.5)
// before it, fp16 keeps nothing of P (below 2^-25) at 2^-41 and lower: a tile further down adds
// no value either way, while its P, as the sum takes it, is still far from FP32's lowest.
constexpr int kLowest = -48;

struct Params {
  LatentPrefillArgs a;
  int T;                // tokens per (sequence, head) in the workspace: max_ctx rounded up to a tile
  int pairs;            // query tile pairs a sequence (attention)
  float scale;          // |scale| log2(e)
  int negative;         // scale < 0
  uint16_t* k;          // [B, Hq, T, DH] bf16
  uint16_t* v;          // [B, Hq, T, DH] fp16, each tile of 128 tokens divided by 2^its exponent
  int32_t* v_exp;       // [B, Hq, T / 128]
  int splits;           // parts of a unit's key tiles; more than one leave records to be merged
  float* acc;           // [units * Hq][splits][2 * kTile][DH]
  float2* ml;           // [units * Hq][splits][2 * kTile]: (reference, sum)
  CUtensorMap wk_map, wv_map, q_map, k_map, v_map;
};

__device__ __forceinline__ int32_t context(const Params& P, int b, bool* bad) {
  const int64_t all = (int64_t)P.a.max_blocks * kBlockTokens;
  return latent_ctx(P.a.ctx[b], all < P.a.max_ctx ? all : (int64_t)P.a.max_ctx, P.a.n_q, bad);
}

// Block j of sequence b: its slab's tensor maps (null outside the pool) and its first row
// there, in eights.  The maps are acquired by the calling lane: a __syncwarp comes between
// the calls and the copies.
__device__ __forceinline__ const uint8_t* block_map(const Params& P, int b, int j, int* y8) {
  const int32_t row = P.a.bt[(int64_t)b * P.a.max_blocks + j];
  if (!latent_row_ok(P.a.lv, row)) {
    atomicOr(P.a.lv.err, ERR_ROW);
    return nullptr;
  }
  const int32_t slab = row / P.a.lv.slab_blocks;
  *y8 = (row - slab * P.a.lv.slab_blocks) * (kBlockTokens / 8);
  const uint8_t* map = P.a.lv.tab.base[(size_t)slab * P.a.lv.tab.stride] + P.a.lv.map_delta;
  latent_maps_acquire(map);
  return map;
}

// ---------------------------------------------------------------------------
// Expansion: [128 tokens x R] x [R x 256] per head (128 key values, 128 value values).
// The items (token tile, head) of all sequences, heads fastest, are split evenly over the
// CTAs.  A tile's latents stay in shared memory over its heads, so only the weights stream
// (from L2, through a ring of 64-wide k-chunks); two accumulators of 256 columns let the
// epilogue of one item run under the products of the next.
//
// Keys are stored in bf16, the type of the queries they meet.  Values meet probabilities,
// which the attention makes itself: both are fp16, whose three more bits halve the output's
// error (relative L2 0.0028 -> 0.0022; the bf16 output alone has 0.0017).  Any magnitude
// fits, as a tile's values are divided by the power of two that puts the largest in
// [2^13, 2^14), and the attention puts the power back into the probabilities' exponent.  A
// tile without any value has the lowest exponent: it bears on no other tile's.
// ---------------------------------------------------------------------------
constexpr int kExpandThreads = 320;  // warps 0..3 store keys, 4..7 values; 8 copies, 9 MMAs
constexpr int kWStages = 3;
constexpr int kWStage = 2 * kSlot;

// The items of one CTA, in order.  Every role walks them by itself.  (Fewer than 2^24 of
// them, as B Hq T < 2^31: 32-bit divisions.)
struct Items {
  uint32_t item, end, base;  // next item; last + 1; tiles before sequence b
  int b, len, tile, h;
  __device__ __forceinline__ void start(const Params& P) {
    const int lane = threadIdx.x & 31;
    bool bad;
    uint32_t n = 0;
    for (int i = lane; i < P.a.B; i += 32) n += (context(P, i, &bad) + kTile - 1) / kTile;
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) n += __shfl_xor_sync(0xffffffffu, n, off);
    n *= P.a.Hq;
    // an even share, the remainder over the first CTAs
    const uint32_t each = n / gridDim.x, more = n - each * gridDim.x;
    item = blockIdx.x * each + min(blockIdx.x, more);
    end = item + each + (blockIdx.x < more ? 1 : 0);
    base = 0;
    b = 0;
  }
  // Whole warp.  new_tile: the tile differs from the item's before.
  __device__ __forceinline__ bool next(const Params& P, bool first, bool* new_tile) {
    if (item >= end) return false;
    const uint32_t t = uniform(item / (uint32_t)P.a.Hq);
    h = (int)(uniform(item) - t * P.a.Hq);
    *new_tile = first || h == 0;
    if (*new_tile) {
      for (;; ++b) {
        bool bad;
        len = uniform(context(P, b, &bad));
        const uint32_t n = (len + kTile - 1) / kTile;
        if (t < base + n) break;
        base += n;
      }
      tile = uniform((int)(t - base));
    }
    ++item;
    return true;
  }
};

template <int R>
struct ExpandSmall {
  uint64_t a_full[R / 64], a_empty[R / 64], w_full[kWStages], w_empty[kWStages], d_full[2], d_free[2], drain;
  float v_max[2][4];  // by parity of the item: the value warps' largest magnitudes
  uint32_t tmem;
  int dead;
};

template <int R>
__global__ void __launch_bounds__(kExpandThreads, 1) latent_expand_kernel(const __grid_constant__ Params P) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
  uint8_t* as = smem;
  uint8_t* ws = as + (R / 64) * kSlot;
  ExpandSmall<R>& sm = *reinterpret_cast<ExpandSmall<R>*>(ws + kWStages * kWStage);
  const int warp = uniform((int)(threadIdx.x >> 5)), lane = threadIdx.x & 31;
  volatile int* dead = &sm.dead;
  int32_t* err = P.a.lv.err;
  constexpr int C = R / 64;  // k-chunks

  if (threadIdx.x == 0) {
    for (int i = 0; i < C; ++i) mbar_init(&sm.a_full[i], 1), mbar_init(&sm.a_empty[i], 1);
    for (int i = 0; i < kWStages; ++i) mbar_init(&sm.w_full[i], 1), mbar_init(&sm.w_empty[i], 1);
    for (int i = 0; i < 2; ++i) mbar_init(&sm.d_full[i], 1), mbar_init(&sm.d_free[i], 256);
    mbar_init(&sm.drain, 1);
    sm.dead = 0;
    fence_mbar_init();
  }
  if (warp == 9) tc_alloc(&sm.tmem, 512);
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = uniform(sm.tmem);
  Items it;
  it.start(P);
  bool new_tile;

  if (warp < 8) {
    const int kind = warp >> 2;  // 0: keys, 1: values
    for (int n = 0; it.next(P, n == 0, &new_tile); ++n) {
      const int t = it.tile * kTile + (threadIdx.x & 127), L = it.len;
      wait_or_die(&sm.d_full[n & 1], (n >> 1) & 1, dead, err);
      tc_fence_after();
      // first of the eight rows that this lane's group of eight stores together
      const int64_t row0 = ((int64_t)it.b * P.a.Hq + it.h) * P.T + (t & ~7);
      const uint32_t acc = tmem + (n & 1) * 256 + kind * DH + ((uint32_t)((warp & 3) * 32) << 16);
      float scale = 1.f;
      if (kind) {
        float mx = 0.f;
#pragma unroll 1
        for (int q = 0; q < 4; ++q) {
          uint32_t r[32];
          tc_ld_rows<32>(acc + q * 32, r);
          tc_wait_ld();
#pragma unroll
          for (int i = 0; i < 32; ++i) mx = fmaxf(mx, fabsf(__uint_as_float(r[i])));
        }
        // a row with an infinity stays one, as documented, but sets no exponent: the tiles
        // beside it keep their bits (fmaxf passes NaN by)
        if (t >= L || mx > 3.402823466e38f) mx = 0.f;
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, off));
        if (lane == 0) sm.v_max[n & 1][warp & 3] = mx;
        named_barrier_sync(1, 128);
#pragma unroll
        for (int i = 0; i < 4; ++i) mx = fmaxf(mx, sm.v_max[n & 1][i]);
        const int e = mx > 0.f ? max(-kMaxExp, min(kMaxExp, (int)(__float_as_uint(mx) >> 23) - 127 - 13)) : -kMaxExp;
        scale = pow2(-e);
        if (threadIdx.x == 128) P.v_exp[((int64_t)it.b * P.a.Hq + it.h) * (P.T / kTile) + it.tile] = e;
      }
#pragma unroll 1
      for (int q = 0; q < 2; ++q) {
        // 64 columns of this thread's row as eight 16-byte pieces.  Rows past the context
        // become zero: their values meet probabilities of zero in the attention, which a
        // NaN would survive.
        uint32_t v[8][4];
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          uint32_t r[32];
          tc_ld_rows<32>(acc + q * 64 + half * 32, r);
          tc_wait_ld();
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            const float lo = __uint_as_float(r[2 * i]), hi = __uint_as_float(r[2 * i + 1]);
            v[4 * half + (i >> 2)][i & 3] = t >= L ? 0u : kind ? fp16x2(lo * scale, hi * scale) : bf2(lo, hi);
          }
        }
        // Transpose the pieces among eight lanes, so that lane l holds piece l of eight rows
        // and a store of the group fills a 128-byte line (one thread's own row, 16 bytes a
        // store, took twice as long as the products).
#pragma unroll
        for (int s = 1; s < 8; s <<= 1) {
          const bool up = lane & s;
#pragma unroll
          for (int i = 0; i < 8; ++i)
            if (!(i & s)) {
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const uint32_t got = __shfl_xor_sync(0xffffffffu, up ? v[i][e] : v[i | s][e], s);
                if (up)
                  v[i][e] = got;
                else
                  v[i | s][e] = got;
              }
            }
        }
        uint16_t* dst = (kind ? P.v : P.k) + row0 * DH + q * 64 + (lane & 7) * 8;
#pragma unroll
        for (int i = 0; i < 8; ++i)
          *reinterpret_cast<uint4*>(dst + i * DH) = make_uint4(v[i][0], v[i][1], v[i][2], v[i][3]);
      }
      tc_fence_before();
      mbar_arrive(&sm.d_free[n & 1]);
    }
  } else if (warp == 8) {
    const uint64_t keep = l2_policy_evict_normal();
    uint32_t nw = 0, na = 0, s = 0, round = 0, tiles = 0;
    const uint8_t* map = nullptr;
    int y0 = 0;
    uint32_t bytes = 0;
    bool alive = true;
    for (int n = 0; alive && it.next(P, n == 0, &new_tile); ++n) {
      if (new_tile) {
        // lane l < 4 looks up block l of the tile
        const int j = it.tile * (kTile / kBlockTokens) + lane;
        map = lane < 4 && j * kBlockTokens < it.len ? block_map(P, it.b, j, &y0) : nullptr;
        __syncwarp();
        bytes = __popc(__ballot_sync(0xffffffffu, map != nullptr)) * kBlockBytes;
        ++tiles;
      }
#pragma unroll 1
      for (int c = 0; c < C; ++c) {
        if (new_tile) {
          if (tiles > 1) alive = warp_wait(&sm.a_empty[c], tiles & 1, dead, err);
          if (!alive) break;
          if (elect_one()) mbar_arrive_expect_tx(&sm.a_full[c], bytes);
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const uint8_t* mk = lane_ptr(map, k);
            const int yk = __shfl_sync(0xffffffffu, y0, k);
            if (mk && elect_one())
              latent_copy_column(as + c * kSlot + k * kBlockBytes, mk, c, yk, &sm.a_full[c], keep);
          }
          ++na;
        }
        if (round > 0) alive = warp_wait(&sm.w_empty[s], (round - 1) & 1, dead, err);
        if (!alive) break;
        if (elect_one()) {
          mbar_arrive_expect_tx(&sm.w_full[s], kWStage);
          tma_load_2d(ws + s * kWStage, &P.wk_map, c * 64, it.h * DH, &sm.w_full[s], keep);
          tma_load_2d(ws + s * kWStage + kSlot, &P.wv_map, c * 64, it.h * DH, &sm.w_full[s], keep);
        }
        ++nw;
        if (++s == kWStages) s = 0, ++round;
      }
    }
    // no copy may be in flight when the CTA ends
    for (uint32_t i = nw > kWStages ? nw - kWStages : 0; i < nw; ++i)
      mbar_wait_bounded(&sm.w_full[i % kWStages], (i / kWStages) & 1, err);
    for (uint32_t i = na > C ? na - C : 0; i < na; ++i) mbar_wait_bounded(&sm.a_full[i % C], (i / C) & 1, err);
  } else {
    constexpr uint32_t id = tc_idesc(128, 256, false, false);
    const uint64_t d_a = tc_desc(smem_u32(as), 16, kAtom), d_w = tc_desc(smem_u32(ws), 16, kAtom);
    uint32_t s = 0, round = 0, tiles = 0;
    bool alive = true;
    for (int n = 0; alive && it.next(P, n == 0, &new_tile); ++n) {
      if (new_tile) ++tiles;
      const bool last_of_tile = it.h == P.a.Hq - 1 || it.item == it.end;
      if (n >= 2) alive = warp_wait(&sm.d_free[n & 1], ((n >> 1) - 1) & 1, dead, err);
#pragma unroll 1
      for (int c = 0; c < C; ++c) {
        if (new_tile) alive = alive && warp_wait(&sm.a_full[c], (tiles - 1) & 1, dead, err);
        alive = alive && warp_wait(&sm.w_full[s], round & 1, dead, err);
        if (!alive) break;
        tc_fence_after();
        if (elect_one()) {
          const uint64_t da = d_a + ((c * kSlot) >> 4), dw = d_w + ((s * kWStage) >> 4);
#pragma unroll
          for (int k = 0; k < 4; ++k)
            tc_mma(tmem + (n & 1) * 256, da + (k * 32 >> 4), dw + (k * 32 >> 4), id, c > 0 || k > 0);
          tc_commit(&sm.w_empty[s]);
          if (last_of_tile) tc_commit(&sm.a_empty[c]);
          if (c == C - 1) tc_commit(&sm.d_full[n & 1]);
        }
        if (++s == kWStages) s = 0, ++round;
      }
    }
    __syncwarp();
    if (elect_one()) tc_commit(&sm.drain);
    mbar_wait_bounded(&sm.drain, 0, err);
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 9) tc_dealloc(tmem, 512);
}

// ---------------------------------------------------------------------------
// Attention: a CTA takes two tiles of 128 queries of one head.  S = Q K^T (12 k-steps)
// and O += P V (8 k-steps) of the two tiles alternate on the tensor cores, so that one
// tile's softmax runs under the other's products.  A thread owns a query: its row of S
// comes from tensor memory into registers, P goes back over it in fp16 and is the next
// product's A operand there.  The reference m, a whole number, moves only when a logit
// passes it by more than 2^8, which is when the row's O is rescaled.  P carries 2^(7 + the
// key tile's exponent - the largest tile's), at most 2^15.5, so that O is in units of
// 2^(largest - 7) throughout; a part of P below 2^-21 of the largest loses bits.  Keys and values arrive in 16 KB
// slots (K: two of 64 dims and one of the position keys, straight from the pool's blocks;
// V: two of 64 keys, so that one MMA covers all 128 value columns), eight in the ring.
//
// Few queries over long contexts make fewer CTAs than there are SMs: the key tiles are then
// split over several CTAs (blockIdx.y), which leave FP32 records (reference, sum, O) for a
// merge kernel (SPLIT; without it the launch has one part and writes the output itself).
// ---------------------------------------------------------------------------
// Warps 0..3 and 4..7: softmax of a tile each; 8: copies; 9: MMAs; 10, 11 fill the third
// warpgroup, which gives registers to the other two: 2 x 200 + 104 = 3 x 168, the launch
// allocation (the launcher checks that the kernel was built with 168).
constexpr int kAttnThreads = 384;
constexpr int kAttnRegs = 168;
constexpr int kSlots = 8;
constexpr int kQTile = 3 * kSlot;

// Two FP32 values in one 64-bit register: one instruction for both.
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

// Units (sequence, 256 queries) up to which a CTA ranks them by their key tiles.
constexpr int kRanked = 384;

struct AttnSmall {
  uint64_t k_full[2], k_empty[2], v_full[2], v_empty[2];  // by parity of the key tile
  uint64_t q_full[2], s_full[2], p_full[2][2], o_full[2], drain, done;
  uint32_t tmem;
  int dead;
  int pick;            // ranked launch: the unit of this CTA
  int cost[kRanked];   // ranked launch: key tiles of each unit
};
static_assert(sizeof(AttnSmall) <= kSmall - 1024, "small state");

template <bool SPLIT>
__global__ void __launch_bounds__(kAttnThreads, 1) latent_prefill_kernel(const __grid_constant__ Params P) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
  uint8_t* qs = smem;
  uint8_t* ring = qs + 2 * kQTile;
  AttnSmall& sm = *reinterpret_cast<AttnSmall*>(ring + kSlots * kSlot);
  const int warp = uniform((int)(threadIdx.x >> 5)), lane = threadIdx.x & 31;
  volatile int* dead = &sm.dead;
  int32_t* err = P.a.lv.err;
  const int R = P.a.R, n_q = P.a.n_q;

  if (threadIdx.x == 0) {
    for (int i = 0; i < 2; ++i) {
      for (uint64_t* bar : {&sm.k_full[i], &sm.k_empty[i], &sm.v_full[i], &sm.v_empty[i]}) mbar_init(bar, 1);
      mbar_init(&sm.q_full[i], 1);
      mbar_init(&sm.s_full[i], 1);
      mbar_init(&sm.p_full[i][0], 128);
      mbar_init(&sm.p_full[i][1], 128);
      mbar_init(&sm.o_full[i], 1);
    }
    mbar_init(&sm.drain, 1);
    mbar_init(&sm.done, 256);
    sm.dead = 0;
    fence_mbar_init();
  }
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  // The units with most key tiles go first (heads fastest).  In one sequence those are the
  // last queries; over several, whose lengths only the device knows, each CTA ranks them.
  const int units = P.pairs * P.a.B;
  const int place = (int)(blockIdx.x / P.a.Hq), h = (int)(blockIdx.x % P.a.Hq);
  int unit = units - 1 - place;  // b fastest
  if (P.a.B > 1 && units <= kRanked) {
    bool bad;
    const int u = threadIdx.x;
    int mine = 0;
    if (u < units) {
      const int32_t L = context(P, u % P.a.B, &bad);
      mine = L == 0 ? 0 : (L - n_q + min(n_q, (u / P.a.B + 1) * 2 * kTile) + kTile - 1) / kTile;
      sm.cost[u] = mine;
    }
    __syncthreads();
    if (u < units) {
      int before = 0;
      for (int k = 0; k < units; ++k) before += sm.cost[k] > mine || (sm.cost[k] == mine && k < u);
      if (before == place) sm.pick = u;
    }
    __syncthreads();
    unit = sm.pick;
  }
  unit = uniform(unit);
  const int pair = unit / P.a.B, b = unit % P.a.B;
  const int i0 = pair * 2 * kTile;
  bool bad;
  const int32_t L = uniform(context(P, b, &bad));
  if (L == 0) {
    if (blockIdx.y > 0) return;
    if (bad && pair == 0 && h == 0 && threadIdx.x == 0) atomicOr(err, ERR_CTX);
    const int n = min(2 * kTile, n_q - i0);
    for (int i = threadIdx.x; i < n * (DH / 8); i += kAttnThreads)
      reinterpret_cast<uint4*>(P.a.out + (((int64_t)b * n_q + i0 + i / (DH / 8)) * P.a.Hq + h) * DH)[i % (DH / 8)] =
          make_uint4(0, 0, 0, 0);
    return;
  }
  if (warp == 9) tc_alloc(&sm.tmem, 512);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = uniform(sm.tmem);  // S of the two tiles, then O of the two
  const int off = L - n_q;        // query i sees off + i + 1 tokens
  // key tiles of each query tile
  auto key_tiles = [&](int t) {
    const int last = min(n_q, i0 + (t + 1) * kTile) - 1;
    return last < i0 + t * kTile ? 0 : uniform((off + last + 1 + kTile - 1) / kTile);
  };
  const int all0 = key_tiles(0), all1 = key_tiles(1), all = max(all0, all1);
  // this CTA's key tiles: from j0 on, numbered from 0 below
  int j0 = 0, nmax = all, nt0 = all0, nt1 = all1;
  if constexpr (SPLIT) {
    const int per = (all + P.splits - 1) / P.splits;
    j0 = uniform((int)blockIdx.y * per);
    nmax = uniform(max(0, min(per, all - j0)));
    nt0 = uniform(max(0, min(nmax, all0 - j0)));
    nt1 = uniform(max(0, min(nmax, all1 - j0)));
  }

  // The warpgroups' paths do not rejoin: each ends in a return.
  if (warp < 8) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 200;");
    // ---------------------------------------------------------------- softmax
    const int t = warp >> 2, ntt = t ? nt1 : nt0;
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t tm_s = tmem + t * kTile + lanes, tm_o = tmem + 2 * kTile + t * kTile + lanes;
    const int i = i0 + t * kTile + (warp & 3) * 32 + lane;
    const int vis = off + i + 1;
    const int vis_first = off + i0 + t * kTile + 1;  // of the tile's first query
    const int32_t* v_exp = P.v_exp + ((int64_t)b * P.a.Hq + h) * (P.T / kTile);
    int top_exp = -kMaxExp;
    for (int k = lane; k < all; k += 32) top_exp = max(top_exp, v_exp[k]);
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) top_exp = max(top_exp, __shfl_xor_sync(0xffffffffu, top_exp, d));
    float m = kNoMax;
    uint64_t l = 0;    // two partial sums
    bool big = false;  // the warp has a reference beyond 2^23
#pragma unroll 1
    for (int j = 0; j < ntt; ++j) {
      const int lift = max(kLowest, v_exp[j0 + j] - top_exp) + 7;  // this tile's power in P
      wait_or_die(&sm.s_full[t], j & 1, dead, err);
      tc_fence_after();
      float x[128];
      {
        uint32_t r[4][32];
#pragma unroll
        for (int q = 0; q < 4; ++q) tc_ld_rows<32>(tm_s + 32 * q, r[q]);
        tc_wait_ld();
#pragma unroll
        for (int c = 0; c < 128; ++c) x[c] = __uint_as_float(r[c >> 5][c & 31]);
      }
      if (P.negative) {
#pragma unroll
        for (int c = 0; c < 128; ++c) x[c] = -x[c];
      }
      if ((j0 + j + 1) * kTile > vis_first) {
        const int n = vis - (j0 + j) * kTile;  // this query sees the tile's first n keys
#pragma unroll
        for (int c = 0; c < 128; ++c)
          if (c >= n) x[c] = -INFINITY;
      }
      float mx[4] = {x[0], x[1], x[2], x[3]};
#pragma unroll
      for (int c = 4; c + 1 < 124; c += 8)
#pragma unroll
        for (int e = 0; e < 4; ++e) mx[e] = max3(mx[e], x[c + e], x[c + 4 + e]);
#pragma unroll
      for (int e = 0; e < 4; ++e) mx[e] = fmaxf(mx[e], x[124 + e]);
      // Rows past the last query hold other sequences' queries and meet slots past the length:
      // they must not move the references of this warp's other rows.
      const float top = i < n_q ? fmaxf(max3(mx[0], mx[1], mx[2]), mx[3]) * P.scale : -INFINITY;
      if (__any_sync(0xffffffffu, top - m > kSlack)) {
        const float mn = fmaxf(m, rintf(top));
        const float f = ex2(m - mn);
        m = mn;
        l = mul2(l, pair2(f, f));
        big = __any_sync(0xffffffffu, fabsf(m) > 8388608.f && m > kNoMax);
        if (j > 0) {
          // the products of the tile before are complete: this S was issued after them
#pragma unroll 1
          for (int q = 0; q < 4; ++q) {
            uint32_t o[32];
            tc_ld_rows<32>(tm_o + 32 * q, o);
            tc_wait_ld();
#pragma unroll
            for (int c = 0; c < 32; ++c) o[c] = __float_as_uint(__uint_as_float(o[c]) * f);
            tc_st_rows<32>(tm_o + 32 * q, o);
          }
        }
      }
      // x scale + (lift - m) in one rounding.  Up to 2^23 lift - m is exact.  Beyond, it would be
      // rounded by a power of two's worth and more, differently from tile to tile: there the
      // product is rounded first, as the reference was, m is taken from it, and then lift added.
      float mul = P.scale, ref = (float)lift - m;
      if (big) {
#pragma unroll
        for (int c = 0; c < 128; ++c) x[c] = __fsub_rn(__fmul_rn(x[c], P.scale), m);
        mul = 1.f;
        ref = (float)lift;
      }
      const uint64_t sc = pair2(mul, mul), mm = pair2(ref, ref);
      uint64_t sum0 = 0, sum1 = 0;
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        uint32_t w[16];
#pragma unroll
        for (int c = 0; c < 16; ++c) {
          float e0, e1;
          split2(fma2(pair2(x[32 * q + 2 * c], x[32 * q + 2 * c + 1]), sc, mm), e0, e1);
          e0 = ex2(e0);
          e1 = ex2(e1);
          uint64_t& s = c & 1 ? sum1 : sum0;
          s = add2(s, pair2(e0, e1));
          w[c] = fp16x2(e0, e1);
        }
        tc_st_rows<16>(tm_s + 16 * q, w);
        if (q & 1) {
          // the product over these 64 keys may start
          tc_wait_st();
          tc_fence_before();
          mbar_arrive(&sm.p_full[t][q >> 1]);
        }
      }
      const float back = pow2(-lift);
      l = fma2(add2(sum0, sum1), pair2(back, back), l);
    }
    float l0, l1;
    split2(l, l0, l1);
    const float sum = l0 + l1;
    int64_t rec = 0;
    if constexpr (SPLIT) {
      rec = (((int64_t)unit * P.a.Hq + h) * P.splits + blockIdx.y) * (2 * kTile) + t * kTile + (warp & 3) * 32 + lane;
      P.ml[rec] = make_float2(m, sum);  // a sum of 0: no tile here, and no O
    }
    if (ntt > 0) {
      wait_or_die(&sm.o_full[t], 0, dead, err);
      tc_fence_after();
      const float unit_o = pow2(top_exp - 7), inv = unit_o / sum;
      uint4* out = reinterpret_cast<uint4*>(P.a.out + (((int64_t)b * n_q + i) * P.a.Hq + h) * DH);
      float4* acc = reinterpret_cast<float4*>(P.acc + rec * DH);
#pragma unroll 1
      for (int q = 0; q < 4; ++q) {
        uint32_t o[32];
        tc_ld_rows<32>(tm_o + 32 * q, o);
        tc_wait_ld();
        if (SPLIT && i < n_q) {
#pragma unroll
          for (int c = 0; c < 8; ++c)
            acc[8 * q + c] =
                make_float4(__uint_as_float(o[4 * c]) * unit_o, __uint_as_float(o[4 * c + 1]) * unit_o,
                            __uint_as_float(o[4 * c + 2]) * unit_o, __uint_as_float(o[4 * c + 3]) * unit_o);
        } else if (i < n_q) {
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            uint32_t w[4];
#pragma unroll
            for (int e = 0; e < 4; ++e)
              w[e] = bf2(__uint_as_float(o[8 * c + 2 * e]) * inv, __uint_as_float(o[8 * c + 2 * e + 1]) * inv);
            out[4 * q + c] = make_uint4(w[0], w[1], w[2], w[3]);
          }
        }
      }
    }
    tc_fence_before();
    mbar_arrive(&sm.done);
    return;
  }
  asm volatile("setmaxnreg.dec.sync.aligned.u32 104;");
  if (warp == 8) {
    // ------------------------------------------------------------------ copies
    const uint64_t keep = l2_policy_evict_normal();
    if (elect_one()) {
#pragma unroll
      for (int t = 0; t < 2; ++t)
        if ((t ? nt1 : nt0) > 0) {
          mbar_arrive_expect_tx(&sm.q_full[t], kQTile);
          for (int c = 0; c < 3; ++c)
            tma_load_3d(qs + t * kQTile + c * kSlot, &P.q_map, c * 64, h, b * n_q + i0 + t * kTile, &sm.q_full[t], keep);
        }
    }
    // Key tile j takes the ring's next five slots: K 0..2, V 3..4.  Eight slots before, slot
    // 0 held the last of K(j - 2), 1 and 2 V(j - 2), 3 and 4 the first of K(j - 1).
    const int row0 = (b * P.a.Hq + h) * P.T + j0 * kTile;
    int nk = 0, nv = 0;  // tiles whose copies were started
    bool alive = true;
    for (int jb = 0; alive && jb < nmax; jb += 8) {
      // lane l looks up block 4 jb + l
      const int blk = 4 * (j0 + jb) + lane;
      int y0 = 0;
      const uint8_t* map = blk < 4 * (j0 + nmax) && blk * kBlockTokens < L ? block_map(P, b, blk, &y0) : nullptr;
      __syncwarp();
      const unsigned have = __ballot_sync(0xffffffffu, map != nullptr);
      const int je = min(jb + 8, nmax);
#pragma unroll 1
      for (int j = jb; j < je; ++j) {
        const int i = 4 * (j - jb), par = j & 1, rd = (j >> 1) & 1;
        auto slot = [&](int c) { return ring + ((5 * (uint32_t)j + c) % kSlots) * kSlot; };
        if (j >= 2) alive = warp_wait(&sm.k_empty[par], rd ^ 1, dead, err);
        if (!alive) break;
        if (elect_one()) {
          mbar_arrive_expect_tx(&sm.k_full[par], 2 * kSlot + __popc((have >> i) & 15u) * kBlockBytes);
          tma_load_2d(slot(0), &P.k_map, 0, row0 + j * kTile, &sm.k_full[par], keep);
        }
        ++nk;
        if (j >= 2) alive = warp_wait(&sm.v_empty[par], rd ^ 1, dead, err);
        if (!alive) break;
        if (elect_one()) tma_load_2d(slot(1), &P.k_map, 64, row0 + j * kTile, &sm.k_full[par], keep);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const uint8_t* mk = lane_ptr(map, i + k);
          const int yk = __shfl_sync(0xffffffffu, y0, i + k);
          if (mk && elect_one()) latent_copy_column(slot(2) + k * kBlockBytes, mk, R / 64, yk, &sm.k_full[par], keep);
        }
        if (j >= 1) alive = warp_wait(&sm.k_empty[par ^ 1], ((j - 1) >> 1) & 1, dead, err);
        if (!alive) break;
        if (elect_one()) {
          mbar_arrive_expect_tx(&sm.v_full[par], 2 * kSlot);
          for (int c = 0; c < 2; ++c)
            for (int k = 0; k < 2; ++k)
              tma_load_2d(slot(3 + c) + k * (kSlot / 2), &P.v_map, k * 64, row0 + j * kTile + c * 64, &sm.v_full[par], keep);
        }
        ++nv;
      }
    }
    // No copy may be in flight when the CTA ends.  (A role that gave up between the copies of
    // one K tile leaves its barrier short of bytes: that wait runs into its limit.)
    for (int j = max(0, nk - 2); j < nk; ++j) mbar_wait_bounded(&sm.k_full[j & 1], (j >> 1) & 1, err);
    for (int j = max(0, nv - 2); j < nv; ++j) mbar_wait_bounded(&sm.v_full[j & 1], (j >> 1) & 1, err);
    if (nt0 > 0) mbar_wait_bounded(&sm.q_full[0], 0, err);
    if (nt1 > 0) mbar_wait_bounded(&sm.q_full[1], 0, err);
  } else if (warp == 9) {
    // -------------------------------------------------------------------- MMAs
    constexpr uint32_t id_s = tc_idesc(128, 128, false, false);
    constexpr uint32_t id_o = tc_idesc(128, 128, false, true, true);
    const uint64_t d_q = tc_desc(smem_u32(qs), 16, 1024), d_k = tc_desc(smem_u32(ring), 16, 1024);
    const uint64_t d_v = tc_desc(smem_u32(ring), kSlot / 2, 1024);  // [2 x 64 values][64 keys], MN-major
    bool alive = true;
    auto ready = [&](uint64_t* bar, int parity) { alive = alive && warp_wait(bar, parity, dead, err); };
    // O_t += P_t(j) V(j), 64 keys at a time: the first half starts under the softmax of the second
    auto add_values = [&](int t, int j, int ntt) {
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        ready(&sm.p_full[t][c], j & 1);
        if (!alive) return;
        tc_fence_after();
        if (elect_one()) {
          const uint64_t v = d_v + ((((5 * (uint32_t)j + 3 + c) % kSlots) * kSlot) >> 4);
#pragma unroll
          for (int k = 0; k < 4; ++k)
            tc_mma_ts(tmem + 2 * kTile + t * kTile, tmem + t * kTile + 32 * c + 8 * k, v + (k * 2048 >> 4), id_o,
                      j > 0 || c > 0 || k > 0);
          if (c == 1 && j == ntt - 1) tc_commit(&sm.o_full[t]);
        }
      }
    };
    // S_t = Q_t K(j)^T
    auto logits = [&](int t, int j) {
      if (j == 0) ready(&sm.q_full[t], 0);
      if (!alive) return;
      tc_fence_after();
      if (elect_one()) {
#pragma unroll
        for (int c = 0; c < 3; ++c) {
          const uint64_t q = d_q + ((t * kQTile + c * kSlot) >> 4);
          const uint64_t k0 = d_k + ((((5 * (uint32_t)j + c) % kSlots) * kSlot) >> 4);
#pragma unroll
          for (int k = 0; k < 4; ++k)
            tc_mma(tmem + t * kTile, q + (k * 32 >> 4), k0 + (k * 32 >> 4), id_s, c > 0 || k > 0);
        }
        tc_commit(&sm.s_full[t]);
      }
    };
#pragma unroll 1
    for (int j = 0; alive && j <= nmax; ++j) {
      const int par = j & 1;
      if (j > 0) ready(&sm.v_full[par ^ 1], ((j - 1) >> 1) & 1);
      if (j > 0 && j - 1 < nt0) add_values(0, j - 1, nt0);
      if (j < nmax) ready(&sm.k_full[par], (j >> 1) & 1);
      if (j < nt0) logits(0, j);
      if (j > 0 && j - 1 < nt1) add_values(1, j - 1, nt1);
      if (j > 0 && alive && elect_one()) tc_commit(&sm.v_empty[par ^ 1]);
      if (j < nt1) logits(1, j);
      if (j < nmax && alive && elect_one()) tc_commit(&sm.k_empty[par]);
    }
    __syncwarp();
    if (elect_one()) tc_commit(&sm.drain);
    mbar_wait_bounded(&sm.drain, 0, err);
    __syncwarp();
    mbar_wait_bounded(&sm.done, 0, err);  // the softmax warps have read their last column
    tc_fence_after();
    __syncwarp();
    tc_dealloc(tmem, 512);
  }
}

// Merge of a row's records, one warp per row.
__global__ void __launch_bounds__(256) latent_prefill_merge_kernel(const __grid_constant__ Params P) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int lane = threadIdx.x & 31;
  const int64_t row = (int64_t)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5);  // (b, i, h)
  if (row >= (int64_t)P.a.B * P.a.n_q * P.a.Hq) return;
  const int h = (int)(row % P.a.Hq), i = (int)(row / P.a.Hq % P.a.n_q), b = (int)(row / P.a.Hq / P.a.n_q);
  const int unit = i / (2 * kTile) * P.a.B + b;
  const int64_t rec = ((int64_t)unit * P.a.Hq + h) * P.splits * (2 * kTile) + i % (2 * kTile);
  bool bad;
  if (context(P, b, &bad) == 0) return;  // zeros are written
  float M = kNoMax;
  for (int k = lane; k < P.splits; k += 32) {
    const float2 ml = P.ml[rec + (int64_t)k * (2 * kTile)];
    if (ml.y != 0.f) M = fmaxf(M, ml.x);
  }
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, off));
  float sum = 0.f;
  float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
  for (int k = 0; k < P.splits; ++k) {
    const int64_t at = rec + (int64_t)k * (2 * kTile);
    const float2 ml = P.ml[at];
    if (ml.y != 0.f) {
      const float w = ex2(ml.x - M);
      const float4 o = reinterpret_cast<const float4*>(P.acc + at * DH)[lane];
      sum += w * ml.y;
      a.x += w * o.x, a.y += w * o.y, a.z += w * o.z, a.w += w * o.w;
    }
  }
  const float inv = 1.f / sum;
  reinterpret_cast<uint2*>(P.a.out + row * DH)[lane] = make_uint2(bf2(a.x * inv, a.y * inv), bf2(a.z * inv, a.w * inv));
}

// Parts of the key tiles: as many as fill the SMs once, each of at least four tiles (a part
// costs about as much as three: its start, its records and their merge).
int prefill_splits(int B, int n_q, int Hq, int max_ctx, int ctas) {
  const int64_t launch = (int64_t)((n_q + 2 * kTile - 1) / (2 * kTile)) * B * Hq;
  const int tiles = (max_ctx + kTile - 1) / kTile;
  const int64_t fill = ctas / launch, most = tiles / 4;
  const int64_t n = fill < most ? fill : most;
  return n > 1 ? (int)(n < 1024 ? n : 1024) : 1;
}

int tile_up(int x) { return (x + kTile - 1) / kTile * kTile; }

}  // namespace

namespace {
// Offsets of the workspace: keys, values and their exponents, records.
struct Layout {
  int splits;
  size_t v, v_exp, acc, ml, total;
};
Layout prefill_layout(int B, int n_q, int Hq, int max_ctx, int ctas) {
  Layout w;
  w.splits = prefill_splits(B, n_q, Hq, max_ctx, ctas);
  w.v = (size_t)B * Hq * (size_t)tile_up(max_ctx) * DH * sizeof(uint16_t);  // a multiple of 256
  w.v_exp = 2 * w.v;
  w.acc = w.v_exp + ((size_t)B * Hq * (size_t)(tile_up(max_ctx) / kTile) * sizeof(int32_t) + 255) / 256 * 256;
  const size_t rows =
      w.splits > 1 ? (size_t)((n_q + 2 * kTile - 1) / (2 * kTile)) * B * Hq * w.splits * (2 * kTile) : 0;
  w.ml = w.acc + rows * DH * sizeof(float);
  w.total = w.ml + rows * sizeof(float2) + 256;
  return w;
}
}  // namespace

size_t latent_prefill_workspace(int B, int n_q, int Hq, int max_ctx, int ctas) {
  return prefill_layout(B, n_q, Hq, max_ctx, ctas).total;
}

cudaError_t launch_latent_prefill(const LatentPrefillArgs& a) {
  Params P;
  P.a = a;
  P.T = tile_up(a.max_ctx);
  const Layout lay = prefill_layout(a.B, a.n_q, a.Hq, a.max_ctx, a.ctas);
  uint8_t* ws = (uint8_t*)a.ws;
  P.k = (uint16_t*)ws;
  P.v = (uint16_t*)(ws + lay.v);
  P.v_exp = (int32_t*)(ws + lay.v_exp);
  P.acc = (float*)(ws + lay.acc);
  P.ml = (float2*)(ws + lay.ml);
  P.splits = lay.splits;
  // -inf (a hidden key) times 0 would be NaN: a scale of 0 becomes a tiny one
  P.scale = fmaxf(fabsf(a.scale_log2), 1e-37f);
  P.negative = a.scale_log2 < 0.f;
  P.pairs = (a.n_q + 2 * kTile - 1) / (2 * kTile);
  const int tiles = P.T / kTile;
  if (tiles > 0) {
    const uint64_t wd[2] = {(uint64_t)a.R, (uint64_t)a.Hq * DH}, wst[1] = {(uint64_t)a.R * 2};
    const uint64_t kd[2] = {DH, (uint64_t)a.B * a.Hq * P.T}, kst[1] = {DH * 2};
    const uint64_t qd[3] = {DH + kRope, (uint64_t)a.Hq, (uint64_t)a.B * a.n_q};
    const uint64_t qst[2] = {(DH + kRope) * 2, (uint64_t)a.Hq * (DH + kRope) * 2};
    const uint32_t box[2] = {64, kTile}, vbox[2] = {64, kTile / 2}, qbox[3] = {64, 1, kTile};
    if (!encode_bf16_map(&P.wk_map, a.wk, 2, wd, wst, box) || !encode_bf16_map(&P.wv_map, a.wv, 2, wd, wst, box) ||
        !encode_bf16_map(&P.k_map, P.k, 2, kd, kst, box) || !encode_bf16_map(&P.v_map, P.v, 2, kd, kst, vbox) ||
        !encode_bf16_map(&P.q_map, a.q, 3, qd, qst, qbox))
      return cudaErrorInvalidValue;
    const int64_t items = (int64_t)tiles * a.B * a.Hq;  // at most
    const dim3 grid((unsigned)(items < a.ctas ? items : a.ctas));
    const size_t smem = kSmall + (size_t)(a.R / 64) * kSlot + kWStages * kWStage;
    static std::atomic<uint64_t> raised[2];
    const cudaError_t e =
        a.R == 512 ? tc_launch(latent_expand_kernel<512>, grid, kExpandThreads, smem, a.stream, P, a.device, &raised[0])
                   : tc_launch(latent_expand_kernel<256>, grid, kExpandThreads, smem, a.stream, P, a.device, &raised[1]);
    if (e != cudaSuccess) return e;
  }
  static const bool regs_ok = [] {
    cudaFuncAttributes f0, f1;
    return cudaFuncGetAttributes(&f0, latent_prefill_kernel<false>) == cudaSuccess && f0.numRegs == kAttnRegs &&
           cudaFuncGetAttributes(&f1, latent_prefill_kernel<true>) == cudaSuccess && f1.numRegs == kAttnRegs;
  }();
  if (!regs_ok) return cudaErrorInvalidDeviceFunction;
  static std::atomic<uint64_t> raised[2];
  const bool split = P.splits > 1;
  const cudaError_t e = tc_launch(split ? latent_prefill_kernel<true> : latent_prefill_kernel<false>,
                                  dim3((unsigned)((int64_t)P.pairs * a.B * a.Hq), (unsigned)P.splits), kAttnThreads,
                                  (size_t)(kSmall + 2 * kQTile + kSlots * kSlot), a.stream, P, a.device, &raised[split]);
  if (e != cudaSuccess || !split) return e;
  const int64_t rows = (int64_t)a.B * a.n_q * a.Hq;
  return tc_launch(latent_prefill_merge_kernel, dim3((unsigned)((rows + 7) / 8)), 256, (size_t)0, a.stream, P, a.device,
                   &raised[0]);
}

}  // namespace pkv
