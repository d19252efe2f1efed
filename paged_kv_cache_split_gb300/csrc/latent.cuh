// latent.cuh — declarations of the latent-pool operators (latent_*.cu): the cache
// write, the absorbed attention and the expanded attention.
//
// A latent pool stores one row per token, shared by every query head: a latent
// vector c (R values) followed by a position key r (kRope values), in bf16.
#pragma once

#include <cuda.h>

#include "pkv_internal.cuh"

namespace pkv {

constexpr int kRope = 64;        // values of the position key
constexpr int kLatentQuad = 4;   // 64-value columns that one copy of a latent block's row moves
constexpr int kLatentHead = 128; // expanded form: values of a head's key part and of its value

// Limits checked at the entry points: they keep every index of the kernels' grids and
// of a launch's rows within 32 bits.
constexpr int kLatentMaxBatch = 4096;
constexpr int kLatentMaxHeads = 1024;
constexpr int64_t kLatentMaxRows = 1 << 24;   // B * n_q * Hq
constexpr int kLatentMaxBlocks = 1 << 20;     // block-table width (2^25 tokens)

enum : int32_t { ERR_POS = 16 };  // a rotary position outside the table (pkv_pool_check_errors)

// Warps of the write per token: one for the latent row, one for every 32 heads.
constexpr int kLatentWriteHeads = 32;
inline int latent_write_units(int Hq) { return 1 + (Hq + kLatentWriteHeads - 1) / kLatentWriteHeads; }

struct LatentWriteArgs {
  LayerView lv;
  int R;                     // 256 or 512
  int n;
  const int32_t* rows;
  const int32_t* slots;
  const uint16_t* kv;        // [n] rows of R + kRope, kv_stride elements apart
  int64_t kv_stride;
  const int32_t* positions;
  const float* cos_sin;      // [n_pos, kRope]: cosines, then sines, of the kRope / 2 angles
  int n_pos;
  const uint16_t* weight;    // [R] or null
  float eps;
  int interleaved;
  int Hq;                    // 0: no queries
  const uint16_t* q;
  int64_t q_tok, q_head;
  uint16_t* qo;
  int64_t o_tok, o_head;
  int per_token;             // set by the launch
  cudaStream_t stream;
};
cudaError_t launch_latent_write(const LatentWriteArgs& a);

struct LatentAttnArgs {
  LayerView lv;
  int R, B, n_q, Hq, max_blocks;
  const uint16_t* ql;        // rows (b, i, h) of R, ql_stride elements apart
  int64_t ql_stride;
  const uint16_t* qr;        // rows (b, i, h) of kRope, qr_stride elements apart
  int64_t qr_stride;
  const int32_t* bt;
  const int32_t* ctx;
  float scale_log2;          // scale * log2(e)
  uint16_t* out;             // [B, n_q, Hq, R]
  void* ws;
  int ctas;                  // CTAs a launch may use at once (one per SM)
  int device;                // the pool's, current at the call
  cudaStream_t stream;
};
size_t latent_attn_workspace(int R, int B, int n_q, int Hq, int ctas);
cudaError_t launch_latent_attn(const LatentAttnArgs& a);

struct LatentPrefillArgs {
  LayerView lv;
  int R, B, n_q, Hq, max_blocks;
  const uint16_t* q;         // [B, n_q, Hq, kLatentHead + kRope]
  const uint16_t* wk;        // [Hq, kLatentHead, R]
  const uint16_t* wv;        // [Hq, kLatentHead, R]
  const int32_t* bt;
  const int32_t* ctx;
  int max_ctx;               // longest context the workspace was sized for
  float scale_log2;
  uint16_t* out;             // [B, n_q, Hq, kLatentHead]
  void* ws;
  int ctas;
  int device;
  cudaStream_t stream;
};
size_t latent_prefill_workspace(int B, int n_q, int Hq, int max_ctx, int ctas);
// A bf16 tensor map of `rank` dimensions (dims[0] contiguous, strides in bytes from the
// second on), read in boxes with the 128-byte swizzle; false if the driver refuses it.
bool encode_bf16_map(CUtensorMap* map, const void* base, int rank, const uint64_t* dims, const uint64_t* strides,
                     const uint32_t* box);
cudaError_t launch_latent_prefill(const LatentPrefillArgs& a);

// Address of one token's row, and whether a block-table entry names a pool row.
__device__ __forceinline__ bool latent_row_ok(const LayerView& lv, int32_t row) {
  return row >= 0 && (int64_t)row < lv.rows_capacity;
}

__device__ __forceinline__ uint8_t* latent_row(const LayerView& lv, int32_t row, int slot) {
  const int32_t slab = row / lv.slab_blocks;
  const int32_t r = row - slab * lv.slab_blocks;
  return lv.tab.base[(size_t)slab * lv.tab.stride] + (size_t)(r * kBlockTokens + slot) * (size_t)lv.row_bytes[0];
}

// Copies of a block's 32 tokens into shared memory: four 64-value columns from column c
// on, as [4 x 8 tokens][4 columns][8][128 bytes] (16 KB), or one column, as [32][128 bytes]
// (4 KB).  `map` is the slab's first tensor map, y8 the block's first row / 8.
__device__ __forceinline__ void latent_copy(void* dst, const void* map, int c, int y8, uint64_t* bar, uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.L2::cache_hint"
      " [%0], [%1, {%2, %2, %3, %4}], [%5], %6;" ::"r"(smem_u32(dst)),
      "l"(map), "r"(0), "r"(c), "r"(y8), "r"(smem_u32(bar)), "l"(policy)
      : "memory");
}
__device__ __forceinline__ void latent_copy_quad(void* dst, const uint8_t* map, int c, int y8, uint64_t* bar,
                                                 uint64_t policy) {
  latent_copy(dst, map, c, y8, bar, policy);
}
__device__ __forceinline__ void latent_copy_column(void* dst, const uint8_t* map, int c, int y8, uint64_t* bar,
                                                   uint64_t policy) {
  latent_copy(dst, map + 128, c, y8, bar, policy);
}
// Both maps become visible to this thread's copies, and, past a __syncwarp, to those of the
// lane that issues them: the fence then lies on the path from the maps' writing to the copy
// (a shuffle of the address alone orders nothing).
__device__ __forceinline__ void latent_maps_acquire(const uint8_t* map) {
  tensormap_acquire(map);
  tensormap_acquire(map + 128);
}

// A context length as the attention uses it: 0 (an unused batch slot) stays 0; a
// negative one, one beyond `lim` or one shorter than the n_q queries is an error and
// counts as 0, so that its output rows are zero.
__device__ __forceinline__ int32_t latent_ctx(int32_t L, int64_t lim, int n_q, bool* bad) {
  *bad = L < 0 || (int64_t)L > lim || (L > 0 && L < n_q);
  return *bad ? 0 : L;
}

}  // namespace pkv
