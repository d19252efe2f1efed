// drafts.cuh — declarations of the operators that verify drafted tokens on the per-head
// pools: the rotated cache write (rotated_write.cu), attention for trees of drafted
// tokens (tree_attn.cu) and the move of accepted tokens (accept.cu).
#pragma once

#include "pkv_internal.cuh"

namespace pkv {

// Limits checked at the entry points: they keep every index of the kernels' grids and of
// a launch's rows within 32 bits.
constexpr int kDraftMaxBatch = 4096;
constexpr int kDraftMaxHeads = 1024;          // query heads
constexpr int kDraftMaxQueries = 1024;        // drafted tokens a sequence
constexpr int64_t kDraftMaxRows = 1 << 24;    // B * n_q * Hq
constexpr int kDraftMaxBlocks = 1 << 20;      // block-table width (2^25 tokens)

enum : int32_t { ERR_PATH = 32 };  // an accepted path outside its tree or not rising

struct RotatedWriteArgs {
  LayerView lv;
  int fmt, D, group;
  int n;
  const int32_t* rows;
  const int32_t* slots;
  const uint16_t* k;
  int64_t k_tok, k_head;     // strides in values
  const uint16_t* v;
  int64_t v_tok, v_head;
  const int32_t* positions;
  const float* cos_sin;      // [n_pos, rot]: cosines, then sines, of the rot / 2 angles
  int n_pos;
  int rot;                   // values of a head that are turned: a multiple of 32, at most D
  int interleaved;
  const uint16_t* k_norm;    // [D] or null
  const uint16_t* q_norm;
  float eps;
  int Hq;                    // 0: no queries
  const uint16_t* q;
  int64_t q_tok, q_head;
  uint16_t* qo;
  int64_t o_tok, o_head;
  const float* signs;        // [D] +-1 (packed)
  cudaStream_t stream;
};
// Warps that one token takes at most (the grid's bound).
int rotated_write_units(int hkv, int Hq);
cudaError_t launch_rotated_write(const RotatedWriteArgs& a);

struct TreeAttnArgs {
  LayerView lv;
  int fmt, D, group;
  int B, n_q, Hq, max_blocks;
  const uint16_t* q;         // [B, n_q, Hq, D]
  const uint32_t* mask;      // [n_q, words] a sequence, mask_stride words apart
  int64_t mask_stride;
  const int32_t* bt;
  const int32_t* ctx;
  float scale_log2;          // scale * log2(e)
  const float* signs;        // [D] +-1 (packed)
  uint16_t* out;             // [B, n_q, Hq, D]
  void* ws;
  int ctas;                  // CTAs a launch may use at once (one per SM)
  int device;                // the pool's, current at the call
  cudaStream_t stream;
};
size_t tree_attn_workspace(int D, int hkv, int B, int n_q, int Hq, int ctas);
cudaError_t launch_tree_attn(const TreeAttnArgs& a);

struct AcceptArgs {
  const uint8_t* const* table;  // slab pointers: [slab][layer][kind]
  int n_layers, n_kinds;
  int64_t token_bytes[4];       // stored bytes of a token (all heads) per kind
  int slab_blocks;
  int64_t rows_capacity;
  int B, n_q, max_path, max_blocks;
  const int32_t* path;          // [B, max_path]
  const int32_t* path_lens;     // [B]
  const int32_t* bt;
  const int32_t* ctx;
  int32_t* new_lens;            // [B] or null
  int32_t* err;
  cudaStream_t stream;
};
cudaError_t launch_accept(const AcceptArgs& a);

// A context length with n_q drafted tokens at its end: 0 (an unused batch slot) stays 0; a
// negative one, one beyond `lim` or one shorter than the drafted tokens is an error and
// counts as 0.
__device__ __forceinline__ int32_t draft_ctx(int32_t L, int64_t lim, int n_q, bool* bad) {
  *bad = L < 0 || (int64_t)L > lim || (L > 0 && L < n_q);
  return *bad ? 0 : L;
}

__device__ __forceinline__ bool draft_row_ok(const LayerView& lv, int32_t row) {
  return row >= 0 && (int64_t)row < lv.rows_capacity;
}

// Address of one (token, head) row of a stored tensor.
__device__ __forceinline__ uint8_t* draft_row(const LayerView& lv, int kind, int32_t row, int slot, int head) {
  const int32_t slab = row / lv.slab_blocks;
  const int32_t r = row - slab * lv.slab_blocks;
  return lv.tab.base[(size_t)slab * lv.tab.stride + kind] +
         ((size_t)(r * kBlockTokens + slot) * lv.hkv + head) * (size_t)lv.row_bytes[kind];
}

}  // namespace pkv
