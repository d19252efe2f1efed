// pool.cu — host runtime of the chunked-slab pool and the C ABI entry points.
//
// Storage follows mlxcel issue #235 ("chunked slab storage for the paged pool"):
// per layer and stored tensor a vector of fixed-size slabs
// [slab_blocks, block_size, n_kv_heads, row]; row -> (row / slab_blocks,
// row % slab_blocks); growth appends fresh zeroed slabs, never copying or
// freeing existing ones (Proposed solution, bullets 1-2), and the slab-append
// counter and reserved bytes are sums over slabs (touch point 5).  Block ids,
// refcounts and free-row reuse stay row-level concepts (Behavioral invariants).
//
// One allocation ("slab group") holds slab s of every layer and tensor; the
// device pointer table still has one entry per (slab, layer, tensor), which is
// what every kernel reads (touch point 4: per-slab base pointers; touch point 7:
// one mapping helper).
#include <cuda.h>
#include <cuda_runtime.h>

#include <cfloat>
#include <cmath>
#include <cstdio>
#include <cstring>
#include <new>
#include <string>
#include <vector>

#include "drafts.cuh"
#include "latent.cuh"
#include "pkv_internal.cuh"

using namespace pkv;

struct pkv_pool {
  pkv_pool_config cfg{};
  pkv_allocator alloc{};
  bool default_alloc = true;
  int device = 0;
  int n_sm = 0;
  size_t smem_optin = 0;
  int n_kinds = 2;
  int n_maps = 2;                        // tensor maps per slab and layer (latent: two of its one tensor)
  int64_t row_bytes[4] = {0, 0, 0, 0};
  int64_t slab_bytes[4] = {0, 0, 0, 0};  // one slab of one layer, per kind
  int64_t group_bytes = 0;               // one slab index across layers and kinds
  int64_t layer_bytes = 0;               // one slab of one layer, all kinds
  int64_t maps_offset = 0;               // tensor maps at the group's tail
  std::vector<void*> groups;             // allocation per slab index
  uint8_t** table_host = nullptr;        // pinned [max_slabs][n_layers][n_kinds]
  uint8_t** table_dev = nullptr;
  int32_t* err_dev = nullptr;
  float* signs_dev = nullptr;            // [head_dim] +-1
  double inv_sqrt_d = 0.0;
  std::vector<int32_t> refcount;
  std::vector<int32_t> free_rows;        // LIFO
  int64_t rows_in_use = 0;
  int64_t append_events = 0;
  int decode_ctas = 0;
  cudaStream_t last_stream = nullptr;
};

static thread_local std::string g_last_error;

namespace pkv {
// Defined in write.cu.
cudaError_t launch_expand_prefill(int B, int n_q, int nq, int max_blocks, const int32_t* bt, const int32_t* ctx,
                                  int32_t* bt_out, int32_t* ctx_out, int32_t* err, cudaStream_t s);
cudaError_t launch_serde_blocks(const uint8_t* const* table, int n_layers, int n_kinds, const int64_t* block_bytes,
                               int slab_blocks, int64_t rows_capacity, int n, const int32_t* rows, uint8_t* buf,
                               int64_t rec_bytes, int to_pool, int32_t* err, cudaStream_t s);
void set_last_error(const char* msg) { g_last_error = msg ? msg : ""; }
}  // namespace pkv

static pkv_status cuda_fail(cudaError_t e, const char* where) {
  g_last_error = std::string(where) + ": " + cudaGetErrorString(e);
  return PKV_ERR_CUDA;
}

#define PKV_CUDA(call, where)                      \
  do {                                             \
    cudaError_t e_ = (call);                       \
    if (e_ != cudaSuccess) return cuda_fail(e_, where); \
  } while (0)

// splitmix64 (Steele, Lea & Flood 2014): output for state x.
static uint64_t splitmix64(uint64_t x) {
  uint64_t z = x + 0x9E3779B97F4A7C15ull;
  z = (z ^ (z >> 30)) * 0xBF58476D1CE4E5B9ull;
  z = (z ^ (z >> 27)) * 0x94D049BB133111EBull;
  return z ^ (z >> 31);
}

static LayerView layer_view(const pkv_pool* p, int layer) {
  LayerView lv;
  lv.tab.base = p->table_dev + (size_t)layer * p->n_kinds;
  lv.tab.stride = p->cfg.n_layers * p->n_kinds;
  lv.n_kinds = p->n_kinds;
  lv.hkv = p->cfg.n_kv_heads;
  lv.slab_blocks = p->cfg.slab_blocks;
  lv.rows_capacity = (int64_t)p->groups.size() * p->cfg.slab_blocks;
  for (int k = 0; k < 4; ++k) lv.row_bytes[k] = (int)p->row_bytes[k];
  lv.err = p->err_dev;
  lv.map_delta = p->maps_offset - (int64_t)layer * p->layer_bytes + (int64_t)layer * p->n_maps * 128;
  for (int k = 0; k < 4; ++k)
    lv.box_bytes[k] = k < p->n_kinds ? tma_box_bytes(p->row_bytes[k] * p->cfg.n_kv_heads) : 0;
  return lv;
}

// cuTensorMapEncodeTiled, looked up once through the runtime's driver entry point.
typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                  const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                  CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

static EncodeTiledFn encode_tiled_fn() {
  static EncodeTiledFn fn = nullptr;
  static bool tried = false;
  if (!tried) {
    tried = true;
    void* f = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<EncodeTiledFn>(f);
    else
      cudaGetLastError();
  }
  return fn;
}

bool pkv::encode_bf16_map(CUtensorMap* map, const void* base, int rank, const uint64_t* dims, const uint64_t* strides,
                          const uint32_t* box) {
  EncodeTiledFn enc = encode_tiled_fn();
  if (!enc) return false;
  const cuuint32_t estr[3] = {1u, 1u, 1u};
  cuuint64_t d[3], st[2];
  cuuint32_t bx[3];
  for (int i = 0; i < rank; ++i) d[i] = dims[i], bx[i] = box[i];
  for (int i = 0; i + 1 < rank; ++i) st[i] = strides[i];
  return enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, (cuuint32_t)rank, const_cast<void*>(base), d, st, bx, estr,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Tensor maps of one slab group: for every layer and stored tensor, the slab
// [slab_blocks * 32 tokens][Hkv * row] bytes viewed in 3-D as [column block][token]
// [W bytes] (W = box_bytes), read in boxes of 16 tokens x the whole row, which land
// as row/W boxes of 16 x W bytes with the matching shared-memory swizzle.  A latent
// slab has two maps, of the same [token][row] bytes in 4-D as [eight tokens][column
// block][token of the eight][128 bytes]: a copy of 32 tokens x `cols` column blocks lands
// as [4][cols][8][128], each eight tokens of a column block a 1024-byte swizzle atom.
// The first map copies four column blocks at a time, the second one.
static bool encode_group_maps(const pkv_pool* p, uint8_t* group, std::vector<CUtensorMap>& maps) {
  EncodeTiledFn enc = encode_tiled_fn();
  if (!enc) return false;
  const int L = p->cfg.n_layers, K = p->n_kinds;
  maps.resize((size_t)L * p->n_maps);
  int64_t off = 0;
  if (p->cfg.format == PKV_FMT_LATENT) {
    const cuuint64_t row = (cuuint64_t)p->row_bytes[PKV_KIND_K];
    const cuuint64_t dims[4] = {128, 8, row / 128, (cuuint64_t)p->cfg.slab_blocks * kBlockTokens / 8};
    const cuuint64_t strides[3] = {row, 128, 8 * row};
    const cuuint32_t estr[4] = {1u, 1u, 1u, 1u};
    for (int l = 0; l < L; ++l, off += p->slab_bytes[PKV_KIND_K])
      for (int m = 0; m < 2; ++m) {
        const cuuint32_t boxd[4] = {128u, 8u, m == 0 ? (cuuint32_t)kLatentQuad : 1u, kBlockTokens / 8};
        if (enc(&maps[(size_t)l * 2 + m], CU_TENSOR_MAP_DATA_TYPE_UINT8, 4, group + off, dims, strides, boxd, estr,
                CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
          return false;
      }
    return true;
  }
  for (int l = 0; l < L; ++l)
    for (int k = 0; k < K; ++k) {
      const int64_t row = p->row_bytes[k] * p->cfg.n_kv_heads;
      const int box = tma_box_bytes(row);
      const CUtensorMapSwizzle sw = box == 128 ? CU_TENSOR_MAP_SWIZZLE_128B
                                    : box == 64 ? CU_TENSOR_MAP_SWIZZLE_64B
                                    : box == 32 ? CU_TENSOR_MAP_SWIZZLE_32B
                                                : CU_TENSOR_MAP_SWIZZLE_NONE;
      // 3-D view [column block][token][W bytes] of the [token][row] tensor: one copy
      // moves 16 tokens of the whole row and lands as nx boxes of 16 x W bytes.
      const cuuint64_t nx = (cuuint64_t)(row / box);
      const cuuint64_t dims[3] = {(cuuint64_t)box, (cuuint64_t)p->cfg.slab_blocks * kBlockTokens, nx};
      const cuuint64_t strides[2] = {(cuuint64_t)row, (cuuint64_t)box};
      const cuuint32_t boxd[3] = {(cuuint32_t)box, 16u, (cuuint32_t)nx};
      const cuuint32_t estr[3] = {1u, 1u, 1u};
      if (enc(&maps[(size_t)l * K + k], CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, group + off, dims, strides, boxd, estr,
              CU_TENSOR_MAP_INTERLEAVE_NONE, sw, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
        return false;
      off += p->slab_bytes[k];
    }
  return true;
}

extern "C" {

const char* pkv_status_string(pkv_status s) {
  switch (s) {
    case PKV_OK: return "ok";
    case PKV_ERR_INVALID: return "invalid argument";
    case PKV_ERR_OOM: return "allocation failed (pool unchanged)";
    case PKV_ERR_CUDA: return "CUDA runtime error";
    case PKV_ERR_FORMAT: return "storage identity / format mismatch";
    case PKV_ERR_RANGE: return "index out of range";
    case PKV_ERR_DEVICE: return "device error word set";
  }
  return "unknown status";
}

const char* pkv_last_error(void) { return g_last_error.c_str(); }

pkv_status pkv_pool_create(const pkv_pool_config* cfg, const pkv_allocator* alloc, void* stream,
                           pkv_pool** out) {
  if (!cfg || !out) return PKV_ERR_INVALID;
  *out = nullptr;
  const FormatBits fb = format_bits(cfg->format);
  const int D = cfg->head_dim;
  const bool latent = cfg->format == PKV_FMT_LATENT;
  if (latent && (cfg->n_kv_heads != 1 || cfg->group_size != kRope || !(D == 256 || D == 512)))
    return PKV_ERR_INVALID;
  if ((!latent && (fb.k == 0 || !(D == 64 || D == 128 || D == 256))) || cfg->n_layers < 1 || cfg->n_kv_heads < 1 ||
      cfg->n_kv_heads > 8 || cfg->block_size != kBlockTokens || cfg->slab_blocks < 1 || cfg->slab_blocks > 4096 ||
      cfg->max_slabs < 1)
    return PKV_ERR_INVALID;
  // Groups of 32 for every packed format; groups of 64 (the five-bit K4/V4 layout)
  // for K4/V4 with head_dim >= 128, so a (token, head) metadata row stays a whole
  // number of 16-byte chunks.
  if (!latent && cfg->format != PKV_FMT_BF16 && cfg->group_size != kGroup &&
      !(cfg->group_size == kGroupWide && cfg->format == PKV_FMT_K4V4 && D >= 128))
    return PKV_ERR_INVALID;
  if (alloc && (!alloc->alloc || !alloc->release)) return PKV_ERR_INVALID;

  pkv_pool* p = new (std::nothrow) pkv_pool();
  if (!p) return PKV_ERR_OOM;
  p->cfg = *cfg;
  if (cfg->format == PKV_FMT_BF16) p->cfg.group_size = cfg->group_size;
  if (alloc) {
    p->alloc = *alloc;
    p->default_alloc = false;
  }
  p->last_stream = (cudaStream_t)stream;
  auto fail = [&](pkv_status st) {
    pkv_pool_destroy(p);
    return st;
  };
  cudaError_t e = cudaGetDevice(&p->device);
  if (e != cudaSuccess) return fail(cuda_fail(e, "cudaGetDevice"));
  e = cudaDeviceGetAttribute(&p->n_sm, cudaDevAttrMultiProcessorCount, p->device);
  if (e != cudaSuccess) return fail(cuda_fail(e, "cudaDeviceGetAttribute(SM count)"));
  int optin = 0;
  e = cudaDeviceGetAttribute(&optin, cudaDevAttrMaxSharedMemoryPerBlockOptin, p->device);
  if (e != cudaSuccess) return fail(cuda_fail(e, "cudaDeviceGetAttribute(smem)"));
  p->smem_optin = (size_t)optin;

  p->n_kinds = latent ? 1 : (cfg->format == PKV_FMT_BF16) ? 2 : 4;
  p->n_maps = latent ? 2 : p->n_kinds;
  p->row_bytes[PKV_KIND_K] = latent ? (int64_t)(D + kRope) * 2 : (int64_t)D * fb.k / 8;
  p->row_bytes[PKV_KIND_V] = latent ? 0 : (int64_t)D * fb.v / 8;
  if (p->n_kinds == 4) {
    p->row_bytes[PKV_KIND_KMETA] = (int64_t)(D / cfg->group_size) * 2 * sizeof(float);
    p->row_bytes[PKV_KIND_VMETA] = p->row_bytes[PKV_KIND_KMETA];
  }
  const int64_t per_row_tokens = (int64_t)cfg->slab_blocks * kBlockTokens * cfg->n_kv_heads;
  p->layer_bytes = 0;
  for (int k = 0; k < p->n_kinds; ++k) {
    p->slab_bytes[k] = per_row_tokens * p->row_bytes[k];
    p->layer_bytes += p->slab_bytes[k];
  }
  p->group_bytes = p->layer_bytes * cfg->n_layers;
  // Tensor maps (128 bytes each, 64-byte aligned) after the slab data.
  p->maps_offset = (p->group_bytes + 127) / 128 * 128;
  p->group_bytes = p->maps_offset + (int64_t)cfg->n_layers * p->n_maps * 128;
  for (int k = 0; k < p->n_kinds; ++k)
    if (tma_box_bytes(p->row_bytes[k] * cfg->n_kv_heads) == 0) return fail(PKV_ERR_INVALID);

  const size_t table_entries = (size_t)cfg->max_slabs * cfg->n_layers * p->n_kinds;
  e = cudaMallocHost((void**)&p->table_host, table_entries * sizeof(uint8_t*));
  if (e != cudaSuccess) return fail(cuda_fail(e, "cudaMallocHost(slab table)"));
  memset(p->table_host, 0, table_entries * sizeof(uint8_t*));
  e = cudaMalloc((void**)&p->table_dev, table_entries * sizeof(uint8_t*));
  if (e != cudaSuccess) return fail(cuda_fail(e, "cudaMalloc(slab table)"));
  e = cudaMemset(p->table_dev, 0, table_entries * sizeof(uint8_t*));
  if (e != cudaSuccess) return fail(cuda_fail(e, "cudaMemset(slab table)"));
  e = cudaMalloc((void**)&p->err_dev, 64);
  if (e != cudaSuccess) return fail(cuda_fail(e, "cudaMalloc(error word)"));
  e = cudaMemset(p->err_dev, 0, 64);
  if (e != cudaSuccess) return fail(cuda_fail(e, "cudaMemset(error word)"));

  // Fixed signed Hadamard basis: s_i = -1 iff the top bit of splitmix64(seed + i)
  // is set (mlx-swift-lm #142, Summary: Q and K share one signed Hadamard basis that
  // never changes).
  std::vector<float> signs((size_t)D);
  for (int i = 0; i < D; ++i) signs[i] = (splitmix64(cfg->hadamard_seed + (uint64_t)i) >> 63) ? -1.f : 1.f;
  e = cudaMalloc((void**)&p->signs_dev, sizeof(float) * (size_t)D);
  if (e != cudaSuccess) return fail(cuda_fail(e, "cudaMalloc(signs)"));
  e = cudaMemcpy(p->signs_dev, signs.data(), sizeof(float) * (size_t)D, cudaMemcpyHostToDevice);
  if (e != cudaSuccess) return fail(cuda_fail(e, "cudaMemcpy(signs)"));
  p->inv_sqrt_d = 1.0 / std::sqrt((double)D);
  *out = p;
  return PKV_OK;
}

void pkv_pool_destroy(pkv_pool* p) {
  if (!p) return;
  // Work enqueued on any stream may still read the slabs: wait for the device.
  if (!p->groups.empty()) cudaDeviceSynchronize();
  for (size_t i = 0; i < p->groups.size(); ++i) {
    if (!p->groups[i]) continue;
    if (p->default_alloc)
      cudaFree(p->groups[i]);
    else
      p->alloc.release(p->alloc.ctx, p->groups[i], (void*)p->last_stream);
  }
  if (p->table_dev) cudaFree(p->table_dev);
  if (p->table_host) cudaFreeHost(p->table_host);
  if (p->err_dev) cudaFree(p->err_dev);
  if (p->signs_dev) cudaFree(p->signs_dev);
  delete p;
}

pkv_status pkv_append_slab(pkv_pool* p, int n_slabs, void* stream) {
  if (!p || n_slabs < 0) return PKV_ERR_INVALID;
  if (n_slabs == 0) return PKV_OK;
  const int have = (int)p->groups.size();
  if (have + n_slabs > p->cfg.max_slabs) return PKV_ERR_RANGE;
  cudaStream_t s = (cudaStream_t)stream;
  std::vector<void*> fresh;
  fresh.reserve((size_t)n_slabs);
  for (int i = 0; i < n_slabs; ++i) {
    void* ptr = nullptr;
    if (p->default_alloc) {
      if (cudaMallocAsync(&ptr, (size_t)p->group_bytes, s) != cudaSuccess) {
        cudaGetLastError();
        ptr = nullptr;
      }
    } else {
      ptr = p->alloc.alloc(p->alloc.ctx, (size_t)p->group_bytes, stream);
    }
    if (!ptr) {
      for (void* q : fresh) {
        if (p->default_alloc)
          cudaFreeAsync(q, s);
        else
          p->alloc.release(p->alloc.ctx, q, stream);
      }
      return PKV_ERR_OOM;
    }
    fresh.push_back(ptr);
  }
  // Tensor maps of the new slabs, encoded before anything is enqueued so that a
  // failure leaves the pool unchanged.
  std::vector<std::vector<CUtensorMap>> maps(fresh.size());
  for (size_t i = 0; i < maps.size(); ++i) {
    if (!encode_group_maps(p, (uint8_t*)fresh[i], maps[i])) {
      for (void* q : fresh) {
        if (p->default_alloc)
          cudaFreeAsync(q, s);
        else
          p->alloc.release(p->alloc.ctx, q, stream);
      }
      g_last_error = "cuTensorMapEncodeTiled unavailable or rejected a slab";
      return PKV_ERR_CUDA;
    }
  }
  // Zero the new slabs (a fresh zeros slab), then publish their base pointers.
  for (void* ptr : fresh) PKV_CUDA(cudaMemsetAsync(ptr, 0, (size_t)p->group_bytes, s), "cudaMemsetAsync(slab)");
  // The maps are copied from pageable memory: the call stages the bytes before it
  // returns, so the vectors may go out of scope at once.
  for (size_t i = 0; i < maps.size(); ++i)
    PKV_CUDA(cudaMemcpyAsync((uint8_t*)fresh[i] + p->maps_offset, maps[i].data(),
                             maps[i].size() * sizeof(CUtensorMap), cudaMemcpyHostToDevice, s),
             "cudaMemcpyAsync(tensor maps)");
  const int L = p->cfg.n_layers, K = p->n_kinds;
  for (int i = 0; i < n_slabs; ++i) {
    uint8_t* g = (uint8_t*)fresh[(size_t)i];
    int64_t off = 0;
    for (int l = 0; l < L; ++l)
      for (int k = 0; k < K; ++k) {
        p->table_host[((size_t)(have + i) * L + l) * K + k] = g + off;
        off += p->slab_bytes[k];
      }
  }
  // The pinned host entries of these slabs are never rewritten, so the copy may
  // run asynchronously.
  const size_t first = (size_t)have * L * K, count = (size_t)n_slabs * L * K;
  PKV_CUDA(cudaMemcpyAsync(p->table_dev + first, p->table_host + first, count * sizeof(uint8_t*),
                           cudaMemcpyHostToDevice, s),
           "cudaMemcpyAsync(slab table)");
  for (int i = 0; i < n_slabs; ++i) p->groups.push_back(fresh[(size_t)i]);
  const int64_t old_rows = (int64_t)have * p->cfg.slab_blocks;
  const int64_t new_rows = (int64_t)p->groups.size() * p->cfg.slab_blocks;
  p->refcount.resize((size_t)new_rows, 0);
  // The free list is a stack: released rows sit on top and are reused first
  // (LIFO).  Fresh rows go underneath them, in descending order, so that once the
  // released rows are used up the fresh rows come out in ascending order.
  std::vector<int32_t> fresh_rows;
  for (int64_t r = new_rows - 1; r >= old_rows; --r) fresh_rows.push_back((int32_t)r);
  p->free_rows.insert(p->free_rows.begin(), fresh_rows.begin(), fresh_rows.end());
  p->append_events += n_slabs;
  p->last_stream = s;
  return PKV_OK;
}

pkv_status pkv_alloc_rows(pkv_pool* p, int n, int32_t* rows_host, void* stream) {
  if (!p || n < 0 || (n > 0 && !rows_host)) return PKV_ERR_INVALID;
  if ((int64_t)p->free_rows.size() < n) {
    const int64_t deficit = n - (int64_t)p->free_rows.size();
    const int need = (int)((deficit + p->cfg.slab_blocks - 1) / p->cfg.slab_blocks);
    pkv_status st = pkv_append_slab(p, need, stream);
    if (st != PKV_OK) return st;
  }
  for (int i = 0; i < n; ++i) {
    int32_t r = p->free_rows.back();
    p->free_rows.pop_back();
    p->refcount[(size_t)r] = 1;
    rows_host[i] = r;
  }
  p->rows_in_use += n;
  return PKV_OK;
}

pkv_status pkv_retain_row(pkv_pool* p, int32_t row) {
  if (!p) return PKV_ERR_INVALID;
  if (row < 0 || (size_t)row >= p->refcount.size() || p->refcount[(size_t)row] <= 0) return PKV_ERR_RANGE;
  p->refcount[(size_t)row] += 1;
  return PKV_OK;
}

pkv_status pkv_release_row(pkv_pool* p, int32_t row) {
  if (!p) return PKV_ERR_INVALID;
  if (row < 0 || (size_t)row >= p->refcount.size() || p->refcount[(size_t)row] <= 0) return PKV_ERR_RANGE;
  if (--p->refcount[(size_t)row] == 0) {
    p->free_rows.push_back(row);
    p->rows_in_use -= 1;
  }
  return PKV_OK;
}

int pkv_slab_runs(const int32_t* rows, int n, int slab_blocks, int32_t* run_start) {
  if (n <= 0) return 0;
  if (!rows || !run_start || slab_blocks < 1) return -1;
  int runs = 0;
  int32_t prev_slab = -1;
  for (int i = 0; i < n; ++i) {
    const int32_t s = rows[i] / slab_blocks;
    if (i == 0 || s != prev_slab) run_start[runs++] = i;
    prev_slab = s;
  }
  return runs;
}

pkv_status pkv_write_block(pkv_pool* p, int layer, int n, const int32_t* rows, const int32_t* slots,
                           const void* k, const void* v, void* stream) {
  if (!p || n < 0 || layer < 0 || layer >= p->cfg.n_layers) return PKV_ERR_INVALID;
  if (p->cfg.format == PKV_FMT_LATENT) return PKV_ERR_FORMAT;
  if (n == 0) return PKV_OK;
  if (!rows || !slots || !k || !v) return PKV_ERR_INVALID;
  if (((uintptr_t)k & 15u) != 0 || ((uintptr_t)v & 15u) != 0) return PKV_ERR_INVALID;
  cudaStream_t s = (cudaStream_t)stream;
  LayerView lv = layer_view(p, layer);
  PKV_CUDA(launch_write(lv, p->cfg.format, p->cfg.head_dim, p->cfg.group_size, n, rows, slots, (const uint16_t*)k,
                        (const uint16_t*)v, p->signs_dev, p->inv_sqrt_d, s),
           "write_block launch");
  p->last_stream = s;
  return PKV_OK;
}

pkv_status pkv_copy_on_write_block(pkv_pool* p, int n, const int32_t* src, const int32_t* dst, void* stream) {
  if (!p || n < 0) return PKV_ERR_INVALID;
  if (n == 0) return PKV_OK;
  if (!src || !dst) return PKV_ERR_INVALID;
  cudaStream_t s = (cudaStream_t)stream;
  int64_t block_bytes[4] = {0, 0, 0, 0};
  for (int k = 0; k < p->n_kinds; ++k) block_bytes[k] = p->row_bytes[k] * kBlockTokens * p->cfg.n_kv_heads;
  PKV_CUDA(launch_copy_blocks(p->table_dev, p->cfg.n_layers, p->n_kinds, block_bytes, p->cfg.slab_blocks,
                              (int64_t)p->groups.size() * p->cfg.slab_blocks, n, src, dst, p->err_dev, s),
           "copy_on_write_block launch");
  p->last_stream = s;
  return PKV_OK;
}

// Bytes of one block record: every layer, every stored tensor.
static size_t record_bytes(const pkv_pool* p, int64_t* block_bytes) {
  size_t per_layer = 0;
  for (int k = 0; k < 4; ++k) block_bytes[k] = 0;
  for (int k = 0; k < p->n_kinds; ++k) {
    block_bytes[k] = p->row_bytes[k] * kBlockTokens * p->cfg.n_kv_heads;
    per_layer += (size_t)block_bytes[k];
  }
  return per_layer * (size_t)p->cfg.n_layers;
}

pkv_status pkv_pool_get_config(const pkv_pool* p, pkv_pool_config* out) {
  if (!p || !out) return PKV_ERR_INVALID;
  *out = p->cfg;
  return PKV_OK;
}

pkv_status pkv_block_record_bytes(const pkv_pool* p, size_t* bytes) {
  if (!p || !bytes) return PKV_ERR_INVALID;
  int64_t bb[4];
  *bytes = record_bytes(p, bb);
  return PKV_OK;
}

static pkv_status serde_blocks(pkv_pool* p, int n, const int32_t* rows, uint8_t* buf, size_t buf_bytes, int to_pool,
                               cudaStream_t s) {
  if (n == 0) return PKV_OK;
  if (!rows || !buf || ((uintptr_t)buf & 15u) != 0) return PKV_ERR_INVALID;
  int64_t bb[4];
  const size_t rec = record_bytes(p, bb);
  if (buf_bytes / rec < (size_t)n) return PKV_ERR_RANGE;
  PKV_CUDA(launch_serde_blocks(p->table_dev, p->cfg.n_layers, p->n_kinds, bb, p->cfg.slab_blocks,
                               (int64_t)p->groups.size() * p->cfg.slab_blocks, n, rows, buf, (int64_t)rec, to_pool,
                               p->err_dev, s),
           to_pool ? "import_blocks launch" : "export_blocks launch");
  p->last_stream = s;
  return PKV_OK;
}

pkv_status pkv_export_blocks(pkv_pool* p, int n, const int32_t* rows_dev, void* out_dev, size_t out_bytes,
                             void* stream) {
  if (!p || n < 0) return PKV_ERR_INVALID;
  return serde_blocks(p, n, rows_dev, (uint8_t*)out_dev, out_bytes, 0, (cudaStream_t)stream);
}

pkv_status pkv_import_blocks(pkv_pool* p, const pkv_pool_config* identity, int n, const int32_t* rows_dev,
                             const void* in_dev, size_t in_bytes, void* stream) {
  if (!p || !identity || n < 0) return PKV_ERR_INVALID;
  // The records' storage identity (and layer count) must be this pool's, checked
  // before any device work.
  if (pkv_pool_check_identity(p, identity) != PKV_OK || identity->n_layers != p->cfg.n_layers) return PKV_ERR_FORMAT;
  return serde_blocks(p, n, rows_dev, (uint8_t*)const_cast<void*>(in_dev), in_bytes, 1, (cudaStream_t)stream);
}

pkv_status pkv_gather_visible(pkv_pool* p, int layer, const int32_t* bt_row, int ctx, void* k_out,
                              void* v_out, void* kmeta_out, void* vmeta_out, void* stream) {
  if (!p || layer < 0 || layer >= p->cfg.n_layers || ctx < 0) return PKV_ERR_INVALID;
  if (ctx == 0) return PKV_OK;  // nothing visible; output pointers may be NULL
  const bool packed = p->n_kinds == 4;
  const bool latent = p->n_kinds == 1;  // one stored tensor
  if (packed != (kmeta_out != nullptr) || packed != (vmeta_out != nullptr) || (latent && v_out)) return PKV_ERR_FORMAT;
  if (!bt_row || !k_out || (!latent && !v_out)) return PKV_ERR_INVALID;
  for (void* o : {k_out, v_out, kmeta_out, vmeta_out})
    if (((uintptr_t)o & 15u) != 0) return PKV_ERR_INVALID;
  cudaStream_t s = (cudaStream_t)stream;
  uint8_t* outs[4] = {(uint8_t*)k_out, (uint8_t*)v_out, (uint8_t*)kmeta_out, (uint8_t*)vmeta_out};
  PKV_CUDA(launch_gather(layer_view(p, layer), bt_row, ctx, outs, s), "gather_visible launch");
  p->last_stream = s;
  return PKV_OK;
}

static int decode_grid(const pkv_pool* p) { return p->decode_ctas > 0 ? p->decode_ctas : p->n_sm; }

static size_t align_up(size_t x, size_t a) { return (x + a - 1) / a * a; }

static size_t workspace_bytes(const pkv_pool* p, int B, int Hq) {
  const int D = p->cfg.head_dim;
  return align_up((size_t)B * sizeof(int32_t), 256) +
         (size_t)(decode_grid(p) + B) * (size_t)Hq * (size_t)(D + 4) * sizeof(float);
}

pkv_status pkv_decode_workspace_bytes(const pkv_pool* p, int B, int Hq, int max_ctx, size_t* bytes) {
  (void)max_ctx;
  if (!p || !bytes || B < 0 || Hq < 1) return PKV_ERR_INVALID;
  if (p->cfg.format == PKV_FMT_LATENT) return PKV_ERR_FORMAT;
  *bytes = workspace_bytes(p, B, Hq);
  return PKV_OK;
}

pkv_status pkv_decode_set_ctas(pkv_pool* p, int n_ctas) {
  if (!p || n_ctas < 0) return PKV_ERR_INVALID;
  p->decode_ctas = n_ctas;
  return PKV_OK;
}

static pkv_status decode_impl(pkv_pool* p, int layer, int B, int Hq, const void* q, const int32_t* bt,
                              int max_blocks, const int32_t* ctx, float scale, void* out, void* ws, size_t ws_bytes,
                              void* stream, int kv_reuse, int nq) {
  if (!p || layer < 0 || layer >= p->cfg.n_layers || B < 0 || Hq < 1 || max_blocks < 0)
    return PKV_ERR_INVALID;
  if (p->cfg.format == PKV_FMT_LATENT) return PKV_ERR_FORMAT;
  if (B == 0) return PKV_OK;
  const int hkv = p->cfg.n_kv_heads;
  if (Hq % hkv) return PKV_ERR_INVALID;
  const int G = Hq / hkv;  // with nq > 1: rows of the tile per kv head (nq x heads per kv head)
  if (!(G == 1 || G == 2 || G == 4 || G == 8 || (nq > 1 && G == 16))) return PKV_ERR_INVALID;
  if (!q || !bt || !ctx || !out || !ws) return PKV_ERR_INVALID;
  if (!std::isfinite(scale)) return PKV_ERR_INVALID;
  if (ws_bytes < workspace_bytes(p, B, Hq)) return PKV_ERR_INVALID;
  if (((uintptr_t)ws & 255u) != 0 || ((uintptr_t)q & 15u) != 0 || ((uintptr_t)out & 15u) != 0)
    return PKV_ERR_INVALID;
  DecodePlan plan;
  if (!plan_decode(p->cfg.format, p->cfg.head_dim, G, hkv, B, p->cfg.group_size, &plan) ||
      plan.smem_bytes > p->smem_optin)
    return PKV_ERR_INVALID;
  DecodeArgs a;
  a.lv = layer_view(p, layer);
  a.fmt = p->cfg.format;
  a.D = p->cfg.head_dim;
  a.G = G;
  a.B = B;
  a.Hq = Hq;
  a.max_blocks = max_blocks;
  a.q = (const uint16_t*)q;
  a.bt = bt;
  a.ctx = ctx;
  a.scale_log2 = (float)((double)scale * 1.4426950408889634);
  a.inv_sqrt_d = (float)p->inv_sqrt_d;
  a.signs = p->signs_dev;
  a.out = (uint16_t*)out;
  a.counters = (int32_t*)ws;
  a.partials = (float*)((uint8_t*)ws + align_up((size_t)B * sizeof(int32_t), 256));
  a.grid = decode_grid(p);
  a.tokens_per_stage = plan.tokens_per_stage;
  a.n_stages = plan.n_stages;
  a.dim_split = plan.dim_split;
  a.group = p->cfg.group_size;
  a.kv_reuse = kv_reuse;
  a.nq = nq;
  // what a sequence start costs a CTA, in quarter units (the CTA split weighs it; the
  // values measured best on the bench workloads): bf16 only reads q's fragments; the
  // packed kernels rotate q at each start (worth more units where units are cheap, at
  // head_dim 64), and with 16 tile rows rotate 16 rows and write two row sets
  const int D = p->cfg.head_dim;
  a.seg_cost = p->cfg.format == PKV_FMT_BF16 ? 2 : (G > 8 ? 16 : (D <= 64 ? 8 : 4));
  a.smem_bytes = plan.smem_bytes;
  a.stream = (cudaStream_t)stream;
  cudaError_t e;
  switch (p->cfg.format) {
    case PKV_FMT_BF16: e = launch_decode_bf16(a); break;
    case PKV_FMT_K4V4: e = launch_decode_k4v4(a); break;
    case PKV_FMT_K8V4: e = launch_decode_k8v4(a); break;
    default: e = launch_decode_k8v8(a); break;
  }
  if (e != cudaSuccess) return cuda_fail(e, "paged_decode_attention launch");
  p->last_stream = (cudaStream_t)stream;
  return PKV_OK;
}

pkv_status pkv_paged_decode_attention(pkv_pool* p, int layer, int B, int Hq, const void* q,
                                      const int32_t* bt, int max_blocks, const int32_t* ctx, int max_ctx,
                                      float scale, void* out, void* ws, size_t ws_bytes, void* stream) {
  (void)max_ctx;
  return decode_impl(p, layer, B, Hq, q, bt, max_blocks, ctx, scale, out, ws, ws_bytes, stream, 0, 1);
}

// Chunked prefill: queries per virtual sequence.  The kernels serve nq queries of
// one sequence per tile when nq x (query heads per kv head) fits the tile's 16 rows
// (8 at head_dim 256) and nq divides the chunk: the bf16 kernel for any such power
// of two, the packed kernels for the tile's full 16 rows or 8 rows.
static int prefill_nq(const pkv_pool* p, int n_q, int Hq) {
  if (Hq % p->cfg.n_kv_heads) return 1;
  const int G = Hq / p->cfg.n_kv_heads;
  const int rows = p->cfg.head_dim <= 128 ? 16 : 8;
  if (p->cfg.format != PKV_FMT_BF16) {
    for (int r = rows; r >= 8; r >>= 1) {
      const int nq = r / G;
      if (nq > 1 && n_q % nq == 0) return nq;
    }
    return 1;
  }
  for (int nq = 16; nq > 1; nq >>= 1)
    if (nq * G <= rows && n_q % nq == 0) return nq;
  return 1;
}

// The expanded block table and context lengths, then the decode workspace of the
// B * n_q / nq virtual sequences (nq queries' heads each).
static void prefill_layout(const pkv_pool* p, int B, int n_q, int Hq, int max_blocks, size_t* bt_off, size_t* ctx_off,
                           size_t* dec_off, size_t* total) {
  const int nq = prefill_nq(p, n_q, Hq);
  const size_t nv = (size_t)B * (size_t)(n_q / nq);
  *bt_off = 0;
  *ctx_off = align_up(nv * (size_t)(max_blocks > 0 ? max_blocks : 1) * sizeof(int32_t), 256);
  *dec_off = *ctx_off + align_up(nv * sizeof(int32_t), 256);
  *total = *dec_off + workspace_bytes(p, (int)nv, Hq * nq);
}

pkv_status pkv_prefill_workspace_bytes(const pkv_pool* p, int B, int n_q, int Hq, int max_blocks, size_t* bytes) {
  if (!p || !bytes || B < 0 || n_q < 1 || Hq < 1 || max_blocks < 0 || (int64_t)B * n_q > 4096)
    return PKV_ERR_INVALID;
  if (p->cfg.format == PKV_FMT_LATENT) return PKV_ERR_FORMAT;
  size_t a, b, c;
  prefill_layout(p, B, n_q, Hq, max_blocks, &a, &b, &c, bytes);
  return PKV_OK;
}

pkv_status pkv_paged_prefill_attention(pkv_pool* p, int layer, int B, int n_q, int Hq, const void* q,
                                       const int32_t* bt, int max_blocks, const int32_t* ctx, int max_ctx,
                                       float scale, void* out, void* ws, size_t ws_bytes, void* stream) {
  (void)max_ctx;
  if (!p || layer < 0 || layer >= p->cfg.n_layers || B < 0 || n_q < 1 || Hq < 1 || max_blocks < 0 ||
      (int64_t)B * n_q > 4096)
    return PKV_ERR_INVALID;
  if (p->cfg.format == PKV_FMT_LATENT) return PKV_ERR_FORMAT;
  if (B == 0) return PKV_OK;
  if (Hq % p->cfg.n_kv_heads) return PKV_ERR_INVALID;
  const int G = Hq / p->cfg.n_kv_heads;
  if (!(G == 1 || G == 2 || G == 4 || G == 8)) return PKV_ERR_INVALID;
  if (!q || !bt || !ctx || !out || !ws || !std::isfinite(scale)) return PKV_ERR_INVALID;
  if (((uintptr_t)ws & 255u) != 0 || ((uintptr_t)q & 15u) != 0 || ((uintptr_t)out & 15u) != 0)
    return PKV_ERR_INVALID;
  const int nq = prefill_nq(p, n_q, Hq);
  const int Bv = B * (n_q / nq);
  size_t bt_off, ctx_off, dec_off, total;
  prefill_layout(p, B, n_q, Hq, max_blocks, &bt_off, &ctx_off, &dec_off, &total);
  if (ws_bytes < total) return PKV_ERR_INVALID;
  DecodePlan plan;
  if (!plan_decode(p->cfg.format, p->cfg.head_dim, G * nq, p->cfg.n_kv_heads, Bv, p->cfg.group_size, &plan) ||
      plan.smem_bytes > p->smem_optin)
    return PKV_ERR_INVALID;
  // q [B, n_q, Hq, D] and out [B, n_q, Hq, D] are [Bv, nq * Hq, D]: virtual sequence v
  // holds queries nq * (v mod (n_q / nq)) .. + nq - 1 of its sequence.  The K/V blocks
  // of a sequence are read by all of its virtual sequences: normal L2 priority.  A
  // chunk of several queries that fits one tile (nq = n_q > 1) is its own virtual
  // sequence: the caller's block table and context lengths serve as they are (the
  // kernels treat a length below nq as a context error and the sequence as empty, as
  // the expansion does).
  const int32_t* bt_v = bt;
  const int32_t* ctx_v = ctx;
  if (nq != n_q || nq == 1) {
    int32_t* bt2 = (int32_t*)((uint8_t*)ws + bt_off);
    int32_t* ctx2 = (int32_t*)((uint8_t*)ws + ctx_off);
    PKV_CUDA(launch_expand_prefill(B, n_q, nq, max_blocks, bt, ctx, bt2, ctx2, p->err_dev, (cudaStream_t)stream),
             "prefill expansion launch");
    bt_v = bt2;
    ctx_v = ctx2;
  }
  return decode_impl(p, layer, Bv, Hq * nq, q, bt_v, max_blocks, ctx_v, scale, out, (uint8_t*)ws + dec_off,
                     ws_bytes - dec_off, stream, 1, nq);
}

// ---------------------------------------------------------------------------
// Latent pools
// ---------------------------------------------------------------------------

// What every latent entry point checks first: a latent pool, the layer, and the
// pool's device as the current one (the kernels launch there).
static pkv_status latent_check(const pkv_pool* p, int layer) {
  if (!p || layer < 0 || layer >= p->cfg.n_layers) return PKV_ERR_INVALID;
  if (p->cfg.format != PKV_FMT_LATENT) return PKV_ERR_FORMAT;
  int dev = -1;
  PKV_CUDA(cudaGetDevice(&dev), "cudaGetDevice");
  if (dev != p->device) return PKV_ERR_INVALID;
  return PKV_OK;
}

// scale log2(e), as the kernels take it; false where fp32 does not hold it.
static bool latent_scale(float scale, float* out) {
  const double s = (double)scale * 1.4426950408889634;
  if (!(std::fabs(s) <= (double)FLT_MAX)) return false;
  *out = (float)s;
  return true;
}

static bool misaligned(const void* ptr, uintptr_t a) { return ((uintptr_t)ptr & (a - 1)) != 0; }

// Whether output rows of `width` values, Hq a token, do not overlap one another: a token's
// heads lie within its span, or a head's tokens within the head's.
static bool rows_disjoint(int n, int Hq, int64_t token_stride, int64_t head_stride, int width) {
  const int64_t t = n > 1 ? token_stride : 0, h = Hq > 1 ? head_stride : 0;
  if ((n > 1 && t < width) || (Hq > 1 && h < width)) return false;
  if (n > 1 && Hq > 1) {
    // (n - 1) t + width <= h, without the product's overflow
    const bool tokens_inside = t <= (h - width) / (n - 1), heads_inside = h <= (t - width) / (Hq - 1);
    if (!tokens_inside && !heads_inside) return false;
  }
  return true;
}

pkv_status pkv_write_latent(pkv_pool* p, int layer, int n, const int32_t* rows, const int32_t* slots, const void* kv,
                            int64_t kv_stride, const int32_t* positions, const float* cos_sin, int n_positions,
                            const void* norm_weight, float eps, int interleaved, int Hq, const void* q_rope,
                            int64_t q_token_stride, int64_t q_head_stride, void* q_out, int64_t out_token_stride,
                            int64_t out_head_stride, void* stream) {
  pkv_status st = latent_check(p, layer);
  if (st != PKV_OK) return st;
  const int R = p->cfg.head_dim;
  if (n < 0 || Hq < 0 || Hq > kLatentMaxHeads || n_positions < 0) return PKV_ERR_INVALID;
  if ((int64_t)n * latent_write_units(Hq) >= (int64_t)1 << 31) return PKV_ERR_INVALID;
  if (n == 0) return PKV_OK;
  if (!rows || !slots || !kv || !positions || !cos_sin) return PKV_ERR_INVALID;
  if (misaligned(kv, 16) || misaligned(cos_sin, 16) || misaligned(norm_weight, 16) || misaligned(q_rope, 16) ||
      misaligned(q_out, 16))
    return PKV_ERR_INVALID;
  if (kv_stride < R + kRope || kv_stride % 8) return PKV_ERR_INVALID;
  if (norm_weight && !(std::isfinite(eps) && eps >= 0.f)) return PKV_ERR_INVALID;
  if (Hq > 0) {
    if (!q_rope || !q_out) return PKV_ERR_INVALID;
    for (int64_t x : {q_token_stride, q_head_stride, out_token_stride, out_head_stride})
      if (x < 0 || x % 8) return PKV_ERR_INVALID;
    if (!rows_disjoint(n, Hq, out_token_stride, out_head_stride, kRope)) return PKV_ERR_INVALID;
    const int64_t t = n > 1 ? out_token_stride : 0, h = Hq > 1 ? out_head_stride : 0;
    // in place, a row's output is its own input
    if (q_out == q_rope && ((n > 1 && t != q_token_stride) || (Hq > 1 && h != q_head_stride))) return PKV_ERR_INVALID;
  }
  LatentWriteArgs a;
  a.lv = layer_view(p, layer);
  a.R = R;
  a.n = n;
  a.rows = rows;
  a.slots = slots;
  a.kv = (const uint16_t*)kv;
  a.kv_stride = kv_stride;
  a.positions = positions;
  a.cos_sin = cos_sin;
  a.n_pos = n_positions;
  a.weight = (const uint16_t*)norm_weight;
  a.eps = eps;
  a.interleaved = interleaved != 0;
  a.Hq = Hq;
  a.q = (const uint16_t*)q_rope;
  a.q_tok = q_token_stride;
  a.q_head = q_head_stride;
  a.qo = (uint16_t*)q_out;
  a.o_tok = out_token_stride;
  a.o_head = out_head_stride;
  a.per_token = 0;
  a.stream = (cudaStream_t)stream;
  PKV_CUDA(launch_latent_write(a), "write_latent launch");
  p->last_stream = a.stream;
  return PKV_OK;
}

static bool latent_sizes_ok(int B, int n_q, int Hq) {
  return B >= 0 && B <= kLatentMaxBatch && n_q >= 1 && Hq >= 1 && Hq <= kLatentMaxHeads &&
         (int64_t)B * n_q * Hq <= kLatentMaxRows;
}

pkv_status pkv_latent_workspace_bytes(const pkv_pool* p, int B, int n_q, int Hq, size_t* bytes) {
  if (!p || !bytes || !latent_sizes_ok(B, n_q, Hq)) return PKV_ERR_INVALID;
  if (p->cfg.format != PKV_FMT_LATENT) return PKV_ERR_FORMAT;
  *bytes = latent_attn_workspace(p->cfg.head_dim, B, n_q, Hq, decode_grid(p));
  return PKV_OK;
}

pkv_status pkv_paged_latent_attention(pkv_pool* p, int layer, int B, int n_q, int Hq, const void* q_latent,
                                      int64_t q_latent_stride, const void* q_rope, int64_t q_rope_stride,
                                      const int32_t* bt, int max_blocks, const int32_t* ctx, int max_ctx, float scale,
                                      void* out, void* ws, size_t ws_bytes, void* stream) {
  (void)max_ctx;
  pkv_status st = latent_check(p, layer);
  if (st != PKV_OK) return st;
  const int R = p->cfg.head_dim;
  float scale_log2;
  if (!latent_sizes_ok(B, n_q, Hq) || max_blocks < 0 || max_blocks > kLatentMaxBlocks ||
      !latent_scale(scale, &scale_log2))
    return PKV_ERR_INVALID;
  if (B == 0) return PKV_OK;
  if (!q_latent || !q_rope || (!bt && max_blocks > 0) || !ctx || !out || !ws) return PKV_ERR_INVALID;
  if (q_latent_stride < R || q_latent_stride % 8 || q_rope_stride < kRope || q_rope_stride % 8) return PKV_ERR_INVALID;
  if (misaligned(q_latent, 16) || misaligned(q_rope, 16) || misaligned(out, 16) || misaligned(ws, 256))
    return PKV_ERR_INVALID;
  LatentAttnArgs a;
  a.ctas = decode_grid(p);
  a.device = p->device;
  if (ws_bytes < latent_attn_workspace(R, B, n_q, Hq, a.ctas)) return PKV_ERR_INVALID;
  a.lv = layer_view(p, layer);
  a.R = R;
  a.B = B;
  a.n_q = n_q;
  a.Hq = Hq;
  a.max_blocks = max_blocks;
  a.ql = (const uint16_t*)q_latent;
  a.ql_stride = q_latent_stride;
  a.qr = (const uint16_t*)q_rope;
  a.qr_stride = q_rope_stride;
  a.bt = bt;
  a.ctx = ctx;
  a.scale_log2 = scale_log2;
  a.out = (uint16_t*)out;
  a.ws = ws;
  a.stream = (cudaStream_t)stream;
  PKV_CUDA(launch_latent_attn(a), "paged_latent_attention launch");
  p->last_stream = a.stream;
  return PKV_OK;
}

// The bound on context lengths that the expanded form's workspace is sized by.
static int latent_prefill_ctx(int max_blocks, int max_ctx) {
  const int64_t all = (int64_t)max_blocks * kBlockTokens;
  return (int)(max_ctx > 0 && max_ctx < all ? max_ctx : all);
}

// The expanded rows (per sequence and head) are numbered in 32 bits.
static bool latent_prefill_fits(int B, int Hq, int max_ctx) {
  return (int64_t)B * Hq * ((int64_t)max_ctx + 128) < (int64_t)1 << 31;
}

pkv_status pkv_latent_prefill_workspace_bytes(const pkv_pool* p, int B, int n_q, int Hq, int max_blocks, int max_ctx,
                                              size_t* bytes) {
  if (!p || !bytes || !latent_sizes_ok(B, n_q, Hq) || max_blocks < 0 || max_blocks > kLatentMaxBlocks || max_ctx < 0)
    return PKV_ERR_INVALID;
  if (p->cfg.format != PKV_FMT_LATENT) return PKV_ERR_FORMAT;
  if (!latent_prefill_fits(B, Hq, latent_prefill_ctx(max_blocks, max_ctx))) return PKV_ERR_INVALID;
  *bytes = latent_prefill_workspace(B, n_q, Hq, latent_prefill_ctx(max_blocks, max_ctx), decode_grid(p));
  return PKV_OK;
}

pkv_status pkv_latent_prefill_attention(pkv_pool* p, int layer, int B, int n_q, int Hq, const void* q, const void* w_k,
                                        const void* w_v, const int32_t* bt, int max_blocks, const int32_t* ctx,
                                        int max_ctx, float scale, void* out, void* ws, size_t ws_bytes, void* stream) {
  pkv_status st = latent_check(p, layer);
  if (st != PKV_OK) return st;
  float scale_log2;
  if (!latent_sizes_ok(B, n_q, Hq) || max_blocks < 0 || max_blocks > kLatentMaxBlocks || max_ctx < 0 ||
      !latent_scale(scale, &scale_log2))
    return PKV_ERR_INVALID;
  if (B == 0) return PKV_OK;
  if (!q || !w_k || !w_v || (!bt && max_blocks > 0) || !ctx || !out || !ws) return PKV_ERR_INVALID;
  if (misaligned(q, 16) || misaligned(w_k, 16) || misaligned(w_v, 16) || misaligned(out, 16) || misaligned(ws, 256))
    return PKV_ERR_INVALID;
  LatentPrefillArgs a;
  a.max_ctx = latent_prefill_ctx(max_blocks, max_ctx);
  if (!latent_prefill_fits(B, Hq, a.max_ctx)) return PKV_ERR_INVALID;
  a.ctas = decode_grid(p);
  if (ws_bytes < latent_prefill_workspace(B, n_q, Hq, a.max_ctx, a.ctas)) return PKV_ERR_INVALID;
  a.lv = layer_view(p, layer);
  a.R = p->cfg.head_dim;
  a.B = B;
  a.n_q = n_q;
  a.Hq = Hq;
  a.max_blocks = max_blocks;
  a.q = (const uint16_t*)q;
  a.wk = (const uint16_t*)w_k;
  a.wv = (const uint16_t*)w_v;
  a.bt = bt;
  a.ctx = ctx;
  a.scale_log2 = scale_log2;
  a.out = (uint16_t*)out;
  a.ws = ws;
  a.device = p->device;
  a.stream = (cudaStream_t)stream;
  PKV_CUDA(launch_latent_prefill(a), "latent_prefill_attention launch");
  p->last_stream = a.stream;
  return PKV_OK;
}

// ---------------------------------------------------------------------------
// Drafted tokens on the per-head pools
// ---------------------------------------------------------------------------

// What the entry points of this part check first: the layer, and the pool's device as the
// current one (the kernels launch there).
static pkv_status draft_check(const pkv_pool* p, int layer) {
  if (!p || layer < 0 || layer >= p->cfg.n_layers) return PKV_ERR_INVALID;
  if (p->cfg.format == PKV_FMT_LATENT) return PKV_ERR_FORMAT;
  int dev = -1;
  PKV_CUDA(cudaGetDevice(&dev), "cudaGetDevice");
  if (dev != p->device) return PKV_ERR_INVALID;
  return PKV_OK;
}

pkv_status pkv_write_rotated(pkv_pool* p, int layer, int n, const int32_t* rows, const int32_t* slots, const void* k,
                             int64_t k_token_stride, int64_t k_head_stride, const void* v, int64_t v_token_stride,
                             int64_t v_head_stride, const int32_t* positions, const float* cos_sin, int n_positions,
                             int rotary_dim, int interleaved, const void* k_norm, const void* q_norm, float eps, int Hq,
                             const void* q, int64_t q_token_stride, int64_t q_head_stride, void* q_out,
                             int64_t out_token_stride, int64_t out_head_stride, void* stream) {
  pkv_status st = draft_check(p, layer);
  if (st != PKV_OK) return st;
  const int D = p->cfg.head_dim;
  if (n < 0 || Hq < 0 || Hq > kDraftMaxHeads || n_positions < 0) return PKV_ERR_INVALID;
  if ((int64_t)n * rotated_write_units(p->cfg.n_kv_heads, Hq) >= (int64_t)1 << 31) return PKV_ERR_INVALID;
  if (rotary_dim < 32 || rotary_dim > D || rotary_dim % 32) return PKV_ERR_INVALID;
  if (n == 0) return PKV_OK;
  if (!rows || !slots || !k || !v || !positions || !cos_sin) return PKV_ERR_INVALID;
  for (const void* x : {k, v, (const void*)cos_sin, k_norm, q_norm, q, (const void*)q_out})
    if (misaligned(x, 16)) return PKV_ERR_INVALID;
  for (int64_t x : {k_token_stride, k_head_stride, v_token_stride, v_head_stride})
    if (x < 0 || x % 8) return PKV_ERR_INVALID;
  if ((k_norm || q_norm) && !(std::isfinite(eps) && eps >= 0.f)) return PKV_ERR_INVALID;
  if (Hq > 0) {
    if (!q || !q_out) return PKV_ERR_INVALID;
    for (int64_t x : {q_token_stride, q_head_stride, out_token_stride, out_head_stride})
      if (x < 0 || x % 8) return PKV_ERR_INVALID;
    if (!rows_disjoint(n, Hq, out_token_stride, out_head_stride, D)) return PKV_ERR_INVALID;
    // in place, a row's output is its own input
    if (q_out == q && ((n > 1 && out_token_stride != q_token_stride) || (Hq > 1 && out_head_stride != q_head_stride)))
      return PKV_ERR_INVALID;
  }
  RotatedWriteArgs a;
  a.lv = layer_view(p, layer);
  a.fmt = p->cfg.format;
  a.D = D;
  a.group = p->cfg.group_size;
  a.n = n;
  a.rows = rows;
  a.slots = slots;
  a.k = (const uint16_t*)k;
  a.k_tok = k_token_stride;
  a.k_head = k_head_stride;
  a.v = (const uint16_t*)v;
  a.v_tok = v_token_stride;
  a.v_head = v_head_stride;
  a.positions = positions;
  a.cos_sin = cos_sin;
  a.n_pos = n_positions;
  a.rot = rotary_dim;
  a.interleaved = interleaved != 0;
  a.k_norm = (const uint16_t*)k_norm;
  a.q_norm = Hq > 0 ? (const uint16_t*)q_norm : nullptr;
  a.eps = eps;
  a.Hq = Hq;
  a.q = (const uint16_t*)q;
  a.q_tok = q_token_stride;
  a.q_head = q_head_stride;
  a.qo = (uint16_t*)q_out;
  a.o_tok = out_token_stride;
  a.o_head = out_head_stride;
  a.signs = p->signs_dev;
  a.stream = (cudaStream_t)stream;
  PKV_CUDA(launch_rotated_write(a), "write_rotated launch");
  p->last_stream = a.stream;
  return PKV_OK;
}

static bool tree_sizes_ok(const pkv_pool* p, int B, int n_q, int Hq) {
  return B >= 0 && B <= kDraftMaxBatch && n_q >= 1 && n_q <= kDraftMaxQueries && Hq >= 1 && Hq <= kDraftMaxHeads &&
         Hq % p->cfg.n_kv_heads == 0 && (int64_t)B * n_q * Hq <= kDraftMaxRows;
}

pkv_status pkv_tree_workspace_bytes(const pkv_pool* p, int B, int n_q, int Hq, size_t* bytes) {
  if (!p || !bytes) return PKV_ERR_INVALID;
  if (p->cfg.format == PKV_FMT_LATENT) return PKV_ERR_FORMAT;
  if (!tree_sizes_ok(p, B, n_q, Hq)) return PKV_ERR_INVALID;
  *bytes = tree_attn_workspace(p->cfg.head_dim, p->cfg.n_kv_heads, B, n_q, Hq, decode_grid(p));
  return PKV_OK;
}

pkv_status pkv_paged_tree_attention(pkv_pool* p, int layer, int B, int n_q, int Hq, const void* q, const uint32_t* mask,
                                    int64_t mask_stride, const int32_t* bt, int max_blocks, const int32_t* ctx,
                                    int max_ctx, float scale, void* out, void* ws, size_t ws_bytes, void* stream) {
  (void)max_ctx;
  pkv_status st = draft_check(p, layer);
  if (st != PKV_OK) return st;
  float scale_log2;
  if (!tree_sizes_ok(p, B, n_q, Hq) || max_blocks < 0 || max_blocks > kDraftMaxBlocks || !latent_scale(scale, &scale_log2))
    return PKV_ERR_INVALID;
  if (B == 0) return PKV_OK;
  if (!q || !mask || (!bt && max_blocks > 0) || !ctx || !out || !ws) return PKV_ERR_INVALID;
  if (mask_stride != 0 && mask_stride < (int64_t)n_q * ((n_q + 31) / 32)) return PKV_ERR_INVALID;
  if (misaligned(q, 16) || misaligned(out, 16) || misaligned(mask, 4) || misaligned(ws, 256)) return PKV_ERR_INVALID;
  TreeAttnArgs a;
  a.fmt = p->cfg.format;
  a.D = p->cfg.head_dim;
  a.group = p->cfg.group_size;
  a.ctas = decode_grid(p);
  if (ws_bytes < tree_attn_workspace(a.D, p->cfg.n_kv_heads, B, n_q, Hq, a.ctas)) return PKV_ERR_INVALID;
  a.lv = layer_view(p, layer);
  a.B = B;
  a.n_q = n_q;
  a.Hq = Hq;
  a.max_blocks = max_blocks;
  a.q = (const uint16_t*)q;
  a.mask = mask;
  a.mask_stride = mask_stride;
  a.bt = bt;
  a.ctx = ctx;
  a.scale_log2 = scale_log2;
  a.signs = p->signs_dev;
  a.out = (uint16_t*)out;
  a.ws = ws;
  a.device = p->device;
  a.stream = (cudaStream_t)stream;
  PKV_CUDA(launch_tree_attn(a), "paged_tree_attention launch");
  p->last_stream = a.stream;
  return PKV_OK;
}

pkv_status pkv_accept_drafts(pkv_pool* p, int B, int n_q, int max_path, const int32_t* path, const int32_t* path_lens,
                             const int32_t* bt, int max_blocks, const int32_t* ctx, int32_t* new_lens, void* stream) {
  if (!p || B < 0 || B > kDraftMaxBatch || n_q < 1 || n_q > kDraftMaxQueries || max_path < 0 || max_blocks < 0 ||
      max_blocks > kDraftMaxBlocks)
    return PKV_ERR_INVALID;
  const int64_t ctas = (int64_t)B * p->cfg.n_layers * p->n_kinds;
  if (ctas >= (int64_t)1 << 31) return PKV_ERR_INVALID;
  int dev = -1;
  PKV_CUDA(cudaGetDevice(&dev), "cudaGetDevice");
  if (dev != p->device) return PKV_ERR_INVALID;
  if (B == 0) return PKV_OK;
  if ((!path && max_path > 0) || !path_lens || (!bt && max_blocks > 0) || !ctx) return PKV_ERR_INVALID;
  // the lengths are read while the new ones are written
  if (new_lens && new_lens < ctx + B && ctx < new_lens + B) return PKV_ERR_INVALID;
  if (new_lens && new_lens < path_lens + B && path_lens < new_lens + B) return PKV_ERR_INVALID;
  AcceptArgs a;
  a.table = p->table_dev;
  a.n_layers = p->cfg.n_layers;
  a.n_kinds = p->n_kinds;
  for (int k = 0; k < 4; ++k) a.token_bytes[k] = p->row_bytes[k] * p->cfg.n_kv_heads;
  a.slab_blocks = p->cfg.slab_blocks;
  a.rows_capacity = (int64_t)p->groups.size() * p->cfg.slab_blocks;
  a.B = B;
  a.n_q = n_q;
  a.max_path = max_path;
  a.max_blocks = max_blocks;
  a.path = path;
  a.path_lens = path_lens;
  a.bt = bt;
  a.ctx = ctx;
  a.new_lens = new_lens;
  a.err = p->err_dev;
  a.stream = (cudaStream_t)stream;
  PKV_CUDA(launch_accept(a), "accept_drafts launch");
  p->last_stream = a.stream;
  return PKV_OK;
}

// What every price has in common: the storage growth and the pages of the new blocks.
static pkv_status price_storage(const pkv_pool* p, const pkv_request* r, pkv_price* out) {
  const int64_t free_rows = (int64_t)p->free_rows.size();
  const int64_t deficit = r->new_blocks > free_rows ? r->new_blocks - free_rows : 0;
  const int64_t slabs = (deficit + p->cfg.slab_blocks - 1) / p->cfg.slab_blocks;
  if ((int64_t)p->groups.size() + slabs > p->cfg.max_slabs) return PKV_ERR_RANGE;
  int64_t block_bytes = 0;  // one block of one layer, every stored tensor
  for (int k = 0; k < p->n_kinds; ++k) block_bytes += p->row_bytes[k] * kBlockTokens * p->cfg.n_kv_heads;
  memset(out, 0, sizeof *out);
  out->slabs_to_append = (int32_t)slabs;
  out->free_rows = free_rows;
  out->storage_bytes = (uint64_t)slabs * (uint64_t)p->group_bytes;
  out->page_bytes = (uint64_t)r->new_blocks * (uint64_t)block_bytes * (uint64_t)p->cfg.n_layers;
  return PKV_OK;
}

pkv_status pkv_price_request(const pkv_pool* p, const pkv_request* r, pkv_price* out) {
  if (!p || !r || !out || r->new_blocks < 0 || r->B < 1 || r->Hq < 1 || r->n_q < 1 || r->max_blocks < 0)
    return PKV_ERR_INVALID;
  if (r->Hq % p->cfg.n_kv_heads) return PKV_ERR_INVALID;
  const bool latent = p->cfg.format == PKV_FMT_LATENT;
  if (!latent && r->n_q > 1 && (int64_t)r->B * r->n_q > 4096) return PKV_ERR_INVALID;
  if (latent && (!latent_sizes_ok(r->B, r->n_q, r->Hq) || r->max_blocks > kLatentMaxBlocks)) return PKV_ERR_INVALID;
  const pkv_status st = price_storage(p, r, out);
  if (st != PKV_OK) return st;
  const uint64_t q_out = 2ull * (uint64_t)p->cfg.head_dim + (latent ? kRope : 0);  // values of a q and an output row
  out->fixed_bytes = (uint64_t)r->max_blocks * 4u + 4u + (uint64_t)r->n_q * (uint64_t)r->Hq * q_out * 2u;
  if (latent) {
    out->workspace_bytes = latent_attn_workspace(p->cfg.head_dim, r->B, r->n_q, r->Hq, decode_grid(p));
  } else if (r->n_q == 1) {
    out->workspace_bytes = workspace_bytes(p, r->B, r->Hq);
  } else {
    size_t a, b, c, t;
    prefill_layout(p, r->B, r->n_q, r->Hq, r->max_blocks, &a, &b, &c, &t);
    out->workspace_bytes = t;
  }
  return PKV_OK;
}

pkv_status pkv_price_latent_prefill(const pkv_pool* p, const pkv_request* r, int max_ctx, pkv_price* out) {
  if (!p || !r || !out || r->new_blocks < 0 || r->B < 1) return PKV_ERR_INVALID;
  size_t ws = 0;
  pkv_status st = pkv_latent_prefill_workspace_bytes(p, r->B, r->n_q, r->Hq, r->max_blocks, max_ctx, &ws);
  if (st == PKV_OK) st = price_storage(p, r, out);
  if (st != PKV_OK) return st;
  out->fixed_bytes = (uint64_t)r->max_blocks * 4u + 4u +
                     (uint64_t)r->n_q * (uint64_t)r->Hq * (2ull * kLatentHead + kRope) * 2u;
  out->workspace_bytes = ws;
  return PKV_OK;
}

pkv_status pkv_pool_stats(const pkv_pool* p, pkv_stats* out) {
  if (!p || !out) return PKV_ERR_INVALID;
  memset(out, 0, sizeof *out);
  out->n_slabs = (int32_t)p->groups.size();
  out->n_kinds = p->n_kinds;
  out->slab_append_events = p->append_events;
  out->rows_capacity = (int64_t)p->groups.size() * p->cfg.slab_blocks;
  out->rows_in_use = p->rows_in_use;
  out->bytes_reserved = (int64_t)p->groups.size() * p->layer_bytes * p->cfg.n_layers;  // slab data only
  for (int k = 0; k < 4; ++k) out->row_bytes[k] = p->row_bytes[k];
  return PKV_OK;
}

pkv_status pkv_slab_address(const pkv_pool* p, int layer, int kind, int slab, void** addr) {
  if (!p || !addr) return PKV_ERR_INVALID;
  if (layer < 0 || layer >= p->cfg.n_layers || kind < 0 || kind >= p->n_kinds || slab < 0 ||
      slab >= (int)p->groups.size())
    return PKV_ERR_RANGE;
  *addr = p->table_host[((size_t)slab * p->cfg.n_layers + layer) * p->n_kinds + kind];
  return PKV_OK;
}

pkv_status pkv_pool_check_identity(const pkv_pool* p, const pkv_pool_config* c) {
  if (!p || !c) return PKV_ERR_INVALID;
  const pkv_pool_config& a = p->cfg;
  bool same = a.format == c->format && a.head_dim == c->head_dim && a.n_kv_heads == c->n_kv_heads &&
              a.block_size == c->block_size && a.slab_blocks == c->slab_blocks;
  if (a.format != PKV_FMT_BF16) same = same && a.group_size == c->group_size;
  if (a.format != PKV_FMT_BF16 && a.format != PKV_FMT_LATENT) same = same && a.hadamard_seed == c->hadamard_seed;
  return same ? PKV_OK : PKV_ERR_FORMAT;
}

pkv_status pkv_pool_check_errors(pkv_pool* p, void* stream, int32_t* word_out) {
  if (!p) return PKV_ERR_INVALID;
  cudaStream_t s = (cudaStream_t)stream;
  int32_t w = 0;
  PKV_CUDA(cudaMemcpyAsync(&w, p->err_dev, sizeof w, cudaMemcpyDeviceToHost, s), "read error word");
  PKV_CUDA(cudaStreamSynchronize(s), "cudaStreamSynchronize");
  if (word_out) *word_out = w;
  if (w) {
    PKV_CUDA(cudaMemsetAsync(p->err_dev, 0, sizeof w, s), "clear error word");
    PKV_CUDA(cudaStreamSynchronize(s), "cudaStreamSynchronize");
    return PKV_ERR_DEVICE;
  }
  return PKV_OK;
}

}  // extern "C"
