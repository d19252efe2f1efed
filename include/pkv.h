/*
 * pkv.h — C ABI of the GB300 paged-KV decode-attention library (libpkv.so).
 *
 * A pool stores the K/V cache of every layer in chunked slab storage: for each
 * layer and stored tensor, a vector of fixed-size slabs shaped
 *   [slab_blocks, block_size, n_kv_heads, row]
 * (row = head_dim bf16 values, or packed codes, or (scale, offset) pairs).  A
 * physical row (one block of block_size tokens) maps to slab = row / slab_blocks,
 * row_in_slab = row % slab_blocks.  Growth appends fresh zeroed slabs and never
 * copies or frees an existing one.
 *   [mlxcel issue #235, "chunked slab storage for the paged pool", Proposed
 *    solution: bullets 1-3]
 *
 * Stored formats: native bf16, or packed K4/V4, K8/V4, K8/V8 with token-local
 * affine groups of group_size values and an FP32 (scale, offset) pair per group;
 * K (and Q at attention time) is expressed in a fixed signed Hadamard basis.
 *   [mlx-swift-lm PR #142, "packed paged KV formats with bounded workspace
 *    admission", Summary]
 *
 * Conventions for every call
 *  - All pointers named *_dev are device pointers; *_host are host pointers.
 *    Device buffers passed in are owned by the caller and must stay valid until
 *    the work enqueued on `stream` has finished.
 *  - `stream` is a cudaStream_t passed as void*; NULL means the legacy default
 *    stream.  Every call that touches device memory is asynchronous on that
 *    stream unless stated otherwise; none synchronises the device except
 *    pkv_pool_check_errors and pkv_pool_destroy.
 *  - Host-checkable errors (NULL pointers, sizes out of range, a layer index out
 *    of range, workspace too small, allocation failure) are returned
 *    synchronously, before any state changes or work is enqueued.
 *  - Device-detected range errors (a block-table row beyond the pool's rows, a
 *    context length beyond max_blocks*block_size, a slot beyond block_size) set
 *    the pool's device error word; the offending block/token is skipped (the
 *    result is then undefined but no memory outside the pool is touched).  Read
 *    and clear it with pkv_pool_check_errors.
 *  - A pool is not thread-safe; callers serialise calls on one pool.
 */
#ifndef PKV_H_
#define PKV_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef struct pkv_pool pkv_pool; /* opaque; owns slabs, pointer tables, row allocator */

typedef enum {
  PKV_FMT_BF16 = 0, /* native: K and V rows are head_dim bf16 values            */
  PKV_FMT_K4V4 = 1, /* K 4-bit codes (Hadamard basis), V 4-bit codes           */
  PKV_FMT_K8V4 = 2, /* K 8-bit codes (Hadamard basis), V 4-bit codes           */
  PKV_FMT_K8V8 = 3, /* K 8-bit codes (Hadamard basis), V 8-bit codes           */
  PKV_FMT_LATENT = 4 /* one bf16 row a token for every head: a latent vector of
                      * head_dim values, then a position key of group_size values */
} pkv_format;

typedef enum {
  PKV_OK = 0,
  PKV_ERR_INVALID = -1, /* bad argument (NULL, size, layer, alignment)          */
  PKV_ERR_OOM = -2,     /* the allocator returned NULL; the pool is unchanged    */
  PKV_ERR_CUDA = -3,    /* a CUDA runtime call failed (message: pkv_last_error)  */
  PKV_ERR_FORMAT = -4,  /* storage identity does not match the request           */
  PKV_ERR_RANGE = -5,   /* a host-visible index is out of range                  */
  PKV_ERR_DEVICE = -6   /* the device error word was set (pkv_pool_check_errors) */
} pkv_status;

/* Tensor kinds stored per layer. */
enum { PKV_KIND_K = 0, PKV_KIND_V = 1, PKV_KIND_KMETA = 2, PKV_KIND_VMETA = 3 };

typedef struct {
  int32_t n_layers;      /* >= 1                                                */
  int32_t n_kv_heads;    /* 1..8 (one decode consumer warp per kv head); latent: 1 */
  int32_t head_dim;      /* 64, 128 or 256; latent: the latent vector's width, 256 or 512 */
  int32_t block_size;    /* tokens per block; must be 32                        */
  int32_t slab_blocks;   /* blocks per slab (POOL_SLAB_BLOCKS); 1..4096, 32 is the default */
  int32_t group_size;    /* values per affine group (ignored for bf16): 32, or 64 for K4/V4 with
                          * head_dim 128 or 256 (one FP32 scale/offset pair per 64 values: five
                          * bits per value, 3.2x against bf16)
                          *   [mlx-swift-lm #142, Summary: K4/V4 at five bits per value,
                          *    metadata included]; latent: the position key's width, 64 */
  int32_t format;        /* pkv_format                                          */
  int32_t max_slabs;     /* capacity of the slab pointer table (>= 1)           */
  uint64_t hadamard_seed;/* signs s_i = -1 iff top bit of splitmix64(seed + i)  */
} pkv_pool_config;

/* Stream-ordered allocator used for slabs.  alloc returns NULL on failure.  With
 * a NULL allocator the pool uses cudaMallocAsync / cudaFreeAsync on the stream. */
typedef struct {
  void* (*alloc)(void* ctx, size_t bytes, void* stream);
  void (*release)(void* ctx, void* ptr, void* stream);
  void* ctx;
} pkv_allocator;

typedef struct {
  int32_t n_slabs;            /* slabs per (layer, tensor) currently held          */
  int32_t n_kinds;            /* 2 (bf16), 4 (packed: K, V, K meta, V meta) or 1 (latent) */
  int64_t slab_append_events; /* slabs appended since create (never a copy)        */
  int64_t rows_capacity;      /* n_slabs * slab_blocks                             */
  int64_t rows_in_use;        /* rows with a nonzero reference count               */
  int64_t bytes_reserved;     /* sum over every slab of every layer and tensor     */
  int64_t row_bytes[4];       /* bytes of one (token, head) row per tensor kind    */
} pkv_stats;

/* Create a pool with no slabs on the current device: per layer and stored tensor an
 * empty vector of slabs, the pointer table for up to max_slabs of them, the row
 * allocator and the device error word.  The allocator struct is copied.  *out
 * receives the pool (owned by the caller until pkv_pool_destroy).  Errors:
 * PKV_ERR_INVALID for an unsupported configuration (n_kv_heads outside 1..8,
 * head_dim not 64/128/256, block_size not 32, group_size not allowed for the
 * format; latent: n_kv_heads not 1, head_dim not 256/512, group_size not 64),
 * PKV_ERR_CUDA if the device cannot be used.  Synchronous.
 *   [mlxcel #235, Proposed solution, bullet 1: the single pool tensor of a layer
 *    becomes a vector of fixed-size slabs] */
pkv_status pkv_pool_create(const pkv_pool_config* cfg, const pkv_allocator* alloc, void* stream,
                           pkv_pool** out);

/* Wait for the device, then release every slab (through the pool's allocator) and
 * the pool itself.  NULL is ignored.  Slabs are freed only here, never while the
 * pool lives.
 *   [mlxcel #235, Proposed solution, bullet 2: growth never frees a slab] */
void pkv_pool_destroy(pkv_pool* pool);

/* Append n_slabs fresh zeroed slabs to every layer and tensor, in one step
 * (presize_for_span).  Existing slabs are neither copied nor freed; their base
 * addresses stay valid.  All-or-nothing: on PKV_ERR_OOM the pool is unchanged.
 *   [mlxcel #235, Proposed solution, bullet 2] */
pkv_status pkv_append_slab(pkv_pool* pool, int n_slabs, void* stream);

/* Take n rows from the free list (LIFO reuse of released rows, then rows of
 * appended slabs in ascending order), appending slabs when it is empty.  Each
 * returned row has reference count 1.  rows_host: n int32.
 *   [mlxcel #235, Behavioral invariants: block identities, reference counts and the
 *    reuse of freed rows remain row-level bookkeeping] */
pkv_status pkv_alloc_rows(pkv_pool* pool, int n, int32_t* rows_host, void* stream);

/* Reference counting of rows (host bookkeeping only).  retain requires a live
 * row; release returns a row to the free list when its count reaches 0.
 * PKV_ERR_RANGE for a row outside the pool or not live. */
pkv_status pkv_retain_row(pkv_pool* pool, int32_t row);
pkv_status pkv_release_row(pkv_pool* pool, int32_t row);

/* Maximal same-slab runs of a block-table row list, in logical order: writes the
 * starting index of each run to run_start_host (capacity n) and returns the number
 * of runs (0 for n <= 0, -1 for bad arguments).  Host only; no pool needed.
 *   [mlxcel #235, touch point 3, gather_visible] */
int pkv_slab_runs(const int32_t* rows_host, int n, int slab_blocks, int32_t* run_start_host);

/* write_block: token i of k/v goes to (rows_dev[i], slots_dev[i]) of `layer`.
 * k_bf16_dev, v_bf16_dev: [n_tokens, n_kv_heads, head_dim] bf16, row-major.
 * Packed formats quantise here, once: K is rotated into the Hadamard basis,
 * then every group of group_size values gets scale = (max-min)/(2^bits-1),
 * offset = min, code = round-half-even((x-min)/scale) (0 when scale is 0).
 *   [mlxcel #235, touch point 1; mlx-swift-lm #142, After flowchart: new K/V are
 *    quantised a single time, when written] */
pkv_status pkv_write_block(pkv_pool* pool, int layer, int n_tokens, const int32_t* rows_dev,
                           const int32_t* slots_dev, const void* k_bf16_dev, const void* v_bf16_dev,
                           void* stream);

/* copy_on_write_block: copy every byte of block src_rows_dev[i] to block
 * dst_rows_dev[i], for every layer and stored tensor.  Pairs must not overlap.
 *   [mlxcel #235, touch point 2] */
pkv_status pkv_copy_on_write_block(pkv_pool* pool, int n, const int32_t* src_rows_dev,
                                   const int32_t* dst_rows_dev, void* stream);

/* gather_visible: the visible context of one sequence (tokens [0, ctx_len)) as
 * dense arrays in logical order, equal to concatenating the maximal same-slab
 * runs of its block-table row.  bt_row_dev: ceil(ctx_len/block_size) rows.
 * Outputs (device): k_out, v_out [n_kv_heads, ctx_len, row_bytes(kind)];
 * kmeta_out, vmeta_out [n_kv_heads, ctx_len, head_dim/group_size, 2] float32,
 * which must be NULL for bf16 and non-NULL for packed (else PKV_ERR_FORMAT);
 * with ctx_len 0 nothing is written and every output may be NULL.  A latent pool has
 * one stored tensor: its rows go to k_out and the other outputs must be NULL.
 *   [mlxcel #235, touch point 3] */
pkv_status pkv_gather_visible(pkv_pool* pool, int layer, const int32_t* bt_row_dev, int ctx_len,
                              void* k_out_dev, void* v_out_dev, void* kmeta_out_dev,
                              void* vmeta_out_dev, void* stream);

/* Workspace bytes needed by pkv_paged_decode_attention for batches of up to B
 * sequences with Hq query heads (max_ctx is the caller's bound on any context
 * length; it is accepted for interface stability and does not change the size).
 * The workspace holds the split-K partials and per-sequence arrival counters; it
 * must be zero-filled once before its first use (the kernel leaves it reusable).
 * Host only; PKV_ERR_INVALID for a NULL pool or bytes, B < 0 or Hq < 1.
 *   [mlx-swift-lm #142, Summary: the workspace a step is guaranteed is priced on
 *    its own, apart from storage] */
pkv_status pkv_decode_workspace_bytes(const pkv_pool* pool, int B, int Hq, int max_ctx,
                                      size_t* bytes);

/* Batched single-token decode attention with GQA (query head h reads KV head
 * h / (Hq / n_kv_heads)), no mask, over tokens [0, ctx_lens[b]) of each
 * sequence:  out[b,h] = softmax(scale * q[b,h] . K_b^T) V_b.
 * For packed formats q is rotated into K's Hadamard basis inside the kernel and
 * K/V are dequantised in registers (no dequantised history is materialised).
 *   q_bf16_dev:      [B, Hq, head_dim] bf16 (un-rotated)
 *   block_table_dev: [B, max_blocks] int32 rows
 *   ctx_lens_dev:    [B] int32; 0 gives a zero output row
 *   max_ctx:         host bound on ctx_lens (used only to size the launch)
 *   out_bf16_dev:    [B, Hq, head_dim] bf16
 *   workspace_dev:   ws_bytes >= pkv_decode_workspace_bytes(B, Hq), zeroed once
 * Deterministic: bitwise identical results for identical inputs on one device.
 * Limits: 1 <= B <= 4096 (the batch's unit prefix is staged in shared memory);
 * n_kv_heads <= 8 (one consumer warp per kv head, fixed at pool creation);
 * G = Hq / n_kv_heads in {1, 2, 4, 8}.
 * Range: q and K of any magnitude whose logits (scale * q.k) are finite in fp32
 * (|q| below 2^100), and V of magnitudes within about 2^-50..2^40, are handled at
 * the same accuracy as values near 1: the packed kernels keep their 16-bit tensor
 * operands in range with powers of two that are removed exactly in fp32 (the
 * rotated q per tile row, in fp16; the probabilities times the V scales with a fixed
 * 2^64, in bf16).  Slots of a block past a sequence's context are never read into
 * the result, whatever bytes they hold.
 * B = 0 returns PKV_OK with no device work.  PKV_ERR_INVALID, before any work,
 * when B > 4096, Hq is not n_kv_heads x G with G in {1, 2, 4, 8}, scale is not
 * finite, the workspace is smaller than pkv_decode_workspace_bytes or not 256-byte
 * aligned, or q / out are not 16-byte aligned.
 *   [mlxcel issue #2171, "one KV storage abstraction": Proposed Solution
 *    (KVCache::attend -> paged_batch_decode_attention) and Implementation Notes,
 *    edge cases (single token, no mask); mlx-swift-lm #142, Summary: packed pages
 *    are attended to directly, with no expanded copy of the history] */
pkv_status pkv_paged_decode_attention(pkv_pool* pool, int layer, int B, int Hq,
                                      const void* q_bf16_dev, const int32_t* block_table_dev,
                                      int max_blocks, const int32_t* ctx_lens_dev, int max_ctx,
                                      float scale, void* out_bf16_dev, void* workspace_dev,
                                      size_t ws_bytes, void* stream);

/* Size of the fixed device scratch array used by pkv_paged_decode_attention_noalloc. */
#define PKV_STATIC_SCRATCH_BYTES (8u * 1024u * 1024u)

/* Decode attention without any device allocation by the caller or the library.
 * The source pages have no counterpart to this call.  It exists for callers that
 * cannot call cudaMalloc or borrow an allocator: for example a serving loop that
 * reserved all of its device memory at start-up and may not allocate during a
 * decode step, or a plugin whose host framework owns the device allocator.
 * Arguments and results are those of pkv_paged_decode_attention, minus the
 * workspace: the split-K partials and arrival counters live instead in a fixed
 * array of PKV_STATIC_SCRATCH_BYTES (8 MiB) compiled into the library, which every
 * GPU that loads the library holds until the process exits.
 *  - The first call on each device looks up that device's copy of the array
 *    (cudaGetSymbolAddress, with the device current); make that first call before
 *    any stream capture.
 *  - Each call clears the arrival counters on `stream` (a cudaMemsetAsync, not an
 *    allocation), then launches the same kernel as pkv_paged_decode_attention.
 *  - All calls on a device share the one array, which keeps the last call's
 *    contents: calls whose GPU work overlaps (different streams, or different
 *    pools) race on it and give undefined results; serialise them.
 *  - PKV_ERR_RANGE, with a message from pkv_last_error, when (B, Hq, head_dim)
 *    need more scratch than the array holds (pkv_decode_workspace_bytes tells). */
pkv_status pkv_paged_decode_attention_noalloc(pkv_pool* pool, int layer, int B, int Hq,
                                              const void* q_bf16_dev, const int32_t* block_table_dev,
                                              int max_blocks, const int32_t* ctx_lens_dev, int max_ctx,
                                              float scale, void* out_bf16_dev, void* stream);

/* Number of CTAs a decode launch uses (0 = one per SM, the default).  Changing it
 * changes the split-K partition (results agree to rounding) and the workspace
 * size, those of the latent calls included.  PKV_ERR_INVALID for n < 0.  Host only.
 * (A tuning and test knob; the pages have no counterpart.) */
pkv_status pkv_decode_set_ctas(pkv_pool* pool, int n_ctas);

/* Pool statistics (host bookkeeping; no device access): slab count, the
 * slab-append counter (one per appended slab; no slab is ever copied), row
 * capacity and rows in use, and bytes_reserved as the sum over every slab of every
 * layer and tensor.  PKV_ERR_INVALID for NULL arguments.
 *   [mlxcel #235, Proposed solution, bullet 2 (the growth counter counts slab
 *    appends) and touch point 5 (reserved bytes summed over slabs)] */
pkv_status pkv_pool_stats(const pkv_pool* pool, pkv_stats* out);

/* Device base address of slab `slab` of (layer, kind); PKV_ERR_RANGE if absent.
 * Host only.
 *   [mlxcel #235, touch point 4: per-slab base pointers] */
pkv_status pkv_slab_address(const pkv_pool* pool, int layer, int kind, int slab, void** addr);

/* A request's price for admission into a step: the three costs that an admission
 * policy weighs separately.  Host only; nothing is allocated or changed.
 *   in  new_blocks:  blocks (rows) the request needs that it does not share with a
 *                    sequence already in the pool (e.g. ceil(tokens / 32) minus the
 *                    blocks of a shared prefix); >= 0
 *   in  B, Hq, n_q:  the step it joins: sequences (the request included), query
 *                    heads, queries per sequence (1 for decode, > 1 for a chunked
 *                    prefill of n_q tokens)
 *   in  max_blocks:  block-table width of that step
 *   out slabs_to_append: slabs pkv_alloc_rows(new_blocks) would append now (0
 *                    while the free list holds enough rows), the same count
 *                    pkv_append_slab(n) takes to presize for the span
 *   out free_rows:   rows on the free list now
 *   out storage_bytes: growing storage: the bytes the allocator is asked for by
 *                    those appends (every layer and tensor of each slab, plus the
 *                    slab's 128-byte tensor maps)
 *   out page_bytes:  page cost: the stored bytes of the request's new blocks, every
 *                    layer and tensor (pkv_block_record_bytes x new_blocks); this is
 *                    space inside the pool's capacity, not a further allocation
 *   out fixed_bytes: fixed per-request cost of a step: its block-table row
 *                    (max_blocks int32), context length (int32), and q and output
 *                    rows (n_q x Hq x head_dim bf16 each)
 *   out workspace_bytes: the step's guaranteed workspace for (B, Hq, n_q,
 *                    max_blocks): pkv_decode_workspace_bytes(B, Hq) when n_q == 1,
 *                    else pkv_prefill_workspace_bytes(B, n_q, Hq, max_blocks)
 * A request fits a device budget of free bytes F when storage_bytes + fixed_bytes
 * plus the growth of the step's workspace over what the caller already holds is at
 * most F.  Errors: PKV_ERR_INVALID for NULL pointers, negative or zero sizes, Hq
 * not a multiple of n_kv_heads or B * n_q > 4096 with n_q > 1 (latent pools have
 * their own limits, given with their calls); PKV_ERR_RANGE when
 * the slabs to append would exceed max_slabs (the pool can never hold the request).
 *   [mlx-swift-lm #142, Summary: admission prices the growth of storage, the page
 *    and fixed costs and the step's guaranteed workspace each on its own; After:
 *    admission = storage plus guaranteed workspace; mlxcel #235, Proposed
 *    solution, bullet 2: presize_for_span appends the slabs a span needs at once] */
typedef struct {
  int32_t new_blocks;
  int32_t B;
  int32_t Hq;
  int32_t n_q;
  int32_t max_blocks;
} pkv_request;

typedef struct {
  int32_t slabs_to_append;
  int64_t free_rows;
  uint64_t storage_bytes;
  uint64_t page_bytes;
  uint64_t fixed_bytes;
  uint64_t workspace_bytes;
} pkv_price;

pkv_status pkv_price_request(const pkv_pool* pool, const pkv_request* req, pkv_price* out);

/* Storage identity check: PKV_OK if cfg describes the same stored layout as the
 * pool (format, head_dim, n_kv_heads, block_size, slab_blocks and, except for bf16,
 * group_size and, for packed formats, hadamard_seed), else PKV_ERR_FORMAT.  Used to reject an
 * incompatible storage identity before any allocation or copy.
 *   [mlx-swift-lm #142, Summary: a checkpoint of another storage identity is
 *    refused before anything is allocated] */
pkv_status pkv_pool_check_identity(const pkv_pool* pool, const pkv_pool_config* cfg);

/* Workspace bytes for pkv_paged_prefill_attention with B sequences, n_q new tokens
 * each, Hq query heads and block tables of max_blocks entries.  B * n_q <= 4096.
 * Synchronous, host only. */
pkv_status pkv_prefill_workspace_bytes(const pkv_pool* pool, int B, int n_q, int Hq, int max_blocks, size_t* bytes);

/* Causal chunked-prefill attention over the pool: sequence b holds ctx_lens[b]
 * tokens (its chunk of n_q new tokens already written with pkv_write_block, as the
 * last n_q), and query i of the chunk attends to tokens [0, ctx_lens[b] - n_q + i].
 * q_bf16: [B, n_q, Hq, head_dim] bf16, un-rotated (packed formats rotate q
 * internally); out_bf16: [B, n_q, Hq, head_dim]; block_table, ctx_lens and the GQA
 * mapping as for pkv_paged_decode_attention.  The workspace (caller-owned, 256-byte
 * aligned, pkv_prefill_workspace_bytes) holds, for each run of NQ consecutive
 * queries of a sequence, a view of the sequence (the same block-table row, the
 * last of those queries' causal length; when NQ = n_q > 1 the caller's block table
 * and lengths serve directly) and the split-K partials.  The attention kernels
 * serve the NQ queries in one tensor-core tile, each masked at its own causal
 * limit: up to 16 (query, head) rows per kv head at head_dim <= 128 and 8 at 256;
 * NQ is the largest such count dividing n_q (bf16), or the one filling 16 rows, else
 * 8 rows (packed formats), else 1.
 * A sequence with fewer than n_q tokens sets the device error word (bit 2) and its
 * rows are zero.
 * Errors as for pkv_paged_decode_attention; PKV_ERR_INVALID when B * n_q > 4096.
 * Asynchronous.
 *   [mlxcel #2171, Proposed Solution: attend = update the storage, then attention;
 *    mlx-swift-lm #142, Summary: packed pages are attended to directly] */
pkv_status pkv_paged_prefill_attention(pkv_pool* pool, int layer, int B, int n_q, int Hq, const void* q_bf16,
                                       const int32_t* block_table, int max_blocks, const int32_t* ctx_lens,
                                       int max_ctx, float scale, void* out_bf16, void* workspace, size_t ws_bytes,
                                       void* stream);

/* The pool's configuration (its storage identity plus n_layers and max_slabs), for
 * a checkpoint header.  Synchronous, host only.
 *   [mlx-swift-lm #142, After: a packed checkpoint carries its format identity] */
pkv_status pkv_pool_get_config(const pkv_pool* pool, pkv_pool_config* out);

/* Bytes of one block record: every stored byte of one block (row) of every layer,
 * layer-major, then tensor kind (K, V, K meta, V meta), each the block's
 * [block_size, n_kv_heads, row_bytes(kind)] bytes exactly as stored.  Equals
 * n_layers * block_size * n_kv_heads * sum over kinds of row_bytes(kind).
 * Synchronous, host only. */
pkv_status pkv_block_record_bytes(const pkv_pool* pool, size_t* bytes);

/* export_blocks: write the records of blocks rows_dev[0..n) to out_dev, one after
 * another in list order (n records; packed codes and FP32 metadata are copied
 * bit for bit, nothing is dequantised).  rows_dev: n int32 on the device; out_dev:
 * caller-owned device buffer, 16-byte aligned, at least n records long
 * (out_bytes).  Errors: PKV_ERR_INVALID for null or misaligned pointers,
 * PKV_ERR_RANGE when out_bytes is too small; a row outside the pool sets the
 * device error word (bit 1) and its record is left unwritten.  Asynchronous.
 *   [mlxcel #235, touch point 6: a block's content is read from the slab that holds
 *    its row, through the shared mapping helper; mlx-swift-lm #142, Summary: a full
 *    checkpoint keeps the packed bytes as they are] */
pkv_status pkv_export_blocks(pkv_pool* pool, int n, const int32_t* rows_dev, void* out_dev, size_t out_bytes,
                             void* stream);

/* import_blocks: the restore path.  Copy n records from in_dev (layout of
 * pkv_export_blocks) into blocks rows_dev[0..n) of this pool (live, distinct rows;
 * the caller allocates them).  `identity` is the configuration of the pool the
 * records came from: when its storage identity (pkv_pool_check_identity) or its
 * n_layers differs from this pool's, PKV_ERR_FORMAT is returned before any device
 * work, so an incompatible checkpoint is rejected before anything is written.
 * Other errors as for export.  Asynchronous.
 *   [mlxcel #235, touch point 6: restore path; mlx-swift-lm #142, Summary: a
 *    checkpoint of another storage identity is refused before anything is
 *    allocated; After: the packed checkpoint is exact and carries its format] */
pkv_status pkv_import_blocks(pkv_pool* pool, const pkv_pool_config* identity, int n, const int32_t* rows_dev,
                             const void* in_dev, size_t in_bytes, void* stream);

/* ---------------------------------------------------------------------------
 * Latent pools (PKV_FMT_LATENT): attention with keys and values from one latent
 * vector a token, shared by every query head.  R = head_dim (the latent vector),
 * P = group_size = 64 (the position key, rotated before it is stored).
 *
 * Rows, slabs, copy-on-write, gather, block records and pricing work as for the
 * other formats; write_block and the decode / prefill calls with per-head K/V
 * return PKV_ERR_FORMAT on a latent pool, and the calls below do so on any other.
 * Stored rows and queries are expected to be finite: a row that holds a NaN or an
 * infinity reaches the outputs of every query it shares a tile with, those that do not
 * see it included (rows past a sequence's length are no such rows, and the queries of an
 * unused batch slot may hold anything).
 * Outputs and workspaces overlap no input, but for write_latent's q_out, and a
 * workspace belongs to one call at a time (two streams or graphs take one each).
 * The pages describe no such format: the operators are written from the formulas
 * given with each call.  They require the pool's device to be the current one
 * (PKV_ERR_INVALID otherwise).  pkv_price_request prices a step in absorbed form: the
 * workspace as pkv_latent_workspace_bytes, under that call's limits, and the q and
 * output rows as R + P and R values.  pkv_price_latent_prefill prices one in expanded
 * form, whose workspace is far larger.
 * --------------------------------------------------------------------------- */

/* write_latent: token i's row goes to (rows_dev[i], slots_dev[i]) of `layer`:
 *   c' = c * rsqrt(mean(c^2) + eps) * w   (c' = c, copied bit for bit, if
 *                                          norm_weight is NULL)
 *   r' = r with each pair (a, b) turned to (a cos t - b sin t, a sin t + b cos t),
 * and, with Hq > 0, the P position values of token i's query heads turned by the same
 * angles into q_out.  Pair j is (2j, 2j + 1) when `interleaved`, else (j, j + P/2);
 * its angle's cosine and sine are cos_sin[positions_dev[i]][j] and [P/2 + j].
 *   kv_bf16:       [n_tokens] rows of R + P values (c, then r), kv_stride values apart
 *   positions_dev: [n_tokens] int32, each in [0, n_positions)
 *   cos_sin:       [n_positions, P] float32, on the device
 *   norm_weight:   [R] bf16, or NULL
 *   q_rope, q_out: bf16, head h of token i at i * token_stride + h * head_stride;
 *                  q_out may be q_rope with the same strides (in place)
 * Arithmetic in fp32, one rounding to bf16 per stored value.  Pointers 16-byte
 * aligned; strides in values, non-negative multiples of 8, kv_stride >= R + P; rows of
 * q_out that do not overlap (a token's heads together, or a head's tokens together);
 * 0 <= Hq <= 1024, n_tokens * (1 + ceil(Hq / 32)) < 2^31 (else PKV_ERR_INVALID).  Two
 * tokens with the same (row, slot) leave a mix of their values there: each 16-byte piece
 * of the row is one token's or the other's.  A row, slot or position out of range sets
 * the device error word (bit 1, 4 or 16): the row is then not written and, for a bad
 * position, neither are the token's q_out rows.  n_tokens 0 returns PKV_OK.
 * Asynchronous. */
pkv_status pkv_write_latent(pkv_pool* pool, int layer, int n_tokens, const int32_t* rows_dev,
                            const int32_t* slots_dev, const void* kv_bf16, int64_t kv_stride,
                            const int32_t* positions_dev, const float* cos_sin, int n_positions,
                            const void* norm_weight, float eps, int interleaved, int Hq, const void* q_rope,
                            int64_t q_token_stride, int64_t q_head_stride, void* q_out, int64_t out_token_stride,
                            int64_t out_head_stride, void* stream);

/* Workspace bytes of pkv_paged_latent_attention for batches of B sequences with n_q
 * queries of Hq heads each (split-K partials; no initialisation needed).  Host only;
 * the limits are those of that call. */
pkv_status pkv_latent_workspace_bytes(const pkv_pool* pool, int B, int n_q, int Hq, size_t* bytes);

/* Absorbed attention over the latent rows themselves, for decode (n_q = 1) and for
 * several newest tokens of each sequence (n_q > 1: drafted tokens, short chunks):
 *   x[t] = scale * (q_latent[b,i,h] . c_t + q_rope[b,i,h] . r_t)
 *   out[b,i,h] = sum_t softmax(x)[t] c_t      over t in [0, ctx_lens[b] - n_q + i]
 * The caller has multiplied the heads' queries by the key projection, and multiplies
 * the output by the value projection.
 *   q_latent, q_rope: bf16 rows (b, i, h) of R and of P values, row (b n_q + i) Hq + h
 *                     at that many strides (q_latent_stride >= R, q_rope_stride >= P;
 *                     multiples of 8)
 *   block_table_dev:  [B, max_blocks] int32 rows; ctx_lens_dev: [B] int32
 *   out_bf16:         [B, n_q, Hq, R] bf16, contiguous
 *   workspace:        256-byte aligned, ws_bytes >= pkv_latent_workspace_bytes
 * A length of 0 (an unused batch slot) gives zero rows.  A negative length, one
 * beyond max_blocks * 32 or one in (0, n_q) sets the device error word (bit 2) and
 * gives zero rows; a block-table row outside the pool sets bit 1 (the sequence's
 * result is then undefined).  Slots past a sequence's length are never read into the
 * result, whatever they hold.  max_ctx is accepted for interface stability.
 * Probabilities enter the second product in bf16; sums and softmax state are fp32, and
 * the logits times log2(e) are expected to be finite in fp32.
 * Deterministic.  Limits: B <= 4096, Hq <= 1024, B * n_q * Hq <= 2^24, max_blocks <=
 * 2^20, |scale| log2(e) finite in fp32, pointers 16-byte aligned.  B = 0 returns PKV_OK.  Asynchronous. */
pkv_status pkv_paged_latent_attention(pkv_pool* pool, int layer, int B, int n_q, int Hq, const void* q_latent,
                                      int64_t q_latent_stride, const void* q_rope, int64_t q_rope_stride,
                                      const int32_t* block_table_dev, int max_blocks, const int32_t* ctx_lens_dev,
                                      int max_ctx, float scale, void* out_bf16, void* workspace, size_t ws_bytes,
                                      void* stream);

/* Workspace bytes of pkv_latent_prefill_attention: the expanded keys and values of B
 * contexts of at most max_ctx tokens (0 or above max_blocks * 32: max_blocks * 32), and,
 * where few queries leave SMs idle, the partial results of a split over the context.
 * Host only; the limits are those of that call. */
pkv_status pkv_latent_prefill_workspace_bytes(const pkv_pool* pool, int B, int n_q, int Hq, int max_blocks,
                                              int max_ctx, size_t* bytes);

/* pkv_price_request for a step in expanded form (a prompt or a long chunk) on a latent
 * pool, with the same meaning of every field but these: workspace_bytes is
 * pkv_latent_prefill_workspace_bytes of (B, n_q, Hq, max_blocks, max_ctx), and the q and
 * output rows in fixed_bytes have 128 + P and 128 values.  Limits and errors are those of
 * that query, B >= 1 and new_blocks >= 0 (PKV_ERR_INVALID), PKV_ERR_FORMAT on a pool of
 * another format and PKV_ERR_RANGE as for pkv_price_request.  Host only. */
pkv_status pkv_price_latent_prefill(const pkv_pool* pool, const pkv_request* req, int max_ctx, pkv_price* out);

/* Expanded attention, for prompts and long chunks: every visible latent row becomes
 * per-head keys and values, then ordinary causal attention runs over them:
 *   k[t,h] = (w_k[h] c_t, r_t)   v[t,h] = w_v[h] c_t
 *   out[b,i,h] = sum_t softmax(scale * q[b,i,h] . k[t,h])[t] v[t,h]
 * over t in [0, ctx_lens[b] - n_q + i], for the n_q newest tokens of each sequence
 * (already written with pkv_write_latent).
 *   q_bf16:   [B, n_q, Hq, 128 + P], each head's 128 values and then its rotated P
 *   w_k, w_v: [Hq, 128, R] bf16;  out_bf16: [B, n_q, Hq, 128]
 *   max_ctx:  bound on ctx_lens (0: max_blocks * 32); a longer context is an error
 *   workspace: 256-byte aligned, ws_bytes >= pkv_latent_prefill_workspace_bytes of the
 *              same arguments, not initialised
 * Lengths, errors, limits, alignment and B = 0 as for pkv_paged_latent_attention, and
 * B * Hq * (the bound on ctx_lens + 128) < 2^31.  Expanded keys are rounded to bf16, and
 * expanded values and the probabilities to fp16, once; sums and softmax state are fp32.
 * The fp16 operands carry a power of two for every 128 tokens, so that any magnitude fits
 * but very uneven ones lose bits: besides their own rounding, values are off by up to 2^-38
 * of the largest of their 128 tokens (positions 128 j to 128 j + 127, seen by the query or
 * not), and probabilities by up to 2^(k - 31) of the query's largest in 128 tokens whose
 * largest value is 2^-k of the largest that any of 256 consecutive queries sees (the
 * 128 tokens it lies in included).  Deterministic.
 * Asynchronous. */
pkv_status pkv_latent_prefill_attention(pkv_pool* pool, int layer, int B, int n_q, int Hq, const void* q_bf16,
                                        const void* w_k, const void* w_v, const int32_t* block_table_dev,
                                        int max_blocks, const int32_t* ctx_lens_dev, int max_ctx, float scale,
                                        void* out_bf16, void* workspace, size_t ws_bytes, void* stream);

/* ---------------------------------------------------------------------------
 * Drafted tokens on the per-head pools (bf16 and packed): a step that verifies a tree of
 * drafted tokens writes their keys and values, attends with the tree's mask, and moves
 * the accepted ones into place.  pkv_write_rotated serves prompts and single tokens as
 * well.
 *
 * The n_q drafted tokens of a sequence are its last ones: ctx_lens counts them, and drafted
 * token j lies at position ctx_lens[b] - n_q + j of the block table.  A sequence with fewer
 * drafts than the batch's n_q still has n_q places; the unused ones are named by no mask.
 * Outputs and workspaces overlap no input, but for write_rotated's q_out, and a workspace
 * belongs to one call at a time (two streams or graphs take one each).  These calls require
 * the pool's device to be the current one (PKV_ERR_INVALID otherwise).  pkv_price_request
 * prices such a step but for its workspace, which is pkv_tree_workspace_bytes.  The pages describe
 * none of them: they are written from the formulas given here.
 * --------------------------------------------------------------------------- */

/* write_rotated: token i's keys and values go to (rows_dev[i], slots_dev[i]) of `layer`:
 *   x' = x * rsqrt(mean(x^2) + eps) * w     (w = k_norm or q_norm; x' = x if it is NULL)
 *   the pairs (a, b) of the first rotary_dim values of x' become
 *   (a cos t - b sin t, a sin t + b cos t)
 * for x each of the token's keys and, with Hq > 0, its queries, which go to q_out; values are
 * stored as they are.  Pair j is (2j, 2j + 1) when `interleaved`, else (j, j + rotary_dim/2);
 * its angle's cosine and sine are cos_sin[positions_dev[i]][j] and [rotary_dim/2 + j].
 *   k_bf16, v_bf16: [n_tokens, n_kv_heads, head_dim], head h of token i at i * token_stride +
 *                  h * head_stride (views of one projection's output, for instance)
 *   positions_dev: [n_tokens] int32, each in [0, n_positions)
 *   cos_sin:       [n_positions, rotary_dim] float32, on the device
 *   k_norm, q_norm: [head_dim] bf16, or NULL
 *   q_bf16, q_out: [n_tokens, Hq, head_dim], strided likewise; q_out may be q_bf16 with the
 *                  same strides (in place)
 * Arithmetic in fp32, one rounding to bf16 per value of a bf16 pool and of q_out; keys of a
 * packed pool are not rounded before they are quantised (as pkv_write_block says, but for the
 * scale, which is (max-min) times the rounded 1/(2^bits-1): an ulp apart at most; the turned
 * key and its Hadamard transform carry about 40 bits).  Pointers 16-byte aligned;
 * strides in values, non-negative multiples of 8; rows of q_out that do not overlap (a
 * token's heads together, or a head's tokens together); rotary_dim a multiple of 32 in
 * [32, head_dim]; 0 <= Hq <= 1024, n_tokens * (2 n_kv_heads + Hq) < 2^31 (else
 * PKV_ERR_INVALID).  Two tokens with the same (row, slot) leave a mix of their values there.
 * A row, slot or position out of range sets the device error word (bit 1, 4 or 16): nothing of
 * the token is then stored and, for a bad position, its q_out rows are not written either.
 * PKV_ERR_FORMAT on a latent pool (pkv_write_latent).  n_tokens 0 returns PKV_OK.
 * Asynchronous. */
pkv_status pkv_write_rotated(pkv_pool* pool, int layer, int n_tokens, const int32_t* rows_dev,
                             const int32_t* slots_dev, const void* k_bf16, int64_t k_token_stride,
                             int64_t k_head_stride, const void* v_bf16, int64_t v_token_stride,
                             int64_t v_head_stride, const int32_t* positions_dev, const float* cos_sin,
                             int n_positions, int rotary_dim, int interleaved, const void* k_norm,
                             const void* q_norm, float eps, int Hq, const void* q_bf16, int64_t q_token_stride,
                             int64_t q_head_stride, void* q_out, int64_t out_token_stride,
                             int64_t out_head_stride, void* stream);

/* Workspace bytes of pkv_paged_tree_attention for batches of B sequences with n_q queries of
 * Hq heads each (split-K partials; no initialisation needed).  Host only; the limits are
 * those of that call. */
pkv_status pkv_tree_workspace_bytes(const pkv_pool* pool, int B, int n_q, int Hq, size_t* bytes);

/* Attention of the n_q drafted tokens of each sequence, arranged as a tree (or in any other
 * way that a mask says):
 *   out[b,i,h] = sum_t softmax_t(scale * q[b,i,h] . k_t) v_t
 * over the tokens t < ctx_lens[b] - n_q, all of them, and the drafted tokens j for which bit
 * j % 32 of word j / 32 of query i's mask row is set (its own bit too, if it is to see itself).
 * A row that sees nothing gives zeros.
 *   q_bf16:      [B, n_q, Hq, head_dim] (packed formats rotate it into K's basis internally)
 *   tree_mask:   uint32 [n_q, ceil(n_q / 32)] a sequence, mask_stride words apart; 0: one
 *                tree for the batch.  Bits from n_q on are not read.
 *   block_table_dev: [B, max_blocks] int32 rows; ctx_lens_dev: [B] int32
 *   out_bf16:    [B, n_q, Hq, head_dim]
 *   workspace:   256-byte aligned, ws_bytes >= pkv_tree_workspace_bytes
 * A length of 0 (an unused batch slot) gives zero rows.  A negative length, one beyond
 * max_blocks * 32 or one in (0, n_q) sets the device error word (bit 2) and gives zero rows; a
 * block-table row outside the pool sets bit 1 (the sequence's result is then undefined).
 * Slots past a sequence's length, and drafted tokens that no query of the sequence sees, are
 * never read into a result, whatever they hold; a drafted token whose value (packed: key or
 * value, scales and offsets among them) holds a NaN or an infinity may reach queries that do not
 * see it, once one does.  max_ctx is not read (the other attention calls take it).  Probabilities
 * enter the second product in 16 bits (bf16, for packed pools fp16), sums and softmax state are
 * fp32 (bf16 pools: 2^8 times the sum of a sequence's values' magnitudes has to fit).  A packed pool's keys,
 * values and rotated queries are expanded to fp16 (c s + o with s and o rounded to fp16), keys and
 * values under a power of two for each 64 tokens (positions 64 j to 64 j + 63), so that any magnitude
 * fits, in every 64 another one, but what is below 2^-27 of the largest of its 64, or below 2^-114, loses
 * bits; the logits times log2(e) are expected to be finite in fp32.  A chain of few drafts in a packed pool goes faster
 * through pkv_paged_prefill_attention (8 drafts of 16 / 8 heads behind 16 x 16384 tokens in K4/V4: 144 us
 * there, 195 here).  Deterministic.  Limits: B <= 4096, n_q <= 1024, Hq <= 1024 and a multiple of
 * n_kv_heads, B * n_q * Hq <= 2^24, max_blocks <= 2^20, |scale| log2(e) finite in fp32, pointers
 * 16-byte aligned.  PKV_ERR_FORMAT on a latent pool.  B = 0 returns PKV_OK.  Asynchronous. */
pkv_status pkv_paged_tree_attention(pkv_pool* pool, int layer, int B, int n_q, int Hq, const void* q_bf16,
                                    const uint32_t* tree_mask, int64_t mask_stride,
                                    const int32_t* block_table_dev, int max_blocks, const int32_t* ctx_lens_dev,
                                    int max_ctx, float scale, void* out_bf16, void* workspace, size_t ws_bytes,
                                    void* stream);

/* accept_drafts: the accepted path of each sequence's tree moves behind the tokens before
 * it.  With first = ctx_lens[b] - n_q, the token at position first + path[b][k] goes to
 * position first + k, for k < path_lens[b], in every layer and stored tensor (bit for bit), and
 * new_lens[b] = first + path_lens[b], the length to go on with.  Places from there up to
 * ctx_lens[b] keep what they held, or hold copies of moved tokens.
 *   path_dev:  [B, max_path] int32, rising along a row, each in [0, n_q); path_lens_dev: [B]
 *              int32 in [0, min(max_path, n_q)]
 *   new_lens_dev: [B] int32, or NULL; must not overlap ctx_lens or path_lens
 * Any format, latent pools included.  The blocks that hold a sequence's drafted tokens belong
 * to it alone.  Lengths as for pkv_paged_tree_attention (a bad one sets bit 2, nothing moves and
 * the new length is 0); a path that does not rise, an entry or a length out of range sets bit
 * 32, nothing of the sequence moves and its new length is `first`; a block-table row outside
 * the pool sets bit 1 and the token is not moved.  Limits: B <= 4096, n_q <= 1024, max_blocks <=
 * 2^20.  Asynchronous. */
pkv_status pkv_accept_drafts(pkv_pool* pool, int B, int n_q, int max_path, const int32_t* path_dev,
                             const int32_t* path_lens_dev, const int32_t* block_table_dev, int max_blocks,
                             const int32_t* ctx_lens_dev, int32_t* new_lens_dev, void* stream);

/* Synchronise `stream`, read and clear the device error word.  PKV_ERR_DEVICE if it
 * was set (bits: 1 row out of range, 2 context too long, 4 slot out of range,
 * 8 wait limit reached, 16 rotary position out of range, 32 accepted path out of range or
 * not rising); *word_out (optional) receives the bits.  The kernels record
 * errors on the device instead of returning them, so that a decode step needs no
 * host synchronisation; the caller checks when it chooses.
 *   [mlxcel #2171, Implementation Notes: a decode step adds no host sync] */
pkv_status pkv_pool_check_errors(pkv_pool* pool, void* stream, int32_t* word_out);

/* Static description of a status code, and the last CUDA error message seen by
 * this thread (empty if none).  Never NULL; the strings belong to the library.
 * (C-ABI conveniences with no counterpart on the pages.) */
const char* pkv_status_string(pkv_status status);
const char* pkv_last_error(void);

#ifdef __cplusplus
}
#endif

#endif /* PKV_H_ */
