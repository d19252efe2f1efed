// accept.cu — accept_drafts: the drafted tokens on the accepted path move, in every layer
// and stored tensor, to the places behind the tokens before them.
//
//   token first + path[k] -> first + k, k = 0 .. len - 1, first = ctx - n_q
//
// A path rises (path[k] >= k, each entry above the one before), so a token's new place is
// never the old place of a later one: moved in order, nothing that is still needed is
// overwritten.  A thread owns 16 bytes of a token and moves them for all of the path, a
// batch of loads before the batch's stores; no other thread touches those bytes.  A CTA takes one
// (sequence, layer, tensor).  What bounds it is each CTA's chain of reads that hang on one another (length,
// path length, path, block rows, slab bases, bytes) for the few tokens that move: 64 sequences, paths of up
// to 9 tokens of 2 KB, 28 layers, bf16, on one GB300, about 285 moved tokens, 65 MB read and written: 15.9 us, 4.1 TB/s, with
// eight pools in turn (more than L2 holds), 10.8 replayed on one pool; 8 sequences 4.8 and 3.7 us.
#include <cuda_runtime.h>

#include "drafts.cuh"
#include "tcgen05.cuh"

namespace pkv {
namespace {

constexpr int kThreads = 256;
constexpr int kBatch = 8;    // tokens in flight
constexpr int kHeld = 64;    // tokens whose addresses are held at a time

__global__ void __launch_bounds__(kThreads) accept_kernel(const __grid_constant__ AcceptArgs a) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  __shared__ const uint4* from[kHeld];
  __shared__ uint4* to[kHeld];
  const int ppb = a.n_layers * a.n_kinds;
  const int b = blockIdx.x / ppb, lk = blockIdx.x - b * ppb;
  const int kind = lk % a.n_kinds;
  bool bad;
  const int32_t L = draft_ctx(a.ctx[b], (int64_t)a.max_blocks * kBlockTokens, a.n_q, &bad);
  const int32_t first = L - a.n_q;
  int len = a.path_lens[b];
  const int32_t* path = a.path + (int64_t)b * a.max_path;
  bool wrong = len < 0 || len > a.max_path || len > a.n_q;
  if (!wrong)
    for (int k = threadIdx.x; k < len; k += blockDim.x) {
      const int32_t p = path[k];
      if (p < 0 || p >= a.n_q || (k > 0 && path[k - 1] >= p)) wrong = true;
    }
  wrong = __syncthreads_or(wrong);
  if (threadIdx.x == 0 && lk == 0) {
    if (bad) atomicOr(a.err, ERR_CTX);
    if (wrong && L > 0) atomicOr(a.err, (int32_t)ERR_PATH);
    if (a.new_lens) a.new_lens[b] = L == 0 ? 0 : first + (wrong ? 0 : len);
  }
  if (wrong || L == 0) return;
  const int64_t bytes = a.token_bytes[kind];
  const int chunks = (int)(bytes / 16);
  auto place = [&](int32_t t, bool* ok) -> uint8_t* {
    const int32_t row = a.bt[(int64_t)b * a.max_blocks + t / kBlockTokens];
    if (row < 0 || (int64_t)row >= a.rows_capacity) {
      *ok = false;
      return nullptr;
    }
    const int32_t slab = row / a.slab_blocks;
    return const_cast<uint8_t*>(a.table[(size_t)slab * ppb + lk]) +
           ((int64_t)(row - slab * a.slab_blocks) * kBlockTokens + t % kBlockTokens) * bytes;
  };
  for (int k0 = 0; k0 < len; k0 += kHeld) {
    const int n = min(kHeld, len - k0);
    for (int k = threadIdx.x; k < n; k += blockDim.x) {
      const int32_t p = path[k0 + k];
      bool ok = true;
      const uint8_t* s = place(first + p, &ok);
      uint8_t* d = place(first + k0 + k, &ok);
      if (!ok) atomicOr(a.err, ERR_ROW);
      // in place already, or outside the pool: nothing to move
      from[k] = ok && p != k0 + k ? reinterpret_cast<const uint4*>(s) : nullptr;
      to[k] = reinterpret_cast<uint4*>(d);
    }
    __syncthreads();
    for (int c = threadIdx.x; c < chunks; c += blockDim.x)
      for (int i = 0; i < n; i += kBatch) {
        uint4 v[kBatch];
#pragma unroll
        for (int j = 0; j < kBatch; ++j)
          if (i + j < n && from[i + j]) v[j] = from[i + j][c];
#pragma unroll
        for (int j = 0; j < kBatch; ++j)
          if (i + j < n && from[i + j]) to[i + j][c] = v[j];
      }
    __syncthreads();
  }
}

}  // namespace

cudaError_t launch_accept(const AcceptArgs& a) {
  int64_t most = 0;
  for (int k = 0; k < a.n_kinds; ++k) most = most > a.token_bytes[k] / 16 ? most : a.token_bytes[k] / 16;
  const int threads = most >= kThreads ? kThreads : most <= 64 ? 64 : (int)((most + 31) / 32 * 32);
  static std::atomic<uint64_t> none{0};
  return tc_launch(accept_kernel, dim3((unsigned)((int64_t)a.B * a.n_layers * a.n_kinds)), threads, (size_t)0, a.stream, a,
                   0, &none);
}

}  // namespace pkv
