// latent_attn.cu — absorbed attention over a latent pool.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "latent.cuh"

namespace pkv {
namespace {

__device__ __forceinline__ float bf(uint16_t x) { return __uint_as_float((uint32_t)x << 16); }

// One warp per query row (b, i, h): lane l holds dims l, l + 32, ... of q and of the
// output; a token costs one dot product, five shuffles and an online-softmax step.
template <int R>
__global__ void __launch_bounds__(256) latent_attn_simple_kernel(const LatentAttnArgs a) {
  constexpr int E = R / 32, EP = kRope / 32;
  const int lane = threadIdx.x & 31;
  const int64_t row = ((int64_t)blockIdx.x * blockDim.x + threadIdx.x) >> 5;
  if (row >= (int64_t)a.B * a.n_q * a.Hq) return;
  const int b = (int)(row / ((int64_t)a.n_q * a.Hq));
  const int i = (int)(row / a.Hq % a.n_q);
  bool bad;
  const int32_t L = latent_ctx(a.ctx[b], (int64_t)a.max_blocks * kBlockTokens, a.n_q, &bad);
  if (bad && lane == 0) atomicOr(a.lv.err, ERR_CTX);
  const int32_t vis = L == 0 ? 0 : L - a.n_q + i + 1;
  float q[E + EP], acc[E];
#pragma unroll
  for (int e = 0; e < E; ++e) q[e] = bf(a.ql[row * a.ql_stride + lane + 32 * e]), acc[e] = 0.f;
#pragma unroll
  for (int e = 0; e < EP; ++e) q[E + e] = bf(a.qr[row * a.qr_stride + lane + 32 * e]);
  float m = -INFINITY, l = 0.f;
  for (int32_t t = 0; t < vis; ++t) {
    const int32_t r = a.bt[(int64_t)b * a.max_blocks + t / kBlockTokens];
    if (!latent_row_ok(a.lv, r)) {
      if (lane == 0) atomicOr(a.lv.err, ERR_ROW);
      continue;
    }
    const uint16_t* kv = reinterpret_cast<const uint16_t*>(latent_row(a.lv, r, t % kBlockTokens));
    float c[E], s = 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e) c[e] = bf(kv[lane + 32 * e]), s += q[e] * c[e];
#pragma unroll
    for (int e = 0; e < EP; ++e) s += q[E + e] * bf(kv[R + lane + 32 * e]);
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) s += __shfl_xor_sync(0xffffffffu, s, off);
    s *= a.scale_log2;
    const float mn = fmaxf(m, s);
    const float k = exp2f(m - mn), p = exp2f(s - mn);
    l = l * k + p;
    m = mn;
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] = acc[e] * k + p * c[e];
  }
  const float inv = vis > 0 ? 1.f / l : 0.f;
#pragma unroll
  for (int e = 0; e < E; ++e)
    a.out[row * R + lane + 32 * e] = __bfloat16_as_ushort(__float2bfloat16_rn(acc[e] * inv));
}

}  // namespace

size_t latent_attn_workspace(int R, int B, int n_q, int Hq, int ctas) { return 256; }

cudaError_t launch_latent_attn(const LatentAttnArgs& a) {
  const int64_t rows = (int64_t)a.B * a.n_q * a.Hq;
  const unsigned grid = (unsigned)((rows + 7) / 8);
  if (a.R == 512)
    latent_attn_simple_kernel<512><<<grid, 256, 0, a.stream>>>(a);
  else
    latent_attn_simple_kernel<256><<<grid, 256, 0, a.stream>>>(a);
  return cudaGetLastError();
}

}  // namespace pkv
