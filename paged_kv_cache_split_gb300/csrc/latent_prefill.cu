// latent_prefill.cu — expanded attention over a latent pool.
//
// The latent rows of every sequence are expanded to per-head keys and values in the
// workspace ([B, Hq, max_ctx, kLatentHead] each, bf16), then ordinary causal attention
// runs over (k, r) and v.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "latent.cuh"

namespace pkv {
namespace {

constexpr int DH = kLatentHead;

__device__ __forceinline__ float bf(uint16_t x) { return __uint_as_float((uint32_t)x << 16); }

// One thread per expanded value.
__global__ void __launch_bounds__(256) latent_expand_simple_kernel(const LatentPrefillArgs a, uint16_t* ko, uint16_t* vo) {
  const int d = threadIdx.x & 127, kind = threadIdx.x >> 7;
  const int h = blockIdx.y, b = blockIdx.z;
  bool bad;
  const int64_t lim = min((int64_t)a.max_blocks * kBlockTokens, (int64_t)a.max_ctx);
  const int32_t L = latent_ctx(a.ctx[b], lim, a.n_q, &bad);
  if (bad && threadIdx.x == 0) atomicOr(a.lv.err, ERR_CTX);
  const uint16_t* w = (kind ? a.wv : a.wk) + ((int64_t)h * DH + d) * a.R;
  uint16_t* o = kind ? vo : ko;
  for (int t = blockIdx.x; t < L; t += gridDim.x) {
    const int32_t r = a.bt[(int64_t)b * a.max_blocks + t / kBlockTokens];
    float s = 0.f;
    if (latent_row_ok(a.lv, r)) {
      const uint16_t* c = reinterpret_cast<const uint16_t*>(latent_row(a.lv, r, t % kBlockTokens));
      for (int e = 0; e < a.R; ++e) s += bf(c[e]) * bf(w[e]);
    } else if (d == 0) {
      atomicOr(a.lv.err, ERR_ROW);
    }
    o[(((int64_t)b * a.Hq + h) * a.max_ctx + t) * DH + d] = __bfloat16_as_ushort(__float2bfloat16_rn(s));
  }
}

// One warp per query row (b, i, h).
__global__ void __launch_bounds__(256) latent_prefill_simple_kernel(const LatentPrefillArgs a, const uint16_t* ki,
                                                                    const uint16_t* vi) {
  constexpr int E = DH / 32, EP = kRope / 32;
  const int lane = threadIdx.x & 31;
  const int64_t row = ((int64_t)blockIdx.x * blockDim.x + threadIdx.x) >> 5;
  if (row >= (int64_t)a.B * a.n_q * a.Hq) return;
  const int b = (int)(row / ((int64_t)a.n_q * a.Hq));
  const int i = (int)(row / a.Hq % a.n_q), h = (int)(row % a.Hq);
  bool bad;
  const int64_t lim = min((int64_t)a.max_blocks * kBlockTokens, (int64_t)a.max_ctx);
  const int32_t L = latent_ctx(a.ctx[b], lim, a.n_q, &bad);
  const int32_t vis = L == 0 ? 0 : L - a.n_q + i + 1;
  float q[E + EP], acc[E];
#pragma unroll
  for (int e = 0; e < E + EP; ++e) q[e] = bf(a.q[row * (DH + kRope) + lane + 32 * e]);
#pragma unroll
  for (int e = 0; e < E; ++e) acc[e] = 0.f;
  float m = -INFINITY, l = 0.f;
  const int64_t base = ((int64_t)b * a.Hq + h) * a.max_ctx;
  for (int32_t t = 0; t < vis; ++t) {
    const int32_t r = a.bt[(int64_t)b * a.max_blocks + t / kBlockTokens];
    if (!latent_row_ok(a.lv, r)) continue;
    const uint16_t* rp = reinterpret_cast<const uint16_t*>(latent_row(a.lv, r, t % kBlockTokens)) + a.R;
    const uint16_t* kp = ki + (base + t) * DH;
    float s = 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e) s += q[e] * bf(kp[lane + 32 * e]);
#pragma unroll
    for (int e = 0; e < EP; ++e) s += q[E + e] * bf(rp[lane + 32 * e]);
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) s += __shfl_xor_sync(0xffffffffu, s, off);
    s *= a.scale_log2;
    const float mn = fmaxf(m, s);
    const float k = exp2f(m - mn), p = exp2f(s - mn);
    l = l * k + p;
    m = mn;
    const uint16_t* vp = vi + (base + t) * DH;
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] = acc[e] * k + p * bf(vp[lane + 32 * e]);
  }
  const float inv = vis > 0 ? 1.f / l : 0.f;
#pragma unroll
  for (int e = 0; e < E; ++e)
    a.out[row * DH + lane + 32 * e] = __bfloat16_as_ushort(__float2bfloat16_rn(acc[e] * inv));
}

}  // namespace

size_t latent_prefill_workspace(int B, int Hq, int max_ctx) {
  return 256 + (size_t)2 * B * Hq * (size_t)max_ctx * DH * sizeof(uint16_t);
}

cudaError_t launch_latent_prefill(const LatentPrefillArgs& a) {
  uint16_t* k = (uint16_t*)a.ws;
  uint16_t* v = k + (size_t)a.B * a.Hq * a.max_ctx * DH;
  dim3 grid((unsigned)max(1, min(a.max_ctx, 4096)), (unsigned)a.Hq, (unsigned)a.B);
  latent_expand_simple_kernel<<<grid, 256, 0, a.stream>>>(a, k, v);
  const int64_t rows = (int64_t)a.B * a.n_q * a.Hq;
  latent_prefill_simple_kernel<<<(unsigned)((rows + 7) / 8), 256, 0, a.stream>>>(a, k, v);
  return cudaGetLastError();
}

}  // namespace pkv
