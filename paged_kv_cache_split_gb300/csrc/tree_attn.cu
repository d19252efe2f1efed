// tree_attn.cu — attention of drafted token trees over the per-head pools.
//
//   o[i, h] = sum_t p[t] v_t,  p = softmax_t(scale q[i, h] . k_t)
//
// over the tokens t < len - n_q and the drafted tokens (the last n_q) that bit t - (len -
// n_q) of query i's mask row names.
//
// One warp takes a (query, head) row and walks the context with the running maximum and
// sum of the softmax; a lane holds D / 32 of the row's values.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "drafts.cuh"
#include "tcgen05.cuh"

namespace pkv {
namespace {

template <int E>
__device__ __forceinline__ void load_row(const uint8_t* codes, const uint8_t* meta, int bits, int group, int lane, float (&x)[E]) {
  if (bits == 16) {
#pragma unroll
    for (int e = 0; e < E; ++e)
      x[e] = __uint_as_float((uint32_t) reinterpret_cast<const uint16_t*>(codes)[lane * E + e] << 16);
    return;
  }
  const float2 m = reinterpret_cast<const float2*>(meta)[lane * E / group];
#pragma unroll
  for (int e = 0; e < E; ++e) {
    const int i = lane * E + e;
    const int c = bits == 8 ? codes[i] : (codes[i / 2] >> (4 * (i & 1))) & 15;
    x[e] = m.x * (float)c + m.y;
  }
}

template <int D>
__global__ void __launch_bounds__(256) tree_attn_kernel(const __grid_constant__ TreeAttnArgs a) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  constexpr int E = D / 32;
  const int lane = threadIdx.x & 31;
  const int64_t r = (int64_t)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5);
  if (r >= (int64_t)a.B * a.n_q * a.Hq) return;
  const int h = (int)(r % a.Hq), i = (int)(r / a.Hq % a.n_q), b = (int)(r / a.Hq / a.n_q);
  const int kvh = h / (a.Hq / a.lv.hkv);
  bool bad;
  const int32_t L = draft_ctx(a.ctx[b], (int64_t)a.max_blocks * kBlockTokens, a.n_q, &bad);
  if (bad && i == 0 && h == 0 && lane == 0) atomicOr(a.lv.err, ERR_CTX);
  const uint32_t* mask = a.mask + b * a.mask_stride + (int64_t)i * ((a.n_q + 31) / 32);
  const int kbits = a.fmt == PKV_FMT_BF16 ? 16 : a.fmt == PKV_FMT_K4V4 ? 4 : 8;
  const int vbits = a.fmt == PKV_FMT_BF16 ? 16 : a.fmt == PKV_FMT_K8V8 ? 8 : 4;
  float q[E], o[E];
#pragma unroll
  for (int e = 0; e < E; ++e) {
    q[e] = __uint_as_float((uint32_t)a.q[r * D + lane * E + e] << 16);
    o[e] = 0.f;
  }
  if (kbits < 16) {
#pragma unroll
    for (int e = 0; e < E; ++e) q[e] *= a.signs[lane * E + e];
#pragma unroll
    for (int hs = 1; hs < E; hs <<= 1)
#pragma unroll
      for (int e = 0; e < E; ++e)
        if ((e & hs) == 0) {
          const float x = q[e], y = q[e + hs];
          q[e] = x + y;
          q[e + hs] = x - y;
        }
#pragma unroll
    for (int m = 1; m < 32; m <<= 1)
#pragma unroll
      for (int e = 0; e < E; ++e) {
        const float other = __shfl_xor_sync(0xffffffffu, q[e], m);
        q[e] = lane & m ? other - q[e] : q[e] + other;
      }
#pragma unroll
    for (int e = 0; e < E; ++e) q[e] *= D == 64 ? 0.125f : D == 128 ? 0.08838834764831845f : 0.0625f;
  }
  float m = -INFINITY, l = 0.f;
  for (int t = 0; t < L; ++t) {
    const int j = t - (L - a.n_q);
    if (j >= 0 && !(mask[j >> 5] >> (j & 31) & 1u)) continue;
    const int32_t row = a.bt[(int64_t)b * a.max_blocks + t / kBlockTokens];
    if (!draft_row_ok(a.lv, row)) {
      if (lane == 0) atomicOr(a.lv.err, ERR_ROW);
      continue;
    }
    const int slot = t % kBlockTokens;
    float k[E], v[E];
    load_row<E>(draft_row(a.lv, PKV_KIND_K, row, slot, kvh), kbits < 16 ? draft_row(a.lv, PKV_KIND_KMETA, row, slot, kvh) : nullptr,
                kbits, a.group, lane, k);
    load_row<E>(draft_row(a.lv, PKV_KIND_V, row, slot, kvh), kbits < 16 ? draft_row(a.lv, PKV_KIND_VMETA, row, slot, kvh) : nullptr,
                vbits, a.group, lane, v);
    float x = 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e) x += q[e] * k[e];
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) x += __shfl_xor_sync(0xffffffffu, x, off);
    x *= a.scale_log2;
    if (x > m) {
      const float f = exp2f(m - x);
      m = x;
      l *= f;
#pragma unroll
      for (int e = 0; e < E; ++e) o[e] *= f;
    }
    const float p = exp2f(x - m);
    l += p;
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] += p * v[e];
  }
  const float inv = l > 0.f ? 1.f / l : 0.f;
#pragma unroll
  for (int e = 0; e < E; ++e) a.out[r * D + lane * E + e] = __bfloat16_as_ushort(__float2bfloat16_rn(o[e] * inv));
}

}  // namespace

size_t tree_attn_workspace(int D, int hkv, int B, int n_q, int Hq, int ctas) { return 256; }

cudaError_t launch_tree_attn(const TreeAttnArgs& a) {
  const dim3 grid((unsigned)(((int64_t)a.B * a.n_q * a.Hq + 7) / 8));
  static std::atomic<uint64_t> none{0};
  return tc_launch(a.D == 64 ? tree_attn_kernel<64> : a.D == 128 ? tree_attn_kernel<128> : tree_attn_kernel<256>, grid, 256,
                   (size_t)0, a.stream, a, a.device, &none);
}

}  // namespace pkv
