// latent_write.cu — write_latent: normalise, rotate and store the latent rows of new
// tokens, and rotate the query heads' position parts by the same angles.
//
//   c' = c * rsqrt(mean(c^2) + eps) * w      (skipped without a weight)
//   (r'_a, r'_b) = (r_a cos t - r_b sin t, r_a sin t + r_b cos t)
//
// over the pairs (2j, 2j+1) or (j, j + kRope/2), t the j-th angle of the token's
// position, read from a table.  Sums and products are FP32, one rounding to bf16.
//
// Bound by HBM: every input byte is read once and every output byte written once.
// A warp takes either one token's latent row (16-byte chunks, R/8/32 of them per
// lane, the sum of squares by shuffles) or 32 heads of one token's queries: eight
// lanes hold a head's 128 bytes, so a warp has 4 heads per load and eight independent
// 16-byte loads per lane in flight before the first is used.
//
// Measured (one GB300): 16384 tokens with 128 heads 84.3 us, 6.87 TB/s of input and output
// bytes (the card copies at 6.79); 4999 tokens with 16 heads, turned by halves, 10.1 us, 3.3
// TB/s, bound by latency: 79 registers (61 interleaved) leave 24 warps to an SM, nearly
// three waves of 9998, half of a query warp's loads are off with 16 heads, and the table's
// rows are gathered from 33 MB; 8 tokens 1.9 us.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "latent.cuh"
#include "tcgen05.cuh"

namespace pkv {
namespace {

constexpr int kHeadsPerUnit = kLatentWriteHeads;

struct Vec8 {
  float x[8];
};

__device__ __forceinline__ Vec8 unpack8(const uint4& v) {
  Vec8 o;
  bf16x2_to_f32(v.x, o.x[0], o.x[1]);
  bf16x2_to_f32(v.y, o.x[2], o.x[3]);
  bf16x2_to_f32(v.z, o.x[4], o.x[5]);
  bf16x2_to_f32(v.w, o.x[6], o.x[7]);
  return o;
}

__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  __nv_bfloat162 t = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<uint32_t*>(&t);
}

__device__ __forceinline__ uint4 pack8(const Vec8& v) {
  return make_uint4(pack2(v.x[0], v.x[1]), pack2(v.x[2], v.x[3]), pack2(v.x[4], v.x[5]), pack2(v.x[6], v.x[7]));
}

// The angles of one lane's eight values (lane j of the eight that hold a 64-value
// row): interleaved, four pairs in the lane; by halves, eight values whose partners
// sit in lane j ^ 4.
template <bool IL>
struct Angles {
  float c[IL ? 4 : 8], s[IL ? 4 : 8];
  __device__ __forceinline__ void load(const float* tab, int j) {
    constexpr int N = IL ? 4 : 8;
    const int first = IL ? 4 * j : 8 * (j & 3);
#pragma unroll
    for (int e = 0; e < N; e += 4) {
      const float4 a = *reinterpret_cast<const float4*>(tab + first + e);
      const float4 b = *reinterpret_cast<const float4*>(tab + kRope / 2 + first + e);
      c[e] = a.x, c[e + 1] = a.y, c[e + 2] = a.z, c[e + 3] = a.w;
      s[e] = b.x, s[e + 1] = b.y, s[e + 2] = b.z, s[e + 3] = b.w;
    }
  }
  // every lane of the warp takes part (shuffles)
  __device__ __forceinline__ Vec8 turn(const Vec8& v, int j) const {
    Vec8 o;
    if constexpr (IL) {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        o.x[2 * e] = v.x[2 * e] * c[e] - v.x[2 * e + 1] * s[e];
        o.x[2 * e + 1] = v.x[2 * e] * s[e] + v.x[2 * e + 1] * c[e];
      }
    } else {
      const bool second = (j & 4) != 0;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float other = __shfl_xor_sync(0xffffffffu, v.x[e], 4);
        o.x[e] = second ? other * s[e] + v.x[e] * c[e] : v.x[e] * c[e] - other * s[e];
      }
    }
    return o;
  }
};

template <int R, bool IL>
__global__ void __launch_bounds__(256) latent_write_kernel(const __grid_constant__ LatentWriteArgs a) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int lane = threadIdx.x & 31;
  const uint32_t u = blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5);
  const uint32_t i = u / (uint32_t)a.per_token;
  if (i >= (uint32_t)a.n) return;
  const int part = (int)(u - i * a.per_token);
  // What is loaded from the token's own rows is asked for before its position and place are
  // checked: one memory latency instead of three.
  const int32_t pos = a.positions[i];
  const bool pos_ok = pos >= 0 && pos < a.n_pos;
  const int j = lane & 7;
  Angles<IL> ang;
  if (part == 0) {
    constexpr int CH = R / 8 / 32;  // 16-byte chunks of the latent per lane
    const uint4* src = reinterpret_cast<const uint4*>(a.kv + (int64_t)i * a.kv_stride);
    uint4 raw[CH];
#pragma unroll
    for (int k = 0; k < CH; ++k) raw[k] = src[lane + 32 * k];
    const uint4 rr = src[R / 8 + j];  // the eight lanes of a row, four copies of it
    const int32_t row = a.rows[i], slot = a.slots[i];
    const bool row_ok = latent_row_ok(a.lv, row), slot_ok = slot >= 0 && slot < kBlockTokens;
    if (!pos_ok || !row_ok || !slot_ok) {
      if (lane == 0) atomicOr(a.lv.err, !pos_ok ? ERR_POS : row_ok ? ERR_SLOT : ERR_ROW);
      return;
    }
    uint4* dst = reinterpret_cast<uint4*>(latent_row(a.lv, row, slot));
    ang.load(a.cos_sin + (int64_t)pos * kRope, j);
    if (a.weight) {
      Vec8 v[CH];
      float ss = 0.f;
#pragma unroll
      for (int k = 0; k < CH; ++k) {
        v[k] = unpack8(raw[k]);
#pragma unroll
        for (int e = 0; e < 8; ++e) ss += v[k].x[e] * v[k].x[e];
      }
#pragma unroll
      for (int off = 16; off > 0; off >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, off);
      const float rs = rsqrtf(ss * (1.0f / R) + a.eps);
      const uint4* w = reinterpret_cast<const uint4*>(a.weight);
#pragma unroll
      for (int k = 0; k < CH; ++k) {
        const Vec8 g = unpack8(w[lane + 32 * k]);
#pragma unroll
        for (int e = 0; e < 8; ++e) v[k].x[e] = v[k].x[e] * rs * g.x[e];
        raw[k] = pack8(v[k]);
      }
    }
#pragma unroll
    for (int k = 0; k < CH; ++k) dst[lane + 32 * k] = raw[k];
    const uint4 turned = pack8(ang.turn(unpack8(rr), j));
    if (lane < 8) dst[R / 8 + j] = turned;
    return;
  }
  const int h0 = (part - 1) * kHeadsPerUnit + (lane >> 3);
  const uint16_t* q = a.q + (int64_t)i * a.q_tok + 8 * j;
  uint16_t* qo = a.qo + (int64_t)i * a.o_tok + 8 * j;
  uint4 v[kHeadsPerUnit / 4];
#pragma unroll
  for (int k = 0; k < kHeadsPerUnit / 4; ++k) {
    const int h = h0 + 4 * k;
    v[k] = h < a.Hq ? *reinterpret_cast<const uint4*>(q + h * a.q_head) : make_uint4(0, 0, 0, 0);
  }
  if (!pos_ok) return;  // flagged with the token's row
  ang.load(a.cos_sin + (int64_t)pos * kRope, j);
#pragma unroll
  for (int k = 0; k < kHeadsPerUnit / 4; ++k) {
    const int h = h0 + 4 * k;
    const uint4 o = pack8(ang.turn(unpack8(v[k]), j));
    if (h < a.Hq) *reinterpret_cast<uint4*>(qo + h * a.o_head) = o;
  }
}

template <int R>
cudaError_t launch_r(const LatentWriteArgs& a) {
  const int64_t units = (int64_t)a.n * a.per_token;
  // a step's few tokens spread over the SMs, one warp per CTA
  const int threads = units < 2048 ? 32 : 256;
  const dim3 grid((unsigned)((units * 32 + threads - 1) / threads));
  static std::atomic<uint64_t> none{0};
  return tc_launch(a.interleaved ? latent_write_kernel<R, true> : latent_write_kernel<R, false>, grid, threads, (size_t)0,
                   a.stream, a, 0, &none);
}

}  // namespace

cudaError_t launch_latent_write(const LatentWriteArgs& args) {
  LatentWriteArgs a = args;
  a.per_token = latent_write_units(a.Hq);
  return a.R == 512 ? launch_r<512>(a) : launch_r<256>(a);
}

}  // namespace pkv
