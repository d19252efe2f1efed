// rotated_write.cu — write_rotated: normalise, turn and store the keys of new tokens with
// their values, and turn the query heads by the same angles.
//
//   x' = x * rsqrt(mean(x^2) + eps) * w                    (skipped without a weight)
//   (y_a, y_b) = (x'_a cos t - x'_b sin t, x'_a sin t + x'_b cos t)
//
// over the pairs (2j, 2j+1) or (j, j + rot/2) of a head's first `rot` values, t the j-th
// angle of the token's position, read from a table.  Sums and products are FP32; queries
// and the keys of a bf16 pool are rounded to bf16 once.
//
// Packed pools quantise on the way, without a rounding before: the key goes into the
// Hadamard basis as it was turned.  Codes hang on the sums' last bits where a value lies
// near a border, so the turned value is kept as an unevaluated sum of two FP32 (products
// and sums with their exact remainders) and the butterflies run on two parts: the leading
// 16 bits relative to the row's largest value, whose sums FP32 holds exactly, and the
// rest.  That carries 40 bits relative to the largest value at twice the FP32 additions;
// FP64 (2 lanes a cycle and SM) would take thirty times as long.
//
// Measured on one GB300, over six sets of buffers in turn (more than L2 holds): 16384 tokens of 8 kv and 32 query
// heads of 128, half of each turned, norms, bf16 71.5 us, 5.7 TB/s (HBM); 5001 tokens, heads of 64, 15.5 us,
// 4.1 TB/s (11.2 replayed on one set, whose 63 MB stay in L2); 8 tokens 2.9 us (latency); 1512 tokens into a K4/V4
// pool 12.3 us (11.0 on one set), 16384 108 us (K8/V4 108, K8/V8 110): 3.8 and 3.1 times the bytes' time.  Issue is 63%
// active there, with the butterflies and the quantiser; the rest was not taken apart (the stages of shuffles
// follow one another).
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "drafts.cuh"
#include "latent.cuh"
#include "tcgen05.cuh"

namespace pkv {
namespace {

constexpr int kLoads = 4;  // 16-byte loads a lane has in flight

struct Params {
  RotatedWriteArgs a;
  int kv_units;        // warps that a token's keys take, and its values
  int per_token;       // warps a token: keys, values and queries; packed: queries
  int64_t pack_units;  // packed: warps that quantise keys (and as many values), before the queries' warps
};

__device__ __forceinline__ void unpack8(const uint4& v, float (&x)[8]) {
  bf16x2_to_f32(v.x, x[0], x[1]);
  bf16x2_to_f32(v.y, x[2], x[3]);
  bf16x2_to_f32(v.z, x[4], x[5]);
  bf16x2_to_f32(v.w, x[6], x[7]);
}
__device__ __forceinline__ uint4 pack8(const float (&x)[8]) {
  return make_uint4(bf2(x[0], x[1]), bf2(x[2], x[3]), bf2(x[4], x[5]), bf2(x[6], x[7]));
}

__device__ __forceinline__ bool place_ok(const LayerView& lv, int32_t row, int32_t slot) {
  return draft_row_ok(lv, row) && slot >= 0 && slot < kBlockTokens;
}
__device__ __forceinline__ void flag(const LayerView& lv, bool pos_ok, int32_t row) {
  atomicOr(lv.err, !pos_ok ? (int32_t)ERR_POS : draft_row_ok(lv, row) ? ERR_SLOT : ERR_ROW);
}

// The angles of one lane's eight values (chunk c of the D / 8 that hold a head).
template <bool IL>
struct Angles {
  float c[IL ? 4 : 8], s[IL ? 4 : 8];
  __device__ __forceinline__ void load(const float* tab, int chunk, int rot) {
    constexpr int N = IL ? 4 : 8;
    const int half = rot / 2;
    const int first = IL ? 4 * chunk : 8 * chunk < half ? 8 * chunk : 8 * chunk - half;
#pragma unroll
    for (int e = 0; e < N; e += 4) {
      const float4 a = *reinterpret_cast<const float4*>(tab + first + e);
      const float4 b = *reinterpret_cast<const float4*>(tab + half + first + e);
      c[e] = a.x, c[e + 1] = a.y, c[e + 2] = a.z, c[e + 3] = a.w;
      s[e] = b.x, s[e + 1] = b.y, s[e + 2] = b.z, s[e + 3] = b.w;
    }
  }
  // every lane of the warp takes part (shuffles); src: the lane that holds the partners
  __device__ __forceinline__ void turn(float (&x)[8], int src, bool second) const {
    if constexpr (IL) {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float a = x[2 * e], b = x[2 * e + 1];
        x[2 * e] = a * c[e] - b * s[e];
        x[2 * e + 1] = a * s[e] + b * c[e];
      }
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float other = __shfl_sync(0xffffffffu, x[e], src);
        x[e] = second ? other * s[e] + x[e] * c[e] : x[e] * c[e] - other * s[e];
      }
    }
  }
};

enum Kind { kKeys, kValues, kQueries };

// Heads r0 .. of one kind of token i, 32 / (D / 8) of them a load.  NORM: k_norm or q_norm is given.
template <int D, bool IL, bool NORM>
__device__ __forceinline__ void copy_heads(const RotatedWriteArgs& a, int i, Kind kind, int r0) {
  constexpr int LPH = D / 8;     // lanes a head
  constexpr int HPL = 32 / LPH;  // heads a load
  const int lane = threadIdx.x & 31, c = lane % LPH, sub = lane / LPH;
  const int heads = kind == kQueries ? a.Hq : a.lv.hkv;
  const int64_t step = kind == kKeys ? a.k_head : kind == kValues ? a.v_head : a.q_head;
  const uint16_t* src = kind == kKeys     ? a.k + (int64_t)i * a.k_tok
                        : kind == kValues ? a.v + (int64_t)i * a.v_tok
                                          : a.q + (int64_t)i * a.q_tok;
  uint4 raw[kLoads];
#pragma unroll
  for (int u = 0; u < kLoads; ++u) {
    const int r = r0 + u * HPL + sub;
    raw[u] = r < heads ? reinterpret_cast<const uint4*>(src + r * step)[c] : make_uint4(0, 0, 0, 0);
  }
  const int32_t pos = a.positions[i];
  const bool pos_ok = pos >= 0 && pos < a.n_pos;
  uint4* dst;
  int64_t dst_step;  // in 16-byte pieces
  if (kind == kQueries) {
    if (!pos_ok) return;  // flagged with the keys
    dst = reinterpret_cast<uint4*>(a.qo + (int64_t)i * a.o_tok);
    dst_step = a.o_head / 8;
  } else {
    const int32_t row = a.rows[i], slot = a.slots[i];
    if (!pos_ok || !place_ok(a.lv, row, slot)) {
      if (kind == kKeys && r0 == 0 && lane == 0) flag(a.lv, pos_ok, row);
      return;
    }
    dst = reinterpret_cast<uint4*>(draft_row(a.lv, kind == kKeys ? PKV_KIND_K : PKV_KIND_V, row, slot, 0));
    dst_step = LPH;
  }
  if (kind == kValues) {
#pragma unroll
    for (int u = 0; u < kLoads; ++u) {
      const int r = r0 + u * HPL + sub;
      if (r < heads) dst[r * dst_step + c] = raw[u];
    }
    return;
  }
  const int half = a.rot / 16;  // chunks of half of the turned part
  const bool turned = c < 2 * half, second = c >= half;
  const int from = lane + (turned ? (second ? -half : half) : 0);
  Angles<IL> ang;
  // (chunks that are not turned take the first angles and drop the result)
  ang.load(a.cos_sin + (int64_t)pos * a.rot, turned ? c : 0, a.rot);
  const uint16_t* w = kind == kKeys ? a.k_norm : a.q_norm;
  float g[8];
  if (NORM && w) unpack8(reinterpret_cast<const uint4*>(w)[c], g);
#pragma unroll
  for (int u = 0; u < kLoads; ++u) {
    const int r = r0 + u * HPL + sub;
    float x[8];
    unpack8(raw[u], x);
    uint4 o = raw[u];  // untouched values keep their bits
    if (NORM && w) {
      float ss = 0.f;
#pragma unroll
      for (int e = 0; e < 8; ++e) ss += x[e] * x[e];
#pragma unroll
      for (int off = 1; off < LPH; off <<= 1) ss += __shfl_xor_sync(0xffffffffu, ss, off);
      const float rs = rsqrtf(ss * (1.0f / D) + a.eps);
#pragma unroll
      for (int e = 0; e < 8; ++e) x[e] = x[e] * rs * g[e];
      if (a.rot < D) o = pack8(x);
    }
    ang.turn(x, from, second);
    if (turned) o = pack8(x);
    if (r < heads) dst[r * dst_step + c] = o;
  }
}

template <int D, bool IL, bool NORM>
__global__ void __launch_bounds__(256, !IL && NORM ? 3 : 4) rotated_write_kernel(const __grid_constant__ Params P) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const uint32_t u = blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5);
  const uint32_t i = u / (uint32_t)P.per_token;
  if (i >= (uint32_t)P.a.n) return;
  int part = (int)(u - i * P.per_token);
  const Kind kind = part < P.kv_units ? kKeys : part < 2 * P.kv_units ? kValues : kQueries;
  part -= kind == kKeys ? 0 : kind == kValues ? P.kv_units : 2 * P.kv_units;
  copy_heads<D, IL, NORM>(P.a, (int)i, kind, part * kLoads * (256 / D));
}

// ---------------------------------------------------------------------------
// Packed pools
// ---------------------------------------------------------------------------
constexpr int E = 16;  // values a lane

__device__ __forceinline__ void load16(const uint16_t* src, float (&x)[E]) {
  const uint4 a = reinterpret_cast<const uint4*>(src)[0], b = reinterpret_cast<const uint4*>(src)[1];
  float lo[8], hi[8];
  unpack8(a, lo);
  unpack8(b, hi);
#pragma unroll
  for (int e = 0; e < 8; ++e) x[e] = lo[e], x[8 + e] = hi[e];
}

// Codes and (scale, offset) of a row's groups, lane `c` of the row's D / 16.  IEEE single
// precision, one rounding an operation.  The scale is the range times the rounded 1 / TOP: an
// ulp from the quotient at most (the codes are the nearest for the scale that is stored).
template <int BITS, int GS>
__device__ __forceinline__ void quantise(const float (&x)[E], uint8_t* codes, uint8_t* meta, int c, bool store) {
  float mn = x[0], mx = x[0];
#pragma unroll
  for (int e = 1; e < E; ++e) mn = fminf(mn, x[e]), mx = fmaxf(mx, x[e]);
#pragma unroll
  for (int off = 1; off < GS / E; off <<= 1) {
    mn = fminf(mn, __shfl_xor_sync(0xffffffffu, mn, off));
    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, off));
  }
  constexpr int TOP = (1 << BITS) - 1;
  const float scale = __fmul_rn(__fsub_rn(mx, mn), 1.0f / TOP);
  uint32_t w[E * BITS / 32];
#pragma unroll
  for (int k = 0; k < E * BITS / 32; ++k) w[k] = 0;
  // The code is that of the IEEE quotient.  A product with the reciprocal is off by less than
  // 2^-21 TOP steps: where it lies further than that from a border, it gives the same code.
  const float inv = scale > 1e-37f && scale < 1e37f ? __frcp_rn(scale) : 0.f;  // (0: divides)
  constexpr float kClear = 0.5f - TOP * 4.76837158e-7f;
#pragma unroll
  for (int e = 0; e < E; ++e) {
    const float d = __fsub_rn(x[e], mn);
    const float t = __fmul_rn(d, inv);
    float code = rintf(t);
    if (inv == 0.f || !(fabsf(__fsub_rn(t, code)) < kClear)) code = scale != 0.f ? rintf(__fdiv_rn(d, scale)) : 0.f;
    const int q = min(max((int)code, 0), TOP);
    w[e * BITS / 32] |= (uint32_t)q << (e * BITS % 32);
  }
  if (!store) return;
  if constexpr (BITS == 8)
    reinterpret_cast<uint4*>(codes)[c] = make_uint4(w[0], w[1], w[2], w[3]);
  else
    reinterpret_cast<uint2*>(codes)[c] = make_uint2(w[0], w[1]);
  if (c % (GS / E) == 0) reinterpret_cast<float2*>(meta)[c / (GS / E)] = make_float2(scale, mn);
}

// x = the exact product a b, x = (h, l)
__device__ __forceinline__ void two_prod(float& h, float& l, float a, float b) {
  h = __fmul_rn(a, b);
  l = __fmaf_rn(a, b, -h);
}
// x += the exact product a b
__device__ __forceinline__ void two_prod_add(float& h, float& l, float a, float b) {
  const float p = __fmul_rn(a, b), pe = __fmaf_rn(a, b, -p);
  const float s = __fadd_rn(h, p), t = __fsub_rn(s, h);
  const float se = __fadd_rn(__fsub_rn(h, __fsub_rn(s, t)), __fsub_rn(p, t));
  h = s;
  l = __fadd_rn(l, __fadd_rn(se, pe));
}

template <int D>
__device__ __forceinline__ void butterflies(float (&x)[E], int c) {
#pragma unroll
  for (int hs = 1; hs < E; hs <<= 1)
#pragma unroll
    for (int e = 0; e < E; ++e)
      if ((e & hs) == 0) {
        const float a = x[e], b = x[e + hs];
        x[e] = a + b;
        x[e + hs] = a - b;
      }
#pragma unroll
  for (int m = 1; m < D / E; m <<= 1) {
    const bool upper = (c & m) != 0;
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const float other = __shfl_xor_sync(0xffffffffu, x[e], m);
      x[e] = upper ? other - x[e] : x[e] + other;
    }
  }
}

// A lane group's (token, head) row of keys: normalise, turn, into the Hadamard basis,
// quantise.  Lanes past the last row take part in the shuffles with row 0's data.
template <int D, bool IL, int BITS, int GS>
__device__ __forceinline__ void pack_keys(const RotatedWriteArgs& a, int64_t r, bool live) {
  constexpr int LPR = D / E;
  const int lane = threadIdx.x & 31, c = lane % LPR;
  const int i = (int)(r / a.lv.hkv), h = (int)(r - (int64_t)i * a.lv.hkv);
  float x[E], l[E];
  load16(a.k + (int64_t)i * a.k_tok + h * a.k_head + c * E, x);
  const int32_t pos = a.positions[i], row = a.rows[i], slot = a.slots[i];
  const bool pos_ok = pos >= 0 && pos < a.n_pos, ok = live && pos_ok && place_ok(a.lv, row, slot);
  if (live && !ok && h == 0 && c == 0) flag(a.lv, pos_ok, row);
  if (a.k_norm) {
    float ss = 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e) ss += x[e] * x[e];
#pragma unroll
    for (int off = 1; off < LPR; off <<= 1) ss += __shfl_xor_sync(0xffffffffu, ss, off);
    const float rs = rsqrtf(ss * (1.0f / D) + a.eps);
    float g[E];
    load16(a.k_norm + c * E, g);
#pragma unroll
    for (int e = 0; e < E; ++e) x[e] = x[e] * rs * g[e];
  }
  const int half = a.rot / 2;
  const bool turned = c * E < a.rot && pos_ok, second = c * E >= half;
  const float* tab = a.cos_sin + (pos_ok ? (int64_t)pos * a.rot : 0);
  if constexpr (IL) {
#pragma unroll
    for (int e = 0; e < E; e += 8) {
      float4 cs = make_float4(1.f, 1.f, 1.f, 1.f), sn = make_float4(0.f, 0.f, 0.f, 0.f);
      if (turned) {
        cs = *reinterpret_cast<const float4*>(tab + (c * E + e) / 2);
        sn = *reinterpret_cast<const float4*>(tab + half + (c * E + e) / 2);
      }
      const float cc[4] = {cs.x, cs.y, cs.z, cs.w}, ss[4] = {sn.x, sn.y, sn.z, sn.w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float u = x[e + 2 * j], v = x[e + 2 * j + 1];
        float h0, l0, h1, l1;
        two_prod(h0, l0, u, cc[j]);
        two_prod_add(h0, l0, -v, ss[j]);
        two_prod(h1, l1, u, ss[j]);
        two_prod_add(h1, l1, v, cc[j]);
        x[e + 2 * j] = h0, l[e + 2 * j] = l0;
        x[e + 2 * j + 1] = h1, l[e + 2 * j + 1] = l1;
      }
    }
  } else {
    const int src = lane + (c * E < a.rot ? (second ? -half / E : half / E) : 0);
    const int first = second ? c * E - half : c * E;
#pragma unroll
    for (int e = 0; e < E; e += 4) {
      float4 cs = make_float4(1.f, 1.f, 1.f, 1.f), sn = make_float4(0.f, 0.f, 0.f, 0.f);
      if (turned) {
        cs = *reinterpret_cast<const float4*>(tab + first + e);
        sn = *reinterpret_cast<const float4*>(tab + half + first + e);
      }
      const float cc[4] = {cs.x, cs.y, cs.z, cs.w}, ss[4] = {sn.x, sn.y, sn.z, sn.w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float other = __shfl_sync(0xffffffffu, x[e + j], src);
        float hh, ll;
        two_prod(hh, ll, x[e + j], cc[j]);
        two_prod_add(hh, ll, second ? other : -other, ss[j]);
        x[e + j] = hh, l[e + j] = ll;
      }
    }
  }
  // the leading part: multiples of 2^(ex - 15), ex the exponent of the row's largest value
  float mx = 0.f;
#pragma unroll
  for (int e = 0; e < E; ++e) mx = fmaxf(mx, fabsf(x[e]));
#pragma unroll
  for (int off = 1; off < LPR; off <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, off));
  const int ex = max(-118, min(118, (int)(__float_as_uint(mx) >> 23) - 127));
  const float big = __uint_as_float((uint32_t)(127 + ex + 8) << 23 | 0x400000u);  // 1.5 2^(ex + 8)
#pragma unroll
  for (int e = 0; e < E; ++e) {
    const float sign = a.signs[c * E + e];
    const float lead = __fsub_rn(__fadd_rn(x[e], big), big);
    l[e] = sign * __fadd_rn(__fsub_rn(x[e], lead), l[e]);
    x[e] = sign * lead;
  }
  butterflies<D>(x, c);
  butterflies<D>(l, c);
  // times 1 / sqrt(D), as a sum of two FP32
  constexpr double inv = D == 64 ? 0.125 : D == 128 ? 0.08838834764831845 : 0.0625;
  constexpr float i0 = (float)inv, i1 = (float)(inv - (double)(float)inv);
#pragma unroll
  for (int e = 0; e < E; ++e) {
    const float p = __fmul_rn(x[e], i0), pe = __fmaf_rn(x[e], i0, -p);
    x[e] = __fadd_rn(p, __fadd_rn(__fmaf_rn(x[e], i1, pe), __fmul_rn(l[e], i0)));
  }
  quantise<BITS, GS>(x, ok ? draft_row(a.lv, PKV_KIND_K, row, slot, h) : nullptr,
                     ok ? draft_row(a.lv, PKV_KIND_KMETA, row, slot, h) : nullptr, c, ok);
}

template <int D, int BITS, int GS>
__device__ __forceinline__ void pack_values(const RotatedWriteArgs& a, int64_t r, bool live) {
  const int c = (threadIdx.x & 31) % (D / E);
  const int i = (int)(r / a.lv.hkv), h = (int)(r - (int64_t)i * a.lv.hkv);
  float x[E];
  load16(a.v + (int64_t)i * a.v_tok + h * a.v_head + c * E, x);
  const int32_t pos = a.positions[i], row = a.rows[i], slot = a.slots[i];
  const bool ok = live && pos >= 0 && pos < a.n_pos && place_ok(a.lv, row, slot);
  quantise<BITS, GS>(x, ok ? draft_row(a.lv, PKV_KIND_V, row, slot, h) : nullptr,
                     ok ? draft_row(a.lv, PKV_KIND_VMETA, row, slot, h) : nullptr, c, ok);
}

template <int D, bool IL, int KBITS, int VBITS, int GS>
__global__ void __launch_bounds__(256) rotated_pack_kernel(const __grid_constant__ Params P) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  constexpr int RPW = 32 / (D / E);  // rows a warp
  int64_t u = (int64_t)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5);
  if (u < 2 * P.pack_units) {
    const bool values = u >= P.pack_units;
    const int64_t r = (values ? u - P.pack_units : u) * RPW + (threadIdx.x & 31) / (D / E);
    const bool live = r < (int64_t)P.a.n * P.a.lv.hkv;
    if (values)
      pack_values<D, VBITS, GS>(P.a, live ? r : 0, live);
    else
      pack_keys<D, IL, KBITS, GS>(P.a, live ? r : 0, live);
    return;
  }
  u -= 2 * P.pack_units;
  const int64_t i = u / P.per_token;
  if (i >= P.a.n || P.a.Hq == 0) return;
  copy_heads<D, IL, true>(P.a, (int)i, kQueries, (int)(u - i * P.per_token) * kLoads * (256 / D));
}

template <int D, bool IL>
cudaError_t launch_di(const RotatedWriteArgs& a) {
  Params P;
  P.a = a;
  constexpr int per_warp = kLoads * (256 / D);
  const int q_units = (a.Hq + per_warp - 1) / per_warp;
  int64_t units;
  void (*kern)(Params);
  if (a.fmt == PKV_FMT_BF16) {
    P.pack_units = 0;
    P.kv_units = (a.lv.hkv + per_warp - 1) / per_warp;
    P.per_token = 2 * P.kv_units + q_units;
    units = (int64_t)a.n * P.per_token;
    kern = a.k_norm || a.q_norm ? rotated_write_kernel<D, IL, true> : rotated_write_kernel<D, IL, false>;
  } else {
    constexpr int RPW = 32 / (D / E);
    P.pack_units = ((int64_t)a.n * a.lv.hkv + RPW - 1) / RPW;
    P.kv_units = 0;
    P.per_token = q_units > 0 ? q_units : 1;
    units = 2 * P.pack_units + (int64_t)a.n * q_units;
    if (a.fmt == PKV_FMT_K4V4)
      kern = D >= 128 && a.group == kGroupWide ? rotated_pack_kernel<D, IL, 4, 4, (D >= 128 ? kGroupWide : kGroup)>
                                               : rotated_pack_kernel<D, IL, 4, 4, kGroup>;
    else if (a.fmt == PKV_FMT_K8V4)
      kern = rotated_pack_kernel<D, IL, 8, 4, kGroup>;
    else
      kern = rotated_pack_kernel<D, IL, 8, 8, kGroup>;
  }
  // a step's few tokens spread over the SMs, one warp per CTA
  const int threads = units < 2048 ? 32 : 256;
  const dim3 grid((unsigned)((units * 32 + threads - 1) / threads));
  static std::atomic<uint64_t> none{0};
  return tc_launch(kern, grid, threads, (size_t)0, a.stream, P, 0, &none);
}

}  // namespace

int rotated_write_units(int hkv, int Hq) { return 2 * hkv + Hq; }  // of any head_dim, packed or not, at most

cudaError_t launch_rotated_write(const RotatedWriteArgs& a) {
  switch (a.D) {
    case 64: return a.interleaved ? launch_di<64, true>(a) : launch_di<64, false>(a);
    case 128: return a.interleaved ? launch_di<128, true>(a) : launch_di<128, false>(a);
    default: return a.interleaved ? launch_di<256, true>(a) : launch_di<256, false>(a);
  }
}

}  // namespace pkv
