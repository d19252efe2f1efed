// tree_attn.cu — attention of drafted token trees: the merge of split units, and the launch.
// The attention kernels are described in tree_attn.cuh.
#include "tree_attn.cuh"

namespace pkv {
namespace tree {
namespace {

// Merge of a row's records, one warp per row, in order.  Also the zero rows of unused or bad
// sequences.
template <int D>
__global__ void __launch_bounds__(256) tree_merge_kernel(const __grid_constant__ Params P) {
  constexpr int V = D / 32;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int lane = threadIdx.x & 31;
  const int64_t row = (int64_t)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5);  // (b, i, h)
  if (row >= (int64_t)P.a.B * P.a.n_q * P.a.Hq) return;
  const int h = (int)(row % P.a.Hq), i = (int)(row / P.a.Hq % P.a.n_q), b = (int)(row / P.a.Hq / P.a.n_q);
  const int kvh = h / P.G, r = i * P.G + h % P.G;
  const int64_t unit = ((int64_t)b * P.a.lv.hkv + kvh) * P.n_rt + r / P.tile_rows;
  const int2 meta = P.meta[unit];  // (garbage where the length is 0)
  bool bad;
  const int32_t len = draft_ctx(P.a.ctx[b], (int64_t)P.a.max_blocks * kBlockTokens, P.a.n_q, &bad);
  uint16_t* out = P.a.out + row * D + lane * V;
  float o[V];
#pragma unroll
  for (int e = 0; e < V; ++e) o[e] = 0.f;
  float inv = 0.f;
  if (len == 0) {
    if (bad && i == 0 && h == 0 && lane == 0) atomicOr(P.a.lv.err, ERR_CTX);
  } else {
    if (meta.x < 0) return;
    const int n = meta.y - meta.x + 1, rr = r % P.tile_rows;
    // records: the first in its CTA's second slot, then the first slot of every later CTA
    auto at = [&](int k) { return (2 * (int64_t)(meta.x + k) + (k == 0 ? 1 : 0)) * P.rec_rows + rr; };
    constexpr int U = D == 256 ? 4 : 8;  // records in flight
    float v[U][V];
    float2 ml[U];
    auto load = [&](int k0) {
#pragma unroll
      for (int k = 0; k < U; ++k)
        if (k0 + k < n) {
          const int64_t a = at(k0 + k);
          ml[k] = P.ml[a];
          const float* src = P.acc + a * D + lane * V;
          if constexpr (V == 2) {
            const float2 x = *reinterpret_cast<const float2*>(src);
            v[k][0] = x.x, v[k][1] = x.y;
          } else {
#pragma unroll
            for (int e = 0; e < V; e += 4) {
              const float4 x = *reinterpret_cast<const float4*>(src + e);
              v[k][e] = x.x, v[k][e + 1] = x.y, v[k][e + 2] = x.z, v[k][e + 3] = x.w;
            }
          }
        }
    };
    load(0);
    float M = kNoMax;
    for (int k = lane; k < n; k += 32) M = fmaxf(M, P.ml[at(k)].x);
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, off));
    float sum = 0.f;
    for (int k0 = 0; k0 < n; k0 += U) {
      if (k0 > 0) load(k0);
#pragma unroll
      for (int k = 0; k < U; ++k)
        if (k0 + k < n) {
          const float w = ex2(ml[k].x - M);
          sum = fmaf(w, ml[k].y, sum);
#pragma unroll
          for (int e = 0; e < V; ++e) o[e] = fmaf(w, v[k][e], o[e]);
        }
    }
    inv = sum > 0.f ? 1.f / sum : 0.f;
  }
  if constexpr (V == 2) {
    *reinterpret_cast<uint32_t*>(out) = bf2(o[0] * inv, o[1] * inv);
  } else if constexpr (V == 4) {
    *reinterpret_cast<uint2*>(out) = make_uint2(bf2(o[0] * inv, o[1] * inv), bf2(o[2] * inv, o[3] * inv));
  } else {
    *reinterpret_cast<uint4*>(out) = make_uint4(bf2(o[0] * inv, o[1] * inv), bf2(o[2] * inv, o[3] * inv),
                                                bf2(o[4] * inv, o[5] * inv), bf2(o[6] * inv, o[7] * inv));
  }
}

// How a call is laid out: rows of a (sequence, kv head), 128 or 256 of them a unit.
struct Geometry {
  int G, rows, mode, tile_rows, n_rt, rec_rows;
  size_t ml, acc, total;  // workspace offsets
};

Geometry geometry(int D, int hkv, int B, int n_q, int Hq, int ctas) {
  Geometry g;
  g.G = Hq / hkv;
  g.rows = n_q * g.G;
  g.mode = D == 256 ? kSolo : g.rows > kRows ? kPair : kTurns;
  g.tile_rows = g.mode == kPair ? 2 * kRows : kRows;
  g.n_rt = (g.rows + g.tile_rows - 1) / g.tile_rows;
  g.rec_rows = g.rows < g.tile_rows ? g.rows : g.tile_rows;
  auto up = [](size_t x) { return (x + 255) / 256 * 256; };
  const size_t records = 2 * (size_t)ctas * g.rec_rows;
  g.ml = up(sizeof(int2) * (size_t)B * hkv * g.n_rt);
  g.acc = g.ml + up(sizeof(float2) * records);
  g.total = g.acc + sizeof(float) * records * D;
  return g;
}

template <int D>
cudaError_t merge(const Params& P) {
  static std::atomic<uint64_t> none{0};
  const int64_t rows = (int64_t)P.a.B * P.a.n_q * P.a.Hq;
  return tc_launch(tree_merge_kernel<D>, dim3((unsigned)((rows + 7) / 8)), 256, (size_t)0, P.a.stream, P, P.a.device, &none);
}

}  // namespace
}  // namespace tree

size_t tree_attn_workspace(int D, int hkv, int B, int n_q, int Hq, int ctas) {
  return tree::geometry(D, hkv, B, n_q, Hq, ctas).total;
}

cudaError_t launch_tree_attn(const TreeAttnArgs& a) {
  const tree::Geometry g = tree::geometry(a.D, a.lv.hkv, a.B, a.n_q, a.Hq, a.ctas);
  tree::Params P;
  P.a = a;
  P.G = g.G;
  P.rows = g.rows;
  P.tile_rows = g.tile_rows;
  P.n_rt = g.n_rt;
  P.rec_rows = g.rec_rows;
  P.words = (a.n_q + 31) / 32;
  P.group_log = a.group == kGroupWide ? 6 : 5;
  P.meta = reinterpret_cast<int2*>(a.ws);
  P.ml = reinterpret_cast<float2*>((uint8_t*)a.ws + g.ml);
  P.acc = reinterpret_cast<float*>((uint8_t*)a.ws + g.acc);
  cudaError_t e;
  switch (a.fmt) {
    case PKV_FMT_BF16: e = launch_tree_bf16(P, g.mode); break;
    case PKV_FMT_K4V4: e = launch_tree_k4v4(P, g.mode); break;
    case PKV_FMT_K8V4: e = launch_tree_k8v4(P, g.mode); break;
    default: e = launch_tree_k8v8(P, g.mode); break;
  }
  if (e != cudaSuccess) return e;
  return a.D == 64 ? tree::merge<64>(P) : a.D == 128 ? tree::merge<128>(P) : tree::merge<256>(P);
}

}  // namespace pkv
