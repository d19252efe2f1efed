// tree_attn.cu — attention of drafted token trees: the merge of split units, and the launch.
// The attention kernels are described in tree_attn.cuh.
#include "tree_attn.cuh"

namespace pkv {
namespace tree {
namespace {

// A sum is below 2^kSlack times 2^25 tokens: under this the weights sum to less than 1, so that the
// values' weighted sum is no larger than they are.
constexpr float kWeight = 5.8207660913467407e-11f;  // 2^-34

// Merge of the records of split units, in order: a record's output counts by exp2(m) times its sum.  A
// warp takes 4 V columns of 32 rows, a lane a row of them.  Also the zero rows of unused or bad
// sequences.  U records are in flight: few units over many CTAs leave many records each, whose latency
// counts (U = 16, V = 1: 8 units with 19 records 26.9 us a call against 28.6), many units many warps
// (U = 8, V = 2: 128 units of 128 rows 185 us against 191).
template <int D, int U, int V>
__global__ void __launch_bounds__(256) tree_merge_kernel(const __grid_constant__ Params P, int row_blocks) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  constexpr int C = D / (4 * V);  // groups of columns
  const int lane = threadIdx.x & 31;
  const int64_t item = (int64_t)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5);
  const int c = (int)(item % C), rb = (int)(item / C % row_blocks);
  const int64_t unit = item / C / row_blocks;  // (sequence, kv head, group of rows)
  if (unit >= (int64_t)P.a.B * P.a.lv.hkv * P.n_rt) return;
  const int rt = (int)(unit % P.n_rt), kvh = (int)(unit / P.n_rt % P.a.lv.hkv), b = (int)(unit / P.n_rt / P.a.lv.hkv);
  const int2 meta = P.meta[unit];  // (garbage where the length is 0)
  bool bad;
  const int32_t len = draft_ctx(P.a.ctx[b], (int64_t)P.a.max_blocks * kBlockTokens, P.a.n_q, &bad);
  const int rr = rb * 32 + lane, r = rt * P.tile_rows + rr;
  const bool mine = rr < P.tile_rows && r < P.rows;
  float o[4 * V] = {};
  float inv = 0.f;
  if (len == 0) {
    if (bad && kvh == 0 && rt == 0 && rb == 0 && c == 0 && lane == 0) atomicOr(P.a.lv.err, ERR_CTX);
  } else {
    if (meta.x < 0) return;
    if (mine) {
      const int n = meta.y - meta.x + 1;
      // records: the first in its CTA's second slot, then the first slot of every later CTA
      auto slot = [&](int k) { return 2 * (int64_t)(meta.x + k) + (k == 0 ? 1 : 0); };
      float m = kNoMax, sum = 0.f;
      for (int k0 = 0; k0 < n; k0 += U) {
        float2 ml[U];
        float4 v[U][V];
#pragma unroll
        for (int k = 0; k < U; ++k) {
          ml[k] = make_float2(kNoMax, 0.f);
#pragma unroll
          for (int e = 0; e < V; ++e) v[k][e] = make_float4(0.f, 0.f, 0.f, 0.f);
          if (k0 + k < n) {
            const int64_t s = slot(k0 + k);
            ml[k] = P.ml[s * P.rec_rows + rr];
            const float4* acc = reinterpret_cast<const float4*>(P.acc) + (s * (D / 4) + V * c) * P.rec_rows + rr;
#pragma unroll
            for (int e = 0; e < V; ++e) v[k][e] = acc[e * P.rec_rows];
          }
        }
        float top = m;
#pragma unroll
        for (int k = 0; k < U; ++k) top = fmaxf(top, ml[k].x);
        const float f = ex2(m - top);
        m = top;
        sum *= f;
#pragma unroll
        for (int e = 0; e < 4 * V; ++e) o[e] *= f;
#pragma unroll
        for (int k = 0; k < U; ++k) {
          const float w = ex2(ml[k].x - m) * ml[k].y * kWeight;
          sum += w;
#pragma unroll
          for (int e = 0; e < V; ++e) {
            o[4 * e] = fmaf(w, v[k][e].x, o[4 * e]);
            o[4 * e + 1] = fmaf(w, v[k][e].y, o[4 * e + 1]);
            o[4 * e + 2] = fmaf(w, v[k][e].z, o[4 * e + 2]);
            o[4 * e + 3] = fmaf(w, v[k][e].w, o[4 * e + 3]);
          }
        }
      }
      inv = sum > 0.f ? 1.f / sum : 0.f;
    }
  }
  if (!mine) return;
  const int i = r / P.G, g = r - i * P.G;
  uint16_t* out = P.a.out + (((int64_t)b * P.a.n_q + i) * P.a.Hq + kvh * P.G + g) * D + 4 * V * c;
#pragma unroll
  for (int e = 0; e < V; ++e)
    reinterpret_cast<uint2*>(out)[e] =
        make_uint2(bf2(o[4 * e] * inv, o[4 * e + 1] * inv), bf2(o[4 * e + 2] * inv, o[4 * e + 3] * inv));
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

// Launched with programmatic dependence, as tc_launch does, with a second argument.
template <int D>
cudaError_t merge(const Params& P) {
  const int row_blocks = (P.rec_rows + 31) / 32;
  const int64_t units = (int64_t)P.a.B * P.a.lv.hkv * P.n_rt;
  const bool many = P.a.ctas >= 4 * units;  // records a unit
  const int64_t warps = units * row_blocks * (many ? D / 4 : D / 8);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((warps + 7) / 8));
  cfg.blockDim = dim3(256);
  cfg.stream = P.a.stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, many ? tree_merge_kernel<D, 16, 1> : tree_merge_kernel<D, 8, 2>, P, row_blocks);
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
  P.cols = a.ctas >= a.lv.hkv ? a.lv.hkv : 1;
  P.col_ctas = a.ctas / P.cols;
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
