// Launches of dsa_tree_attn: the attention kernel (tree_kernel.cuh) and the merge of split row tiles.
#include "tree_kernel.cuh"

namespace dsa {
namespace {

// Merges the chunks of each split row: out = sum_j 2^(m_j - M) o_j / sum_j 2^(m_j - M) l_j.  A CTA takes eight
// rows, a thread one row, four values and every G-th chunk, B chunks' loads in flight.  G = 16 (and 32 value columns
// per CTA) for launches of few row tiles, which have many chunks each, G = 1 (and 128) for others: one token over 2K, 33
// chunks: 17.3 us the call with G = 1, 14.7 with 16; 8 row tiles of 9 chunks: 91 with 1, 95 to 97 with 2 and 4.
template <int G>
__global__ void __launch_bounds__(G > 1 ? 64 * G : 256) tree_combine_kernel(const TreeAttnParams p, const TreePlan pl) {
  constexpr int B = G > 1 ? 4 : 8, T = G > 1 ? 64 : 256;  // threads that share out rows and columns
  __shared__ float2 part_ml[G][T];
  __shared__ float4 part_o[G][T];
  const int rows = p.q_per_seq * p.H, at = threadIdx.x % T, g = threadIdx.x / T;
  const int seq = blockIdx.y, row = blockIdx.x * 8 + (at & 7), c4 = blockIdx.z * (T / 8) + (at >> 3);
  int ctx, fresh, len;
  seq_facts(p, seq, ctx, fresh, len);  // (the lengths were there before the attention kernel began)
  pdl_wait();
  const int live = live_row_tiles(p, fresh);
  const int rt = row / kRows, r = row - rt * kRows;
  const int plan = pl.head[0], nt = (len + kKeys - 1) / kKeys, base = pl.head[1 + seq];
  int chunks, slot0, slot1, stride;  // the unit's partials: slot0 holds the first, slot1, slot1 + stride, ... the others
  if (plan > 0) {
    chunks = nt ? (nt + plan - 1) / plan : 1;
    slot0 = base + rt, slot1 = slot0 + live, stride = live;
    if (rt >= live || chunks == 1) return;  // written by the attention kernel
  } else {
    // tiles [begin, begin + nt) over spans of W: the last item of the first span, the first ones of the others
    const int W = -plan, begin = base + rt * nt, first = begin / W;
    chunks = rt < live && nt ? (begin + nt - 1) / W - first + 1 : 0;
    slot0 = 2 * first + 1, slot1 = 2 * (first + 1), stride = 2;
    if (chunks == 1) return;
  }
  if (row / p.H >= fresh) chunks = 0;  // a padding node: zeros
  if (row >= rows) chunks = 0;
  float M = -INFINITY, l = 0.f;
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
  auto add = [&](const float2* ml, const float4* v, int n) {  // n partial results to (M, l, o)
    float Mb = M;
    for (int k = 0; k < n; ++k) Mb = fmaxf(Mb, ml[k].x);
    const float mu = Mb == -INFINITY ? 0.f : Mb;
    const float f = exp2f(M - mu);
    l *= f;
    o.x *= f, o.y *= f, o.z *= f, o.w *= f;
    for (int k = 0; k < n; ++k) {
      const float w = exp2f(ml[k].x - mu);
      l += w * ml[k].y;
      o.x += w * v[k].x, o.y += w * v[k].y, o.z += w * v[k].z, o.w += w * v[k].w;
    }
    M = Mb;
  };
  for (int j0 = g; j0 < chunks; j0 += G * B) {
    float2 ml[B];
    float4 v[B];
#pragma unroll
    for (int k = 0; k < B; ++k) {
      const int j = j0 + k * G;
      const int64_t s = j == 0 ? slot0 : slot1 + (j - 1) * stride;
      const bool in = j < chunks;
      ml[k] = in ? pl.part_ml[(s * 2 + (c4 >> 6)) * kRows + r] : make_float2(-INFINITY, 0.f);
      v[k] = in ? pl.part_o[(s * (kDv / 4) + c4) * kRows + r] : make_float4(0.f, 0.f, 0.f, 0.f);
    }
    add(ml, v, B);
  }
  if (G > 1) {
    if (g > 0) part_ml[g][at] = make_float2(M, l), part_o[g][at] = o;
    __syncthreads();
  }
  if (g > 0 || row >= rows) return;
#pragma unroll
  for (int k = 1; k < G; ++k) add(&part_ml[k][at], &part_o[k][at], 1);
  const int64_t to = (int64_t)seq * rows + row;
  const float inv = l == 0.f ? 0.f : 1.f / l;
  *reinterpret_cast<uint2*>(p.out + to * kDv + 4 * c4) =
      make_uint2(pack_bf16(o.x * inv, o.y * inv), pack_bf16(o.z * inv, o.w * inv));
  if (p.lse && c4 == 0) p.lse[to] = l == 0.f ? -INFINITY : (M + log2f(l)) * kLn2;
}

__global__ void tree_nothing_kernel(const TreeAttnParams p, int64_t rows) {
  const int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
  if (i < rows * (kDv / 8)) reinterpret_cast<uint4*>(p.out)[i] = make_uint4(0u, 0u, 0u, 0u);
  if (p.lse && i < rows) p.lse[i] = -INFINITY;
}

constexpr int kPairs = 76;  // of CTAs: two of the 152 SMs each

// A launch of more units than the lists of items hold has no plan: pairs take whole units in turn.  Its many rounds of the
// grid are full enough where the contexts are alike; a single long one among short ones is walked by one pair.
TreePlan plan_of(const TreeAttnParams& p) {
  TreePlan pl = {};
  pl.row_tiles = (p.q_per_seq * p.H + kRows - 1) / kRows;
  pl.units = p.n_seq * pl.row_tiles;
  pl.cap = pl.units <= kMaxItems * kPairs ? kSlotsPerPair * kPairs : 0;
  pl.grid = pl.cap ? kPairs : (pl.units < kPairs ? pl.units : kPairs);
  return pl;
}

bool long_contexts(const TreeAttnParams& p) { return p.L > kLong * kKeys; }
constexpr size_t kPartBytes = (size_t)kRows * (2 * sizeof(float2) + kDv * sizeof(float));     // of a partial result
constexpr size_t kSumBytes = (size_t)kRows * (2 * sizeof(float2) + kDv / 2 * sizeof(float));  // a CTA's sums

size_t head_bytes(const TreeAttnParams& p) { return align_up((size_t)(1 + p.n_seq) * sizeof(int), 256); }

template <int FMT, bool LONG>
cudaError_t launch_form(const TreeAttnParams& p, TreePlan pl, void* ws, cudaStream_t stream) {
  using C = Cfg<FMT>;
  CUtensorMap tm;
  cudaError_t e = cache_map<FMT>(&tm, p);
  if (e != cudaSuccess) return e;
  uint8_t* w = reinterpret_cast<uint8_t*>(ws);
  if (pl.cap) {
    pl.head = reinterpret_cast<int*>(w);
    w += head_bytes(p);
    pl.part_ml = reinterpret_cast<float2*>(w);
    pl.part_o = reinterpret_cast<float4*>(w + (size_t)pl.cap * 2 * kRows * sizeof(float2));
    w += pl.cap * kPartBytes;
  }
  if (LONG) {
    pl.sum_ml = reinterpret_cast<float2*>(w);
    pl.sum_o = reinterpret_cast<float4*>(w + (size_t)2 * pl.grid * 2 * kRows * sizeof(float2));
  }
  auto kern = tree_attn_kernel<FMT, LONG>;
  static std::atomic<uint64_t> allowed{0};
  e = allow_smem_once(&allowed, reinterpret_cast<const void*>(kern), C::SMEM);
  if (e != cudaSuccess) return e;
  e = launch_kernel(kern, dim3(2 * pl.grid), dim3(C::THREADS), C::SMEM, stream, false, tm, p, pl);
  if (e != cudaSuccess || !pl.cap) return e;
  const unsigned rows8 = (p.q_per_seq * p.H + 7) / 8;
  if (16 * pl.units <= kPairs)
    return launch_kernel(tree_combine_kernel<16>, dim3(rows8, p.n_seq, 16), dim3(1024), 0, stream, true, p, pl);
  return launch_kernel(tree_combine_kernel<1>, dim3(rows8, p.n_seq, 4), dim3(256), 0, stream, true, p, pl);
}

template <int FMT>
cudaError_t launch_fmt(const TreeAttnParams& p, const TreePlan& pl, void* ws, cudaStream_t stream) {
  return long_contexts(p) ? launch_form<FMT, true>(p, pl, ws, stream) : launch_form<FMT, false>(p, pl, ws, stream);
}

}  // namespace

size_t tree_attn_ws_bytes(const TreeAttnParams& p) {
  const TreePlan pl = plan_of(p);
  if (p.L == 0) return 0;
  return (pl.cap ? head_bytes(p) + pl.cap * kPartBytes : 0) + (long_contexts(p) ? 2 * pl.grid * kSumBytes : 0);
}

cudaError_t launch_tree_attn(const TreeAttnParams& p, void* ws, cudaStream_t stream) {
  const int64_t rows = (int64_t)p.n_seq * p.q_per_seq * p.H;
  if (p.L == 0) {
    const int64_t n = rows * (kDv / 8);
    return launch_kernel(tree_nothing_kernel, dim3((unsigned)((n + 255) / 256)), dim3(256), 0, stream, false, p, rows);
  }
  const TreePlan pl = plan_of(p);
  if (!p.kv_fp8) return launch_fmt<kBf16>(p, pl, ws, stream);
  return p.nsc == 1 ? launch_fmt<kFp8Row>(p, pl, ws, stream) : launch_fmt<kFp8Tile>(p, pl, ws, stream);
}

}  // namespace dsa
