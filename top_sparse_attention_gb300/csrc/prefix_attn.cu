// Attention over a latent cache for groups of sequences that share a prefix (dsa_prefix_attn): out and lse are those of
// dsa_tree_attn, whose kernel this is (tree_kernel.cuh), with other items of work.
//
// A group's prefix is taken once for the rows (heads of nodes) of all of its sequences, packed in 128s as the queries lie in
// memory, and what follows it per sequence:
//   softmax over both parts = (sum_j 2^(m_j - M) o_j) / (sum_j 2^(m_j - M) l_j)  over the partial results j of a row.
// With 16 rows a sequence that is an eighth of the tiles that the sequences alone would take over the prefix (a tile of 128
// rows costs the same however many of them are used), and its rows are read once instead of once per sequence.
//
// The shared part ends at a whole tile of 64 positions; the rest of the prefix is taken with the tails.  Units of work
// are the row tiles of the groups' prefixes, then those of the sequences' tails; laid end to end, each with a fixed cost
// (the fill and drain of the pipeline) before its tiles, they are cut into one span for each pair of CTAs.  prefix_plan_kernel writes
// each pair's list of items; prefix_merge_kernel finds a row's partial results from the same numbers.  No atomics: the
// results of a call repeat.
//
// Measured (device us): 64 sequences x 16 heads behind 32768 shared positions, E4M3 rows in a paged cache, tails of up to 512:
// 110, of which the attention 99 (1100 cycles of tensor cores in a tile of 2200; the sequences alone, with dsa_tree_attn, walk
// eight times the tiles); 48 sequences x 4 nodes behind three prefixes of up to 8192, tile scales: 138 (the tile-scale form's turns, see
// tree_kernel.cuh); four behind 1024, bf16: 17.7, of which the plan and the merge take about 3 each.  Bound as dsa_tree_attn.
#include "tree_kernel.cuh"

namespace dsa {
namespace {

struct PrefixParams {
  const int32_t* group_start;  // [n_groups + 1]
  const int32_t* n_shared;     // [n_groups]
  int n_groups, unit_cost;
};

// The plan, in the workspace.
struct Group {
  int lo, hi, lead, tiles;     // sequences [lo, hi), the one whose cache is read, tiles of the prefix taken once
  int first_unit, base;        // units, and cost, before its own
};
struct PrefixPlan {
  int* width;                  // [0]: of a span; [1]: the fixed cost of a unit
  Group* groups;               // [n_groups]
  int2* seqs;                  // [n_seq]: cost before a sequence's units, its group (-1: none)
  SharedItem* list;
  int2* list_place;            // [pairs]
};

constexpr int kPairs = 76;
constexpr int kMaxGroups = 4096, kMaxSeq = 4096;
constexpr int kPlanThreads = 1024;
// Fill, query rows and partial results of a unit, in tiles: about 10 us, of tiles of 1.2 us (tile scales: 2.6).  Device us with 2, 4,
// 8 and 16, tails of up to 256 to 1500 positions:
//                                               bf16                  row scales            tile scales
//   64 x 16 rows behind 32768 positions         125, 111, 115, 125    160, 129, 112, 121    215, 205, 214, 236
//   32 x 128 rows behind two of up to 16384     180, 154, 137, 145    201, 170, 136, 141    286, 248, 255, 273
//   48 x 64 rows behind three of up to 8192      87,  82,  85,  95    100,  89,  84,  93    142, 138, 149, 169
//   256 x 16 rows behind 32 of up to 1024        74,  77,  81,  82     94,  84,  87,  87    106, 115, 126, 126
// and the same for 16 x 16 rows behind 4096 (37, 44, 47) and 8 x 128 behind 2048 (36, 41, 46), where a CTA has one tile or two and
// the cost is taken as one tile at most (prefix_plan_kernel).
constexpr int kUnitCost = 8, kUnitCostTiled = 4;

__host__ __device__ __forceinline__ int row_tiles(int rows) { return (rows + kRows - 1) / kRows; }
__device__ __forceinline__ int up8(int x) { return (x + 7) & ~7; }

// A sequence's tail: tiles [from, from + tiles), for `live` row tiles.
struct Tail {
  int ctx, fresh, len, live, from, tiles;
};
__device__ __forceinline__ Tail tail_of(const TreeAttnParams& p, int seq, int from) {
  Tail t;
  seq_facts(p, seq, t.ctx, t.fresh, t.len);
  t.live = live_row_tiles(p, t.fresh);
  t.from = from;
  t.tiles = t.live ? max((t.len + kKeys - 1) / kKeys - from, 0) : 0;
  return t;
}
__device__ __forceinline__ int unit_cost(int tiles, int fixed) { return tiles ? tiles + fixed : 0; }  // (all of them: below 2^31)

// First row of partial results of a unit (rounded up to eights, the groups' before the sequences'), without the spans cut
// before it: 128 rows are kept for the part behind each cut.
__device__ __forceinline__ int group_slot(const TreeAttnParams& p, const Group& g, int gi, int rt) {
  return up8(g.lo * p.q_per_seq * p.H) + 8 * gi + kRows * rt;
}
__device__ __forceinline__ int tail_slot(const TreeAttnParams& p, int n_groups, int seq, int rt) {
  const int rows = p.q_per_seq * p.H;
  return up8(p.n_seq * rows) + 8 * (n_groups + 1) + seq * up8(rows) + kRows * rt;
}

// Running sums of two numbers over the CTA's threads; `all` gets the wholes.
__device__ int2 block_scan(int2 x, int2* warps, int2& all) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int2 incl = x;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int a = __shfl_up_sync(0xffffffffu, incl.x, o), b = __shfl_up_sync(0xffffffffu, incl.y, o);
    if (lane >= o) incl.x += a, incl.y += b;
  }
  __syncthreads();  // (the last sums have been read)
  if (lane == 31) warps[warp] = incl;
  __syncthreads();
  int2 mine = warps[lane], run = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int a = __shfl_up_sync(0xffffffffu, run.x, o), b = __shfl_up_sync(0xffffffffu, run.y, o);
    if (lane >= o) run.x += a, run.y += b;
  }
  all = make_int2(__shfl_sync(0xffffffffu, run.x, 31), __shfl_sync(0xffffffffu, run.y, 31));
  const int bx = __shfl_sync(0xffffffffu, run.x - mine.x, warp), by = __shfl_sync(0xffffffffu, run.y - mine.y, warp);
  return make_int2(bx + incl.x - x.x, by + incl.y - x.y);
}

// The last of n entries whose key is at most x (key(0) <= x).
template <class Key>
__device__ __forceinline__ int last_at_most(int n, int x, Key&& key) {
  int lo = 0, hi = n - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (key(mid) <= x) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

// What is searched lies in shared memory: the groups, and per sequence its cost before, its tail's tiles and its group.
struct PlanSmem {
  Group* groups;
  int* base;
  int* tiles;
  int* group_of;
};
size_t plan_smem(int n_groups, int n_seq) { return sizeof(Group) * n_groups + 3 * sizeof(int) * n_seq; }

__global__ void __launch_bounds__(kPlanThreads) prefix_plan_kernel(const TreeAttnParams p, const PrefixParams pp, const PrefixPlan pl) {
  extern __shared__ int plan_s[];
  __shared__ int2 warps[32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int rows = p.q_per_seq * p.H;
  PlanSmem sm;
  sm.groups = reinterpret_cast<Group*>(plan_s);
  sm.base = reinterpret_cast<int*>(sm.groups + pp.n_groups);
  sm.tiles = sm.base + p.n_seq;
  sm.group_of = sm.tiles + p.n_seq;

  // ---- the groups: a warp each
  bool disorder = false;  // group_start decreases: groups would overlap, and their units be more than there is room for
  for (int g = warp; g < pp.n_groups; g += kPlanThreads / 32) {
    const int lo = min(max(pp.group_start[g], 0), p.n_seq), end = min(max(pp.group_start[g + 1], 0), p.n_seq), hi = max(end, lo);
    disorder |= end < lo;
    int least = INT_MAX, lead = INT_MAX, members = 0;
    for (int s = lo + lane; s < hi; s += 32) {
      int ctx, fresh, len;
      seq_facts(p, s, ctx, fresh, len);
      if (fresh) least = min(least, ctx), lead = min(lead, s), ++members;  // (one without queries has no say)
    }
    const int shared = pp.n_shared[g];
    least = __reduce_min_sync(0xffffffffu, least);
    lead = __reduce_min_sync(0xffffffffu, lead);
    members = __reduce_add_sync(0xffffffffu, members);
    if (lane == 0) {
      Group x = {};
      x.lo = lo, x.hi = hi, x.lead = lead;
      x.tiles = members > 1 ? min(max(shared, 0), least) / kKeys : 0;
      sm.groups[g] = x;
    }
  }
  if (__syncthreads_or(disorder)) {  // nothing is shared
    if (tid == 0) record_error(p.err, DSA_DEVERR_INDEX_RANGE);
    for (int g = tid; g < pp.n_groups; g += kPlanThreads) sm.groups[g] = Group{};
    __syncthreads();
  }
  // ---- the sequences' groups and tails, and all tiles
  int2 sum = make_int2(0, 0), all;
  for (int s = tid; s < p.n_seq; s += kPlanThreads) {
    int g = -1;
    if (pp.n_groups > 0) {
      const int k = last_at_most(pp.n_groups, s, [&](int i) { return sm.groups[i].lo; });
      if (sm.groups[k].lo <= s && s < sm.groups[k].hi) g = k;
    }
    const Tail t = tail_of(p, s, g >= 0 ? sm.groups[g].tiles : 0);
    sm.group_of[s] = g;
    sm.tiles[s] = t.tiles;
    sm.base[s] = t.live;  // (until the costs are known)
    sum.x += t.tiles * t.live;
  }
  for (int g = tid; g < pp.n_groups; g += kPlanThreads) sum.x += sm.groups[g].tiles * row_tiles((sm.groups[g].hi - sm.groups[g].lo) * rows);
  block_scan(sum, warps, all);
  // A unit's fixed cost: its own where spans are long, nothing where there is less than a tile for each pair
  // (then the time is that of the longest item).
  const int fixed = min(all.x / (2 * kPairs), pp.unit_cost);
  // ---- the units' places: groups, then sequences
  int run = 0, units = 0;
  for (int g0 = 0; g0 < pp.n_groups; g0 += kPlanThreads) {
    const int g = g0 + tid;
    int2 c = make_int2(0, 0);
    if (g < pp.n_groups) {
      c.y = row_tiles((sm.groups[g].hi - sm.groups[g].lo) * rows);
      c.x = c.y * unit_cost(sm.groups[g].tiles, fixed);
    }
    const int2 before = block_scan(c, warps, all);
    if (g < pp.n_groups) {
      sm.groups[g].base = run + before.x, sm.groups[g].first_unit = units + before.y;
      pl.groups[g] = sm.groups[g];
    }
    run += all.x, units += all.y;
  }
  for (int s0 = 0; s0 < p.n_seq; s0 += kPlanThreads) {
    const int s = s0 + tid;
    int2 c = make_int2(0, 0);
    if (s < p.n_seq) c.x = sm.base[s] * unit_cost(sm.tiles[s], fixed);
    const int2 before = block_scan(c, warps, all);
    if (s < p.n_seq) {
      sm.base[s] = run + before.x;
      pl.seqs[s] = make_int2(run + before.x, sm.group_of[s]);
    }
    run += all.x;
  }
  const int W = max((int)(((long long)run + kPairs - 1) / kPairs), 1);
  if (tid == 0) pl.width[0] = W, pl.width[1] = fixed;
  __syncthreads();
  // ---- the pairs' lists: a warp each.  Entry of unit u in span k: u + k
  const int per_seq = row_tiles(rows);
  auto unit_at = [&](int x) {  // the unit that holds cost x
    if (x < sm.base[0]) {
      const Group g = sm.groups[last_at_most(pp.n_groups, x, [&](int i) { return sm.groups[i].base; })];
      return g.first_unit + (x - g.base) / unit_cost(g.tiles, fixed);
    }
    const int s = last_at_most(p.n_seq, x, [&](int i) { return sm.base[i]; });
    return units + s * per_seq + (x - sm.base[s]) / unit_cost(sm.tiles[s], fixed);
  };
  for (int k = warp; k < kPairs; k += kPlanThreads / 32) {
    const long long from = (long long)k * W;
    if (from >= run) {
      if (lane == 0) pl.list_place[k] = make_int2(0, 0);
      continue;
    }
    const int x0 = (int)from, x1 = (int)min(from + W, (long long)run);
    const int u0 = unit_at(x0), u1 = unit_at(x1 - 1);
    if (lane == 0) pl.list_place[k] = make_int2(u0 + k, u1 - u0 + 1);
    for (int u = u0 + lane; u <= u1; u += 32) {
      SharedItem it = {};
      int b = 0;  // cost before the unit
      int tiles = 0, from_tile = 0;
      if (u < units) {
        const int gi = last_at_most(pp.n_groups, u, [&](int i) { return sm.groups[i].first_unit; });
        const Group g = sm.groups[gi];
        const int rt = u - g.first_unit;
        tiles = g.tiles;
        b = g.base + rt * unit_cost(tiles, fixed);
        it.seq = g.lead;
        it.at = g.lo * rows + rt * kRows;
        it.nrows = min(kRows, (g.hi - g.lo) * rows - rt * kRows);
        it.ctx = it.len = tiles * kKeys;
        it.slot = group_slot(p, g, gi, rt);
      } else {
        const int s = (u - units) / per_seq, rt = (u - units) % per_seq, g = sm.group_of[s];
        const Tail t = tail_of(p, s, g >= 0 ? sm.groups[g].tiles : 0);
        tiles = rt < t.live ? t.tiles : 0;
        from_tile = t.from;
        b = sm.base[s] + rt * unit_cost(t.tiles, fixed);
        it.seq = s;
        it.row_lo = rt * kRows;
        it.at = s * rows + it.row_lo;
        it.nrows = min(kRows, rows - it.row_lo);
        it.ctx = t.ctx, it.fresh = t.fresh, it.len = t.len;
        it.slot = tail_slot(p, pp.n_groups, s, rt);
      }
      const int first = b + fixed;
      const int t0 = min(max(x0 - first, 0), tiles), t1 = min(max(x1 - first, 0), tiles);
      it.t0 = from_tile + t0, it.t1 = from_tile + max(t1, t0);
      // the parts of a unit behind its first one follow it, as many rows each
      it.slot += kRows * (b / W) + (k - first / W) * up8(it.nrows);
      pl.list[u + k] = it;
    }
  }
}

// Merges each row's partial results, those over the prefix and those over the tail.  A CTA takes eight rows, a thread one
// row, four values and every G-th part.
template <int G>
__global__ void __launch_bounds__(G > 1 ? 64 * G : 256) prefix_merge_kernel(const TreeAttnParams p, const PrefixParams pp, const PrefixPlan pl,
                                                                           const float4* part_o, const float2* part_ml) {
  constexpr int B = G > 1 ? 2 : 4, T = G > 1 ? 64 : 256;  // parts whose loads are in flight; threads that share out rows and columns
  __shared__ float2 sum_ml[G][T];
  __shared__ float4 sum_o[G][T];
  const int rows = p.q_per_seq * p.H, at = threadIdx.x % T, g = threadIdx.x / T;
  const int row = blockIdx.x * 8 + (at & 7), c4 = blockIdx.z * (T / 8) + (at >> 3);
  pdl_wait();
  int parts_a = 0, parts = 0, r_a = 0, r_b = 0, size_a = 0, size_b = 0;
  int slot_a = 0, slot_b = 0;
  if (row < p.n_seq * rows) {
    const int s = row / rows, in = row - s * rows;
    const int W = pl.width[0], fixed = pl.width[1];
    const int2 place = pl.seqs[s];
    const int gi = place.y;
    Group x = {};
    if (gi >= 0) x = pl.groups[gi];
    const Tail t = tail_of(p, s, x.tiles);
    if (in / p.H < t.fresh) {  // (a padding node: zeros)
      if (x.tiles > 0) {
        const int ra = (s - x.lo) * rows + in, rt = ra / kRows;
        const int b = x.base + rt * unit_cost(x.tiles, fixed);
        parts_a = (b + fixed + x.tiles - 1) / W - (b + fixed) / W + 1;
        r_a = ra - rt * kRows;
        size_a = up8(min(kRows, (x.hi - x.lo) * rows - rt * kRows));
        slot_a = group_slot(p, x, gi, rt) + kRows * (b / W);
      }
      parts = parts_a;
      if (t.tiles > 0) {
        const int rt = in / kRows;
        const int b = place.x + rt * unit_cost(t.tiles, fixed);
        parts += (b + fixed + t.tiles - 1) / W - (b + fixed) / W + 1;
        r_b = in - rt * kRows;
        size_b = up8(min(kRows, rows - rt * kRows));
        slot_b = tail_slot(p, pp.n_groups, s, rt) + kRows * (b / W);
      }
    }
  }
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
  for (int j0 = g; j0 < parts; j0 += G * B) {
    float2 ml[B];
    float4 v[B];
#pragma unroll
    for (int k = 0; k < B; ++k) {
      const int j = j0 + k * G;
      ml[k] = make_float2(-INFINITY, 0.f);
      v[k] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (j < parts) {
        const bool a = j < parts_a;
        const int size = a ? size_a : size_b, r = a ? r_a : r_b;
        const int64_t first = a ? slot_a + j * size : slot_b + (j - parts_a) * size;
        ml[k] = part_ml[first * 2 + (c4 >> 6) * size + r];
        v[k] = part_o[first * (kDv / 4) + c4 * size + r];
      }
    }
    add(ml, v, B);
  }
  if (G > 1) {
    if (g > 0) sum_ml[g][at] = make_float2(M, l), sum_o[g][at] = o;
    __syncthreads();
  }
  if (g > 0 || row >= p.n_seq * rows) return;
#pragma unroll
  for (int k = 1; k < G; ++k) add(&sum_ml[k][at], &sum_o[k][at], 1);
  const float inv = l == 0.f ? 0.f : 1.f / l;
  *reinterpret_cast<uint2*>(p.out + (int64_t)row * kDv + 4 * c4) =
      make_uint2(pack_bf16(o.x * inv, o.y * inv), pack_bf16(o.z * inv, o.w * inv));
  if (p.lse && c4 == 0) p.lse[row] = l == 0.f ? -INFINITY : (M + log2f(l)) * kLn2;
}

// ---- the workspace
constexpr size_t kSumBytes = (size_t)kRows * (2 * sizeof(float2) + kDv / 2 * sizeof(float));  // a CTA's sums of long walks

struct Layout {
  size_t width, groups, seqs, place, list, part_ml, part_o, sum, total;
};
Layout layout_of(const TreeAttnParams& p, int n_groups) {
  const int64_t rows = (int64_t)p.q_per_seq * p.H, all = rows * p.n_seq;
  const int64_t units = all / kRows + n_groups + 1 + (int64_t)p.n_seq * ((rows + kRows - 1) / kRows) + kPairs;
  const int64_t parts = (all + 7) / 8 * 8 + 8 * (n_groups + 2) + p.n_seq * ((rows + 7) / 8 * 8) + kRows * (kPairs + 1);
  Layout l;
  l.width = 0;
  l.groups = 256;
  l.seqs = align_up(l.groups + sizeof(Group) * n_groups, 256);
  l.place = align_up(l.seqs + sizeof(int2) * p.n_seq, 256);
  l.list = align_up(l.place + sizeof(int2) * kPairs, 256);
  l.part_ml = align_up(l.list + sizeof(SharedItem) * units, 256);
  l.part_o = align_up(l.part_ml + sizeof(float2) * 2 * parts, 256);
  l.sum = align_up(l.part_o + sizeof(float) * kDv * parts, 256);
  l.total = l.sum + (p.L > kLong * kKeys ? 2 * kPairs * kSumBytes : 0);
  return l;
}

template <int FMT, bool LONG>
cudaError_t launch_form(const TreeAttnParams& p, const PrefixParams& pp, void* ws, cudaStream_t stream) {
  using C = Cfg<FMT>;
  CUtensorMap tm;
  cudaError_t e = cache_map<FMT>(&tm, p);
  if (e != cudaSuccess) return e;
  const Layout l = layout_of(p, pp.n_groups);
  uint8_t* w = reinterpret_cast<uint8_t*>(ws);
  PrefixPlan plan;
  plan.width = reinterpret_cast<int*>(w + l.width);
  plan.groups = reinterpret_cast<Group*>(w + l.groups);
  plan.seqs = reinterpret_cast<int2*>(w + l.seqs);
  plan.list = reinterpret_cast<SharedItem*>(w + l.list);
  plan.list_place = reinterpret_cast<int2*>(w + l.place);
  TreePlan pl = {};
  pl.grid = kPairs;
  pl.part_ml = reinterpret_cast<float2*>(w + l.part_ml);
  pl.part_o = reinterpret_cast<float4*>(w + l.part_o);
  pl.sum_ml = reinterpret_cast<float2*>(w + l.sum);
  pl.sum_o = reinterpret_cast<float4*>(w + l.sum + (size_t)2 * kPairs * 2 * kRows * sizeof(float2));
  pl.list = plan.list;
  pl.list_place = plan.list_place;
  auto kern = tree_attn_kernel<FMT, LONG, true>;
  static std::atomic<uint64_t> allowed{0};
  if ((e = allow_smem_once(&allowed, reinterpret_cast<const void*>(kern), C::SMEM)) != cudaSuccess) return e;
  static std::atomic<uint64_t> allowed_plan{0};
  if ((e = allow_smem_once(&allowed_plan, reinterpret_cast<const void*>(prefix_plan_kernel), (int)plan_smem(kMaxGroups, kMaxSeq))) != cudaSuccess)
    return e;
  if ((e = launch_kernel(prefix_plan_kernel, dim3(1), dim3(kPlanThreads), plan_smem(pp.n_groups, p.n_seq), stream, false, p, pp, plan)) != cudaSuccess) return e;
  if ((e = launch_kernel(kern, dim3(2 * kPairs), dim3(C::THREADS), C::SMEM, stream, true, tm, p, pl)) != cudaSuccess) return e;
  const int64_t rows = (int64_t)p.n_seq * p.q_per_seq * p.H;
  const unsigned rows8 = (unsigned)((rows + 7) / 8);
  // few rows have many parts each
  if (rows <= kRows * kPairs / 16)
    return launch_kernel(prefix_merge_kernel<16>, dim3(rows8, 1, 16), dim3(1024), 0, stream, true, p, pp, plan, (const float4*)pl.part_o,
                         (const float2*)pl.part_ml);
  return launch_kernel(prefix_merge_kernel<1>, dim3(rows8, 1, 4), dim3(256), 0, stream, true, p, pp, plan, (const float4*)pl.part_o,
                       (const float2*)pl.part_ml);
}

template <int FMT>
cudaError_t launch_fmt(const TreeAttnParams& p, const PrefixParams& pp, void* ws, cudaStream_t stream) {
  return p.L > kLong * kKeys ? launch_form<FMT, true>(p, pp, ws, stream) : launch_form<FMT, false>(p, pp, ws, stream);
}

dsa_status check_prefix(const dsa_tree_args* a, const int32_t* group_start, const int32_t* n_shared, int n_groups) {
  const dsa_status s = check_tree_args(a);
  if (s != DSA_OK) return s;
  if (n_groups < 0 || (n_groups > 0 && (!group_start || !n_shared))) return DSA_ERR_INVALID_ARG;
  if (((reinterpret_cast<uintptr_t>(group_start) | reinterpret_cast<uintptr_t>(n_shared)) & 3) != 0) return DSA_ERR_INVALID_ARG;
  const int64_t rows = (int64_t)a->q_per_seq * a->H;
  if (n_groups > kMaxGroups || a->n_seq > kMaxSeq || a->n_seq * rows > 1 << 26) return DSA_ERR_UNSUPPORTED;
  // the plan's costs have 31 bits: tiles of positions x row tiles, of the sequences' and of the groups' units
  const int64_t units = a->n_seq * ((rows + kRows - 1) / kRows) + a->n_seq * rows / kRows + n_groups + 1;
  if (units * ((int64_t)a->L / kKeys + 1 + kUnitCost) >= 1ll << 31) return DSA_ERR_UNSUPPORTED;
  return DSA_OK;
}

}  // namespace
}  // namespace dsa

using namespace dsa;

extern "C" {

dsa_status dsa_prefix_attn_workspace_size(const dsa_tree_args* a, const int32_t* group_start, const int32_t* n_shared, int n_groups,
                                          size_t* bytes) {
  if (!bytes) return DSA_ERR_INVALID_ARG;
  const dsa_status s = check_prefix(a, group_start, n_shared, n_groups);
  if (s != DSA_OK) return s;
  *bytes = a->n_seq == 0 ? 0 : n_groups == 0 || a->L == 0 ? tree_attn_ws_bytes(tree_attn_params(*a)) : layout_of(tree_attn_params(*a), n_groups).total;
  return DSA_OK;
}

dsa_status dsa_prefix_attn(const dsa_tree_args* a, const int32_t* group_start, const int32_t* n_shared, int n_groups, void* ws,
                           size_t ws_bytes, void* stream) {
  size_t need = 0;
  dsa_status s = dsa_prefix_attn_workspace_size(a, group_start, n_shared, n_groups, &need);
  if (s != DSA_OK || a->n_seq == 0) return s;
  if (n_groups == 0 || a->L == 0) return dsa_tree_attn(a, ws, ws_bytes, stream);
  if (!ws || ws_bytes < need || (reinterpret_cast<uintptr_t>(ws) & 255) != 0) return DSA_ERR_WORKSPACE;
  if ((s = check_device_arch()) != DSA_OK) return s;
  TreeAttnParams p = tree_attn_params(*a);
  p.err = device_error_word();
  const PrefixParams pp = {group_start, n_shared, n_groups, p.nsc > 1 ? kUnitCostTiled : kUnitCost};
  const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const cudaError_t e = !p.kv_fp8      ? launch_fmt<kBf16>(p, pp, ws, st)
                        : p.nsc == 1 ? launch_fmt<kFp8Row>(p, pp, ws, st)
                                     : launch_fmt<kFp8Tile>(p, pp, ws, st);
  return e == cudaSuccess ? DSA_OK : DSA_ERR_CUDA;
}

}  // extern "C"
