// Attention of drafted tokens over the latent cache (dsa_tree_attn): query node i of sequence s sees
// the n_ctx[s] cached positions and the drafted positions n_ctx[s] + j whose bit j is set in its row
// of the tree mask,
//   logit[p] = sm_scale * q[i, h] . Kv[p],  out[i, h] = sum_p softmax(logit)[p] * Kv[p, :512].
//
// A "row" is one head of one node; the rows of a sequence are consecutive in q and share its cache.
// Two CTAs take 128 rows and walk tiles of 64 positions; each takes the first product of all of them and the second
// one for half of the value columns, on its own (no cluster: nothing is exchanged):
//   * S[128 x 64] = Q K^T, 36 steps: A = the rows (M = 128; 320 of their columns in tensor memory, 128 with tile
//     scales, the others in shared memory), B = the positions (K-major);
//   * one pass over the positions keeps a reference maximum m and a sum l per row,
//       l' = l 2^(m - m') + sum_p 2^(x_p - m'),   o' = o 2^(m - m') + sum_p 2^(x_p - m') v_p,
//     where m is moved only when a tile's maximum exceeds it by more than 2^8 (weights stay below 2^8,
//     fp32 sums and bf16 weights lose nothing by it), so o in tensor memory is rescaled rarely;
//   * O_c[128 x 256] += P V_c: A = the weights, bf16, in tensor memory, B = 256 value columns of the positions, read
//     MN-major (values along N), 4 steps of K = 16 with N = 256.
// Why two CTAs: o for 128 rows x 512 values fills a tensor memory (512 columns), which leaves no room for S; with half
// of the values it takes 256 columns, q 160, S 64, the weights 32.  Why both take the whole first product: an MMA of
// N = 64 with A in tensor memory takes 32 cycles, one of N = 32 33, so that sharing the 64 positions of a tile out
// saves nothing (a tile of 128 shared out would take N = 64 each; that was not built).
// Measured (8 x 64 nodes at 32K, E4M3 rows; 8 x 8 nodes at 32K, bf16; device us): this form 611 and 91.  The forms before
// it, as they were when they gave way: the positions of the first product shared out and weights exchanged through
// distributed shared memory 1002 and 105; columns shared out and partial S exchanged 1090 and 120; one CTA with 64 rows
// and q in shared memory 1805 and 149.
//
// Weights are rounded to bf16 for the second product (as the bf16 cache is); sums, maxima, logits and outputs are
// fp32.  E4M3 codes enter the first product as they are: q's bf16 values, scaled by a power of two per row, are the sum
// of an E4M3 and an E5M2 value, exactly down to 2^-13 of the row's largest value and to 2^-20 of it below, and the
// 8-bit MMAs (K = 32, both parts) cost what bf16 ones would, at half of the shared memory.  For the second product the
// codes of a CTA's own value columns are widened to bf16 exactly.  (Widening all of them: 1002 us instead of 803 at the
// time, 8 x 64 nodes.)  The positions' scales are applied in fp32 to the logit and to the weight (128-column scales:
// one S accumulation per scale tile, one P per value tile).
//
// Bound: with few rows the memory, with many the tensor cores: 36 x 32 to 48 + 512 cycles per tile are 1920 of the
// measured 2500; with tile scales the softmax warps' turn from one accumulation to the next (6200).
//
// Warp roles: producer (TMA), MMA issuer, scale loader, eight softmax warps (a row and 32 positions per thread; also
// the query load, the rescale and the epilogue), for E4M3 four warps that widen the value columns.
//
// Work split: items (sequence, chunk of its tiles, row tile) for pairs of CTAs.  The lengths are on the device:
// every CTA evaluates the same cost model over them (plan_items); partial results are merged by
// tree_combine_kernel.
#pragma once

#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <string.h>

#include "tc_common.cuh"

namespace dsa {
namespace {

constexpr float kLn2 = 0.6931471805599453f;
constexpr int kDqk = 576, kDv = 512;
constexpr int kRows = 128;                // query rows per pair of CTAs
constexpr int kKeys = 64;                 // positions per tile
constexpr int kBox = kKeys * 128;         // 64 columns of a tile: 64 rows x 128 bytes
constexpr int kSlotV = 4 * kBox;          // a CTA's value columns
constexpr int kBoxC = kKeys * 64;         // 64 columns of a tile's E4M3 codes
constexpr int kSlotC = 9 * kBoxC;
constexpr int kSmemMax = 227 * 1024;
constexpr float kLazy = 8.f;              // log2 growth of a row's maximum that is left unscaled
constexpr int kMaxItems = 8;              // of a pair of CTAs, in a planned launch
constexpr int kSlotsPerPair = 3;          // partial results
// The tensor cores truncate their sums, four to a tile, so o loses up to 2^-23 of itself each time, always in the same
// direction: 0.037 % over 1024 tiles, 0.34 % over 8192, 2.7 % over 65536 (measured).  Launches whose contexts may be longer
// than kLong tiles walk an item in stretches of kStretch tiles, whose o and l are added up in fp32, in memory: 0.02 % at
// any length.  They are a form of the kernel of their own, because it costs something where nothing is long too (device us
// without and with it, contexts of 32K: 8 x 8 nodes bf16 98.5 and 99.5, 8 x 64 E4M3 rows 606 and 624, 8 x 64 tile scales
// 1280 and 1309; contexts of 60K, two stretches: 8 x 64 bf16 1300 and 1312, E4M3 1161 and 1170, tile scales 2301 and 2372).
// (A break inside the tile loop cost up to 9 %, stretches as an outer loop around it 11 %: the loop's registers.)
constexpr int kLong = 1024, kStretch = 512;
constexpr int kAhead = 2;                 // tiles between the request to L2 and the load into shared memory
constexpr int kColO = 0;                  // tensor-memory columns: O, then boxes of q, S and the weights

enum { kBf16 = 0, kFp8Row = 1, kFp8Tile = 2 };

struct Aux {
  uint64_t v_full[3], v_empty[3], k_full[7], k_empty[7], c_full[2], c_empty[2], s_full[2], s_empty[2], p_full, pv_done;
  uint64_t o_done, o_free, q_full, sc_full[2], sc_empty[2], drain;
  uint32_t tmem;
  int abort;
  int n_items;
  int tile_bad[8];
  int items[kMaxItems][8];
  alignas(16) float mx[2][2][kRows];  // the rows' maxima over half of a tile
  float sum[2][kRows];                // and, at an item's end, their sums
  uint32_t clear[2][8];               // positions to clear
  int list_first;                     // of a launch with shared prefixes
};

template <int FMT>
struct Cfg {
  static constexpr bool FP8 = FMT != kBf16;
  static constexpr int NSC = FMT == kFp8Tile ? 5 : FMT == kFp8Row ? 1 : 0;
  static constexpr bool TILED = FMT == kFp8Tile;
  static constexpr int THREADS = FP8 ? 512 : 384;
  // bf16: slots of this CTA's value columns (held from the first product to the second) and boxes of the others
  // (first product only).  E4M3: slots of a tile's codes, and of the value columns widened to bf16.
  static constexpr int VS = TILED ? 1 : FP8 ? 2 : 3, KS = FP8 ? 0 : 7, CS = FP8 ? 2 : 0;
  static constexpr int SB = TILED ? 2 : 1;                // S buffers
  static constexpr int BT = TILED ? 2 : 5;                // q's boxes in tensor memory (the others are in shared memory)
  static constexpr int COL_Q = 256, COL_S = COL_Q + 32 * BT, COL_P = COL_S + kKeys * SB;
  static constexpr int GROUPS = TILED ? 5 : 1;            // S accumulations per tile
  static constexpr int PC = TILED ? 2 : 1;                // copies of P (one per 128 values)
  static constexpr int SC_BYTES = NSC * kKeys * 4;
  static constexpr int Q_BOX = kRows * 128, Q_BYTES = (9 - BT) * Q_BOX;
  static constexpr int OFF_K = VS * kSlotV;
  static constexpr int OFF_C = OFF_K + KS * kBox;
  static constexpr int OFF_Q = OFF_C + CS * kSlotC;
  static constexpr int OFF_SC = OFF_Q + Q_BYTES;
  static constexpr int OFF_AUX = OFF_SC + 2 * SC_BYTES;
  static constexpr int SMEM = OFF_AUX + (int)sizeof(Aux) + 1024;
  static_assert(SMEM <= kSmemMax, "shared memory");
  static_assert(COL_P + 32 * PC <= 512, "tensor memory");
};

struct Item {
  int seq, rt, t0, t1;     // tiles [t0, t1) of row tile rt
  int ctx, fresh, len;     // cached and drafted positions, the sequence's end
  int slot;                // partial slot, or -1: the whole range, written to the output
};

// An item of a launch with shared prefixes: rows [at, at + nrows) of all queries, which may be several sequences' (of a
// group, over its prefix) or one's (over what follows it), against the cache of sequence `seq`.
struct SharedItem : Item {
  int at, nrows, row_lo;   // row_lo: the first row's number within its sequence (rows of one sequence only)
  int pad;
};
static_assert(sizeof(SharedItem) == 48, "three 16-byte loads");
// An item's first row: its number within the sequence, that in out and lse; and its rows.
__device__ __forceinline__ int first_row(const Item& it) { return it.rt * kRows; }
__device__ __forceinline__ int first_row(const SharedItem& it) { return it.row_lo; }
__device__ __forceinline__ int64_t first_in_out(const Item& it, int rows, int lo) { return (int64_t)it.seq * rows + lo; }
__device__ __forceinline__ int64_t first_in_out(const SharedItem& it, int, int) { return it.at; }
__device__ __forceinline__ int rows_of(const Item&, int rows, int lo) { return min(kRows, rows - lo); }
__device__ __forceinline__ int rows_of(const SharedItem& it, int, int) { return it.nrows; }
template <bool SHARED>
struct ItemOf {
  using type = Item;
};
template <>
struct ItemOf<true> {
  using type = SharedItem;
};

// The launch's fixed facts (host) and the split plan in the workspace (device).
struct TreePlan {
  int row_tiles;           // per sequence
  int units;               // n_seq * row_tiles
  int cap;                 // partial slots; 0: a launch of many units, without a plan
  int grid;                // pairs of CTAs
  int* head;               // [0]: tiles of a chunk, or minus those of a span; [1 + s]: first item or tile of sequence s
  float4* part_o;          // [cap][128 groups of four values][128 rows]
  float2* part_ml;         // [cap][half of the values][128 rows]
  // per CTA of a launch with long contexts: the sums of an item's stretches so far
  float4* sum_o;           // [2 grid][64 groups of four values][128 rows]
  float2* sum_ml;          // [2 grid][half of a tile's positions][128 rows]: the reference maximum, the sum of weights
  // a launch with shared prefixes: each pair's items (prefix_attn.cu), `slot` the first row of its partial results
  const SharedItem* list;
  const int2* list_place;  // [grid]: the pair's first entry and their number
};

__device__ __forceinline__ void seq_facts(const TreeAttnParams& p, int seq, int& ctx, int& fresh, int& len) {
  ctx = min(max(p.n_ctx[seq], 0), p.L);
  fresh = p.n_new ? min(max(p.n_new[seq], 0), p.q_per_seq) : p.q_per_seq;
  len = min(ctx + fresh, p.L);
}

__device__ __forceinline__ int live_row_tiles(const TreeAttnParams& p, int fresh) {
  return (fresh * p.H + kRows - 1) / kRows;  // row tiles that hold a node below `fresh`
}

// Barriers of the eight softmax warps, and of the two that share 32 rows (ids 2 to 5).
__device__ __forceinline__ void softmax_bar() {
  __syncwarp();
  asm volatile("bar.sync 1, 256;" ::: "memory");
}
__device__ __forceinline__ void pair_bar(int quarter) {
  __syncwarp();
  asm volatile("bar.sync %0, 64;" ::"r"(2 + quarter) : "memory");
}

// Two bf16 values, times mul (a power of two that brings them below 2^8), as E4M3 plus E5M2: the first takes four of
// the eight significant bits, what is left is a multiple of the last bit of at most eight of them, which three bits
// hold.  So v = e4 + e5 exactly for |v| >= 2^-6, and to 2^-13 below (fp16 holds the values between, to 2^-25).
__device__ __forceinline__ void split_fp8(uint32_t x, float mul, uint32_t& e4, uint32_t& e5) {
  const __half2 v = __floats2half2_rn(__uint_as_float(x << 16) * mul, __uint_as_float(x & 0xFFFF0000u) * mul);
  const __nv_fp8x2_storage_t a = __nv_cvt_halfraw2_to_fp8x2(v, __NV_SATFINITE, __NV_E4M3);
  e4 = a;
  e5 = __nv_cvt_halfraw2_to_fp8x2(__hsub2(v, __half2(__nv_cvt_fp8x2_to_halfraw2(a, __NV_E4M3))), __NV_SATFINITE, __NV_E5M2);
}

// Bits of the tile's 64 positions (first at t * 64) that `node` sees, for a tile that holds drafted
// positions or the sequence's end.
__device__ __forceinline__ uint64_t seen_bits(const TreeAttnParams& p, const Item& it, int node, int t) {
  const int start = t * kKeys - it.ctx;  // drafted index of the tile's first position (negative: cached)
  const int end = it.len - t * kKeys;    // positions of the tile that exist
  uint64_t v;
  if (!p.mask) {
    const int n = node + 1 - start;      // the chain's nodes 0 .. node
    v = n >= 64 ? ~0ull : n <= 0 ? 0ull : (1ull << n) - 1;
  } else {
    const uint32_t* w = p.mask + ((int64_t)it.seq * p.q_per_seq + node) * p.mask_words;
    auto word = [&](int i) -> uint64_t { return i >= 0 && i < p.mask_words ? w[i] : 0u; };
    if (start >= 0) {
      const int i = start >> 5, s = start & 31;
      v = (word(i) | word(i + 1) << 32) >> s;
      if (s) v |= word(i + 2) << (64 - s);
    } else if (start > -64) {
      v = (word(0) | word(1) << 32) << -start | ((1ull << -start) - 1);
    } else {
      v = ~0ull;
    }
  }
  // only drafted tokens below `fresh` exist: the sequence's end says so too (len <= ctx + fresh)
  if (end < 64) v &= end <= 0 ? 0ull : (1ull << end) - 1;
  return v;
}

// Splits the sequences' tiles into items, for each pair of CTAs a list.  Two kinds of plan:
//   * chunks of CH tiles of every unit (a row tile of a sequence), dealt out in turn: pairs that run together read
//     the same positions;
//   * spans of W tiles, a pair's share, of the units' tiles laid end to end: no pair waits for another.  Only the
//     first and the last item of a span are parts of a unit.  (Units of W / 6 at least: kMaxItems.  One that is shorter
//     leaves the launch to chunks.)
// The cost of each in tiles: the fullest pair's items and the fill and drain of its pipeline for each, and for a split
// the merge.  (8 x 64 nodes at 32K, E4M3: 64 units of 512 tiles on 76 pairs, 710 us whole, 630 us as spans.)
// CTA 0 leaves the plan for the merge.  Scratch: 3 n_seq + 160 ints of shared memory.
__device__ void plan_items(const TreeAttnParams& p, const TreePlan& pl, Aux* a, int* scratch) {
  constexpr float kItemCost = 4.f, kMergeCost = 4.f, kMergePerItem = 0.02f;  // in tiles
  const int tid = threadIdx.x, n = p.n_seq;
  int* nt = scratch;            // tiles of each sequence
  int* live = scratch + n;      // its live row tiles
  int* base = scratch + 2 * n;  // its first item
  float* cost = reinterpret_cast<float*>(scratch + 3 * n);  // [64]
  int* chunk = scratch + 3 * n + 64;                        // [64], then [0] the choice, [1] the longest
  for (int s = tid; s < n; s += blockDim.x) {
    int ctx, fresh, len;
    seq_facts(p, s, ctx, fresh, len);
    live[s] = live_row_tiles(p, fresh);
    nt[s] = live[s] ? (len + kKeys - 1) / kKeys : 0;
  }
  __syncthreads();
  long long total = 0;  // (in the first warp) all units' tiles
  int least = INT_MAX;  // of a unit that has any
  if (tid < 32) {
    int m = 1;
    for (int s = tid; s < n; s += 32) {
      m = max(m, nt[s]);
      if (nt[s]) least = min(least, nt[s]);
      total += (long long)nt[s] * live[s];
    }
    m = __reduce_max_sync(0xffffffffu, m);
    least = __reduce_min_sync(0xffffffffu, least);
#pragma unroll
    for (int o = 16; o; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
    if (tid == 0) chunk[65] = m;
  }
  __syncthreads();
  const int longest = chunk[65];
  if (tid < 256) {
    // 64 candidates, four threads each: 1 .. 32 chunks of the longest sequence, and as many as make 1 .. 32
    // rounds of the grid
    const int c = tid >> 2;
    const int k = c < 32 ? c + 1 : max(1, (c - 31) * pl.grid / pl.units);
    const int ch = (longest + k - 1) / k;
    int items = 0;
    bool split = false;
    for (int s = tid & 3; s < n; s += 4) {
      const int chunks = nt[s] ? (nt[s] + ch - 1) / ch : 1;
      items += live[s] * chunks + (pl.row_tiles - live[s]);
      split |= chunks > 1;
    }
    items += __shfl_xor_sync(0xffffffffu, items, 1);
    items += __shfl_xor_sync(0xffffffffu, items, 2);
    int sp = split;
    sp |= __shfl_xor_sync(0xffffffffu, sp, 1);
    sp |= __shfl_xor_sync(0xffffffffu, sp, 2);
    const int rounds = (items + pl.grid - 1) / pl.grid;
    float v = rounds * (ch + kItemCost) + (sp ? kMergeCost + kMergePerItem * items : 0.f);
    if ((sp && items > pl.cap) || rounds > kMaxItems) v = INFINITY;
    if ((tid & 3) == 0) cost[c] = v, chunk[c] = ch;
  }
  __syncthreads();
  if (tid < 32) {
    const float c0 = cost[tid], c1 = cost[tid + 32];
    float best = fminf(c0, c1);
#pragma unroll
    for (int o = 16; o; o >>= 1) best = fminf(best, __shfl_xor_sync(0xffffffffu, best, o));
    const uint32_t m0 = __ballot_sync(0xffffffffu, c0 == best), m1 = __ballot_sync(0xffffffffu, c1 == best);
    const int ch = chunk[m0 ? __ffs(m0) - 1 : 31 + __ffs(m1)];
    const long long share = (total + pl.grid - 1) / pl.grid;
    const bool spans = total > 0 && total <= INT_MAX - 4096 && (kMaxItems - 2ll) * least >= share &&
                       share + kItemCost * (2 + pl.units / pl.grid) + kMergeCost + 2 * kMergePerItem * pl.grid < best;
    const int W = (int)share;
    int run = 0;  // items, or tiles
    for (int s0 = 0; s0 < n; s0 += 32) {
      const int s = s0 + tid;
      const int c = s >= n ? 0
                    : spans ? nt[s] * live[s]
                            : live[s] * (nt[s] ? (nt[s] + ch - 1) / ch : 1) + (pl.row_tiles - live[s]);
      int incl = c;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(0xffffffffu, incl, o);
        if (tid >= o) incl += u;
      }
      if (s < n) base[s] = run + incl - c;
      run += __shfl_sync(0xffffffffu, incl, 31);
    }
    __syncwarp();
    // this pair's items: tiles [pair W, (pair + 1) W), or the items of its number, + grid, ...
    const int pair = (int)(blockIdx.x >> 1), mine = spans ? pair * W : pair + tid * pl.grid;
    auto sequence = [&](int at) {  // whose tiles or items hold number `at`
      int lo = 0, hi = n - 1;
      while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (base[mid] <= at) lo = mid;
        else hi = mid - 1;
      }
      return lo;
    };
    if (spans) {
      if (tid == 0) {
        const int end = min(run - mine, W) + mine;
        int count = 0;
        for (int at = mine; at < end; ++count) {
          Item it;
          it.seq = sequence(at);
          seq_facts(p, it.seq, it.ctx, it.fresh, it.len);
          const int tiles = nt[it.seq];
          it.rt = (at - base[it.seq]) / tiles;
          const int unit = base[it.seq] + it.rt * tiles;
          it.t0 = at - unit;
          it.t1 = min(tiles, end - unit);
          it.slot = it.t0 > 0 ? 2 * pair : it.t1 < tiles ? 2 * pair + 1 : -1;
          memcpy(a->items[count], &it, sizeof(it));
          at = unit + it.t1;
        }
        a->n_items = count;
      }
    } else {
      if (tid < kMaxItems && mine < run) {
        const int s = sequence(mine), at = mine - base[s];
        const int chunks = nt[s] ? (nt[s] + ch - 1) / ch : 1;
        Item it;
        seq_facts(p, s, it.ctx, it.fresh, it.len);
        it.seq = s;
        it.slot = -1;
        it.t0 = it.t1 = 0;
        if (at < live[s] * chunks) {
          const int j = at / live[s];
          it.rt = at - j * live[s];
          it.t0 = min(j * ch, nt[s]);
          it.t1 = min(it.t0 + ch, nt[s]);
          if (chunks > 1) it.slot = mine;
        } else {
          it.rt = live[s] + at - live[s] * chunks;
        }
        memcpy(a->items[tid], &it, sizeof(it));
      }
      if (tid == 0) a->n_items = pair < run ? (run - pair + pl.grid - 1) / pl.grid : 0;
    }
    if (blockIdx.x == 0) {
      if (tid == 0) pl.head[0] = spans ? -W : ch;
      for (int s = tid; s < n; s += 32) pl.head[1 + s] = base[s];
    }
  }
  __syncthreads();
}

// Item i of this pair in a launch with shared prefixes (empty ones have t0 = t1).
__device__ __forceinline__ bool get_item(const TreeAttnParams& p, const TreePlan& pl, const Aux* a, int i, SharedItem& it) {
  if (i >= a->n_items) return false;
  const int4* src = reinterpret_cast<const int4*>(pl.list + a->list_first + i);
  int4 v[3] = {src[0], src[1], src[2]};
  memcpy(&it, v, sizeof(it));
  return true;
}

// Item i of this pair: from the list of a split launch, or the unit of number pair + i * grid whole.
__device__ __forceinline__ bool get_item(const TreeAttnParams& p, const TreePlan& pl, const Aux* a, int i, Item& it) {
  if (pl.cap) {
    if (i >= a->n_items) return false;
    memcpy(&it, a->items[i], sizeof(it));
    return true;
  }
  const int u = (int)(blockIdx.x >> 1) + i * pl.grid;
  if (u >= pl.units) return false;
  it.seq = u / pl.row_tiles;
  it.rt = u - it.seq * pl.row_tiles;
  seq_facts(p, it.seq, it.ctx, it.fresh, it.len);
  it.t0 = 0;
  it.t1 = it.rt < live_row_tiles(p, it.fresh) ? (it.len + kKeys - 1) / kKeys : 0;
  it.slot = -1;
  return true;
}

// The next item, or with LONG the next stretch of one: tiles [t0, t1) of those that end at `st.stop`.
struct Stretch {
  int stop = 0;
  bool first = true;
};
template <bool LONG, class AnyItem>
__device__ __forceinline__ bool next_item(const TreeAttnParams& p, const TreePlan& pl, const Aux* a, int& i, AnyItem& it, Stretch& st) {
  if (!LONG) return get_item(p, pl, a, i, it);
  st.first = it.t1 >= st.stop;
  if (st.first) {
    if (!get_item(p, pl, a, i, it)) return false;
    st.stop = it.t1;
  } else {
    it.t0 = it.t1;
    --i;
  }
  it.t1 = min(st.stop, it.t0 + kStretch);
  return true;
}

template <int N>
struct Int {
  static constexpr int v = N;
};

// SHARED: a launch with shared prefixes, whose items come from a list and all leave partial results.
template <int FMT, bool LONG, bool SHARED = false>
__global__ void __launch_bounds__(Cfg<FMT>::THREADS, 1)
    tree_attn_kernel(const __grid_constant__ CUtensorMap tm, const TreeAttnParams p, const TreePlan pl) {
  using C = Cfg<FMT>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* v_s = smem;
  uint8_t* k_s = smem + C::OFF_K;
  uint8_t* c_s = smem + C::OFF_C;
  uint8_t* q_s = smem + C::OFF_Q;
  float* sc_s = reinterpret_cast<float*>(smem + C::OFF_SC);
  Aux* a = reinterpret_cast<Aux*>(smem + C::OFF_AUX);
  const int tid = threadIdx.x, lane = tid & 31, warp = uniform(tid >> 5);
  const int rank = (int)(blockIdx.x & 1);  // which half of the value columns
  int* err = p.err;

  if (warp == 0) {
    tmem_alloc(&a->tmem, 512);
    tmem_relinquish();
  }
  if (tid == 32) {
    // (the converters' four warps fill the value columns, and read a slot of codes beside the first product)
    for (int i = 0; i < C::VS; ++i) mbar_init(&a->v_full[i], C::FP8 ? 4 : 1), mbar_init(&a->v_empty[i], 1);
    for (int i = 0; i < C::KS; ++i) mbar_init(&a->k_full[i], 1), mbar_init(&a->k_empty[i], 1);
    for (int i = 0; i < C::CS; ++i) mbar_init(&a->c_full[i], 1), mbar_init(&a->c_empty[i], 1 + 4);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&a->s_full[i], 1), mbar_init(&a->s_empty[i], 8);
      mbar_init(&a->sc_full[i], 32), mbar_init(&a->sc_empty[i], 8);
    }
    mbar_init(&a->p_full, 8);
    mbar_init(&a->pv_done, 1);
    mbar_init(&a->o_done, 1);
    mbar_init(&a->o_free, 8);
    mbar_init(&a->q_full, 256);
    mbar_init(&a->drain, 1);
    a->abort = 0;
    fence_mbar_init();
  }
  if constexpr (SHARED) {
    pdl_wait();  // the list
    if (tid == 0) {
      const int2 mine = pl.list_place[blockIdx.x >> 1];
      a->list_first = mine.x, a->n_items = mine.y;
    }
  } else if (pl.cap) {
    plan_items(p, pl, a, reinterpret_cast<int*>(v_s));
  }
  fence_proxy_async_smem();  // the plan's scratch is a slot that the copies write
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = a->tmem;
  pdl_launch_dependents();

  using AnyItem = typename ItemOf<SHARED>::type;
  AnyItem it = {};
  Stretch st;
  if (warp == 0) {
    // ---- producer: boxes of 64 columns x 64 positions by TMA
    if (lane == 0) {
      prefetch_tmap(&tm);
      int vs = 0, vph = 0, ks = 0, kph = 0, cs = 0, cph = 0, tiles = 0;
      bool ok = true;
      // Tiles on their way to L2, this CTA's value columns of them (the other one of the pair asks for the others):
      // the slots alone do not cover the latency of the memory.
      auto ahead = [&](int t) {
        if (t >= it.t1) return;
        int64_t row = t * kKeys;
        if (p.pages.table && (row = tree_row(p, it.seq, (int)row)) < 0) return;
#pragma unroll
        for (int b = 0; b < 4; ++b) tma_prefetch_3d(&tm, 256 * rank + 64 * b, (int)row, p.pages.table ? 0 : it.seq);
        if (rank) tma_prefetch_3d(&tm, 512, (int)row, p.pages.table ? 0 : it.seq);
      };
      // an item's query rows too: the first one's before its tiles queue up at the memory, the others' an item ahead
      auto query = [&](const AnyItem& x) {
        if (rank != 0 || x.t0 >= x.t1) return;
        if constexpr (SHARED) {
          prefetch_l2(p.q + (int64_t)x.at * kDqk, x.nrows * kDqk * 2);
        } else {
          const int lo = x.rt * kRows, n = min(kRows, p.q_per_seq * p.H - lo);
          prefetch_l2(p.q + ((int64_t)x.seq * p.q_per_seq * p.H + lo) * kDqk, n * kDqk * 2);
        }
      };
      AnyItem next;
      if (get_item(p, pl, a, 0, next)) query(next);
      for (int i = 0; ok && next_item<LONG>(p, pl, a, i, it, st); ++i) {
        if (get_item(p, pl, a, i + 1, next)) query(next);
        for (int t = it.t0; !C::FP8 && t < it.t0 + kAhead; ++t) ahead(t);
        for (int t = it.t0; ok && t < it.t1; ++t, ++tiles) {
          if (!C::FP8) ahead(t + kAhead);
          int row = t * kKeys, z = it.seq, bad = 0;
          if (p.pages.table) {
            const int64_t r = tree_row(p, it.seq, row);
            z = 0;
            bad = r < 0;
            // a block id outside the pool: rows past its end, which the copy fills with zeros
            row = bad ? p.pages.num_blocks * p.pages.block_size : (int)r;
            if (bad) record_error(err, DSA_DEVERR_INDEX_RANGE);
          }
          if constexpr (C::FP8) {
            ok = wait_ahead(a, &a->c_empty[cs], cph ^ 1, err);
            if (!ok) break;
            a->tile_bad[tiles & 7] = bad;
            mbar_arrive_expect_tx(&a->c_full[cs], kSlotC);
#pragma unroll
            for (int b = 0; b < 9; ++b)
              tma_load_3d(c_s + cs * kSlotC + b * kBoxC, &tm, &a->c_full[cs], b < 8 ? 64 * (b ^ (rank << 2)) : 512, row, z);
            if (++cs == C::CS) cs = 0, cph ^= 1;
          } else {
            for (int b = 0; b < 5; ++b) {
              ok = wait_ahead(a, &a->k_empty[ks], kph ^ 1, err);
              if (!ok) break;
              mbar_arrive_expect_tx(&a->k_full[ks], kBox);
              tma_load_3d(k_s + ks * kBox, &tm, &a->k_full[ks], b < 4 ? 256 * (rank ^ 1) + 64 * b : 512, row, z);
              if (++ks == C::KS) ks = 0, kph ^= 1;
            }
            ok = ok && wait_ahead(a, &a->v_empty[vs], vph ^ 1, err);
            if (!ok) break;
            a->tile_bad[tiles & 7] = bad;
            mbar_arrive_expect_tx(&a->v_full[vs], kSlotV);
#pragma unroll
            for (int b = 0; b < 4; ++b)
              tma_load_3d(v_s + vs * kSlotV + b * kBox, &tm, &a->v_full[vs], 256 * rank + 64 * b, row, z);
            if (++vs == C::VS) vs = 0, vph ^= 1;
          }
        }
      }
      if (*reinterpret_cast<volatile int*>(&a->abort)) {  // wind down: the copies in flight land first
        for (int s = 0; !C::FP8 && s < C::VS; ++s) mbar_wait(&a->v_full[s], s < vs ? vph : vph ^ 1, err);
        for (int s = 0; s < C::KS; ++s) mbar_wait(&a->k_full[s], s < ks ? kph : kph ^ 1, err);
        for (int s = 0; s < C::CS; ++s) mbar_wait(&a->c_full[s], s < cs ? cph : cph ^ 1, err);
      }
    }
    __syncwarp();
  } else if (warp == 1) {
    // ---- MMA issuer.  The warp stays converged and one elected lane issues; descriptors are sums of
    // 32-bit words (their upper words are constants), so that issuing an instruction costs less than
    // the tensor cores take for it
    constexpr uint32_t idesc_qk = make_idesc(1, 1, kRows, kKeys);  // bf16
    constexpr uint32_t idesc_e4 = make_idesc(0, 0, kRows, kKeys), idesc_e5 = make_idesc(1, 0, kRows, kKeys);
    constexpr uint32_t idesc_pv = make_idesc(1, 1, kRows, C::TILED ? 128 : 256) | (1u << 16);  // B (values) MN-major
    const uint32_t tm_base = (uint32_t)uniform((int)tmem);
    const uint32_t kv_lo = kmajor_lo(smem_u32(v_s)), kk_lo = kmajor_lo(smem_u32(k_s));
    const uint32_t vv_lo = mnmajor_lo(smem_u32(v_s), kBox), c_lo = kmajor_lo(smem_u32(c_s));
    const uint32_t q_lo = kmajor_lo(smem_u32(q_s));
    int vs = 0, vph = 0, ks = 0, kph = 0, cs = 0, cph = 0;  // slots of the first product
    int ps = 0, pph = 0;                                    // of the second
    int tile = 0, qt = 0, items = 0;       // tiles of the second product, of the first
    uint32_t su = 0;                       // uses of the S buffers
    bool ok = true;
    auto commit = [&](uint64_t* bar) {
      if (elect_one()) tc_commit(bar);
      __syncwarp();
    };
    auto all = [&](uint64_t* bar, uint32_t parity) { ok = __all_sync(0xffffffffu, wait(a, bar, parity, err)) && ok; };
    // Box j of q (in the order of the slots: our value columns, the other columns, the rotary ones) against the
    // tile's positions: 4 steps of K = 16.  With E4M3 rows q's bf16 values are E4M3 plus E5M2: two steps of
    // K = 32, each for both parts, at the same cost, and the codes need no widening.
    auto qk_box = [&](uint32_t d, int j, uint32_t B, bool first) {
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const uint32_t acc = first && k == 0 ? 0u : 1u;
        const uint32_t id = !C::FP8 ? idesc_qk : k & 1 ? idesc_e5 : idesc_e4;
        const uint32_t b = B + 2 * (C::FP8 ? k >> 1 : k);
        if (j < C::BT) mma_ts<C::FP8>(d, tm_base + C::COL_Q + 32 * j + 8 * k, b, id, acc);
        else mma_ss<C::FP8>(d, q_lo + (j - C::BT) * (C::Q_BOX >> 4) + 2 * k, b, id, acc);
      }
    };
    // Slot of box j of the K ring, from the next one on, and its phase.
    auto k_slot = [&](int j) { return ks + j >= C::KS ? ks + j - C::KS : ks + j; };
    auto k_phase = [&](int j) { return ks + j >= C::KS ? kph ^ 1 : kph; };
    // Boxes [J0, J1) of the first product into the S buffer of use `su`.  One lane per barrier: a wait costs about
    // 120 cycles even when there is nothing to wait for, and the tensor cores run dry.
    auto qk = [&](auto J0, auto J1) {
      constexpr int j0 = decltype(J0)::v, j1 = decltype(J1)::v;
      const uint32_t d = tm_base + C::COL_S + kKeys * (su % C::SB);
      uint64_t* bar = &a->s_empty[su % C::SB];
      uint32_t parity = ((su / C::SB) & 1) ^ 1;
      if (C::FP8) {
        if (lane == 1) bar = &a->c_full[cs], parity = cph;
        if (!C::TILED && lane == 2) bar = &a->sc_full[qt & 1], parity = (qt >> 1) & 1;  // (the softmax warps rely on it)
      } else {
        if (lane >= 2 && lane < 7) bar = &a->k_full[k_slot(lane - 2)], parity = k_phase(lane - 2);
      }
      all(bar, parity);
      if (!ok) return;
      tc_fence_after();
      if (elect_one()) {
        if (C::FP8) {
          const uint32_t B = c_lo + cs * (kSlotC >> 4);
#pragma unroll
          for (int j = j0; j < j1; ++j) qk_box(d, j, B + (j * kBoxC >> 4), j == j0);
          if (j1 == 9) tc_commit(&a->c_empty[cs]);
          tc_commit(&a->s_full[su % C::SB]);
        } else {
          // those of the K ring first: their slots are the scarcer ones, and loading them again takes longer than
          // the rest of this product
#pragma unroll
          for (int j = 4; j < 9; ++j) {
            qk_box(d, j, kk_lo + k_slot(j - 4) * (kBox >> 4), j == 4);
            tc_commit(&a->k_empty[k_slot(j - 4)]);
          }
        }
      }
      if (!C::FP8) {  // the value columns, waited for while the others are multiplied
        __syncwarp();
        all(&a->v_full[vs], vph);
        if (!ok) return;
        tc_fence_after();
        if (elect_one()) {
          const uint32_t V = kv_lo + vs * (kSlotV >> 4);
#pragma unroll
          for (int j = 0; j < 4; ++j) qk_box(d, j, V + (j * kBox >> 4), false);
          tc_commit(&a->s_full[su % C::SB]);
        }
      }
      __syncwarp();
      ++su;
      if (j1 == 9) {
        ++qt;
        if (C::FP8) {
          if (++cs == C::CS) cs = 0, cph ^= 1;
        } else {
          if (++vs == C::VS) vs = 0, vph ^= 1;
          ks += 5;
          if (ks >= C::KS) ks -= C::KS, kph ^= 1;
        }
      }
    };
    auto pv = [&](bool first) {
      uint64_t* bar = &a->p_full;
      uint32_t parity = tile & 1;
      if (first && lane == 1) bar = &a->o_free, parity = (items & 1) ^ 1;
      if (C::FP8 && lane == 2) bar = &a->v_full[ps], parity = pph;
      all(bar, parity);
      if (!ok) return;
      tc_fence_after();
      const uint32_t acc0 = first ? 0u : 1u, V = vv_lo + ps * (kSlotV >> 4);
      if (elect_one()) {
        constexpr int NB = C::TILED ? 2 : 1;  // value tiles of N = 128 with a P each, or all 256 at once
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
          for (int s = 0; s < 4; ++s)
            mma_ts(tm_base + kColO + 128 * b, tm_base + C::COL_P + 32 * b + 8 * s, V + (2 * b * kBox + 2048 * s) / 16, idesc_pv,
                   s ? 1u : acc0);
        tc_commit(&a->v_empty[ps]);
        tc_commit(&a->pv_done);
      }
      __syncwarp();
      if (++ps == C::VS) ps = 0, pph ^= 1;
      ++tile;
    };
    for (int i = 0; ok && uniform(next_item<LONG>(p, pl, a, i, it, st)); ++i) {
      const int t0 = uniform(it.t0), t1 = uniform(it.t1);
      if (t0 >= t1) continue;
      all(&a->q_full, items & 1);
      if constexpr (C::TILED) {
        // an accumulation per scale tile: two run ahead of the softmax warps
        qk(Int<0>{}, Int<2>{});
        qk(Int<2>{}, Int<4>{});
        for (int t = t0; ok && t < t1; ++t) {
          qk(Int<4>{}, Int<6>{});
          qk(Int<6>{}, Int<8>{});
          qk(Int<8>{}, Int<9>{});
          if (t + 1 < t1) {
            qk(Int<0>{}, Int<2>{});
            qk(Int<2>{}, Int<4>{});
          }
          pv(t == t0);
        }
      } else {
        // the next tile's first product, then this one's second
        qk(Int<0>{}, Int<9>{});
        for (int t = t0; ok && t < t1; ++t) {
          if (t + 1 < t1) qk(Int<0>{}, Int<9>{});
          pv(t == t0);
        }
      }
      if (ok) commit(&a->o_done);
      ++items;
    }
    if (__any_sync(0xffffffffu, *reinterpret_cast<volatile int*>(&a->abort))) {
      commit(&a->drain);  // wind down: what was issued ends before the tensor memory is freed
      mbar_wait(&a->drain, 0, err);
    }
  } else if (warp == 2 && C::FP8) {
    // ---- scales of the tile's positions (1 where there is none: the position is masked)
    int tiles = 0;
    bool ok = true;
    for (int i = 0; ok && next_item<LONG>(p, pl, a, i, it, st); ++i) {
      for (int t = it.t0; ok && t < it.t1; ++t, ++tiles) {
        const int d = tiles & 1;
        int64_t row = tree_row(p, it.seq, t * kKeys);
        const bool bad = row < 0;
        row += p.pages.table ? 0 : (int64_t)it.seq * p.L;
        const int n = min(it.len - t * kKeys, kKeys) * C::NSC;
        const float* src = p.kv_scale + row * C::NSC;
        float v[2 * C::NSC + 1];
#pragma unroll
        for (int k = 0; k < 2 * C::NSC; ++k) v[k] = !bad && lane + 32 * k < n ? __ldg(src + lane + 32 * k) : 1.f;
        ok = __all_sync(0xffffffffu, wait_ahead(a, &a->sc_empty[d], ((tiles >> 1) & 1) ^ 1, err));
        if (!ok) break;
#pragma unroll
        for (int k = 0; k < 2 * C::NSC; ++k) {
          const int e = lane + 32 * k, key = e / (C::NSC + !C::NSC);
          sc_s[(d * C::NSC + e - key * C::NSC) * kKeys + key] = v[k];  // [scale of the row][position]
        }
        mbar_arrive(&a->sc_full[d]);
      }
    }
  } else if (warp >= 12) {
    // ---- converters (E4M3): this CTA's value columns, widened into swizzled bf16 boxes for the second product.
    // 16 codes per lane and step: eight positions of a box, four lanes each, so that eight lanes' 16-byte loads
    // and stores fall into different banks.
    const int w = warp - 12, c = lane & 3;
    int cs = 0, cph = 0, vs = 0, vph = 0;
    bool ok = true;
    for (int i = 0; ok && next_item<LONG>(p, pl, a, i, it, st); ++i) {
      for (int t = it.t0; ok && t < it.t1; ++t) {
        ok = __all_sync(0xffffffffu, wait_ahead(a, &a->c_full[cs], cph, err));
        if (!ok) break;
        const uint8_t* src = c_s + cs * kSlotC;
        uint4 raw[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const int key = 8 * (w + 4 * (k >> 2)) + (lane >> 2);
          raw[k] = *reinterpret_cast<const uint4*>(src + (k & 3) * kBoxC + key * 64 + ((c ^ ((key >> 1) & 3)) << 4));
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&a->c_empty[cs]);
        if (++cs == C::CS) cs = 0, cph ^= 1;
        ok = __all_sync(0xffffffffu, wait_ahead(a, &a->v_empty[vs], vph ^ 1, err));
        if (!ok) break;
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const int key = 8 * (w + 4 * (k >> 2)) + (lane >> 2);
          uint8_t* d = v_s + vs * kSlotV + (k & 3) * kBox + key * 128;
          const uint4 v = raw[k];
          *reinterpret_cast<uint4*>(d + (((2 * c) ^ (key & 7)) << 4)) =
              make_uint4(e4m3x2_to_bf16x2(v.x, 0x1404), e4m3x2_to_bf16x2(v.x, 0x3424), e4m3x2_to_bf16x2(v.y, 0x1404),
                         e4m3x2_to_bf16x2(v.y, 0x3424));
          *reinterpret_cast<uint4*>(d + (((2 * c + 1) ^ (key & 7)) << 4)) =
              make_uint4(e4m3x2_to_bf16x2(v.z, 0x1404), e4m3x2_to_bf16x2(v.z, 0x3424), e4m3x2_to_bf16x2(v.w, 0x1404),
                         e4m3x2_to_bf16x2(v.w, 0x3424));
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&a->v_full[vs]);
        if (++vs == C::VS) vs = 0, vph ^= 1;
      }
    }
  } else if (warp >= 4) {
    // ---- softmax warps: thread = row = tensor-memory lane, half h of the tile's positions
    const int w = warp - 4, h = w >> 2, quarter = w & 3, row = 32 * quarter + lane, tw = tid - 128;
    const uint32_t lane_base = tmem + ((uint32_t)(32 * quarter) << 16);
    const int rows = p.q_per_seq * p.H;
    int tile = 0, items = 0;
    uint32_t su = 0;
    bool ok = true;

    for (int i = 0; next_item<LONG>(p, pl, a, i, it, st); ++i) {
      if (SHARED && it.t0 >= it.t1) continue;
      const int row_lo = first_row(it);
      const int64_t at = first_in_out(it, rows, row_lo);  // the item's first row in out and lse
      const int nrows = rows_of(it, rows, row_lo);
      if (!SHARED && it.t0 >= it.t1) {  // nothing to see: padding nodes, or an empty sequence
        if (rank == 0) {
          for (int k = tw; k < nrows * (kDv / 8); k += 256)
            reinterpret_cast<uint4*>(p.out + at * kDv)[k] = make_uint4(0u, 0u, 0u, 0u);
          if (p.lse && tw < nrows) p.lse[at + tw] = -INFINITY;
        }
        continue;
      }
      float row_scale = p.scale_log2;
      // The query's rows, their boxes in the order of the slots: the first ones into tensor memory, the others into
      // shared memory (the previous item's products are done: its epilogue waited for them).  A warp takes half h of
      // each box of its 32 rows; four lanes read 64 bytes of a row (a lane per row would touch 32 lines per load:
      // 6.7 us for the whole), and 2 KB per warp of the other boxes' memory turn them into rows per lane.
      {
        const int r4 = lane >> 2, c4 = lane & 3;
        const __nv_bfloat16* src = p.q + (at + 32 * quarter) * kDqk + 32 * h + 8 * c4;
        uint8_t* turn = q_s + w * 2048;
        uint32_t top = 0;
        auto load = [&](int j, int i) -> uint4 {  // this lane's chunk of box j, row 8 i + r4 of the warp's
          const int r = 8 * i + r4;
          if (32 * quarter + r >= nrows) return make_uint4(0u, 0u, 0u, 0u);
          return __ldg(reinterpret_cast<const uint4*>(src + r * kDqk + 64 * (j < 8 ? j ^ (rank << 2) : 8)));
        };
        auto greatest = [&](const uint4& u) {
          top = __vmaxu2(top, __vmaxu2(__vmaxu2(u.x & 0x7FFF7FFFu, u.y & 0x7FFF7FFFu), __vmaxu2(u.z & 0x7FFF7FFFu, u.w & 0x7FFF7FFFu)));
        };
        constexpr int kBatch = 3;
#pragma unroll(C::FP8 ? 3 : 1)  // (rolled, bf16: 0.5 us less for the first item, whose code is not in the caches)
        for (int j0 = 0; j0 < 9; j0 += kBatch) {
          uint4 u[kBatch][4];
#pragma unroll
          for (int b = 0; b < kBatch; ++b)
#pragma unroll
            for (int i = 0; i < 4; ++i) u[b][i] = load(j0 + b, i);
#pragma unroll
          for (int b = 0; b < kBatch; ++b) {
            const int j = j0 + b;
            if (j < C::BT) {
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                const int r = 8 * i + r4;
                *reinterpret_cast<uint4*>(turn + r * 64 + ((c4 ^ ((r >> 1) & 3)) << 4)) = u[b][i];
              }
              __syncwarp();
              uint32_t v[16];
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                const uint4 x = *reinterpret_cast<const uint4*>(turn + lane * 64 + ((k ^ ((lane >> 1) & 3)) << 4));
                if (C::FP8) greatest(x);
                v[4 * k] = x.x, v[4 * k + 1] = x.y, v[4 * k + 2] = x.z, v[4 * k + 3] = x.w;
              }
              tmem_st16(lane_base + C::COL_Q + 32 * j + 16 * h, v);
              __syncwarp();
            } else {
              if (j == C::BT) softmax_bar();  // no warp turns rows any more
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                const int r = 32 * quarter + 8 * i + r4;
                *reinterpret_cast<uint4*>(q_s + (j - C::BT) * C::Q_BOX + r * 128 + (((4 * h + c4) ^ (r & 7)) << 4)) = u[b][i];
              }
            }
          }
        }
        if constexpr (C::FP8) {
          // In place: scaled by a power of two, the row's largest value to [2^7, 2^8), and split into two 8-bit parts,
          // per box and half of its columns 32 bytes of the one, then of the other.
          auto mine = [&](int j, int k) {
            return reinterpret_cast<uint4*>(q_s + (j - C::BT) * C::Q_BOX + row * 128 + (((4 * h + k) ^ (row & 7)) << 4));
          };
          __syncwarp();
#pragma unroll
          for (int j = C::BT; j < 9; ++j)
#pragma unroll
            for (int k = 0; k < 4; ++k) greatest(*mine(j, k));
          a->mx[0][h][row] = __uint_as_float(max(top & 0xFFFFu, top >> 16) << 16);
          tmem_wait_st();
          pair_bar(quarter);
          const int e = (__float_as_int(fmaxf(a->mx[0][0][row], a->mx[0][1][row])) >> 23) - 127;
          const int up = min(7 - e, 126);
          const float mul = __int_as_float((up + 127) << 23);
          // (an infinity or NaN in the row: every logit is NaN)
          row_scale = e == 128 ? __int_as_float(0x7FC00000) : p.scale_log2 * __int_as_float((127 - up) << 23);
#pragma unroll 1
          for (int j = 0; j < 9; ++j) {
            float raw[16];
            if (j < C::BT) {
              tmem_ld_sync(lane_base + C::COL_Q + 32 * j + 16 * h, raw);
            } else {
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                const uint4 x = *mine(j, k);
                raw[4 * k] = __uint_as_float(x.x), raw[4 * k + 1] = __uint_as_float(x.y);
                raw[4 * k + 2] = __uint_as_float(x.z), raw[4 * k + 3] = __uint_as_float(x.w);
              }
            }
            uint32_t v[16];
#pragma unroll
            for (int k = 0; k < 8; ++k) {
              uint32_t a0, a1, b0, b1;
              split_fp8(__float_as_uint(raw[2 * k]), mul, a0, b0);
              split_fp8(__float_as_uint(raw[2 * k + 1]), mul, a1, b1);
              v[k] = a0 | a1 << 16;
              v[8 + k] = b0 | b1 << 16;
            }
            if (j < C::BT) {
              tmem_st16(lane_base + C::COL_Q + 32 * j + 16 * h, v);
            } else {
#pragma unroll
              for (int k = 0; k < 4; ++k) *mine(j, k) = make_uint4(v[4 * k], v[4 * k + 1], v[4 * k + 2], v[4 * k + 3]);
            }
          }
          pair_bar(quarter);  // (the maxima have been read)
        }
        tmem_wait_st();
        tc_fence_before();
        fence_proxy_async_smem();
        if (ok) mbar_arrive(&a->q_full);
      }
      const int node = min((row_lo + row) / p.H, p.q_per_seq - 1);
      float m = -INFINITY, l = 0.f;

      for (int t = it.t0; t < it.t1; ++t, ++tile) {
        // ---- logits, scaled and masked
        float x[32];
        const float* sc = sc_s + (tile & 1) * kKeys * C::NSC + 32 * h;
        float4 scale[C::FP8 ? 8 : 1];  // of the positions (tile scales: of one column tile after another)
        auto scales = [&](const float* from) {
          if constexpr (C::FP8) {
#pragma unroll
            for (int k = 0; k < 8; ++k) scale[k] = *reinterpret_cast<const float4*>(from + 4 * k);
          }
        };
        if constexpr (C::TILED) {
#pragma unroll
          for (int k = 0; k < 32; ++k) x[k] = 0.f;
        }
#pragma unroll 1
        for (int g = 0; g < C::GROUPS; ++g, ++su) {
          // (the groups are in the order of the slots, the scales in that of the columns; those are loaded before the
          // wait where the wait for the first accumulation has not shown that they are there)
          if (C::TILED) {
            if (g == 0) ok = wait(a, &a->sc_full[tile & 1], (tile >> 1) & 1, err) && ok;
            scales(sc + kKeys * (g < 4 ? g ^ (rank << 1) : 4));
          }
          ok = wait(a, &a->s_full[su % C::SB], (su / C::SB) & 1, err) && ok;
          if (!C::TILED) scales(sc);
          tc_fence_after();
          float s[32];
          tmem_ld_sync(lane_base + C::COL_S + kKeys * (su % C::SB) + 32 * h, s);
          tc_fence_before();
          __syncwarp();
          if (lane == 0 && ok) mbar_arrive(&a->s_empty[su % C::SB]);
          const float2 rs = make_float2(row_scale, row_scale);
#pragma unroll
          for (int k = 0; k < 32; k += 2) {
            const float2 z = make_float2(s[k], s[k + 1]);
            float2 f = rs, y;
            if constexpr (C::FP8) f = k & 2 ? make_float2(scale[k >> 2].z, scale[k >> 2].w) : make_float2(scale[k >> 2].x, scale[k >> 2].y);
            if constexpr (C::TILED) y = make_float2(fmaf(f.x, z.x, x[k]), fmaf(f.y, z.y, x[k + 1]));
            else if constexpr (C::FP8) y = mul2(z, mul2(f, rs));
            else y = mul2(z, rs);
            x[k] = y.x, x[k + 1] = y.y;
          }
        }
        if constexpr (C::TILED) {
#pragma unroll
          for (int k = 0; k < 32; ++k) x[k] *= row_scale;
        }
        const bool bad = p.pages.table && a->tile_bad[tile & 7];
        const bool edge = (t + 1) * kKeys > it.ctx;  // drafted positions, or the sequence's end
        uint32_t clear = 0;
        if (edge || bad) {
          const uint32_t see = bad ? 0u : (uint32_t)(seen_bits(p, it, node, t) >> (32 * h));
#pragma unroll
          for (int k = 0; k < 32; ++k)
            if (!((see >> k) & 1)) x[k] = -INFINITY;
          clear = ~see;
        }
        // ---- the rows' maxima over the tile
        float mx[4] = {x[0], x[1], x[2], x[3]};
#pragma unroll
        for (int k = 4; k < 32; ++k) mx[k & 3] = fmaxf(mx[k & 3], x[k]);
        const float mine = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
        a->mx[tile & 1][h][row] = mine;
        if (!C::FP8 && edge) {
          // zero the value columns of positions that some row does not see (the logits have been taken), so that 0 * value
          // is 0: a position past the end always, another one only if it holds something that is not finite (and who
          // sees that has no finite logit)
          clear = __reduce_or_sync(0xffffffffu, clear);
          if (lane == 0) a->clear[tile & 1][w] = clear;
          softmax_bar();
          const int key = tw >> 2;  // a position, one of its four boxes
          uint32_t word = 0u;
#pragma unroll
          for (int k = 0; k < 4; ++k) word |= a->clear[tile & 1][(key >> 5) * 4 + k];
          if ((word >> (key & 31)) & 1) {
            uint8_t* line = v_s + (tile % C::VS) * kSlotV + (tw & 3) * kBox + key * 128;
            bool zero = t * kKeys + key >= it.len;
            if (!zero) {
#pragma unroll
              for (int c = 0; c < 8; ++c) {
                const uint4 u = *reinterpret_cast<const uint4*>(line + 16 * c);
                const uint32_t ws[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
                for (int q = 0; q < 4; ++q)
                  zero |= (ws[q] & 0x7F80u) == 0x7F80u || (ws[q] & 0x7F800000u) == 0x7F800000u;
              }
            }
            if (zero) {
#pragma unroll
              for (int c = 0; c < 8; ++c) *reinterpret_cast<uint4*>(line + 16 * c) = make_uint4(0u, 0u, 0u, 0u);
              fence_proxy_async_smem();
            }
          }
          __syncwarp();
        } else {
          pair_bar(quarter);
        }
        const float top = fmaxf(mine, a->mx[tile & 1][h ^ 1][row]);
        // the second product of the tile before is done: O may be rescaled, P written
        if (tile > 0) ok = wait(a, &a->pv_done, (tile - 1) & 1, err) && ok;
        // the reference maximum moves, in both halves' warps alike
        if (__any_sync(0xffffffffu, top > m + kLazy)) {
          float f = 1.f;
          if (top > m + kLazy) {  // (m = -inf: nothing summed yet, the factor is 0)
            f = ex2(m - top);
            m = top;
            l *= f;
          }
          if (t > it.t0) {
            tc_fence_after();
#pragma unroll 1
            for (int c = 128 * h; c < 128 * h + 128; c += 16) {
              float o[16];
              tmem_ld_sync(lane_base + kColO + c, o);
              uint32_t v[16];
#pragma unroll
              for (int k = 0; k < 16; ++k) v[k] = __float_as_uint(o[k] * f);
              tmem_st16(lane_base + kColO + c, v);
            }
            tmem_wait_st();
          }
        }
        // ---- weights, times the positions' scales (a hidden position's weight is 0 whatever its scale holds)
        const float mu = m == -INFINITY ? 0.f : m;
        float2 sum = make_float2(0.f, 0.f);
#pragma unroll
        for (int k = 0; k < 32; k += 2) {
          if constexpr (C::TILED) {
            x[k] = ex2(x[k] - mu), x[k + 1] = ex2(x[k + 1] - mu);
            sum.x += x[k], sum.y += x[k + 1];
          } else {
            const float2 y = add2(make_float2(x[k], x[k + 1]), make_float2(-mu, -mu));
            x[k] = ex2(y.x), x[k + 1] = ex2(y.y);
            sum = add2(sum, make_float2(x[k], x[k + 1]));
          }
        }
        l += sum.x + sum.y;
        const bool hides = C::FP8 && (edge || bad);
#pragma unroll
        for (int b = 0; b < C::PC; ++b) {
          if constexpr (C::TILED) scales(sc + kKeys * (2 * rank + b));
          uint32_t v[16];
#pragma unroll
          for (int k = 0; k < 32; k += 2) {
            float z0 = x[k], z1 = x[k + 1];
            if constexpr (C::FP8) {
              const float4 f = scale[k >> 2];
              const float2 f2 = k & 2 ? make_float2(f.z, f.w) : make_float2(f.x, f.y);
              if constexpr (C::TILED) {
                z0 *= f2.x, z1 *= f2.y;
              } else {
                const float2 z = mul2(make_float2(z0, z1), f2);
                z0 = z.x, z1 = z.y;
              }
              if (hides) z0 = x[k] == 0.f ? 0.f : z0, z1 = x[k + 1] == 0.f ? 0.f : z1;
            }
            v[k >> 1] = pack_bf16(z0, z1);
          }
          tmem_st16(lane_base + C::COL_P + 32 * b + 16 * h, v);
        }
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0 && ok) {
          mbar_arrive(&a->p_full);
          if constexpr (C::FP8) mbar_arrive(&a->sc_empty[tile & 1]);
        }
      }
      // ---- the rows' sums (their halves added in the same order everywhere)
      float now = 1.f, before = 0.f;  // what brings this stretch's sums, and those of the ones before, to their maximum
      float4* sum_o = nullptr;        // this thread's: no other one touches them
      const bool last = !LONG || it.t1 == st.stop;
      if (LONG && !(st.first && last)) {
        sum_o = pl.sum_o + ((int64_t)blockIdx.x * 64 + 32 * h) * kRows + row;
        float2* ml = pl.sum_ml + ((int64_t)blockIdx.x * 2 + h) * kRows + row;
        const float2 old = st.first ? make_float2(-INFINITY, 0.f) : *ml;
        const float M = fmaxf(m, old.x);
        now = m == -INFINITY ? 0.f : ex2(m - M);
        before = old.x == -INFINITY ? 0.f : ex2(old.x - M);
        m = M;
        l = fmaf(old.y, before, l * now);
        if (!last) *ml = make_float2(m, l);
      }
      a->sum[h][row] = l;
      pair_bar(quarter);
      l = a->sum[0][row] + a->sum[1][row];
      const bool live = row < nrows && (SHARED || (row_lo + row) / p.H < it.fresh);
      const int part_rows = SHARED ? (nrows + 7) & ~7 : kRows;  // rows of this partial result
      const float inv = live && l != 0.f ? 1.f / l : 0.f;
      if (h == 0 && last) {
        // (each CTA's own: the two sum the logits' columns in different orders, so that their maxima may differ)
        if (SHARED ? row < nrows : it.slot >= 0) pl.part_ml[SHARED ? (int64_t)it.slot * 2 + rank * part_rows + row : ((int64_t)it.slot * 2 + rank) * kRows + row] = make_float2(m, l);
        else if (!SHARED && rank == 0 && p.lse && row < nrows) p.lse[at + row] = !live || l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
      }
      ok = wait(a, &a->o_done, items & 1, err) && ok;
      tc_fence_after();
#pragma unroll 1
      for (int c = 128 * h; c < 128 * h + 128; c += 32) {
        float o[32];
        tmem_ld_sync(lane_base + kColO + c, o);
        if (LONG && sum_o) {
#pragma unroll
          for (int k = 0; k < 8; ++k, sum_o += kRows) {
            float4 v = st.first ? make_float4(0.f, 0.f, 0.f, 0.f) : *sum_o;
            v.x = fmaf(v.x, before, o[4 * k] * now), v.y = fmaf(v.y, before, o[4 * k + 1] * now);
            v.z = fmaf(v.z, before, o[4 * k + 2] * now), v.w = fmaf(v.w, before, o[4 * k + 3] * now);
            if (!last) *sum_o = v;
            o[4 * k] = v.x, o[4 * k + 1] = v.y, o[4 * k + 2] = v.z, o[4 * k + 3] = v.w;
          }
        }
        if (!last) {
        } else if (row < nrows && (SHARED || it.slot >= 0)) {
          float4* dst = pl.part_o + (SHARED ? (int64_t)it.slot * (kDv / 4) + (256 * rank + c) / 4 * part_rows
                                            : ((int64_t)it.slot * (kDv / 4) + (256 * rank + c) / 4) * kRows) + row;
#pragma unroll
          for (int k = 0; k < 8; ++k) dst[k * part_rows] = make_float4(o[4 * k], o[4 * k + 1], o[4 * k + 2], o[4 * k + 3]);
        } else if (row < nrows) {
          uint4* dst = reinterpret_cast<uint4*>(p.out + (at + row) * kDv + 256 * rank + c);
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            uint32_t v[4];
#pragma unroll
            for (int q = 0; q < 4; ++q)
              v[q] = live ? pack_bf16(o[8 * k + 2 * q] * inv, o[8 * k + 2 * q + 1] * inv) : 0u;
            dst[k] = make_uint4(v[0], v[1], v[2], v[3]);
          }
        }
        __syncwarp();
      }
      pair_bar(quarter);  // the sums have been read
      tc_fence_before();
      if (lane == 0 && ok) mbar_arrive(&a->o_free);
      ++items;
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 0) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// The cache's tensor map: boxes of 64 columns x 64 positions.
template <int FMT>
cudaError_t cache_map(CUtensorMap* tm, const TreeAttnParams& p) {
  using C = Cfg<FMT>;
  const bool paged = p.pages.table != nullptr;
  const cuuint64_t n = paged ? (cuuint64_t)p.pages.num_blocks * p.pages.block_size : (cuuint64_t)p.L;
  const cuuint64_t dims[3] = {(cuuint64_t)kDqk, n, paged ? 1 : (cuuint64_t)p.n_seq};
  const cuuint64_t strides[2] = {(cuuint64_t)p.kv_row_stride,
                                 paged || p.n_seq == 1 ? n * (cuuint64_t)p.kv_row_stride : (cuuint64_t)p.kv_seq_stride};
  memset(tm, 0, sizeof(*tm));
  const cuuint32_t box[3] = {64, kKeys, 1};
  if (encode_tensor_map(tm, C::FP8 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3,
                        const_cast<uint8_t*>(p.kv), dims, strides, box,
                        C::FP8 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B) != CUDA_SUCCESS)
    return cudaErrorInvalidValue;
  return cudaSuccess;
}

}  // namespace
}  // namespace dsa
