// Attention of prompts, or chunks of them, over expanded keys and values (dsa_expanded_attn): head h of query i of sequence s,
// with m queries over n positions,
//   logit[p] = sm_scale (q[:128] . k[p, h] + q[128:] . k_rope[p]),  out = sum_p softmax(logit)[p] v[p, h]
// over the positions p <= n - m + i (causal) or all n.  Sequences are packed, one behind another.
//
// A CTA takes 256 queries of a head, two tiles of 128, and walks tiles of 128 positions, each loaded once for both.  Per tile
// of queries and positions:
//   * S[128 x 128] = Q K^T: 12 steps of K = 16, both operands in shared memory (the rotary columns are a box of K of their
//     own, that all heads read);
//   * one pass over the positions keeps a reference maximum m and a sum l per row as in tree_kernel.cuh: m moves only where
//     a tile's maximum exceeds it by more than 2^8, so that O is rescaled rarely;
//   * P takes the place of S in tensor memory, and O[128 x 128] += P V: 8 steps, A in tensor memory, V MN-major.  P is rounded to
//     bf16: an MMA's operands have one 16-bit type, which is V's (the next wider one, tf32, runs at half the rate and would want V
//     widened too).  A weight is off by at most 2^-8 of itself, as the output is by its own rounding; an output over normal
//     values is 1.2 to 1.4 times as far from 64 bits as one of fp32 weights.
// Tensor memory: S and O of both tiles, 4 x 128 columns.  The two tiles take turns: while eight warps take the softmax of one (a
// thread a row and half of the positions), the tensor cores multiply for the other: O += P V of the last positions, then S
// of the next ones.
// The instructions of one thread execute in order, so that S may follow the P V that reads P in the same columns, and a
// finished S means that the P V before it has finished.
//
// Shared memory: both tiles of Q (96 KB) and a ring of eight boxes of 64 columns x 128 positions (three of K, two of V per
// tile), whose boxes are refilled as soon as their product is done.
//
// Positions that some row of a tile of positions does not see: their logits become -inf; what lies behind the sequence's
// end is cleared from V, and infinities and NaN at positions that only some rows see too (0 * inf is NaN), which are
// added afterwards for the rows that see them.
//
// Work: blocks of 256 queries, each for every head (plan_kernel: the lengths are on the device).  Two ways to share it out:
//   * many blocks: dealt to the CTAs back and forth, the longest first; what is left behind whole rounds is cut for all CTAs;
//   * few: laid end to end and cut into one span of tiles for each CTA; a block that is cut leaves fp32 partial results, which
//     the CTA that finishes the last of them merges, in the order of the positions (so results do not depend on which that is).
// The tensor cores truncate their sums, and O loses up to 2^-23 of itself per step of 16 positions, 0.05 % over 65536.  Longer
// contexts are walked in stretches of 512 tiles, whose O and l are added up in fp32, in memory (a form of the kernel of its own,
// taken where max_len, or without it N, is above 65536; nine prompts of 8192 take 1 to 4 % longer in it, shorter sequences
// the same).
//
// Bound: tensor cores, 12 x 64 + 8 x 64 cycles per tile of 128 x 128, beside shared memory, which the first product's operands
// fill for as long (4 + 4 KB a step).  Measured: one prompt of 8192 x 16 heads 234 us (1470 TFLOP/s of what causality leaves; tensor cores
// busy 61 % of the time); two chunks of 1125 over 12288 positions 252 (1165; K and V, 200 MB, do not fit the L2); seven
// prompts of 150 17.  What is left: two tiles of queries are in flight, and each waits for its softmax (1100 cycles) and the hand-overs
// (three, of 100 to 300 cycles) before its products (1280) go on, so that a pair of tiles takes 4000 cycles where 2560 would do;
// and K arrives about 500 cycles late, because its places in the ring are given back that late (the bytes do not matter: a third
// of them takes as long).
// Without any softmax, hand-overs and products alone take 205 us, the softmax without products 176.
// Tried: P handed over in halves 337 us (at 263 of the whole), K's boxes handed over one by one 307 (at 266), strict turns of the two
// issuers 244, S read twice instead of held in registers 274 (at 266).
#include <limits.h>
#include <stddef.h>
#include <string.h>

#include <initializer_list>

#include "tc_common.cuh"

namespace dsa {
namespace {

constexpr float kLn2 = 0.6931471805599453f;
constexpr int kNope = 128, kRope = 64, kDv = 128;
constexpr int kTile = 128;                  // rows of a tile of queries, positions of a tile of them
constexpr int kBlock = 2 * kTile;
constexpr int kBox = kTile * 128;           // 64 columns of 128 rows
constexpr int kRing = 8;
constexpr int kOffRing = 6 * kBox;          // two tiles of Q first
constexpr int kThreads = 640;
constexpr float kLazy = 8.f;                // log2 growth of a row's maximum that is left unscaled
constexpr int kSms = 152;
constexpr int kStretch = 512;                  // tiles whose products are summed in tensor memory, at most
constexpr int kLengths = 512;                  // that the counting sort tells apart
constexpr int kFixed = 3;                      // what starting on a block costs, in tiles
constexpr int kMinSpan = 4;                    // tiles of a span, at least
constexpr int kMinPart = 16;                   // and of a part of an item of the list's last round
constexpr int kMaxSeq = 4096;
constexpr int kMaxRows = 1 << 24;              // of q, and of k and v: fewer
constexpr uint32_t kColS = 0, kColO = 256;

// What the planning kernel leaves for the others.
constexpr int kSpanItems = 3 * kSms;         // fewer than this many blocks and heads may be cut into spans
struct alignas(16) SpanItem {  // (read as two 16-byte words)
  int seq, q0, t0, t1, head, slot;  // head: with the item's number << 8; slot: of the partial result, -1: the whole block
  int parts;                        // of this head of the block (0: nothing to do here)
  int first;                        // span, or place in the last round, of the first of them
};
struct Plan {
  int done[kSpanItems][2];                   // parts that are finished, of each block and head and each tile of queries
  int4 place[kSms];                           // of each CTA: items of the list of work; its own: first, number
  SpanItem list[kSpanItems + kSms];
};

static_assert(sizeof(SpanItem) == 32 && offsetof(Plan, list) % 16 == 0 && offsetof(Plan, place) % 16 == 0, "vector reads");

struct ExpandedAttnParams {
  const int32_t* q_start;  // [n_seq + 1]
  const int32_t* kv_start; // [n_seq + 1]
  int n_seq, T, N, H;      // rows of q, rows of k and v
  int max_len;             // positions of the longest sequence, at most
  bool causal;
  float scale_log2;        // sm_scale * log2(e)
  const __nv_bfloat16* v;  // (element strides)
  int64_t v_row_stride, v_head_stride;
  __nv_bfloat16* out;      // [T, H, 128]
  float* lse;              // [T, H] or null
  int shift;               // of tiles, to lengths of at most kLengths
  int grid;                // CTAs of the attention kernel
  bool may_span;           // blocks may be cut into spans (see plan_kernel)
  // workspace
  Plan* plan;
  int4* work;              // [max_work]
  int max_work;
  float2* part_ml;         // partial results: reference maximum and sum of weights, output
  float* part_o;
  float2* sum_ml;          // per CTA, of a block in stretches: the same of the stretches so far, a thread's own
  float4* sum_o;
  int* err;                // device error word
};

struct Aux {
  // (k and v: of tiles of positions of even and of odd number)
  uint64_t q_full[2], q_empty[2], k_full[2], k_empty[2], v_full[2], v_ready[2], v_empty[2], s_full[2], p_full[2], o_done[2], o_free[2], drain[2];
  uint32_t tmem;
  int abort;
  int not_finite;  // an infinity or NaN was cleared from V
  int last[2];     // this CTA has finished the last part of a tile's rows
  float rows[2][2][kTile];  // per tile of queries and half of the positions: the rows' maxima, at an item's end their sums
};
constexpr int kOffAux = kOffRing + kRing * kBox;
constexpr int kSmem = kOffAux + (int)sizeof(Aux);  // (without room to align: the array's own alignment does it)
static_assert(kSmem <= 227 * 1024, "shared memory");

struct Work {
  int seq, q0, t0, t1;  // queries q0 ... of the sequence, tiles [t0, t1) of positions
  int entry;            // of the plan's list, -1: of the list of work (its slot, parts and so on are read when they are needed)
  bool begins, ends;    // the first, the last stretch of it
};

struct Facts {
  int q_row, m;   // the sequence's first row of q, its queries
  int k_row, n;   // its first row of k and v, its positions
  int nrows;      // queries of the block
  int first, step;  // row i of the block sees first + i * step positions (clamped to [0, n])
};

__device__ __forceinline__ void seq_facts(const ExpandedAttnParams& p, int seq, Facts& f) {
  f.q_row = min(max(p.q_start[seq], 0), p.T);
  f.m = min(max(p.q_start[seq + 1], f.q_row), p.T) - f.q_row;
  f.k_row = min(max(p.kv_start[seq], 0), p.N);
  f.n = min(min(max(p.kv_start[seq + 1], f.k_row), p.N) - f.k_row, p.max_len);
}
__device__ __forceinline__ Facts block_facts(const ExpandedAttnParams& p, int seq, int q0) {
  Facts f;
  seq_facts(p, seq, f);
  f.nrows = min(kBlock, f.m - q0);
  f.step = p.causal ? 1 : 0;
  f.first = p.causal ? f.n - f.m + q0 + 1 : f.n;
  return f;
}
__device__ __forceinline__ int sees(const Facts& f, int i) { return min(max(f.first + i * f.step, 0), f.n); }
__device__ __forceinline__ int tiles_of(int positions) { return (positions + kTile - 1) / kTile; }
// Tiles of positions of a block: those that its last query sees.
__device__ __forceinline__ int block_tiles(const Facts& f) { return tiles_of(sees(f, f.nrows - 1)); }
// Tiles of [w.t0, w.t1) that tile t of the queries takes.
__device__ __forceinline__ int tiles_for(const Facts& f, const Work& w, int t) {
  if (f.nrows <= t * kTile) return 0;
  return max(min(w.t1, tiles_of(sees(f, min(f.nrows, (t + 1) * kTile) - 1))) - w.t0, 0);
}

// Tiles of positions of an item that are looked through for what some row does not see: of [0, n0) those past what the
// block's first row sees, of [n0, n) those past what the second tile's first row sees.
__device__ __forceinline__ int edges_of(const Facts& f, const Work& w, int n0, int n) {
  return max(n0 - max(sees(f, 0) / kTile - w.t0, 0), 0) + max(n - max(sees(f, kTile) / kTile - w.t0, n0), 0);
}

// ---------------------------------------------------------------------------------------------
// the list of work: blocks, the longest first (a counting sort by tiles)

__global__ void __launch_bounds__(1024) plan_kernel(const ExpandedAttnParams p) {
  __shared__ int base[kMaxSeq + 1];          // blocks before each sequence
  __shared__ int place[kLengths + 2];        // by tiles: how many, then where the next goes (the last entry: of threads without a block)
  __shared__ int longest_block;
  __shared__ int warp_sum[32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  int run = 0;
  for (int s0 = 0; s0 < p.n_seq; s0 += 1024) {  // running sums of the sequences' blocks
    const int s = s0 + tid;
    Facts f;
    int c = 0;
    if (s < p.n_seq) {
      seq_facts(p, s, f);
      c = (f.m + kBlock - 1) / kBlock;
      // a start that decreases or lies outside of the rows, a sequence longer than max_len
      if ((int64_t)p.kv_start[s + 1] - p.kv_start[s] != f.n || (int64_t)p.q_start[s + 1] - p.q_start[s] != f.m)
        record_error(p.err, DSA_DEVERR_INDEX_RANGE);
    }
    int incl = c;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int u = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += u;
    }
    if (lane == 31) warp_sum[warp] = incl;
    __syncthreads();
    if (warp == 0) {
      int v = warp_sum[lane];
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o) v += u;
      }
      warp_sum[lane] = v;
    }
    __syncthreads();
    if (s < p.n_seq) base[s] = run + incl - c + (warp ? warp_sum[warp - 1] : 0);
    run += warp_sum[31];
    __syncthreads();
  }
  if (tid == 0) base[p.n_seq] = run;
  for (int i = tid; i < kLengths + 2; i += 1024) place[i] = 0;
  if (tid == 0) longest_block = 0;
  __syncthreads();
  auto find = [&](int b, int& q0) {  // the sequence of block b, and the block's first query
    int lo = 0, hi = p.n_seq - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (base[mid] <= b) lo = mid;
      else hi = mid - 1;
    }
    q0 = (b - base[lo]) * kBlock;
    return lo;
  };
  if (p.may_span && (int64_t)run * p.H < kSpanItems) {
    // Few blocks: laid end to end, a head of a block after another, each with a fixed cost before its tiles, and cut into one
    // span for each CTA, if that is shorter than dealing them out whole
    int q0 = 0, seq = 0, tiles = 0;
    if (tid < run) {
      seq = find(tid, q0);
      tiles = block_tiles(block_facts(p, seq, q0));
    }
    const int cost = tid < run ? tiles + kFixed : 0;
    int incl = cost, most = cost;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int u = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += u;
    }
    most = __reduce_max_sync(0xffffffffu, most);
    __shared__ int warp_most[32], before[kSpanItems + 1];  // (costs before each block, of one head)
    if (lane == 31) warp_sum[warp] = incl, warp_most[warp] = most;
    __syncthreads();
    int ahead = 0, all = 0, longest = 0;
    for (int i = 0; i < 32; ++i) {
      ahead += i < warp ? warp_sum[i] : 0;
      all += warp_sum[i];
      longest = max(longest, warp_most[i]);
    }
    if (tid < run) before[tid] = ahead + incl - cost;
    if (tid == run) before[run] = all;
    __syncthreads();
    const int items = run * p.H, total = all * p.H, W = max((total + p.grid - 1) / p.grid, kMinSpan);
    static_assert((int64_t)kSpanItems * (kMaxRows / kTile + kFixed) < 1 << 26, "costs are ints");
    const int whole = items <= p.grid ? longest : total / p.grid + longest / 2;
    if (W + 2 * kFixed < whole) {
      // The order: a sequence after another, of it a head after another, of that the blocks, so that the CTAs that read the
      // same keys and values are neighbours and do so at about the same time (two chunks of 1125 tokens over 12K positions,
      // 200 MB of keys and values: 260 us with the heads of a block side by side)
      auto seq_at = [&](auto&& start, int x) {  // the last sequence that starts at or before x
        int lo = 0, hi = p.n_seq - 1;
        while (lo < hi) {
          const int mid = (lo + hi + 1) >> 1;
          if (start(mid) <= x) lo = mid;
          else hi = mid - 1;
        }
        return lo;
      };
      auto item_at = [&](int x) {  // that holds cost x
        const int s = seq_at([&](int i) { return before[base[i]] * p.H; }, x), b0 = base[s], nb = base[s + 1] - b0;
        const int sum = before[b0 + nb] - before[b0], in = x - before[b0] * p.H, h = in / sum;
        int b = 0;
        while (b + 1 < nb && before[b0 + b + 1] - before[b0] <= in - h * sum) ++b;
        return b0 * p.H + h * nb + b;
      };
      if (tid < p.grid) {
        const int x0 = tid * W, x1 = min(x0 + W, total);
        int4 mine = make_int4(0, 0, 0, 0);
        if (x0 < total) {
          const int i0 = item_at(x0);
          mine = make_int4(0, i0 + tid, item_at(x1 - 1) - i0 + 1, 0);
        }
        p.plan->place[tid] = mine;
      }
      if (tid < items) {  // an item's pieces: entry of item i in span k: i + k
        const int s = seq_at([&](int i) { return base[i] * p.H; }, tid), b0 = base[s], nb = base[s + 1] - b0;
        const int head = (tid - b0 * p.H) / nb, b = b0 + (tid - b0 * p.H) % nb;
        SpanItem it = {};
        it.seq = s;
        it.q0 = (b - b0) * kBlock;
        it.head = head | tid << 8;
        p.plan->done[tid][0] = p.plan->done[tid][1] = 0;
        const int c = before[b + 1] - before[b], n = c - kFixed;
        const int begin = before[b0] * p.H + head * (before[b0 + nb] - before[b0]) + before[b] - before[b0], first = begin + kFixed;
        it.first = first / W;
        for (int k = begin / W; k <= (begin + c - 1) / W; ++k) {
          it.t0 = min(max(k * W - first, 0), n), it.t1 = max(min((k + 1) * W - first, n), it.t0);
          it.slot = it.t0 == 0 && it.t1 == n ? -1 : it.t0 == 0 ? 2 * k + 1 : 2 * k;
          it.parts = (n > 0 ? it.t0 == it.t1 : k != begin / W) ? 0 : n > 0 ? (first + n - 1) / W - first / W + 1 : 1;
          p.plan->list[tid + k] = it;
        }
      }
      return;
    }
  }
  // Blocks, the longest first: counted, then placed
  int most = 0;
  for (int b = tid; b < run; b += 1024) {
    int q0;
    const int seq = find(b, q0), n = block_tiles(block_facts(p, seq, q0));
    atomicAdd(&place[min(n >> p.shift, kLengths)], 1);
    most = max(most, n);
  }
  most = __reduce_max_sync(0xffffffffu, most);
  if (lane == 0) atomicMax(&longest_block, most);
  __syncthreads();
  {  // how many are longer, for each length: the running sum from the longest on
    static_assert(kLengths < 1024, "a thread a length");
    const int at = kLengths - tid, c = at >= 0 ? place[at] : 0;
    int incl = c;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int u = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += u;
    }
    if (lane == 31) warp_sum[warp] = incl;
    __syncthreads();
    int ahead = 0;
    for (int i = 0; i < warp; ++i) ahead += warp_sum[i];
    if (at >= 0) place[at] = ahead + incl - c;
    __syncthreads();
  }
  const int items = min(run, p.max_work) * p.H, rounds = items / p.grid, left = items % p.grid;
  // Where what is left behind whole rounds may be cut (below), blocks of equal length stay in the order of their numbers, a warp
  // placing its 32 after another: a block that is cut is summed in another order than one that is not, so which ones are may
  // not go by the warps' speed.  Elsewhere the order does not matter, and they go where an atomic puts them (4096 sequences of
  // 3 tokens of a head: 138 us, 144 in order).
  const bool ordered = left > 0 && p.grid / left > 1 && longest_block >= 2 * kMinPart;
  for (int b0 = 0; b0 < run; b0 += 1024) {
    const int b = b0 + tid;
    int4 item = make_int4(0, 0, 0, 0);
    int key = kLengths + 1, at = p.max_work;
    if (b < run) {
      item.x = find(b, item.y);
      item.w = block_tiles(block_facts(p, item.x, item.y));
      key = min(item.w >> p.shift, kLengths);
    }
    if (!ordered) {
      if (b < run) at = atomicAdd(&place[key], 1);
    } else {
      const uint32_t same = __match_any_sync(0xffffffffu, key), before = same & ((1u << lane) - 1);
      const int turns = min((run - b0 + 31) / 32, 32);
      for (int turn = 0; turn < turns; ++turn) {
        if (warp == turn) {
          at = place[key] + __popc(before);
          __syncwarp();
          if (before == 0) place[key] += __popc(same);
        }
        __syncthreads();
      }
    }
    if (b < run && at < p.max_work) p.work[at] = item;
  }
  __syncthreads();
  // What is left behind whole rounds, where that is half a round or less: its items are cut, into parts of kMinPart tiles at
  // least, for all CTAs (3.4 rounds of 16 heads: 8192 tokens over 20480 positions 1.01 ms, uncut 1.09; over 9216, whose last items
  // are of 8 to 24 tiles, cut into parts of 8 and more 0.419, uncut 0.407)
  if (tid < p.grid) {
    const int ways = left ? max(min(p.grid / left, p.work[rounds * p.grid / p.H].w / kMinPart), 1) : 1;  // (the longest of them)
    const int at = rounds & 1 ? p.grid - 1 - tid : tid, x = at / ways;
    p.plan->done[tid][0] = p.plan->done[tid][1] = 0;
    p.plan->place[tid] = make_int4(rounds + (ways == 1 && at < left), tid, ways > 1 && x < left, 0);
    if (ways > 1 && x < left) {
      const int i = rounds * p.grid + x;
      const int4 v = p.work[i / p.H];
      const int n = v.w, parts = max(min(ways, n / kMinPart), 1), part = at - x * ways;
      SpanItem it = {};
      it.seq = v.x, it.q0 = v.y;
      it.head = i % p.H | x << 8;
      it.parts = part < parts ? parts : 0;
      it.first = x * ways;
      it.t0 = (int)((int64_t)n * part / parts), it.t1 = (int)((int64_t)n * (part + 1) / parts);
      it.slot = parts == 1 ? -1 : 2 * at + (part == 0);
      p.plan->list[tid] = it;
    }
  }
}

// ---------------------------------------------------------------------------------------------

// Item r of this CTA: of the list of work, dealt back and forth, every head of an entry after another; then of its own
// list.
struct Mine {
  int rounds;
  int first, items;  // of its own
};
__device__ __forceinline__ bool get_work(const ExpandedAttnParams& p, const Mine& mine, int r, Work& w, int& head, Facts& f, bool& skip) {
  if (r >= mine.rounds) {
    if (r - mine.rounds >= mine.items) return false;
    w.entry = mine.first + r - mine.rounds;
    const int4* v = reinterpret_cast<const int4*>(p.plan->list + w.entry);
    const int4 a = v[0], b = v[1];
    w.seq = a.x, w.q0 = a.y, w.t0 = a.z, w.t1 = a.w;
    head = b.x & 255;
    skip = b.z == 0;
    f = block_facts(p, w.seq, w.q0);  // (once in each branch: behind both it costs the softmax warps 30 spilled registers)
    return true;
  } else {
    const int g = (int)gridDim.x, c = (int)blockIdx.x, i = r * g + (r & 1 ? g - 1 - c : c);
    const int4 v = p.work[i / p.H];
    head = i % p.H;
    w.seq = v.x, w.q0 = v.y, w.t0 = v.z, w.t1 = v.w, w.entry = -1;
    skip = false;
  }
  f = block_facts(p, w.seq, w.q0);
  return true;
}

// The next item with anything to do, or with LONG the next stretch of one.
struct Walk {
  int r = 0, stop = 0;  // the next item; where the one in hand ends
};
template <bool LONG>
__device__ __forceinline__ bool next_work(const ExpandedAttnParams& p, const Mine& mine, Walk& k, Work& w, int& head, Facts& f) {
  if (LONG && w.t1 < k.stop) {
    w.t0 = w.t1;
    w.begins = false;
  } else {
    bool skip;
    do {
      if (!get_work(p, mine, k.r++, w, head, f, skip)) return false;
    } while (skip);
    k.stop = w.t1;
    w.begins = true;
  }
  if (LONG) w.t1 = min(k.stop, w.t0 + kStretch);
  w.ends = w.t1 == k.stop;
  return true;
}

// Merge of partial results: out = sum_c 2^(m_c - M) o_c / sum_c 2^(m_c - M) l_c.  A warp takes a row, a lane four columns.
__device__ __forceinline__ void write_merged(const ExpandedAttnParams& p, int64_t row, float M, float l, float4 o) {
  const int lane = threadIdx.x & 31;
  const float inv = l == 0.f ? 0.f : 1.f / l;
  reinterpret_cast<uint2*>(p.out + row * kDv)[lane] = make_uint2(pack_bf16(o.x * inv, o.y * inv), pack_bf16(o.z * inv, o.w * inv));
  if (p.lse && lane == 0) p.lse[row] = l == 0.f ? -INFINITY : (M + log2f(l)) * kLn2;
}

// Rows [from, from + 128) of a block that was cut into spans, by eight warps, four rows of each at a time, the parts in order.
__device__ __forceinline__ void merge_parts(const ExpandedAttnParams& p, const Work& w, const Facts& f, int head, int parts, int first, int from, int warp) {
  constexpr int U = 4;
  const int lane = threadIdx.x & 31;
  for (int i0 = from + U * warp; i0 < min(from + kTile, f.nrows); i0 += 8 * U) {
    float M[U], l[U];
    float4 o[U];
#pragma unroll
    for (int u = 0; u < U; ++u) M[u] = -INFINITY, l[u] = 0.f, o[u] = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int q = 0; q < parts; ++q) {
      // the first part ends a span (its second slot), the others begin the spans behind it
      const int64_t slot = 2 * (first + q) + (q == 0);
      float2 ml[U];
      float4 v[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int64_t row = slot * kBlock + min(i0 + u, f.nrows - 1);
        ml[u] = __ldcg(p.part_ml + row);
        v[u] = __ldcg(reinterpret_cast<const float4*>(p.part_o + row * kDv) + lane);
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (ml[u].y == 0.f) continue;  // the row saw nothing there
        const float Mb = fmaxf(M[u], ml[u].x), mu = Mb == -INFINITY ? 0.f : Mb;
        const float a = exp2f(M[u] - mu), g = exp2f(ml[u].x - mu);
        M[u] = Mb;
        l[u] = fmaf(g, ml[u].y, l[u] * a);
        o[u].x = fmaf(g, v[u].x, o[u].x * a), o[u].y = fmaf(g, v[u].y, o[u].y * a);
        o[u].z = fmaf(g, v[u].z, o[u].z * a), o[u].w = fmaf(g, v[u].w, o[u].w * a);
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (i0 + u < f.nrows) write_merged(p, (int64_t)(f.q_row + w.q0 + i0 + u) * p.H + head, M[u], l[u], o[u]);
  }
}

// LONG: contexts of more than kStretch tiles, whose blocks are walked in stretches.
template <bool LONG>
__global__ void __launch_bounds__(kThreads, 1)
    expanded_attn_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                         const __grid_constant__ CUtensorMap tm_r, const __grid_constant__ CUtensorMap tm_v,
                         const ExpandedAttnParams p) {
  extern __shared__ __align__(1024) uint8_t smem[];
  uint8_t* ring = smem + kOffRing;
  Aux* a = reinterpret_cast<Aux*>(smem + kOffAux);
  const int tid = threadIdx.x, lane = tid & 31, warp = uniform(tid >> 5);
  int* err = p.err;

  if (warp == 0) {
    tmem_alloc(&a->tmem, 512);
    tmem_relinquish();
  }
  if (tid == 32) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&a->q_full[i], 1), mbar_init(&a->q_empty[i], 1);
      mbar_init(&a->s_full[i], 1), mbar_init(&a->p_full[i], 8);
      mbar_init(&a->o_done[i], 1), mbar_init(&a->o_free[i], 8);
      mbar_init(&a->k_full[i], 1), mbar_init(&a->k_empty[i], 2);  // (one arrival for each tile of queries)
      mbar_init(&a->v_full[i], 1), mbar_init(&a->v_ready[i], 8), mbar_init(&a->v_empty[i], 2);
      mbar_init(&a->drain[i], 1);
    }
    a->abort = 0;
    a->not_finite = 0;
    fence_mbar_init();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = a->tmem;
  pdl_wait();  // the plan
  Mine mine;
  const int4 place = p.plan->place[blockIdx.x];
  mine.rounds = place.x, mine.first = place.y, mine.items = place.z;

  Work w;
  w.t1 = 0;
  Facts f;
  int head;
  // Registers: 640 x 96 at launch; the softmax warps take what the others leave (128 x 64 + 512 x 104 = 61440)
  if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 64;");
    if (warp == 0) {
      // ---- producer
      if (lane == 0) {
        prefetch_tmap(&tm_q), prefetch_tmap(&tm_k), prefetch_tmap(&tm_r), prefetch_tmap(&tm_v);
        int uses[2] = {0, 0};
        int g = 0;  // tiles of positions so far; their boxes are 5 g (of K) ... 5 g + 4 (of V), in the ring's order
        bool ok = true;
        auto load = [&](const CUtensorMap* tm, uint64_t* bar, int box, int x, int z, bool flat) {
          uint8_t* dst = ring + (uint32_t)box % kRing * kBox;
          if (flat) tma_load_2d(dst, tm, bar, x, z);
          else tma_load_3d(dst, tm, bar, x, head, z);
        };
        // (looked at again at once: the ring holds 1.6 tiles, and what waits for a place arrives just in time; with pauses of 50 ns
        // 239 us instead of 236)
        auto done = [&](uint64_t* empty, int tile) { ok = ok && (tile < 0 || wait_here(a, &empty[tile & 1], (tile >> 1) & 1, err)); };
        auto query = [&](int t) {
          ok = ok && wait_here<50>(a, &a->q_empty[t], (uses[t] & 1) ^ 1, err);
          if (!ok) return;
          ++uses[t];
          mbar_arrive_expect_tx(&a->q_full[t], 3 * kBox);
          for (int b = 0; b < 3; ++b) tma_load_3d(smem + (3 * t + b) * kBox, &tm_q, &a->q_full[t], 64 * b, head, f.q_row + w.q0 + kTile * t);
        };
        for (Walk k; ok && next_work<LONG>(p, mine, k, w, head, f);) {
          const int n0 = tiles_for(f, w, 0), n1 = tiles_for(f, w, 1), n = max(n0, n1);
          if (n0) query(0);
          for (int j = 0; ok && j < n; ++j, ++g) {
            const int row = f.k_row + (w.t0 + j) * kTile;
            // the boxes of K take the places of the last one of K, and of V, two tiles ago
            done(a->k_empty, g - 2);
            if (!ok) break;
            uint64_t* bar = &a->k_full[g & 1];
            mbar_arrive_expect_tx(bar, 3 * kBox);
            load(&tm_k, bar, 5 * g, 0, row, false);
            done(a->v_empty, g - 2);
            if (!ok) break;
            load(&tm_k, bar, 5 * g + 1, 64, row, false);
            load(&tm_r, bar, 5 * g + 2, 0, row, true);
            if (j == 0 && n1) query(1);
            done(a->k_empty, g - 1);  // and V those of the first two of K of the last tile
            if (!ok) break;
            bar = &a->v_full[g & 1];
            mbar_arrive_expect_tx(bar, 2 * kBox);
            load(&tm_v, bar, 5 * g + 3, 0, row, false);
            load(&tm_v, bar, 5 * g + 4, 64, row, false);
          }
        }
        if (*reinterpret_cast<volatile int*>(&a->abort)) {  // wind down: the copies in flight land first
          for (int i = max(g - 2, 0); i <= g; ++i) {        // (of a tile that was not armed there is nothing to wait for but time)
            mbar_wait(&a->k_full[i & 1], (i >> 1) & 1, err);
            mbar_wait(&a->v_full[i & 1], (i >> 1) & 1, err);
          }
          for (int t = 0; t < 2; ++t) mbar_wait(&a->q_full[t], (uses[t] & 1) ^ 1, err);
        }
      }
      __syncwarp();
    } else if (warp <= 2) {
      // ---- MMA issuers, a warp for each tile of queries.  Issuing an instruction waits for the ones before it, but for a few,
      // and between two turns lie about 700 cycles of waits and arithmetic, in which the tensor cores run dry: with two warps
      // the other one's instructions fill them.  (8192-token prompt: one issuer 266 us, two 237.  Strict turns, which keep one
      // tile's products against the other's softmax: 244.)
      constexpr uint32_t idesc_qk = make_idesc(1, 1, kTile, kTile);
      constexpr uint32_t idesc_pv = idesc_qk | (1u << 16), idesc_pv64 = make_idesc(1, 1, kTile, 64) | (1u << 16);  // B (values) MN-major
      const uint32_t t = warp - 1;
      const uint32_t base = (uint32_t)uniform((int)tmem), col_s = base + kColS + kTile * t, col_o = base + kColO + kTile * t;
      const uint32_t q_lo = kmajor_lo(smem_u32(smem)) + 3 * t * (kBox >> 4), k_lo = kmajor_lo(smem_u32(ring));
      const uint32_t v_lo = mnmajor_lo(smem_u32(ring), kBox);
      int g = 0;               // tiles of positions before the item
      int used = 0, soft = 0;  // items and softmax tiles
      int edges = 0;           // tiles of positions that were looked through
      bool ok = true;
      for (Walk k; ok && uniform(next_work<LONG>(p, mine, k, w, head, f));) {
        const int n0 = uniform(tiles_for(f, w, 0)), n1 = uniform(tiles_for(f, w, 1)), n = max(n0, n1), nt = t ? n1 : n0;
        if (n == 0) continue;
        const int least0 = sees(f, 0), least1 = sees(f, kTile);
        // A turn: O += P V over positions j, and S of positions j + 1, as far as there are any.  One wait, a lane per barrier (a
        // wait costs about 120 cycles even when there is nothing to wait for)
        for (int j = -1; ok && j < n; ++j) {
          const bool pv = j >= 0 && j < nt, qk = j + 1 < nt;
          const int gv = g + j, gk = gv + 1;
          const uint32_t v0 = (uint32_t)uniform((5 * gv + 3) & (kRing - 1)), V = v_lo + v0 * (kBox >> 4);
          uint32_t B[3];
#pragma unroll
          for (int b = 0; b < 3; ++b) B[b] = k_lo + (uint32_t)uniform((5 * gk + b) & (kRing - 1)) * (kBox >> 4);
          uint64_t* bar = j + 1 < n ? &a->k_full[gk & 1] : &a->v_full[gv & 1];
          uint32_t parity = j + 1 < n ? (gk >> 1) & 1 : (gv >> 1) & 1;
          if (j >= 0 && lane == 1) bar = &a->v_full[gv & 1], parity = (gv >> 1) & 1;
          if (pv && lane == 2) bar = &a->p_full[t], parity = soft & 1;
          // V is looked through where a row of the first tile that takes it does not see all of it
          const bool edge = j >= 0 && (w.t0 + j + 1) * kTile > (j < n0 ? least0 : least1);
          if (pv && edge && lane == 4) bar = &a->v_ready[edges & 1], parity = (edges >> 1) & 1;
          if (pv && j == 0 && lane == 3) bar = &a->o_free[t], parity = (used & 1) ^ 1;
          if (qk && j < 0 && lane == 3) bar = &a->q_full[t], parity = used & 1;
          ok = __all_sync(0xffffffffu, wait_here(a, bar, parity, err)) && ok;
          if (!ok) break;
          soft += pv;
          edges += edge;
          tc_fence_after();
          const uint32_t acc0 = j > 0 ? 1u : 0u;
          if (elect_one()) {
            if (pv) {
              if (v0 != kRing - 1) {
#pragma unroll
                for (int i = 0; i < 8; ++i) mma_ts(col_o, col_s + 8 * i, V + i * (2048 >> 4), idesc_pv, i ? 1u : acc0);
              } else {  // value columns 64 .. 127 are in the ring's first box, not in the one behind
#pragma unroll
                for (int b = 0; b < 2; ++b)
#pragma unroll
                  for (int i = 0; i < 8; ++i)
                    mma_ts(col_o + 64 * b, col_s + 8 * i, (b ? v_lo : V) + i * (2048 >> 4), idesc_pv64, i ? 1u : acc0);
              }
              tc_commit(&a->v_empty[gv & 1]);
              if (j == nt - 1) tc_commit(&a->o_done[t]);
            } else if (j >= 0) {
              mbar_arrive(&a->v_empty[gv & 1]);
            }
            if (qk) {
#pragma unroll
              for (int b = 0; b < 3; ++b)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                  mma_ss(col_s, q_lo + b * (kBox >> 4) + 2 * i, B[b] + 2 * i, idesc_qk, b || i ? 1u : 0u);
              tc_commit(&a->s_full[t]);
            } else if (j + 1 < n) {
              mbar_arrive(&a->k_empty[gk & 1]);
            }
          }
          __syncwarp();
        }
        g += n;
        used += nt > 0;
      }
      if (__any_sync(0xffffffffu, *reinterpret_cast<volatile int*>(&a->abort))) {  // wind down: what was issued ends first
        if (elect_one()) tc_commit(&a->drain[t]);
        __syncwarp();
        mbar_wait(&a->drain[t], 0, err);
      }
    }
  } else {
    // ---- softmax: eight warps for each tile of queries, a thread a row and half of the positions (four, a thread a row and
    // all of them: 239 us for the 8192-token prompt instead of 237, 17.8 for the short ones instead of 16.7)
    asm volatile("setmaxnreg.inc.sync.aligned.u32 104;");
    const int t = (warp - 4) >> 3, h = (warp >> 2 & 1) ^ 1, quarter = warp & 3, row = 32 * quarter + lane;
    const uint32_t lane_base = tmem + ((uint32_t)(32 * quarter) << 16);
    const uint32_t col_s = lane_base + kColS + kTile * t + 64 * h, col_p = lane_base + kColS + kTile * t + 32 * h;
    const uint32_t col_o = lane_base + kColO + kTile * t + 64 * h;
    auto pair_bar = [&]() {  // the two warps that share 32 rows
      __syncwarp();
      asm volatile("bar.sync %0, 64;" ::"r"(1 + 4 * t + quarter) : "memory");
    };
    const bool teller = (warp & 7) == 4 && lane == 0;  // (the first warp of the tile's eight)
    int g = 0, soft = 0, used = 0, edges = 0;
    bool ok = true;
    for (Walk walk; next_work<LONG>(p, mine, walk, w, head, f);) {
      const int n0 = tiles_for(f, w, 0), n1 = tiles_for(f, w, 1), n = t ? n1 : n0;
      const int i = kTile * t + row;                             // row of the block
      const int see = i < f.nrows ? sees(f, i) : 0;              // positions that it sees
      const int least = sees(f, kTile * t);                      // positions that every row of this tile sees
      const int least0 = sees(f, 0), edges0 = edges;
      const int64_t out_row = (int64_t)(f.q_row + w.q0 + i) * p.H + head;
      float m = -INFINITY, l = 0.f;
      for (int j = 0; j < n; ++j, ++soft) {
        const int pos = (w.t0 + j) * kTile;
        const bool edge = pos + kTile > least;
        ok = wait_here(a, &a->s_full[t], soft & 1, err) && ok;
        tc_fence_after();
        if (teller && ok) {
          // S is finished, and the K (at an item's end also the Q) that it read is free: a thread says so, which saves the issuers a
          // commit of 100 to 250 cycles.  (V too, which then waits for the next S: 296 us instead of 239.)
          mbar_arrive(&a->k_empty[(g + j) & 1]);
          if (j == n - 1) mbar_arrive(&a->q_empty[t]);
        }
        if (pos + kTile > (j < n0 ? least0 : least)) {
          const int gv = g + j;
          if (t == 0 || j >= n0) {
            // a thread a position: half of its values, where some row does not see it (the tile of later queries finds them so)
            const uint32_t vb = 5 * gv + 3;
            ok = wait_here(a, &a->v_full[gv & 1], (gv >> 1) & 1, err) && ok;
            const bool behind = pos + row >= f.n;
            if (ok && pos + row >= least) {
              bool found = false;
#pragma unroll 1
              for (int c = 0; c < 8; ++c) {
                uint4* chunk = reinterpret_cast<uint4*>(ring + ((vb + h) % kRing) * kBox + row * 128 + (((c ^ row) & 7) << 4));
                uint4 v = make_uint4(0u, 0u, 0u, 0u);
                bool bad = behind;
                if (!behind) {
                  v = *chunk;
                  uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                  for (int q = 0; q < 4; ++q) {
                    if ((u[q] & 0x7F80u) == 0x7F80u) u[q] &= 0xFFFF0000u, bad = true;
                    if ((u[q] & 0x7F800000u) == 0x7F800000u) u[q] &= 0xFFFFu, bad = true;
                  }
                  v = make_uint4(u[0], u[1], u[2], u[3]);
                  found |= bad;
                }
                if (bad) *chunk = v;
              }
              if (found) *reinterpret_cast<volatile int*>(&a->not_finite) = 1;
              fence_proxy_async_smem();
            }
            __syncwarp();
            // (of two tiles in turn: an S that is finished means that the one before the last has been multiplied)
            if (lane == 0 && ok) mbar_arrive(&a->v_ready[edges & 1]);
          }
          ++edges;
        }
        const int upto = see - pos;  // positions of the tile that this row sees
        auto hide = [&](int c, float (&x)[32]) {
          if (edge) {
#pragma unroll
            for (int k = 0; k < 32; ++k) x[k] = 64 * h + c + k < upto ? x[k] : -INFINITY;
          }
        };
        float x[2][32];
#pragma unroll
        for (int c = 0; c < 2; ++c) tmem_ld_issue(col_s + 32 * c, x[c]);
        float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          tmem_ld_wait(x[c]);
          hide(32 * c, x[c]);
#pragma unroll
          for (int k = 0; k < 32; k += 2) mx[(k >> 1) & 3] = fmaxf(mx[(k >> 1) & 3], fmaxf(x[c][k], x[c][k + 1]));
        }
        mx[0] = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
        a->rows[t][h][row] = mx[0];
        pair_bar();  // (and both halves of S have been read: P may take their place)
        const float top = fmaxf(mx[0], a->rows[t][h ^ 1][row]) * p.scale_log2;
        if (__any_sync(0xffffffffu, top > m + kLazy)) {
          float g = 1.f;
          if (top > m + kLazy) {  // (m = -inf: nothing summed yet, the factor is 0)
            g = ex2(m - top);
            m = top;
            l *= g;
          }
          if (j > 0) {
#pragma unroll 1
            for (int c = 0; c < kDv / 2; c += 16) {
              float o[16];
              tmem_ld_sync(col_o + c, o);
              uint32_t v[16];
#pragma unroll
              for (int k = 0; k < 16; ++k) v[k] = __float_as_uint(o[k] * g);
              tmem_st16(col_o + c, v);
            }
          }
        }
        const float mu = m == -INFINITY ? 0.f : -m;
        const float2 scale = make_float2(p.scale_log2, p.scale_log2), minus = make_float2(mu, mu);
        float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          float(&y)[32] = x[c];
          uint32_t v[16];
#pragma unroll
          for (int k = 0; k < 32; k += 2) {
            const float2 z = ffma2(make_float2(y[k], y[k + 1]), scale, minus);
            const float2 e = make_float2(ex2(z.x), ex2(z.y));
            sum[k >> 1 & 1] = add2(sum[k >> 1 & 1], e);
            v[k >> 1] = pack_bf16(e.x, e.y);
          }
          tmem_st16(col_p + 16 * c, v);
        }
        l += sum[0].x + sum[0].y + (sum[1].x + sum[1].y);
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0 && ok) mbar_arrive(&a->p_full[t]);
      }
      g += max(n0, n1);
      edges = edges0 + edges_of(f, w, n0, max(n0, n1));
      // ---- the rows' results
      const bool live = i < f.nrows;
      if (n > 0) {
        ok = wait_here(a, &a->o_done[t], used & 1, err) && ok;
        tc_fence_after();
        ++used;
      }
      int4 part_of = make_int4(0, -1, 1, 0);  // head and item, slot, parts, first of them
      if (w.entry >= 0) part_of = reinterpret_cast<const int4*>(p.plan->list + w.entry)[1];
      const int slot = part_of.y, parts = part_of.z;
      float now = 1.f, before = 0.f;  // what brings this stretch's sums, and those of the ones before, to their maximum
      const int64_t own = ((int64_t)blockIdx.x * 2 + t) * 2 + h;  // this thread's: no other one touches them
      const bool adds = LONG && !(w.begins && w.ends);
      if (adds) {
        float2* ml = p.sum_ml + own * kTile + row;
        const float2 old = w.begins ? make_float2(-INFINITY, 0.f) : *ml;
        const float M = fmaxf(m, old.x);
        now = m == -INFINITY ? 0.f : ex2(m - M);
        before = old.x == -INFINITY ? 0.f : ex2(old.x - M);
        m = M;
        l = fmaf(old.y, before, l * now);
        if (!w.ends) *ml = make_float2(m, l);
      }
      a->rows[t][h][row] = l;  // (O is finished: the maxima of the last tile have been read)
      pair_bar();
      l = a->rows[t][0][row] + a->rows[t][1][row];
      const float inv = l != 0.f ? 1.f / l : 0.f;
      const int64_t part = (int64_t)slot * kBlock + i;
      if (live && h == 0 && w.ends) {
        if (slot >= 0) p.part_ml[part] = make_float2(m, l);
        else if (p.lse) p.lse[out_row] = l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
      }
      // (from the first tile of positions that was looked through: of the first queries' where they are multiplied with it)
      const int cleared = sees(f, 0) / kTile * kTile;
      const bool odd = n > 0 && *reinterpret_cast<volatile int*>(&a->not_finite);
#pragma unroll 1
      for (int c0 = 0; c0 < kDv / 2; c0 += 32) {
        const int c = 64 * h + c0;
        float o[32];
        if (n > 0) {
          tmem_ld_sync(col_o + c0, o);
        } else {
#pragma unroll
          for (int k = 0; k < 32; ++k) o[k] = 0.f;
        }
        if (odd && live) {  // what was cleared from V, for the rows that see it (rows before it never read it)
          const int end = min(see, (w.t0 + n) * kTile);
          for (int q = max(cleared, w.t0 * kTile); q < end; ++q) {
            const __nv_bfloat16* v = p.v + (int64_t)(f.k_row + q) * p.v_row_stride + head * p.v_head_stride + c;
#pragma unroll
            for (int k = 0; k < 32; ++k) {
              const float y = __bfloat162float(v[k]);
              if (!(fabsf(y) < INFINITY)) o[k] += y;
            }
          }
        }
        if (adds) {
          float4* sum = p.sum_o + (own * (kDv / 8) + c0 / 4) * kTile + row;
#pragma unroll
          for (int k = 0; k < 8; ++k, sum += kTile) {
            float4 v = w.begins ? make_float4(0.f, 0.f, 0.f, 0.f) : *sum;
            v.x = fmaf(v.x, before, o[4 * k] * now), v.y = fmaf(v.y, before, o[4 * k + 1] * now);
            v.z = fmaf(v.z, before, o[4 * k + 2] * now), v.w = fmaf(v.w, before, o[4 * k + 3] * now);
            if (!w.ends) *sum = v;
            o[4 * k] = v.x, o[4 * k + 1] = v.y, o[4 * k + 2] = v.z, o[4 * k + 3] = v.w;
          }
        }
        if (!live || !w.ends) {
        } else if (slot >= 0) {
          float4* dst = reinterpret_cast<float4*>(p.part_o + part * kDv + c);
#pragma unroll
          for (int k = 0; k < 8; ++k) dst[k] = make_float4(o[4 * k], o[4 * k + 1], o[4 * k + 2], o[4 * k + 3]);
        } else {
          uint4* dst = reinterpret_cast<uint4*>(p.out + out_row * kDv + c);
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            uint32_t v[4];
#pragma unroll
            for (int q = 0; q < 4; ++q) v[q] = pack_bf16(o[8 * k + 2 * q] * inv, o[8 * k + 2 * q + 1] * inv);
            dst[k] = make_uint4(v[0], v[1], v[2], v[3]);
          }
        }
        __syncwarp();
      }
      pair_bar();  // the sums have been read
      if (n > 0) {
        tc_fence_before();
        __syncwarp();
        if (lane == 0 && ok) mbar_arrive(&a->o_free[t]);
      }
      if (w.ends && parts > 1) {  // whoever finishes the last part of the tile's rows merges them
        __threadfence();
        __syncwarp();
        asm volatile("bar.sync %0, 256;" ::"r"(9 + t) : "memory");
        if (row == 0 && h == 0) a->last[t] = atomicAdd(&p.plan->done[part_of.x >> 8][t], 1) == parts - 1;
        asm volatile("bar.sync %0, 256;" ::"r"(9 + t) : "memory");
        if (a->last[t]) {
          __threadfence();
          merge_parts(p, w, f, head, parts, part_of.w, kTile * t, (warp - 4) & 7);
        }
        asm volatile("bar.sync %0, 256;" ::"r"(11 + t) : "memory");  // (`last` has been read)
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 0) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

int blocks_of(const ExpandedAttnParams& p) {  // at most
  const int64_t b = p.n_seq == 1 ? (p.T + kBlock - 1) / kBlock : (int64_t)p.T / kBlock + p.n_seq;
  return (int)(b < p.T ? b : p.T);
}
int longest(const ExpandedAttnParams& p) { return (int)(((int64_t)(p.max_len < p.N ? p.max_len : p.N) + kTile - 1) / kTile); }
// Blocks may be cut into spans where that can pay: where a whole one is longer than a span and two starts.
void set_cuts(ExpandedAttnParams* p) {
  const int64_t items = (int64_t)blocks_of(*p) * p->H;
  p->shift = 0;
  while (longest(*p) >> p->shift > kLengths) ++p->shift;
  p->may_span = longest(*p) > kMinSpan + kFixed;
  int64_t ctas = items;
  if (p->may_span) ctas = (items * (longest(*p) + kFixed) + kMinSpan - 1) / kMinSpan;
  p->grid = (int)(ctas < kSms ? ctas : kSms);
}

struct Layout {
  size_t work, part_ml, part_o, sum_ml, sum_o, total;
};
Layout layout_of(const ExpandedAttnParams& p) {
  Layout l;
  const size_t rows = p.may_span ? (size_t)2 * p.grid * kBlock : 0, sums = longest(p) > kStretch ? (size_t)p.grid * kBlock : 0;
  l.work = align_up(sizeof(Plan), 256);
  l.part_ml = l.work + align_up((size_t)blocks_of(p) * sizeof(int4), 256);
  l.part_o = l.part_ml + align_up(rows * sizeof(float2), 256);
  l.sum_ml = l.part_o + rows * kDv * sizeof(float);
  l.sum_o = l.sum_ml + align_up(2 * sums * sizeof(float2), 256);
  l.total = l.sum_o + sums * kDv * sizeof(float);
  return l;
}

bool map_of(CUtensorMap* tm, const void* base, int cols, int heads, int rows, int64_t head_stride, int64_t row_stride) {
  const cuuint64_t dims[3] = {(cuuint64_t)cols, (cuuint64_t)heads, (cuuint64_t)rows};
  const cuuint64_t strides[2] = {(cuuint64_t)head_stride * 2, (cuuint64_t)row_stride * 2};
  const cuuint32_t box[3] = {64, 1, kTile};
  memset(tm, 0, sizeof(*tm));
  return encode_tensor_map(tm, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B) ==
         CUDA_SUCCESS;
}

cudaError_t launch(ExpandedAttnParams p, const dsa_expanded_attn_args& a, void* ws, cudaStream_t stream) {
  const Layout l = layout_of(p);
  uint8_t* base = reinterpret_cast<uint8_t*>(ws);
  p.plan = reinterpret_cast<Plan*>(base);
  p.work = reinterpret_cast<int4*>(base + l.work);
  p.part_ml = reinterpret_cast<float2*>(base + l.part_ml);
  p.part_o = reinterpret_cast<float*>(base + l.part_o);
  p.sum_ml = reinterpret_cast<float2*>(base + l.sum_ml);
  p.sum_o = reinterpret_cast<float4*>(base + l.sum_o);
  p.max_work = blocks_of(p);
  CUtensorMap tq, tk, tr, tv;
  // (without positions nothing of k and v is loaded: their maps are q's)
  const bool any = p.N > 0;
  const int64_t q_row = (int64_t)p.H * (kNope + kRope);
  if (!map_of(&tq, a.q, kNope + kRope, p.H, p.T, kNope + kRope, q_row) ||
      !(any ? map_of(&tk, a.k, kNope, p.H, p.N, a.k_head_stride, a.k_row_stride) : map_of(&tk, a.q, kNope, p.H, p.T, kNope + kRope, q_row)) ||
      !(any ? map_of(&tv, a.v, kDv, p.H, p.N, a.v_head_stride, a.v_row_stride) : map_of(&tv, a.q, kDv, p.H, p.T, kNope + kRope, q_row)))
    return cudaErrorInvalidValue;
  const cuuint64_t dims[2] = {(cuuint64_t)kRope, (cuuint64_t)(any ? p.N : p.T)}, strides[1] = {(cuuint64_t)kRope * 2};
  const cuuint32_t box[2] = {64, kTile};
  memset(&tr, 0, sizeof(tr));
  if (encode_tensor_map(&tr, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(any ? a.k_rope : a.q), dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B) !=
      CUDA_SUCCESS)
    return cudaErrorInvalidValue;
  const bool stretches = longest(p) > kStretch;
  auto kern = stretches ? expanded_attn_kernel<true> : expanded_attn_kernel<false>;
  static std::atomic<uint64_t> allowed[2];
  cudaError_t e = allow_smem_once(&allowed[stretches], reinterpret_cast<const void*>(kern), kSmem);
  if (e != cudaSuccess) return e;
  if ((e = launch_kernel(plan_kernel, dim3(1), dim3(1024), 0, stream, false, p)) != cudaSuccess) return e;
  return launch_kernel(kern, dim3((unsigned)p.grid), dim3(kThreads), kSmem, stream, true, tq, tk, tr, tv, p);
}

dsa_status check_expanded(const dsa_expanded_attn_args* a) {
  if (!a || a->n_seq < 0 || a->T < 0 || a->N < 0 || a->max_len < 0 || a->H < 1) return DSA_ERR_INVALID_ARG;
  if (!(a->sm_scale > 0.f) || !(a->sm_scale < INFINITY)) return DSA_ERR_INVALID_ARG;
  if (a->H > 128 || a->n_seq > kMaxSeq || a->T >= kMaxRows || a->N >= kMaxRows) return DSA_ERR_UNSUPPORTED;
  if (a->n_seq == 0 || a->T == 0) return DSA_OK;
  auto ok16 = [](const void* p) { return p && (reinterpret_cast<uintptr_t>(p) & 15) == 0; };
  if (!a->q_start || !a->kv_start || !ok16(a->q) || !ok16(a->out)) return DSA_ERR_INVALID_ARG;
  for (const void* p : {(const void*)a->q_start, (const void*)a->kv_start, (const void*)a->lse})
    if ((reinterpret_cast<uintptr_t>(p) & 3) != 0) return DSA_ERR_INVALID_ARG;
  if (a->N == 0) return DSA_OK;
  if (!ok16(a->k) || !ok16(a->k_rope) || !ok16(a->v)) return DSA_ERR_INVALID_ARG;
  for (const int64_t s : {a->k_row_stride, a->v_row_stride, a->k_head_stride, a->v_head_stride}) {
    if (s % 8 != 0 || s < kNope) return DSA_ERR_INVALID_ARG;
    if (s >= 1ll << 39) return DSA_ERR_UNSUPPORTED;
  }
  return DSA_OK;
}

ExpandedAttnParams params_of(const dsa_expanded_attn_args& a) {
  ExpandedAttnParams p = {};
  p.q_start = a.q_start;
  p.kv_start = a.kv_start;
  p.n_seq = a.n_seq;
  p.T = a.T;
  p.N = a.N;
  p.H = a.H;
  p.max_len = a.max_len > 0 && a.max_len < a.N ? a.max_len : a.N;
  p.causal = a.causal != 0;
  p.scale_log2 = a.sm_scale * 1.4426950408889634f;
  p.v = reinterpret_cast<const __nv_bfloat16*>(a.v);
  p.v_row_stride = a.v_row_stride;
  p.v_head_stride = a.v_head_stride;
  p.out = reinterpret_cast<__nv_bfloat16*>(a.out);
  p.lse = a.lse;
  set_cuts(&p);
  return p;
}

}  // namespace
}  // namespace dsa

using namespace dsa;

extern "C" {

dsa_status dsa_expanded_attn_workspace_size(const dsa_expanded_attn_args* a, size_t* bytes) {
  if (!bytes) return DSA_ERR_INVALID_ARG;
  const dsa_status s = check_expanded(a);
  if (s != DSA_OK) return s;
  *bytes = a->n_seq > 0 && a->T > 0 ? layout_of(params_of(*a)).total : 0;
  return DSA_OK;
}

dsa_status dsa_expanded_attn(const dsa_expanded_attn_args* a, void* ws, size_t ws_bytes, void* stream) {
  dsa_status s = check_expanded(a);
  if (s != DSA_OK || a->n_seq == 0 || a->T == 0) return s;
  ExpandedAttnParams p = params_of(*a);
  if (!ws || ws_bytes < layout_of(p).total || (reinterpret_cast<uintptr_t>(ws) & 255) != 0) return DSA_ERR_WORKSPACE;
  if ((s = check_device_arch()) != DSA_OK) return s;
  p.err = device_error_word();
  return launch(p, *a, ws, reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess ? DSA_OK : DSA_ERR_CUDA;
}

}  // extern "C"
