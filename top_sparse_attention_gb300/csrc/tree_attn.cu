// Attention of drafted tokens over the latent cache (dsa_tree_attn): query node i of sequence s sees
// the n_ctx[s] cached positions and the drafted positions n_ctx[s] + j whose bit j is set in its row
// of the tree mask,
//   logit[p] = sm_scale * q[i, h] . Kv[p],  out[i, h] = sum_p softmax(logit)[p] * Kv[p, :512].
//
// A "row" is one head of one node; the rows of a sequence are consecutive in q and share its cache.
// A cluster of two CTAs takes 128 rows and walks tiles of 64 positions.  CTA c takes the first product
// and the softmax of 32 of the positions, and the second product of half of the value columns:
//   * S[128 x 32] = Q K_c^T: A = the rows (M = 128; 448 of their columns in tensor memory, 128 in shared
//     memory), B = its 32 positions (K-major), 36 steps of K = 16;
//   * one pass over the positions keeps a reference maximum m and a sum l per row,
//       l' = l 2^(m - m') + sum_p 2^(x_p - m'),   o' = o 2^(m - m') + sum_p 2^(x_p - m') v_p,
//     where m is moved only when a tile's maximum exceeds it by more than 2^8 (weights stay below 2^8,
//     fp32 sums and bf16 weights lose nothing by it), so o in tensor memory is rescaled rarely.  The CTAs send
//     each other their rows' maxima over their positions a tile ahead, so both move m alike;
//   * each sends the other its P[128 x 32] (bf16): 8 KB per tile through distributed shared memory;
//   * O_c[128 x 256] += P V_c: A = P in shared memory, B = 256 value columns of all 64 positions, read MN-major
//     (values along N), 4 steps of K = 16 with N = 256.  A CTA's own positions are in shared memory whole, of
//     the other's only these 256 columns are loaded besides: 832 of 1152 bytes per position and CTA.
// Why two CTAs: o for 128 rows x 512 values fills a tensor memory (512 columns), which leaves no room for S;
// with half of the values it takes 256 columns, q 224, S 32.  Measured against it (8 x 64 nodes
// at 32K, E4M3 rows; 8 x 8 nodes at 32K, bf16): one CTA with 64 rows, q in shared memory and o
// transposed, 1805 and 149 us (245 KB of shared memory read per tile by the MMAs, room for two tiles);
// columns of the rows split between the CTAs, whose partial S then travel, 1090 and 120 us (16 to 32 KB
// per tile at about 20 bytes per cycle between two SMs).
//
// Weights are rounded to bf16 for the second product (as the bf16 cache is); sums, maxima, logits and
// outputs are fp32.  E4M3 rows are widened to bf16 exactly, and their scales are applied in fp32 to the
// logit and to the weight (128-column scales: one S accumulation per scale tile, one P per value tile).
//
// Warp roles: producer (TMA), MMA issuer, scale loader, credits of the exchange, eight softmax warps (a row and
// 16 positions per thread; also the query load, the rescale and the epilogue), for E4M3 eight warps that
// load, widen and store the tile.
//
// Work split: items (sequence, chunk of its tiles, row tile), in this order, so that clusters that run
// together read the same positions and the cache comes from HBM once.  The lengths are on the device:
// every CTA evaluates the same cost model over them and picks the chunk length (plan_items); partial
// results are merged by tree_combine_kernel.
#include <string.h>

#include "dsa_internal.h"

namespace dsa {
namespace {

constexpr float kLn2 = 0.6931471805599453f;
constexpr int kDqk = 576, kDv = 512;
constexpr int kRows = 128;                // query rows per cluster
constexpr int kKeys = 64;                 // positions per tile, half of them per CTA
constexpr int kBox = 32 * 128;            // 64 columns of 32 positions: 32 rows x 128 bytes
constexpr int kSlotV = 4 * kBox;          // a CTA's value columns of 32 positions (its own, or the other's)
constexpr int kSlotK = 5 * kBox;          // the other columns of its positions: 4 boxes of values, the rotary one
constexpr int kSmemMax = 227 * 1024;
constexpr float kLazy = 8.f;              // log2 growth of a row's maximum that is left unscaled
constexpr int kItemsPerCta = 3;           // split launches are cut into at most this many items per cluster
// tensor-memory columns: O, seven (six) of the nine 64-column boxes of q, one S buffer (two)
constexpr int kColO = 0, kColQ = 256;

enum { kBf16 = 0, kFp8Row = 1, kFp8Tile = 2 };

template <int FMT>
struct Cfg {
  static constexpr bool FP8 = FMT != kBf16;
  static constexpr int NSC = FMT == kFp8Tile ? 5 : FMT == kFp8Row ? 1 : 0;
  static constexpr bool TILED = FMT == kFp8Tile;
  static constexpr int THREADS = FP8 ? 640 : 384;
  // slots: our positions' value columns (held from the first product to the second), their other columns (first
  // product only), the other's positions (second product only)
  static constexpr int AS = TILED ? 3 : 4, KS = 2, BS = TILED ? 2 : 3;
  static constexpr int BT = TILED ? 6 : 7;                // q's boxes in tensor memory (the others are in shared memory)
  static constexpr int SB = TILED ? 2 : 1;                // S buffers
  static constexpr int PB = TILED ? 1 : 2;                // P buffers
  static constexpr int COL_S = kColQ + 32 * BT;
  static constexpr int GROUPS = TILED ? 5 : 1;            // S accumulations per tile
  static constexpr int PC = TILED ? 2 : 1;                // copies of P (one per 128 values)
  static constexpr int SC_DEPTH = 2;
  static constexpr int SC_BYTES = NSC * 32 * 4;           // scales of this CTA's positions
  static constexpr int Q_BOX = kRows * 128, Q_BYTES = (9 - BT) * Q_BOX;
  static constexpr int P_HALF = kRows * 64;               // 128 rows x 32 positions
  static constexpr int P_BYTES = 2 * P_HALF;
  static constexpr int PP_BYTES = TILED ? PC * P_HALF : 0;  // with tile scales: the other's copies of our P, on their way
  static constexpr int AUX = 8192;
  static constexpr int OFF_B = AS * kSlotV;
  static constexpr int OFF_K = OFF_B + BS * kSlotV;
  static constexpr int OFF_Q = OFF_K + KS * kSlotK;
  static constexpr int OFF_P = OFF_Q + Q_BYTES;
  static constexpr int OFF_PP = OFF_P + PB * PC * P_BYTES;
  static constexpr int OFF_SC = OFF_PP + PP_BYTES;
  static constexpr int OFF_AUX = OFF_SC + SC_DEPTH * SC_BYTES;
  static constexpr int SMEM = OFF_AUX + AUX + 1024;
  static_assert(SMEM <= kSmemMax, "shared memory");
};

struct Item {
  int seq, rt, t0, t1;     // tiles [t0, t1) of row tile rt
  int ctx, fresh, len;     // cached and drafted positions, the sequence's end
  int slot;                // partial slot, or -1: the whole range, written to the output
};

// The launch's fixed facts (host) and the split plan in the workspace (device).
struct TreePlan {
  int row_tiles;           // per sequence
  int units;               // n_seq * row_tiles
  int cap;                 // partial slots; 0: no unit is split
  int grid;                // clusters
  int* head;               // [0]: chunk length in tiles (0: not split), [1 + s]: first item of sequence s
  float4* part_o;          // [cap][128 groups of four values][128 rows]
  float2* part_ml;         // [cap][128 rows]
};

__device__ __forceinline__ void seq_facts(const TreeAttnParams& p, int seq, int& ctx, int& fresh, int& len) {
  ctx = min(max(p.n_ctx[seq], 0), p.L);
  fresh = p.n_new ? min(max(p.n_new[seq], 0), p.q_per_seq) : p.q_per_seq;
  len = min(ctx + fresh, p.L);
}

__device__ __forceinline__ int live_row_tiles(const TreeAttnParams& p, int fresh) {
  return (fresh * p.H + kRows - 1) / kRows;  // row tiles that hold a node below `fresh`
}

struct Aux {
  uint64_t a_full[4], a_empty[4], b_full[3], b_empty[3], k_full[2], k_empty[2];
  uint64_t s_full[2], s_empty[2], m_msg[4], p_full[2], p_msg[2], p_free[2], pv_done[2];
  uint64_t stat_full, o_done, o_free, q_full, sc_full[2], sc_empty[2], drain;
  uint32_t tmem;
  int abort;
  int n_items;
  int tile_bad[8];
  int items[kItemsPerCta][8];
  // each half's maxima over its 16 positions, ours (by tile % 2; at an item's end its sums) and the other CTA's (by
  // tile % 4), and the positions to clear
  alignas(16) float mx_own[2][2][kRows];
  alignas(16) float mx[4][2][kRows];
  uint32_t clear_own[4][8], clear[4][8];
  float stat[2][kRows];  // the other's sums, by half
};
static_assert(sizeof(Aux) <= 8192, "Aux");

__device__ __forceinline__ bool mbar_test(uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred P;\n\t"
      "mbarrier.test_wait.parity.shared::cta.b64 P, [%1], %2;\n\t"
      "selp.b32 %0, 1, 0, P;\n\t}"
      : "=r"(ok)
      : "r"(smem_u32(bar)), "r"(parity)
      : "memory");
  return ok != 0;
}

// A bounded wait.  Once one wait of the CTA has run out, the others return at once: the softmax warps then walk
// through the rest of their work (every address stays in range), so that their common barriers still match; the
// other roles leave.  A thread whose wait failed arrives on no mbarrier, arms none and sends nothing any more: an
// arrival is only legal in a phase that the arriving thread has seen begin.
__device__ __noinline__ bool wait_slow(Aux* a, uint64_t* bar, uint32_t parity, int* err, bool cluster);
__device__ __forceinline__ bool wait(Aux* a, uint64_t* bar, uint32_t parity, int* err) {
  return mbar_test(bar, parity) || wait_slow(a, bar, parity, err, false);
}
// The same for a barrier that the other CTA of the cluster arrives on: what it did before is visible after.
__device__ __forceinline__ bool try_wait_cluster(uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred P;\n\t"
      "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 P, [%1], %2;\n\t"
      "selp.b32 %0, 1, 0, P;\n\t}"
      : "=r"(ok)
      : "r"(smem_u32(bar)), "r"(parity)
      : "memory");
  return ok != 0;
}
__device__ __forceinline__ bool test_cluster(uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred P;\n\t"
      "mbarrier.test_wait.parity.acquire.cluster.shared::cta.b64 P, [%1], %2;\n\t"
      "selp.b32 %0, 1, 0, P;\n\t}"
      : "=r"(ok)
      : "r"(smem_u32(bar)), "r"(parity)
      : "memory");
  return ok != 0;
}
__device__ __forceinline__ bool wait_cluster(Aux* a, uint64_t* bar, uint32_t parity, int* err) {
  return test_cluster(bar, parity) || wait_slow(a, bar, parity, err, true);
}
__device__ __noinline__ bool wait_slow(Aux* a, uint64_t* bar, uint32_t parity, int* err, bool cluster) {
  const unsigned long long t0 = globaltimer_ns();
  for (uint32_t i = 0;; ++i) {
    if (*reinterpret_cast<volatile int*>(&a->abort)) return false;
    if (cluster ? try_wait_cluster(bar, parity) : mbar_try_wait(bar, parity)) return true;
    if ((i & 63u) == 63u && globaltimer_ns() - t0 > kWaitLimitNs) {
      record_error(err, DSA_DEVERR_WAIT_TIMEOUT);
      *reinterpret_cast<volatile int*>(&a->abort) = 1;
      return false;
    }
  }
}

__device__ __forceinline__ void arrive_remote(uint32_t bar) {
  asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}

// `bytes` of this CTA's shared memory into the other CTA's, counted on its mbarrier (measured one way: 320
// cycles for 64 bytes, 520 for 4 KB, 1100 for 16 KB).
__device__ __forceinline__ void copy_remote(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
  asm volatile("cp.async.bulk.shared::cluster.shared::cta.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
               "r"(smem_u32(src)), "r"(bytes), "r"(bar)
               : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.bulk.commit_group;" ::: "memory"); }
// All of this thread's copies have read their source.
__device__ __forceinline__ void copy_wait_read() { asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory"); }

__device__ __forceinline__ void st_async4(uint32_t addr, uint32_t v, uint32_t bar) {
  asm volatile("st.async.weak.shared::cluster.mbarrier::complete_tx::bytes.b32 [%0], %1, [%2];" ::"r"(addr), "r"(v), "r"(bar)
               : "memory");
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

// A value that is the same in all lanes, as one the compiler knows to be so (a warp-wide reduction writes
// a uniform register): the MMA issuer's loop bounds and addresses go through it, because operands in
// per-lane registers cost the issue of each instruction more than its execution (67 against 32 to 48
// cycles).
__device__ __forceinline__ int uniform(int x) { return __reduce_max_sync(0xffffffffu, x); }

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 b = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&b);
}

// Low words of shared-memory descriptors with 128-byte swizzle (the upper word, kDescHi, holds the 1024-byte
// stride, the version and the swizzle): K-major operands, and MN-major ones whose 64-element atoms are one
// box apart.  Adding bytes / 16 moves the start address.  P's rows are 64 bytes, with 64-byte swizzle
// (kDescHi64: 8 rows are 512 bytes; 16-byte chunk c of row r lies at chunk c ^ (r / 2 % 4)).
constexpr uint32_t kDescHi = (1024u >> 4) | (1u << 14) | (2u << 29);
constexpr uint32_t kDescHi64 = (512u >> 4) | (1u << 14) | (4u << 29);
__device__ __forceinline__ uint32_t kmajor_lo(uint32_t saddr) { return ((saddr & 0x3FFFFu) >> 4) | (1u << 16); }
__device__ __forceinline__ uint32_t mnmajor_lo(uint32_t saddr) {
  return ((saddr & 0x3FFFFu) >> 4) | ((uint32_t)(kBox >> 4) << 16);
}

// D += A B^T with A in shared memory, or in tensor memory (lane = row, two bf16 per column).
template <uint32_t A_HI = kDescHi>
__device__ __forceinline__ void mma_ss(uint32_t d, uint32_t a_lo, uint32_t b_lo, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 da, db;\n\t"
      "mov.b64 da, {%1, %6};\n\t"
      "mov.b64 db, {%2, %5};\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %3, p;\n\t}" ::"r"(d),
      "r"(a_lo), "r"(b_lo), "r"(idesc), "r"(acc), "r"(kDescHi), "r"(A_HI)
      : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a_tmem, uint32_t b_lo, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 db;\n\t"
      "mov.b64 db, {%2, %5};\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], db, %3, p;\n\t}" ::"r"(d),
      "r"(a_tmem), "r"(b_lo), "r"(idesc), "r"(acc), "r"(kDescHi)
      : "memory");
}

// Registers -> tensor memory: this thread's lane, 16 columns.
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&v)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
      "%15, %16};" ::"r"(taddr),
      "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]),
      "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
      : "memory");
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

// Splits the sequences' tiles into items.  Cost of chunks of CH tiles: the fullest CTA's items, each CH
// tiles plus the fill and drain of its pipeline, and for a split the merge.  Fills this cluster's list;
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
  if (tid < 32) {
    int m = 1;
    for (int s = tid; s < n; s += 32) m = max(m, nt[s]);
    m = __reduce_max_sync(0xffffffffu, m);
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
    if (sp && items > pl.cap) v = INFINITY;
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
    int run = 0;
    for (int s0 = 0; s0 < n; s0 += 32) {
      const int s = s0 + tid;
      const int c = s < n ? live[s] * (nt[s] ? (nt[s] + ch - 1) / ch : 1) + (pl.row_tiles - live[s]) : 0;
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
    // this cluster's items: its number, + grid, ...
    const int first = (int)(blockIdx.x >> 1), mine = first + tid * pl.grid;
    if (tid < kItemsPerCta && mine < run) {
      int lo = 0, hi = n - 1;
      while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (base[mid] <= mine) lo = mid;
        else hi = mid - 1;
      }
      const int s = lo, at = mine - base[s];
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
    if (tid == 0) a->n_items = first < run ? (run - first + pl.grid - 1) / pl.grid : 0;
    if (blockIdx.x == 0) {
      if (tid == 0) pl.head[0] = ch;
      for (int s = tid; s < n; s += 32) pl.head[1 + s] = base[s];
    }
  }
  __syncthreads();
}

// Item i of this cluster: from the list of a split launch, or the unit of number cluster + i * grid whole.
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

template <int FMT>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(Cfg<FMT>::THREADS, 1)
    tree_attn_kernel(const __grid_constant__ CUtensorMap tm, const TreeAttnParams p, const TreePlan pl) {
  using C = Cfg<FMT>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* a_s = smem;
  uint8_t* b_s = smem + C::OFF_B;
  uint8_t* k_s = smem + C::OFF_K;
  uint8_t* q_s = smem + C::OFF_Q;
  uint8_t* p_s = smem + C::OFF_P;
  uint8_t* pp_s = smem + C::OFF_PP;
  float* sc_s = reinterpret_cast<float*>(smem + C::OFF_SC);
  Aux* a = reinterpret_cast<Aux*>(smem + C::OFF_AUX);
  const int tid = threadIdx.x, lane = tid & 31, warp = uniform(tid >> 5);
  const int rank = uniform((int)cluster_rank());  // which 32 positions of a tile, which half of the value columns
  int* err = p.err;

  if (warp == 0) {
    tmem_alloc(&a->tmem, 512);
    tmem_relinquish();
  }
  constexpr uint32_t kMaxBytes = 2 * kRows * 4 + 8 * 4;  // a tile's maxima and clear words
  constexpr uint32_t kPBytes = C::PC * C::P_HALF;    // a tile's P from the other CTA
  if (tid == 32) {
    const int fillers = C::FP8 ? 8 : 1;  // arrivals that fill a slot: converter warps, or the TMA's thread
    for (int i = 0; i < C::AS; ++i) mbar_init(&a->a_full[i], fillers), mbar_init(&a->a_empty[i], 1);
    for (int i = 0; i < C::BS; ++i) mbar_init(&a->b_full[i], fillers), mbar_init(&a->b_empty[i], 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&a->k_full[i], fillers), mbar_init(&a->k_empty[i], 1);
      mbar_init(&a->s_full[i], 1), mbar_init(&a->s_empty[i], 8);
      mbar_init(&a->p_full[i], 8), mbar_init(&a->p_msg[i], 1), mbar_init(&a->p_free[i], 1), mbar_init(&a->pv_done[i], 1);
      mbar_init(&a->sc_full[i], 32), mbar_init(&a->sc_empty[i], 8);
    }
    for (int i = 0; i < 4; ++i) mbar_init(&a->m_msg[i], 9);
    mbar_init(&a->stat_full, 1);
    mbar_init(&a->o_done, 1);
    mbar_init(&a->o_free, 8);
    mbar_init(&a->q_full, 256);
    mbar_init(&a->drain, 1);
    a->abort = 0;
    fence_mbar_init();
    for (int i = 0; i < 4; ++i) mbar_arrive_expect_tx(&a->m_msg[i], kMaxBytes);
    for (int i = 0; i < C::PB; ++i) mbar_arrive_expect_tx(&a->p_msg[i], kPBytes);
    mbar_arrive_expect_tx(&a->stat_full, 2 * kRows * 4);
  }
  if (pl.cap) plan_items(p, pl, a, reinterpret_cast<int*>(a_s));
  fence_proxy_async_smem();  // the plan's scratch is a slot that the copies write
  tc_fence_before();
  __syncthreads();
  cluster_sync();  // the other CTA's barriers are ready too
  tc_fence_after();
  const uint32_t tmem = a->tmem;
  pdl_launch_dependents();

  Item it;
  if (warp == 0) {
    // ---- producer (bf16): boxes of 64 columns x 32 positions by TMA
    if (lane == 0 && !C::FP8) {
      prefetch_tmap(&tm);
      int as = 0, aph = 0, bs = 0, bph = 0, ks = 0, kph = 0, tiles = 0;
      bool ok = true;
      for (int i = 0; ok && get_item(p, pl, a, i, it); ++i) {
        for (int t = it.t0; ok && t < it.t1; ++t, ++tiles) {
          int row = t * kKeys, z = it.seq, bad = 0;
          if (p.pages.table) {
            const int64_t r = tree_row(p, it.seq, row);
            z = 0;
            bad = r < 0;
            // a block id outside the pool: rows past its end, which the copy fills with zeros
            row = bad ? p.pages.num_blocks * p.pages.block_size : (int)r;
            if (bad) record_error(err, DSA_DEVERR_INDEX_RANGE);
          }
          const int mine = row + 32 * rank, other = row + 32 * (rank ^ 1);
          ok = wait(a, &a->a_empty[as], aph ^ 1, err);
          if (!ok) break;
          a->tile_bad[tiles & 7] = bad;
          uint8_t* dst = a_s + as * kSlotV;
          mbar_arrive_expect_tx(&a->a_full[as], kSlotV);
#pragma unroll
          for (int b = 0; b < 4; ++b) tma_load_3d(dst + b * kBox, &tm, &a->a_full[as], 256 * rank + 64 * b, mine, z);
          if (++as == C::AS) as = 0, aph ^= 1;
          ok = wait(a, &a->k_empty[ks], kph ^ 1, err);
          if (!ok) break;
          dst = k_s + ks * kSlotK;
          mbar_arrive_expect_tx(&a->k_full[ks], kSlotK);
#pragma unroll
          for (int b = 0; b < 4; ++b) tma_load_3d(dst + b * kBox, &tm, &a->k_full[ks], 256 * (rank ^ 1) + 64 * b, mine, z);
          tma_load_3d(dst + 4 * kBox, &tm, &a->k_full[ks], 512, mine, z);
          if (++ks == C::KS) ks = 0, kph ^= 1;
          ok = wait(a, &a->b_empty[bs], bph ^ 1, err);
          if (!ok) break;
          dst = b_s + bs * kSlotV;
          mbar_arrive_expect_tx(&a->b_full[bs], kSlotV);
#pragma unroll
          for (int b = 0; b < 4; ++b) tma_load_3d(dst + b * kBox, &tm, &a->b_full[bs], 256 * rank + 64 * b, other, z);
          if (++bs == C::BS) bs = 0, bph ^= 1;
        }
      }
      if (*reinterpret_cast<volatile int*>(&a->abort)) {  // wind down: the copies in flight land first
        for (int s = 0; s < C::AS; ++s) mbar_wait(&a->a_full[s], s < as ? aph : aph ^ 1, err);
        for (int s = 0; s < C::BS; ++s) mbar_wait(&a->b_full[s], s < bs ? bph : bph ^ 1, err);
        for (int s = 0; s < C::KS; ++s) mbar_wait(&a->k_full[s], s < ks ? kph : kph ^ 1, err);
      }
    }
    __syncwarp();
  } else if (warp == 1) {
    // ---- MMA issuer.  The warp stays converged and one elected lane issues; descriptors are sums of
    // 32-bit words (their upper words are constants), so that issuing an instruction costs less than
    // the tensor cores take for it
    constexpr uint32_t idesc_qk = make_idesc(1, 1, kRows, 32);
    constexpr uint32_t idesc_pv = make_idesc(1, 1, kRows, C::TILED ? 128 : 256) | (1u << 16);  // B (values) MN-major
    const uint32_t tm_base = (uint32_t)uniform((int)tmem);
    const uint32_t ka_lo = kmajor_lo(smem_u32(a_s)), kk_lo = kmajor_lo(smem_u32(k_s));
    const uint32_t va_lo = mnmajor_lo(smem_u32(a_s)), vb_lo = mnmajor_lo(smem_u32(b_s));
    const uint32_t q_lo = kmajor_lo(smem_u32(q_s)), p_lo = kmajor_lo(smem_u32(p_s));
    int as = 0, aph = 0, ks = 0, kph = 0;  // slots of the first product
    int ps = 0, bs = 0, bph = 0;           // of the second
    int tile = 0, items = 0;
    uint32_t su = 0;                       // uses of the S buffers
    bool ok = true;
    auto commit = [&](uint64_t* bar) {
      if (elect_one()) tc_commit(bar);
      __syncwarp();
    };
    // Box j of q against this CTA's positions: 4 steps of K = 16.
    auto qk_box = [&](uint32_t d, int j, uint32_t B, bool first) {
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const uint32_t acc = first && k == 0 ? 0u : 1u;
        if (j < C::BT) mma_ts(d, tm_base + kColQ + 32 * j + 8 * k, B + 2 * k, idesc_qk, acc);
        else mma_ss(d, q_lo + (j - C::BT) * (C::Q_BOX >> 4) + 2 * k, B + 2 * k, idesc_qk, acc);
      }
    };
    auto test = [&](uint64_t* bar, uint32_t parity) { return __all_sync(0xffffffffu, mbar_test(bar, parity)); };
    // First product, one accumulation: the whole tile, or with tile scales a pair of boxes (g) after another
    // through the S buffers.  The softmax warps have read what the buffer held.
    auto qk_ready = [&](int g) {
      return test(&a->s_empty[su % C::SB], ((su / C::SB) & 1) ^ 1) &&
             (g > 0 || (test(&a->a_full[as], aph) && test(&a->k_full[ks], kph)));
    };
    auto qk = [&](int g) {
      const uint32_t V = ka_lo + as * (kSlotV >> 4), K = kk_lo + ks * (kSlotK >> 4);
      const uint32_t d = tm_base + C::COL_S + 32 * (su % C::SB);
      const bool last = g == C::GROUPS - 1;
      tc_fence_after();
      if (elect_one()) {
        if (C::TILED) {
          if (g < 4) {
            const uint32_t B = ((g >> 1) == rank ? V : K) + (2 * (g & 1) * kBox >> 4);
            if (g < 3) {
#pragma unroll
              for (int k = 0; k < 8; ++k)
                mma_ts(d, tm_base + kColQ + 64 * g + 8 * k, B + ((k >> 2) * kBox + 32 * (k & 3)) / 16, idesc_qk, k ? 1u : 0u);
            } else {
#pragma unroll
              for (int k = 0; k < 8; ++k)
                mma_ss(d, q_lo + ((k >> 2) * C::Q_BOX + 32 * (k & 3)) / 16, B + ((k >> 2) * kBox + 32 * (k & 3)) / 16, idesc_qk,
                       k ? 1u : 0u);
            }
          } else {
            qk_box(d, 8, K + (4 * kBox >> 4), true);
          }
        } else {
#pragma unroll
          for (int j = 0; j < 8; ++j) qk_box(d, j, ((j >> 2) == rank ? V : K) + ((j & 3) * kBox >> 4), j == 0);
          qk_box(d, 8, K + (4 * kBox >> 4), false);
        }
        tc_commit(&a->s_full[su % C::SB]);
        if (last) tc_commit(&a->k_empty[ks]);
      }
      __syncwarp();
      ++su;
      if (last) {
        if (++as == C::AS) as = 0, aph ^= 1;
        if (++ks == C::KS) ks = 0, kph ^= 1;
      }
    };
    // Second product of a tile: its weights from both CTAs, and the other's positions, are there.
    auto pv_ready = [&](bool first) {
      const int pb = tile % C::PB;
      return test(&a->p_full[tile & 1], (tile >> 1) & 1) &&
             __all_sync(0xffffffffu, test_cluster(&a->p_msg[pb], (tile / C::PB) & 1)) && test(&a->b_full[bs], bph) &&
             (!first || test(&a->o_free, (items & 1) ^ 1));
    };
    auto pv = [&](bool first) {
      if (lane == 0) mbar_arrive_expect_tx(&a->p_msg[tile % C::PB], kPBytes);  // for this buffer's next use
      __syncwarp();
      tc_fence_after();
      const uint32_t acc0 = first ? 0u : 1u, A = va_lo + ps * (kSlotV >> 4), B = vb_lo + bs * (kSlotV >> 4);
      const uint32_t P = p_lo + (tile % C::PB) * (C::PC * C::P_BYTES >> 4);
      if (elect_one()) {
        constexpr int NB = C::TILED ? 2 : 1;  // value tiles of N = 128 with a P each, or all 256 at once
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
          for (int s = 0; s < 4; ++s) {  // two steps over this CTA's positions, two over the other's
            const uint32_t half = (uint32_t)((s >> 1) ^ rank);  // whose P: the halves of the buffer are by CTA
            mma_ss<kDescHi64>(tm_base + kColO + 128 * b, P + (b * C::P_BYTES >> 4) + half * (C::P_HALF >> 4) + 2 * (s & 1),
                              (s < 2 ? A : B) + (2 * b * kBox + 2048 * (s & 1)) / 16, idesc_pv, s ? 1u : acc0);
          }
        tc_commit(&a->a_empty[ps]);
        tc_commit(&a->b_empty[bs]);
        tc_commit(&a->pv_done[tile & 1]);
      }
      __syncwarp();
      if (++ps == C::AS) ps = 0;
      if (++bs == C::BS) bs = 0, bph ^= 1;
    };
    for (int i = 0; ok && uniform(get_item(p, pl, a, i, it)); ++i) {
      const int t0 = uniform(it.t0), t1 = uniform(it.t1);
      if (t0 >= t1) continue;
      ok = __all_sync(0xffffffffu, wait(a, &a->q_full, items & 1, err));
      // whichever product can go: the first one runs ahead as far as S buffers and slots allow
      int t = t0, n = t0, g = 0;  // next tile of the second product; of the first, and its accumulation
      unsigned long long since = 0;
      for (uint32_t idle = 0; ok && t < t1;) {
        if (idle++ == 0) since = 0;
        if (n < t1 && qk_ready(g)) {
          qk(g);
          if (++g == C::GROUPS) g = 0, ++n;
          idle = 0;
        }
        if (t < n && pv_ready(t == t0)) {
          pv(t == t0);
          ++t, ++tile;
          idle = 0;
        }
        if ((idle & 255u) == 255u) {  // a bounded wait, as the others
          const unsigned long long now = globaltimer_ns();
          if (since == 0) since = now;
          const bool late = now - since > kWaitLimitNs;
          if (__any_sync(0xffffffffu, late) && !*reinterpret_cast<volatile int*>(&a->abort)) {
            record_error(err, DSA_DEVERR_WAIT_TIMEOUT);
            *reinterpret_cast<volatile int*>(&a->abort) = 1;
          }
          ok = !__any_sync(0xffffffffu, *reinterpret_cast<volatile int*>(&a->abort));
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
    // ---- scales of this CTA's positions (1 where there is none: the position is masked)
    int tiles = 0;
    bool ok = true;
    for (int i = 0; ok && get_item(p, pl, a, i, it); ++i) {
      for (int t = it.t0; ok && t < it.t1; ++t, ++tiles) {
        const int d = tiles % C::SC_DEPTH, pos = t * kKeys + 32 * rank;
        int64_t row = tree_row(p, it.seq, t * kKeys);
        const bool bad = row < 0;
        row += 32 * rank + (p.pages.table ? 0 : (int64_t)it.seq * p.L);
        const int n = (it.len - pos) * C::NSC;
        const float* src = p.kv_scale + row * C::NSC;
        float v[C::NSC + 1];
#pragma unroll
        for (int k = 0; k < C::NSC; ++k) v[k] = !bad && lane + 32 * k < n ? __ldg(src + lane + 32 * k) : 1.f;
        ok = __all_sync(0xffffffffu, wait(a, &a->sc_empty[d], ((tiles / C::SC_DEPTH) & 1) ^ 1, err));
        if (!ok) break;
#pragma unroll
        for (int k = 0; k < C::NSC; ++k) {
          const int e = lane + 32 * k, key = e / (C::NSC + !C::NSC);
          sc_s[(d * C::NSC + e - key * C::NSC) * 32 + key] = v[k];  // [scale of the row][position]
        }
        if (lane == 0) {
          a->tile_bad[tiles & 7] = bad;
          if (bad) record_error(err, DSA_DEVERR_INDEX_RANGE);
        }
        __syncwarp();
        mbar_arrive(&a->sc_full[d]);
      }
    }
  } else if (warp == 3) {
    // ---- credits of the exchange (here, because a release at cluster scope would hold up the softmax warps):
    // once a second product has read P, the other CTA may send into that buffer again
    int tiles = 0;
    bool ok = true;
    const uint32_t peer_p = dsmem_addr(&a->p_free[0], rank ^ 1);
    for (int i = 0; ok && get_item(p, pl, a, i, it); ++i) {
      for (int t = it.t0; ok && t < it.t1; ++t, ++tiles) {
        ok = __all_sync(0xffffffffu, wait(a, &a->pv_done[tiles & 1], (tiles >> 1) & 1, err));
        if (ok && lane == 0) arrive_remote(peer_p + 8 * (tiles % C::PB));
        __syncwarp();
      }
    }
  } else if (warp >= 12) {
    // ---- converters (E4M3): 16 codes per lane and step, loaded a tile ahead, widened into the swizzled bf16
    // boxes.  Eight lanes take four 16-code chunks of one box from two neighbouring positions: their eight
    // 16-byte stores fall into different banks.  A warp takes one pair of positions of each group of 8 pairs:
    // step k < 4: box k of our value columns, ours; < 8: the other's positions; < 12: our other columns; 12: rotary.
    const int cw = warp - 12;
    int as = 0, aph = 0, bs = 0, bph = 0, ks = 0, kph = 0;
    bool ok = true;
    constexpr int STEPS = 7;  // two boxes per step (lanes 0-15, 16-31), the rotary one alone
    uint4 raw[STEPS];
    // step k: box 2 k + lane / 16; the warp's pair of positions: 2 cw + 16 (lane / 8 % 2) ... (of 32)
    auto place = [&](int k, int& box, int& key, int& c) {
      box = 2 * k + (lane >> 4);
      c = lane & 3;
      key = 2 * cw + ((lane >> 2) & 1) + 16 * ((lane >> 3) & 1);
    };
    auto tile_rows = [&](const Item& x, int t) -> const uint8_t* {
      if (t >= x.t1) return nullptr;
      const int64_t row = tree_row(p, x.seq, t * kKeys);
      if (row < 0) return nullptr;
      return p.kv + (p.pages.table ? 0 : (int64_t)x.seq * p.kv_seq_stride) + row * p.kv_row_stride;
    };
    // of this lane's chunk of step k: its position in the tile and its offset from the tile's first row (boxes 0-3:
    // our value columns of our positions, 4-7: of the other's, 8-11: our positions' other columns, 12: rotary)
    int off[STEPS];
#pragma unroll
    for (int k = 0; k < STEPS; ++k) {
      int box, key, c;
      place(k, box, key, c);
      const int pos = key + 32 * (box >= 4 && box < 8 ? rank ^ 1 : rank);
      const int col = box < 8 ? 256 * rank + 64 * (box & 3) : box < 12 ? 256 * (rank ^ 1) + 64 * (box & 3) : 512;
      off[k] = pos * (int)p.kv_row_stride + col + 16 * c;
    }
    const int at0 = 2 * cw + ((lane >> 2) & 1) + 16 * ((lane >> 3) & 1);
    auto fetch = [&](const uint8_t* r, int n, int k) {
      const bool other = k >= 2 && k < 4;
      bool in = r != nullptr && (k < 6 || lane < 16);
      if (n < kKeys) in = in && at0 + 32 * (other ? rank ^ 1 : rank) < n;
      raw[k] = in ? __ldg(reinterpret_cast<const uint4*>(r + off[k])) : make_uint4(0u, 0u, 0u, 0u);
    };
    auto store = [&](uint8_t* slot, int k) {
      int box, key, c;
      place(k, box, key, c);
      if (box >= 13) return;
      uint8_t* d = slot + (k < 4 ? box & 3 : box - 8) * kBox + key * 128;
      const uint4 v = raw[k];
      *reinterpret_cast<uint4*>(d + (((2 * c) ^ (key & 7)) << 4)) =
          make_uint4(e4m3x2_to_bf16x2(v.x, 0x1404), e4m3x2_to_bf16x2(v.x, 0x3424), e4m3x2_to_bf16x2(v.y, 0x1404),
                     e4m3x2_to_bf16x2(v.y, 0x3424));
      *reinterpret_cast<uint4*>(d + (((2 * c + 1) ^ (key & 7)) << 4)) =
          make_uint4(e4m3x2_to_bf16x2(v.z, 0x1404), e4m3x2_to_bf16x2(v.z, 0x3424), e4m3x2_to_bf16x2(v.w, 0x1404),
                     e4m3x2_to_bf16x2(v.w, 0x3424));
    };
    for (int i = 0; ok && get_item(p, pl, a, i, it); ++i) {
      const uint8_t* r = tile_rows(it, it.t0);
      const uint8_t* r1 = tile_rows(it, it.t0 + 1);  // the block table is read two tiles ahead, the codes one
#pragma unroll
      for (int k = 0; k < STEPS; ++k) fetch(r, it.len - it.t0 * kKeys, k);
      for (int t = it.t0; ok && t < it.t1; ++t) {
        r = r1;
        r1 = tile_rows(it, t + 2);
        const int n = it.len - (t + 1) * kKeys;
        // steps [k0, k1) into a slot
        auto fill = [&](uint8_t* slot, int k0, int k1, uint64_t* full) {
#pragma unroll
          for (int k = 0; k < STEPS; ++k) {
            if (k >= k0 && k < k1) {
              store(slot, k);
              fetch(r, n, k);
            }
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(full);
        };
        ok = __all_sync(0xffffffffu, wait(a, &a->a_empty[as], aph ^ 1, err));
        if (!ok) break;
        fill(a_s + as * kSlotV, 0, 2, &a->a_full[as]);
        if (++as == C::AS) as = 0, aph ^= 1;
        ok = __all_sync(0xffffffffu, wait(a, &a->k_empty[ks], kph ^ 1, err));
        if (!ok) break;
        fill(k_s + ks * kSlotK, 4, STEPS, &a->k_full[ks]);
        if (++ks == C::KS) ks = 0, kph ^= 1;
        ok = __all_sync(0xffffffffu, wait(a, &a->b_empty[bs], bph ^ 1, err));
        if (!ok) break;
        fill(b_s + bs * kSlotV, 2, 4, &a->b_full[bs]);
        if (++bs == C::BS) bs = 0, bph ^= 1;
      }
    }
  } else if (warp >= 4) {
    // ---- softmax warps: thread = row = tensor-memory lane, half h of this CTA's 32 positions
    const int w = warp - 4, h = w >> 2, quarter = w & 3, row = 32 * quarter + lane, st = tid - 128;
    const uint32_t lane_base = tmem + ((uint32_t)(32 * quarter) << 16);
    const uint32_t peer_mx = dsmem_addr(&a->mx[0][h][row], rank ^ 1), peer_mm = dsmem_addr(&a->m_msg[0], rank ^ 1);
    const uint32_t peer_clear = dsmem_addr(&a->clear[0][w], rank ^ 1);
    const uint32_t peer_p = dsmem_addr(p_s, rank ^ 1) + rank * C::P_HALF + 32 * quarter * 64;
    const uint32_t peer_pm = dsmem_addr(&a->p_msg[0], rank ^ 1);
    const uint32_t peer_stat = dsmem_addr(&a->stat[h][row], rank ^ 1), peer_sf = dsmem_addr(&a->stat_full, rank ^ 1);
    const int p_at = row * 64, p_sw = (row >> 1) & 3;  // this row in a half of P, and its swizzle
    int tile = 0, items = 0;
    uint32_t su = 0;
    bool ok = true;
    const int rows = p.q_per_seq * p.H;

    for (int i = 0; get_item(p, pl, a, i, it); ++i) {
      const int row_lo = it.rt * kRows;
      const int64_t at = (int64_t)it.seq * rows + row_lo;  // the item's first row in out and lse
      const int nrows = min(kRows, rows - row_lo);
      if (it.t0 >= it.t1) {  // nothing to see: padding nodes, or an empty sequence
        if (rank == 0) {
          for (int k = st; k < nrows * (kDv / 8); k += 256)
            reinterpret_cast<uint4*>(p.out + at * kDv)[k] = make_uint4(0u, 0u, 0u, 0u);
          if (p.lse && st < nrows) p.lse[at + st] = -INFINITY;
        }
        continue;
      }
      // the query's row: most boxes into tensor memory, the others into shared memory, half of them per half h
      // (the previous item's products are done: its epilogue waited for them)
      {
        const uint4* src = reinterpret_cast<const uint4*>(p.q + (at + (row < nrows ? row : 0)) * kDqk);
        const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
#pragma unroll 4
        for (int k = 0; k < 4 * (9 - C::BT); ++k) {
          const int c = 2 * k + h;
          cp_async16(q_s + (c >> 3) * C::Q_BOX + row * 128 + (((c & 7) ^ (row & 7)) << 4), src + 8 * C::BT + c, row < nrows);
        }
        cp_async_commit();
#pragma unroll 4
        for (int g = 0; g < C::BT; ++g) {
          uint32_t v[16];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const uint4 u = row < nrows ? __ldg(src + 8 * g + 4 * h + k) : zero;
            v[4 * k] = u.x, v[4 * k + 1] = u.y, v[4 * k + 2] = u.z, v[4 * k + 3] = u.w;
          }
          tmem_st16(lane_base + kColQ + 32 * g + 16 * h, v);
        }
        cp_async_wait<0>();
        tmem_wait_st();
        tc_fence_before();
        fence_proxy_async_smem();
        if (ok) mbar_arrive(&a->q_full);
      }
      const int node = min((row_lo + row) / p.H, p.q_per_seq - 1);
      float m = -INFINITY, l = 0.f;

      // Logits of tile n (position tile t) for this row, scaled and masked; their maximum goes to the other
      // half's warp and to the other CTA.
      auto stage = [&](int n, int t, float (&x)[16]) {
        const float* sc = sc_s + (n % C::SC_DEPTH) * 32 * C::NSC + 16 * h;
        if constexpr (C::FP8) ok = wait(a, &a->sc_full[n % C::SC_DEPTH], (n / C::SC_DEPTH) & 1, err) && ok;
        if constexpr (C::TILED) {
#pragma unroll
          for (int k = 0; k < 16; ++k) x[k] = 0.f;
        }
#pragma unroll 1
        for (int g = 0; g < C::GROUPS; ++g, ++su) {
          ok = wait(a, &a->s_full[su % C::SB], (su / C::SB) & 1, err) && ok;
          tc_fence_after();
          float s[16];
          tmem_ld_sync(lane_base + C::COL_S + 32 * (su % C::SB) + 16 * h, s);
          tc_fence_before();
          __syncwarp();
          if (lane == 0 && ok) mbar_arrive(&a->s_empty[su % C::SB]);
#pragma unroll
          for (int k = 0; k < 16; k += 4) {
            float4 f = make_float4(p.scale_log2, p.scale_log2, p.scale_log2, p.scale_log2);
            if constexpr (C::FP8) f = *reinterpret_cast<const float4*>(sc + 32 * g + k);
            if constexpr (C::TILED) {
              x[k] = fmaf(f.x, s[k], x[k]), x[k + 1] = fmaf(f.y, s[k + 1], x[k + 1]);
              x[k + 2] = fmaf(f.z, s[k + 2], x[k + 2]), x[k + 3] = fmaf(f.w, s[k + 3], x[k + 3]);
            } else {
              if constexpr (C::FP8) f.x *= p.scale_log2, f.y *= p.scale_log2, f.z *= p.scale_log2, f.w *= p.scale_log2;
              x[k] = s[k] * f.x, x[k + 1] = s[k + 1] * f.y, x[k + 2] = s[k + 2] * f.z, x[k + 3] = s[k + 3] * f.w;
            }
          }
        }
        if constexpr (C::TILED) {
#pragma unroll
          for (int k = 0; k < 16; ++k) x[k] *= p.scale_log2;
        }
        const bool bad = p.pages.table && a->tile_bad[n & 7];
        uint32_t clear = 0;
        if ((t + 1) * kKeys > it.ctx || bad) {
          const uint32_t see = bad ? 0u : (uint32_t)(seen_bits(p, it, node, t) >> (32 * rank + 16 * h));
#pragma unroll
          for (int k = 0; k < 16; ++k) {
            if (!((see >> k) & 1)) {
              // a hidden position that may hold infinities or NaN (its logit is not finite, or it lies past
              // the end): its values are cleared in the tile, so that 0 * value is 0
              if (!C::FP8 && (!(fabsf(x[k]) < INFINITY) || t * kKeys + 32 * rank + 16 * h + k >= it.len)) clear |= 1u << (16 * h + k);
              x[k] = -INFINITY;
            }
          }
          clear = __reduce_or_sync(0xffffffffu, clear);
        }
        float mx = x[0];
#pragma unroll
        for (int k = 1; k < 16; ++k) mx = fmaxf(mx, x[k]);
        const int slot = n & 3;
        a->mx_own[n & 1][h][row] = mx;
        if (lane == 0) a->clear_own[slot][w] = clear;
        if (ok) {
          st_async4(peer_mx + slot * (2 * kRows * 4), __float_as_uint(mx), peer_mm + 8 * slot);
          if (lane == 0) st_async4(peer_clear + slot * 32, clear, peer_mm + 8 * slot);
        }
        __syncwarp();
        if (lane == 0 && ok) mbar_arrive(&a->m_msg[slot]);
      };

      float x[16], y[16];
      stage(tile, it.t0, x);
      for (int t = it.t0; t < it.t1; ++t, ++tile) {
        // the next tile's logits first, if they are there: their maxima travel while this tile is finished.  (With
        // tile scales always: there an S buffer is refilled only when all eight warps have read it, so they have
        // to take the tiles' steps in one order.)
        const bool more = t + 1 < it.t1;
        bool staged = false;
        if (more && (C::TILED || __all_sync(0xffffffffu, mbar_test(&a->s_full[su % C::SB], (su / C::SB) & 1)))) {
          stage(tile + 1, t + 1, y);
          staged = true;
        }
        const int slot = tile & 3, pb = tile % C::PB;
        ok = wait_cluster(a, &a->m_msg[slot], (tile >> 2) & 1, err) && ok;
        const float top = fmaxf(fmaxf(a->mx_own[tile & 1][0][row], a->mx_own[tile & 1][1][row]),
                                fmaxf(a->mx[slot][0][row], a->mx[slot][1][row]));
        if (!C::FP8 && (t + 1) * kKeys > it.ctx) {
          // zero the value columns of the positions to clear (their logits have been taken): a position past the
          // end always, another one only if it holds something that is not finite
          uint32_t clear[2] = {0u, 0u};  // ours, the other's
#pragma unroll
          for (int k = 0; k < 8; ++k) clear[0] |= a->clear_own[slot][k], clear[1] |= a->clear[slot][k];
          const int who = st >> 7, key = (st >> 2) & 31;  // a position, one of its four boxes
          if ((clear[who] >> key) & 1) {
            uint8_t* line = (who ? b_s + (tile % C::BS) * kSlotV : a_s + (tile % C::AS) * kSlotV) + (st & 3) * kBox + key * 128;
            bool zero = t * kKeys + 32 * (who ? rank ^ 1 : rank) + key >= it.len;
            if (who) ok = wait(a, &a->b_full[tile % C::BS], (tile / C::BS) & 1, err) && ok;  // (loaded for the second product only)
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
            }
          }
          __syncwarp();
        }
        // the reference maximum moves, in both halves' warps and in the other CTA alike
        if (__any_sync(0xffffffffu, top > m + kLazy)) {
          float f = 1.f;
          if (top > m + kLazy) {  // (m = -inf: nothing summed yet, the factor is 0)
            f = ex2(m - top);
            m = top;
            l *= f;
          }
          if (t > it.t0) {
            // the second product of the tile before is done: O may be rescaled (half of its columns per warp)
            ok = wait(a, &a->pv_done[(tile - 1) & 1], ((tile - 1) >> 1) & 1, err) && ok;
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
        // ---- weights
        const float mu = m == -INFINITY ? 0.f : m;
#pragma unroll
        for (int k = 0; k < 16; ++k) {
          x[k] = ex2(x[k] - mu);
          l += x[k];
        }
        // the tile that used this P buffer has been added, here and in the other CTA (so the copies of it have left)
        if (tile >= C::PB) ok = wait(a, &a->pv_done[(tile - C::PB) & 1], ((tile - C::PB) >> 1) & 1, err) && ok;
        ok = wait_cluster(a, &a->p_free[pb], ((tile / C::PB) & 1) ^ 1, err) && ok;
        const float* sc = sc_s + (tile % C::SC_DEPTH) * 32 * C::NSC + 16 * h;
        // P, times the positions' scales (a hidden position's weight is 0 whatever its scale holds)
        const bool hides = C::FP8 && ((t + 1) * kKeys > it.ctx || (p.pages.table && a->tile_bad[tile & 7]));
        auto put = [&](uint8_t* dst, int g) {
#pragma unroll
          for (int j = 0; j < 2; ++j) {  // 16-byte chunks of eight positions
            float z[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) z[k] = x[8 * j + k];
            if constexpr (C::FP8) {
              const float4 f0 = *reinterpret_cast<const float4*>(sc + 32 * g + 8 * j);
              const float4 f1 = *reinterpret_cast<const float4*>(sc + 32 * g + 8 * j + 4);
              z[0] *= f0.x, z[1] *= f0.y, z[2] *= f0.z, z[3] *= f0.w;
              z[4] *= f1.x, z[5] *= f1.y, z[6] *= f1.z, z[7] *= f1.w;
              if (hides) {
#pragma unroll
                for (int k = 0; k < 8; ++k) z[k] = x[8 * j + k] == 0.f ? 0.f : z[k];
              }
            }
            *reinterpret_cast<uint4*>(dst + p_at + (((2 * h + j) ^ p_sw) << 4)) =
                make_uint4(pack_bf16(z[0], z[1]), pack_bf16(z[2], z[3]), pack_bf16(z[4], z[5]), pack_bf16(z[6], z[7]));
          }
        };
#pragma unroll
        for (int pc = 0; pc < C::PC; ++pc) {
          put(p_s + (pb * C::PC + pc) * C::P_BYTES + rank * C::P_HALF, C::TILED ? 2 * rank + pc : 0);
          if (C::TILED) put(pp_s + pc * C::P_HALF, 2 * (rank ^ 1) + pc);  // the scales of the other's value tiles
        }
        fence_proxy_async_smem();
        tc_fence_before();
        pair_bar(quarter);  // both halves of the 32 rows are there
        if (lane == 0 && ok) {
          if (h == 0) {
#pragma unroll
            for (int pc = 0; pc < C::PC; ++pc)
              copy_remote(peer_p + (pb * C::PC + pc) * C::P_BYTES,
                          (C::TILED ? pp_s + pc * C::P_HALF : p_s + pb * C::P_BYTES + rank * C::P_HALF) + 32 * quarter * 64,
                          32 * 64, peer_pm + 8 * pb);
            copy_commit();
          } else if (quarter == 0) {
            mbar_arrive_expect_tx(&a->m_msg[slot], kMaxBytes);  // for the tile four on
          }
          if constexpr (C::FP8) mbar_arrive(&a->sc_empty[tile % C::SC_DEPTH]);
          mbar_arrive(&a->p_full[tile & 1]);
        }
        if (more) {
          if (!staged) stage(tile + 1, t + 1, y);
#pragma unroll
          for (int k = 0; k < 16; ++k) x[k] = y[k];
        }
      }
      // ---- the item's sums, to the other CTA as well
      a->mx_own[0][h][row] = l;
      if (ok) st_async4(peer_stat, __float_as_uint(l), peer_sf);
      ok = wait_cluster(a, &a->stat_full, items & 1, err) && ok;
      softmax_bar();
      {
        // (added in the same order on both sides)
        const float mine = a->mx_own[0][0][row] + a->mx_own[0][1][row], theirs = a->stat[0][row] + a->stat[1][row];
        l = rank ? theirs + mine : mine + theirs;
      }
      if (st == 0 && ok) mbar_arrive_expect_tx(&a->stat_full, 2 * kRows * 4);
      const bool live = row < nrows && (row_lo + row) / p.H < it.fresh;
      const float inv = live && l != 0.f ? 1.f / l : 0.f;
      if (rank == 0 && h == 0) {
        if (it.slot >= 0) pl.part_ml[(int64_t)it.slot * kRows + row] = make_float2(m, l);
        else if (p.lse && row < nrows) p.lse[at + row] = !live || l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
      }
      ok = wait(a, &a->o_done, items & 1, err) && ok;
      tc_fence_after();
#pragma unroll 1
      for (int c = 128 * h; c < 128 * h + 128; c += 32) {
        float o[32];
        tmem_ld_sync(lane_base + kColO + c, o);
        if (row < nrows && it.slot >= 0) {
          float4* dst = pl.part_o + ((int64_t)it.slot * (kDv / 4) + (256 * rank + c) / 4) * kRows + row;
#pragma unroll
          for (int k = 0; k < 8; ++k) dst[k * kRows] = make_float4(o[4 * k], o[4 * k + 1], o[4 * k + 2], o[4 * k + 3]);
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
      softmax_bar();  // the sums have been read
      tc_fence_before();
      if (lane == 0 && ok) mbar_arrive(&a->o_free);
      ++items;
    }
  }
  copy_wait_read();
  tc_fence_before();
  __syncthreads();
  cluster_sync();  // no CTA leaves while the other may still write into its shared memory
  if (warp == 0) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// Merges the chunks of each split row: out = sum_j 2^(m_j - M) o_j / sum_j 2^(m_j - M) l_j.  A CTA takes eight
// rows and 128 value columns, a thread one row and four values, eight chunks' loads in flight.
__global__ void __launch_bounds__(256) tree_combine_kernel(const TreeAttnParams p, const TreePlan pl) {
  pdl_wait();
  const int rows = p.q_per_seq * p.H;
  const int seq = blockIdx.y, row = blockIdx.x * 8 + (threadIdx.x & 7), c4 = blockIdx.z * 32 + (threadIdx.x >> 3);
  if (row >= rows) return;
  int ctx, fresh, len;
  seq_facts(p, seq, ctx, fresh, len);
  const int live = live_row_tiles(p, fresh);
  const int rt = row / kRows, r = row - rt * kRows;
  const int ch = pl.head[0], nt = (len + kKeys - 1) / kKeys;
  int chunks = nt ? (nt + ch - 1) / ch : 1;
  if (rt >= live || chunks == 1) return;  // written by the attention kernel
  if (row / p.H >= fresh) chunks = 0;     // a padding node beside live ones: zeros
  const int item0 = pl.head[1 + seq] + rt;
  float M = -INFINITY, l = 0.f;
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
  constexpr int B = 8;
  for (int j0 = 0; j0 < chunks; j0 += B) {
    float2 ml[B];
    float4 v[B];
#pragma unroll
    for (int k = 0; k < B; ++k) {
      const int64_t s = item0 + (j0 + k) * live;
      const bool in = j0 + k < chunks;
      ml[k] = in ? pl.part_ml[s * kRows + r] : make_float2(-INFINITY, 0.f);
      v[k] = in ? pl.part_o[(s * (kDv / 4) + c4) * kRows + r] : make_float4(0.f, 0.f, 0.f, 0.f);
    }
    float Mb = M;
#pragma unroll
    for (int k = 0; k < B; ++k) Mb = fmaxf(Mb, ml[k].x);
    const float mu = Mb == -INFINITY ? 0.f : Mb;
    const float f = exp2f(M - mu);
    l *= f;
    o.x *= f, o.y *= f, o.z *= f, o.w *= f;
#pragma unroll
    for (int k = 0; k < B; ++k) {
      if (j0 + k >= chunks) continue;
      const float g = exp2f(ml[k].x - mu);
      l += g * ml[k].y;
      o.x += g * v[k].x, o.y += g * v[k].y, o.z += g * v[k].z, o.w += g * v[k].w;
    }
    M = Mb;
  }
  const int64_t at = (int64_t)seq * rows + row;
  const float inv = l == 0.f ? 0.f : 1.f / l;
  *reinterpret_cast<uint2*>(p.out + at * kDv + 4 * c4) =
      make_uint2(pack_bf16(o.x * inv, o.y * inv), pack_bf16(o.z * inv, o.w * inv));
  if (p.lse && c4 == 0) p.lse[at] = l == 0.f ? -INFINITY : (M + log2f(l)) * kLn2;
}

__global__ void tree_nothing_kernel(const TreeAttnParams p, int64_t rows) {
  const int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
  if (i < rows * (kDv / 8)) reinterpret_cast<uint4*>(p.out)[i] = make_uint4(0u, 0u, 0u, 0u);
  if (p.lse && i < rows) p.lse[i] = -INFINITY;
}

constexpr int kClusters = 76;  // two of the 152 SMs each

// A launch with many units needs no split: its rounds of the grid are full enough.
TreePlan plan_of(const TreeAttnParams& p) {
  TreePlan pl = {};
  pl.row_tiles = (p.q_per_seq * p.H + kRows - 1) / kRows;
  pl.units = p.n_seq * pl.row_tiles;
  pl.cap = pl.units <= kItemsPerCta * kClusters ? kItemsPerCta * kClusters : 0;
  pl.grid = pl.cap ? kClusters : (pl.units < kClusters ? pl.units : kClusters);
  return pl;
}

size_t head_bytes(const TreeAttnParams& p) { return align_up((size_t)(1 + p.n_seq) * sizeof(int), 256); }

template <int FMT>
cudaError_t launch_fmt(const TreeAttnParams& p, TreePlan pl, void* ws, cudaStream_t stream) {
  using C = Cfg<FMT>;
  const bool paged = p.pages.table != nullptr;
  const cuuint64_t n = paged ? (cuuint64_t)p.pages.num_blocks * p.pages.block_size : (cuuint64_t)p.L;
  const cuuint64_t dims[3] = {(cuuint64_t)kDqk, n, paged ? 1 : (cuuint64_t)p.n_seq};
  const cuuint64_t strides[2] = {(cuuint64_t)p.kv_row_stride,
                                 paged || p.n_seq == 1 ? n * (cuuint64_t)p.kv_row_stride : (cuuint64_t)p.kv_seq_stride};
  CUtensorMap tm;
  memset(&tm, 0, sizeof(tm));
  const cuuint32_t box[3] = {64, 32, 1};
  if (!C::FP8 && encode_tensor_map(&tm, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<uint8_t*>(p.kv), dims, strides, box,
                                   CU_TENSOR_MAP_SWIZZLE_128B) != CUDA_SUCCESS)
    return cudaErrorInvalidValue;
  if (pl.cap) {
    uint8_t* w = reinterpret_cast<uint8_t*>(ws);
    pl.head = reinterpret_cast<int*>(w);
    w += head_bytes(p);
    pl.part_ml = reinterpret_cast<float2*>(w);
    w += (size_t)pl.cap * kRows * sizeof(float2);
    pl.part_o = reinterpret_cast<float4*>(w);
  }
  auto kern = tree_attn_kernel<FMT>;
  static std::atomic<uint64_t> allowed{0};
  cudaError_t e = allow_smem_once(&allowed, reinterpret_cast<const void*>(kern), C::SMEM);
  if (e != cudaSuccess) return e;
  e = launch_kernel(kern, dim3(2 * pl.grid), dim3(C::THREADS), C::SMEM, stream, false, tm, p, pl);
  if (e != cudaSuccess || !pl.cap) return e;
  return launch_kernel(tree_combine_kernel, dim3((p.q_per_seq * p.H + 7) / 8, p.n_seq, 4), dim3(256), 0, stream, true, p, pl);
}

}  // namespace

size_t tree_attn_ws_bytes(const TreeAttnParams& p) {
  const TreePlan pl = plan_of(p);
  if (!pl.cap || p.L == 0) return 0;
  return head_bytes(p) + (size_t)pl.cap * kRows * (sizeof(float2) + kDv * sizeof(float));
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
