// Attention of drafted tokens over the latent cache (dsa_tree_attn): query node i of sequence s sees
// the n_ctx[s] cached positions and the drafted positions n_ctx[s] + j whose bit j is set in its row
// of the tree mask,
//   logit[p] = sm_scale * q[i, h] . Kv[p],  out[i, h] = sum_p softmax(logit)[p] * Kv[p, :512].
//
// A "row" is one head of one node; the rows of a sequence are consecutive in q and share its cache.
// A cluster of two CTAs takes 128 rows and walks tiles of 64 positions.  The cache row's columns are
// split between the two: CTA c holds value columns 256 c ... 256 c + 255 and half of the 64 rotary
// columns, so every byte of the cache enters one SM's shared memory once and serves both products:
//   * partial S[128 x 64] = Q_c K_c^T: A = the rows in tensor memory (M = 128, 256 columns of q; the rotary
//     half from shared memory), B = the tile (K-major), 18 steps of K = 16;
//   * each CTA takes the softmax of 64 of the rows: the other sends it its partial S of those rows through
//     distributed shared memory (bulk copies, counted on the receiver's mbarrier), and gets their P (bf16)
//     back, so both hold P for all rows: 24 KB per tile each way;
//   * one pass over the positions keeps a reference maximum m and a sum l per row,
//       l' = l 2^(m - m') + sum_p 2^(x_p - m'),   o' = o 2^(m - m') + sum_p 2^(x_p - m') v_p,
//     where m is moved only when a tile's maximum exceeds it by more than 2^8 (weights stay below 2^8,
//     fp32 sums and bf16 weights lose nothing by it), so o in tensor memory is rescaled rarely;
//   * O_c[128 x 256] += P V_c: A = P (bf16) in shared memory; B = the same tile read MN-major (values along
//     N), 4 steps of K = 16 with N = 256.
// Why two CTAs: o for 128 rows x 512 values fills a tensor memory (512 columns), which leaves no room for S;
// with half of the values it takes 256 columns, q 128, two S buffers 128.  One CTA with 64 rows, q in shared
// memory and o transposed read 245 KB of shared memory per tile for the MMAs (2000 cycles at 128 B per
// cycle) and loaded each tile twice as often: 149 us instead of the time below for 8 x 8 nodes at 32K.
//
// Weights are rounded to bf16 for the second product (as the bf16 cache is); sums, maxima, logits and
// outputs are fp32.  E4M3 rows are widened to bf16 exactly, and their scales are applied in fp32 to the
// logit and to the weight (128-column scales: one S accumulator per scale tile, one P per value tile).
//
// Warp roles: producer (TMA), MMA issuer, scale loader, credits of the exchange, eight row warps (four take
// the softmax of this CTA's rows, four send the other's partial logits and take in its P; all of them
// the query load, the rescale and the epilogue), for E4M3 four warps that load, widen and store the tile.
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
constexpr int kKeys = 64;                 // positions per tile
constexpr int kBox = kKeys * 128;         // one 64-column box of a tile: 64 rows x 128 bytes
constexpr int kTile = 5 * kBox;           // four value boxes and the rotary one
constexpr int kSmemMax = 227 * 1024;
constexpr float kLazy = 8.f;              // log2 growth of a row's maximum that is left unscaled
constexpr int kItemsPerCta = 3;           // split launches are cut into at most this many items per cluster
// tensor-memory columns: O, the value columns of q, two S buffers
constexpr int kColO = 0, kColQ = 256, kColS = 384;

enum { kBf16 = 0, kFp8Row = 1, kFp8Tile = 2 };

template <int FMT>
struct Cfg {
  static constexpr bool FP8 = FMT != kBf16;
  static constexpr int NSC = FMT == kFp8Tile ? 5 : FMT == kFp8Row ? 1 : 0;
  static constexpr bool TILED = FMT == kFp8Tile;
  static constexpr int THREADS = FP8 ? 512 : 384;
  static constexpr int STAGES = TILED ? 2 : 3;            // tiles in shared memory
  static constexpr int PC = TILED ? 2 : 1;                // copies of P (one per 128 values)
  static constexpr int PB = TILED ? 1 : 2;                // P buffers
  static constexpr int SC_DEPTH = 2;
  static constexpr int SC_BYTES = NSC * kKeys * 4;
  static constexpr int X_BYTES = kRows / 2 * kKeys * 4;   // the peer's partial S of our rows (two buffers)
  static constexpr int QR_BYTES = kRows * 128;            // q's rotary columns
  static constexpr int P_BYTES = kRows * 128;             // P: 128 rows x 64 positions
  // what a CTA sends of a tile: its rows of P, their rescale factors, the positions to clear
  static constexpr int MSG_BYTES = PC * P_BYTES / 2 + 64 * 4 + 4 * 4;
  static constexpr int OUT_BYTES = X_BYTES;               // our partial S of the peer's rows, on its way there
  static constexpr int PP_BYTES = TILED ? PC * P_BYTES / 2 : 0;  // with tile scales: the peer's copies of our P
  static constexpr int AUX = 2560;
  static constexpr int OFF_X = STAGES * kTile;
  static constexpr int OFF_QR = OFF_X + 2 * X_BYTES;
  static constexpr int OFF_P = OFF_QR + QR_BYTES;
  static constexpr int OFF_OUT = OFF_P + PB * PC * P_BYTES;
  static constexpr int OFF_PP = OFF_OUT + OUT_BYTES;
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
  uint64_t full[3], empty[3];
  uint64_t s_full[2], s_empty[2], x_full[2], x_read[2], x_free[2];
  uint64_t p_full[2], p_msg[2], p_free[2], pv_done[2], stat_full, o_done, o_free, q_full, sc_full[2], sc_empty[2], drain;
  uint32_t tmem;
  int abort;
  int n_items;
  int tile_bad[4];
  int items[kItemsPerCta][8];
  alignas(16) float fac[2][64];  // the peer's rescale factors of its rows
  alignas(16) float fac_own[2][64];  // ours, on their way there
  uint32_t clear[2][4];    // positions to clear, from the peer (quarter, half)
  uint32_t clear_own[2][4];
  float red[2][64];        // per half of our rows: maxima, then sums
  float stat[64];          // the peer's sums
};
static_assert(sizeof(Aux) <= 2560, "Aux");

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

// A bounded wait.  Once one wait of the CTA has run out, the others return at once: the warps then walk
// through the rest of their work without waiting (every address stays in range), so that their common
// barriers still match, and the kernel ends.
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
__device__ __forceinline__ bool wait_cluster(Aux* a, uint64_t* bar, uint32_t parity, int* err) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred P;\n\t"
      "mbarrier.test_wait.parity.acquire.cluster.shared::cta.b64 P, [%1], %2;\n\t"
      "selp.b32 %0, 1, 0, P;\n\t}"
      : "=r"(ok)
      : "r"(smem_u32(bar)), "r"(parity)
      : "memory");
  return ok || wait_slow(a, bar, parity, err, true);
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

// `bytes` of this CTA's shared memory into the other CTA's, counted on its mbarrier.  (Stores of 16 bytes per
// lane, each counted by itself, took 1300 to 1900 cycles for a tile's 16 KB to arrive.)
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

// Barriers: of the two warps that share 32 rows (id 1 or 2), of all eight row warps (id 3).
__device__ __forceinline__ void pair_bar(int id) { asm volatile("bar.sync %0, 64;" ::"r"(id) : "memory"); }
__device__ __forceinline__ bool pair_any(int id, bool pred) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.u32 p, %1, 0;\n\t"
      "bar.red.or.pred q, %2, 64, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"((uint32_t)pred), "r"(id)
      : "memory");
  return r != 0;
}
__device__ __forceinline__ void row_bar() { asm volatile("bar.sync 3, 256;" ::: "memory"); }

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
// box apart.  Adding bytes / 16 moves the start address.
constexpr uint32_t kDescHi = (1024u >> 4) | (1u << 14) | (2u << 29);
__device__ __forceinline__ uint32_t kmajor_lo(uint32_t saddr) { return ((saddr & 0x3FFFFu) >> 4) | (1u << 16); }
__device__ __forceinline__ uint32_t mnmajor_lo(uint32_t saddr) {
  return ((saddr & 0x3FFFFu) >> 4) | ((uint32_t)(kBox >> 4) << 16);
}

// D += A B^T with A in shared memory, or in tensor memory (lane = row, two bf16 per column).
__device__ __forceinline__ void mma_ss(uint32_t d, uint32_t a_lo, uint32_t b_lo, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 da, db;\n\t"
      "mov.b64 da, {%1, %5};\n\t"
      "mov.b64 db, {%2, %5};\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %3, p;\n\t}" ::"r"(d),
      "r"(a_lo), "r"(b_lo), "r"(idesc), "r"(acc), "r"(kDescHi)
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
  uint8_t* tiles_s = smem;
  uint8_t* x_s = smem + C::OFF_X;
  uint8_t* qr_s = smem + C::OFF_QR;
  uint8_t* p_s = smem + C::OFF_P;
  uint8_t* out_s = smem + C::OFF_OUT;
  uint8_t* pp_s = smem + C::OFF_PP;
  float* sc_s = reinterpret_cast<float*>(smem + C::OFF_SC);
  Aux* a = reinterpret_cast<Aux*>(smem + C::OFF_AUX);
  const int tid = threadIdx.x, lane = tid & 31, warp = uniform(tid >> 5);
  const int rank = uniform((int)cluster_rank());  // which half of the columns, and which 64 of the rows
  int* err = p.err;

  if (warp == 0) {
    tmem_alloc(&a->tmem, 512);
    tmem_relinquish();
  }
  if (tid == 32) {
    for (int i = 0; i < 3; ++i) mbar_init(&a->full[i], C::FP8 ? 4 : 1), mbar_init(&a->empty[i], 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&a->s_full[i], 1), mbar_init(&a->s_empty[i], 8);
      mbar_init(&a->x_full[i], 1), mbar_init(&a->x_read[i], 4), mbar_init(&a->x_free[i], 1);
      mbar_init(&a->p_full[i], 8), mbar_init(&a->p_msg[i], 1), mbar_init(&a->p_free[i], 1), mbar_init(&a->pv_done[i], 1);
      mbar_init(&a->sc_full[i], 32), mbar_init(&a->sc_empty[i], C::TILED ? 8 : 4);
    }
    mbar_init(&a->stat_full, 1);
    mbar_init(&a->o_done, 1);
    mbar_init(&a->o_free, 8);
    mbar_init(&a->q_full, 256);
    mbar_init(&a->drain, 1);
    a->abort = 0;
    fence_mbar_init();
    for (int i = 0; i < 2; ++i) {
      mbar_arrive_expect_tx(&a->x_full[i], C::X_BYTES);
      mbar_arrive_expect_tx(&a->p_msg[i], C::MSG_BYTES);
    }
    mbar_arrive_expect_tx(&a->stat_full, 64 * 4);
  }
  if (pl.cap) plan_items(p, pl, a, reinterpret_cast<int*>(tiles_s));
  fence_proxy_async_smem();  // the plan's scratch is a tile that the copies write
  tc_fence_before();
  __syncthreads();
  cluster_sync();  // the peer's barriers are ready too
  tc_fence_after();
  const uint32_t tmem = a->tmem;
  pdl_launch_dependents();

  Item it;
  if (warp == 0) {
    // ---- producer (bf16): this CTA's columns of each tile by TMA
    if (lane == 0 && !C::FP8) {
      prefetch_tmap(&tm);
      int sl = 0, ph = 0, tiles = 0;
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
          ok = wait(a, &a->empty[sl], ph ^ 1, err);
          if (!ok) break;
          a->tile_bad[tiles & 3] = bad;
          uint8_t* dst = tiles_s + sl * kTile;
          mbar_arrive_expect_tx(&a->full[sl], kTile);
#pragma unroll
          for (int b = 0; b < 4; ++b) tma_load_3d(dst + b * kBox, &tm, &a->full[sl], 256 * rank + 64 * b, row, z);
          tma_load_3d(dst + 4 * kBox, &tm, &a->full[sl], 512, row, z);
          if (++sl == C::STAGES) sl = 0, ph ^= 1;
        }
      }
      if (*reinterpret_cast<volatile int*>(&a->abort))  // wind down: the copies in flight land first
        for (int s = 0; s < C::STAGES; ++s) mbar_wait(&a->full[s], s < sl ? ph : ph ^ 1, err);
    }
    __syncwarp();
  } else if (warp == 1) {
    // ---- MMA issuer.  The warp stays converged and one elected lane issues; descriptors are sums of
    // 32-bit words (their upper words are one constant), so that issuing an instruction costs less than
    // the tensor cores take for it
    constexpr uint32_t idesc_qk = make_idesc(1, 1, kRows, kKeys);
    constexpr uint32_t idesc_pv = make_idesc(1, 1, kRows, C::TILED ? 128 : 256) | (1u << 16);  // B (values) MN-major
    const uint32_t tm_base = (uint32_t)uniform((int)tmem);
    const uint32_t k_lo = kmajor_lo(smem_u32(tiles_s)), v_lo = mnmajor_lo(smem_u32(tiles_s));
    const uint32_t qr_lo = kmajor_lo(smem_u32(qr_s)) + 4 * rank;  // this CTA's half: 64 bytes into the row
    const uint32_t p_lo = kmajor_lo(smem_u32(p_s));
    int qs = 0, qph = 0, ps = 0;  // stages of the first and of the second product
    int tile = 0, items = 0;
    uint32_t su = 0;              // uses of the S buffers
    bool ok = true;
    auto all = [&](uint64_t* bar, uint32_t parity) { ok = __all_sync(0xffffffffu, wait(a, bar, parity, err)) && ok; };
    auto commit = [&](uint64_t* bar) {
      if (elect_one()) tc_commit(bar);
      __syncwarp();
    };
    // First product of the next tile, group g of its columns: all of them (-1), or for 128-column scales
    // one accumulation per scale tile (0, 1: 128 value columns; 2: the rotary ones).  The row warps have
    // read what the S buffer held.
    auto qk = [&](int g) {
      if (g <= 0) all(&a->full[qs], qph);
      all(&a->s_empty[su & 1], ((su >> 1) & 1) ^ 1);
      tc_fence_after();
      const uint32_t d = tm_base + kColS + 64 * (su & 1), B = k_lo + qs * (kTile >> 4);
      if (elect_one()) {
        if (g < 2) {
          const uint32_t q0 = tm_base + kColQ + (g > 0 ? 64 : 0), B0 = B + (g > 0 ? 2 * kBox >> 4 : 0);
#pragma unroll
          for (int k = 0; k < (C::TILED ? 8 : 16); ++k)
            mma_ts(d, q0 + 8 * k, B0 + ((k >> 2) * kBox + 32 * (k & 3)) / 16, idesc_qk, k ? 1u : 0u);
        }
        if (g < 0 || g == 2) {
#pragma unroll
          for (int k = 0; k < 2; ++k)
            mma_ss(d, qr_lo + 2 * k, B + (4 * kBox >> 4) + 4 * rank + 2 * k, idesc_qk, k || !C::TILED ? 1u : 0u);
        }
        tc_commit(&a->s_full[su & 1]);
      }
      __syncwarp();
      ++su;
      if (g < 0 || g == 2) {
        if (++qs == C::STAGES) qs = 0, qph ^= 1;
      }
    };
    auto qk_tile = [&]() {
      if (C::TILED) qk(0), qk(1), qk(2);
      else qk(-1);
    };
    auto pv = [&](bool first) {
      const uint32_t acc0 = first ? 0u : 1u, B = v_lo + ps * (kTile >> 4);
      const uint32_t P = p_lo + (tile % C::PB) * (C::PC * C::P_BYTES >> 4);
      if (elect_one()) {
        constexpr int NB = C::TILED ? 2 : 1;  // value tiles of N = 128 with a P each, or all 256 at once
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
          for (int ks = 0; ks < 4; ++ks)
            mma_ss(tm_base + kColO + 128 * b, P + (b * C::P_BYTES + 32 * ks) / 16, B + (2 * b * kBox + 2048 * ks) / 16,
                   idesc_pv, ks ? 1u : acc0);
        tc_commit(&a->empty[ps]);
        tc_commit(&a->pv_done[tile & 1]);
      }
      __syncwarp();
      if (++ps == C::STAGES) ps = 0;
    };
    constexpr int AHEAD = C::TILED ? 1 : 2;  // tiles whose first product is issued before P of this one is there
    for (int i = 0; uniform(get_item(p, pl, a, i, it)); ++i) {
      const int t0 = uniform(it.t0), t1 = uniform(it.t1);
      if (t0 >= t1) continue;
      all(&a->q_full, items & 1);
      tc_fence_after();
      int tq = t0;  // the next tile to start
      for (; tq < t1 && tq < t0 + AHEAD; ++tq) qk_tile();
      for (int t = t0; t < t1; ++t, ++tile) {
        // the tile after next early, if it and its S buffer are ready; P of this one first otherwise
        bool started = tq >= t1;
        if (!started && (C::TILED || __all_sync(0xffffffffu, mbar_test(&a->full[qs], qph) &&
                                                                 mbar_test(&a->s_empty[su & 1], ((su >> 1) & 1) ^ 1)))) {
          qk_tile();
          ++tq;
          started = true;
        }
        all(&a->p_full[tile & 1], (tile >> 1) & 1);
        if (t == t0) all(&a->o_free, (items & 1) ^ 1);
        tc_fence_after();
        pv(t == t0);
        if (!started) {
          qk_tile();
          ++tq;
        }
      }
      commit(&a->o_done);
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
    for (int i = 0; ok && get_item(p, pl, a, i, it); ++i) {
      for (int t = it.t0; ok && t < it.t1; ++t, ++tiles) {
        const int d = tiles % C::SC_DEPTH;
        int64_t row = tree_row(p, it.seq, t * kKeys);
        const bool bad = row < 0;
        if (!p.pages.table) row += (int64_t)it.seq * p.L;
        const int n = min(kKeys, it.len - t * kKeys) * C::NSC;
        const float* src = p.kv_scale + row * C::NSC;
        float v[C::NSC * 2 + 1];
#pragma unroll
        for (int k = 0; k < C::NSC * 2; ++k) v[k] = !bad && lane + 32 * k < n ? __ldg(src + lane + 32 * k) : 1.f;
        ok = __all_sync(0xffffffffu, wait(a, &a->sc_empty[d], ((tiles / C::SC_DEPTH) & 1) ^ 1, err));
        if (!ok) break;
#pragma unroll
        for (int k = 0; k < C::NSC * 2; ++k) sc_s[d * kKeys * C::NSC + lane + 32 * k] = v[k];
        if (lane == 0) {
          a->tile_bad[tiles & 3] = bad;
          if (bad) record_error(err, DSA_DEVERR_INDEX_RANGE);
        }
        __syncwarp();
        mbar_arrive(&a->sc_full[d]);
      }
    }
  } else if (warp == 3) {
    // ---- credits of the exchange (here, because a release at cluster scope would hold up the row warps): once
    // our softmax warps have read the peer's part of S, its buffer is armed for the tile after next and
    // the peer told so; once a second product has read P, the peer may send into that buffer again
    int tiles = 0;
    bool ok = true;
    const uint32_t peer_x = dsmem_addr(&a->x_free[0], rank ^ 1), peer_p = dsmem_addr(&a->p_free[0], rank ^ 1);
    for (int i = 0; ok && get_item(p, pl, a, i, it); ++i) {
      for (int t = it.t0; ok && t < it.t1; ++t, ++tiles) {
        const int b = tiles & 1;
        ok = __all_sync(0xffffffffu, wait(a, &a->x_read[b], (tiles >> 1) & 1, err));
        if (ok && lane == 0) {
          mbar_arrive_expect_tx(&a->x_full[b], C::X_BYTES);
          arrive_remote(peer_x + 8 * b);
        }
        __syncwarp();
        ok = ok && __all_sync(0xffffffffu, wait(a, &a->pv_done[b], (tiles >> 1) & 1, err));
        if (ok && lane == 0) arrive_remote(peer_p + 8 * (tiles % C::PB));
        __syncwarp();
      }
    }
  } else if (warp >= 12) {
    // ---- converters (E4M3): 16 codes per lane and step, loaded a tile ahead, widened into the swizzled bf16
    // boxes.  Eight lanes take four 16-code chunks of one box from two neighbouring positions: their eight
    // 16-byte stores fall into different banks.
    const int ct = tid - 384, cw = warp - 12;
    int st = 0, sph = 0;
    bool ok = true;
    uint4 raw[9];
    auto place = [&](int k, int& key, int& box, int& c) {  // chunk c of 16 codes of a box of 64 columns
      if (k < 8) {
        const int unit = 16 * k + 4 * cw + (lane >> 3);
        box = unit & 3, key = 2 * (unit >> 2) + ((lane >> 2) & 1), c = lane & 3;
      } else {  // the rotary half: 32 codes of a position
        box = 4, key = ct >> 1, c = 2 * rank + (ct & 1);
      }
    };
    auto tile_rows = [&](const Item& x, int t) -> const uint8_t* {
      if (t >= x.t1) return nullptr;
      const int64_t row = tree_row(p, x.seq, t * kKeys);
      if (row < 0) return nullptr;
      return p.kv + (p.pages.table ? 0 : (int64_t)x.seq * p.kv_seq_stride) + row * p.kv_row_stride;
    };
    auto fetch = [&](const uint8_t* r, int n, int k) {
      int key, box, c;
      place(k, key, box, c);
      const int col = (box < 4 ? 256 * rank + 64 * box : 512) + 16 * c;
      raw[k] = r && key < n ? __ldg(reinterpret_cast<const uint4*>(r + (int64_t)key * p.kv_row_stride + col))
                            : make_uint4(0u, 0u, 0u, 0u);
    };
    for (int i = 0; ok && get_item(p, pl, a, i, it); ++i) {
      const uint8_t* r = tile_rows(it, it.t0);
      const uint8_t* r1 = tile_rows(it, it.t0 + 1);  // the block table is read two tiles ahead, the codes one
#pragma unroll
      for (int k = 0; k < 9; ++k) fetch(r, it.len - it.t0 * kKeys, k);
      for (int t = it.t0; ok && t < it.t1; ++t) {
        r = r1;
        r1 = tile_rows(it, t + 2);
        const int n = it.len - (t + 1) * kKeys;
        ok = __all_sync(0xffffffffu, wait(a, &a->empty[st], sph ^ 1, err));
        if (!ok) break;
        uint8_t* dst = tiles_s + st * kTile;
#pragma unroll
        for (int k = 0; k < 9; ++k) {
          int key, box, c;
          place(k, key, box, c);
          uint8_t* d = dst + box * kBox + key * 128;
          const uint4 v = raw[k];
          *reinterpret_cast<uint4*>(d + (((2 * c) ^ (key & 7)) << 4)) =
              make_uint4(e4m3x2_to_bf16x2(v.x, 0x1404), e4m3x2_to_bf16x2(v.x, 0x3424), e4m3x2_to_bf16x2(v.y, 0x1404),
                         e4m3x2_to_bf16x2(v.y, 0x3424));
          *reinterpret_cast<uint4*>(d + (((2 * c + 1) ^ (key & 7)) << 4)) =
              make_uint4(e4m3x2_to_bf16x2(v.z, 0x1404), e4m3x2_to_bf16x2(v.z, 0x3424), e4m3x2_to_bf16x2(v.w, 0x1404),
                         e4m3x2_to_bf16x2(v.w, 0x3424));
          fetch(r, n, k);
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&a->full[st]);
        if (++st == C::STAGES) st = 0, sph ^= 1;
      }
    }
  } else if (warp >= 4) {
    // ---- row warps.  Thread = row (tensor-memory lane) and half h of the tile's positions (32), of the query's
    // columns and of the value columns.  Rows 64 rank ... are ours (softmax), the others the peer's.
    const int w = warp - 4, h = w >> 2, quarter = w & 3, row = 32 * quarter + lane, r64 = row & 63;
    const bool own = (quarter >> 1) == rank;
    const int bar_id = 1 + (quarter & 1);
    const uint32_t lane_base = tmem + ((uint32_t)(32 * quarter) << 16);
    const int unit = 2 * (quarter & 1) + h;  // of the exchanged logits: 32 rows x 32 positions, [8 chunks][32 rows] x 16 B
    const uint32_t peer_x = dsmem_addr(x_s, rank ^ 1) + unit * 4096;
    const uint32_t peer_xf = dsmem_addr(&a->x_full[0], rank ^ 1), peer_msg = dsmem_addr(&a->p_msg[0], rank ^ 1);
    const uint32_t peer_p = dsmem_addr(p_s, rank ^ 1) + 32 * quarter * 128;
    const uint32_t peer_fac = dsmem_addr(&a->fac[0][32 * (quarter & 1)], rank ^ 1);
    const uint32_t peer_clear = dsmem_addr(&a->clear[0][unit], rank ^ 1);
    const float4* my_x = reinterpret_cast<const float4*>(x_s) + unit * 256 + lane;
    int tile = 0, items = 0;
    uint32_t su = 0;
    bool ok = true;
    const int rows = p.q_per_seq * p.H;

    // This CTA's partial logits of tile n (its columns; with tile scales, scaled), 32 positions of this row.
    auto partial = [&](int n, float (&x)[32]) {
      if constexpr (C::TILED) {
        const float* sc = sc_s + (n % C::SC_DEPTH) * kKeys * 5 + 32 * h * 5;
        ok = wait(a, &a->sc_full[n % C::SC_DEPTH], (n / C::SC_DEPTH) & 1, err) && ok;
#pragma unroll
        for (int k = 0; k < 32; ++k) x[k] = 0.f;
#pragma unroll 1
        for (int g = 0; g < 3; ++g, ++su) {
          ok = wait(a, &a->s_full[su & 1], (su >> 1) & 1, err) && ok;
          tc_fence_after();
          float s[32];
          tmem_ld_sync(lane_base + kColS + 64 * (su & 1) + 32 * h, s);
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&a->s_empty[su & 1]);
          const float* f = sc + (g < 2 ? 2 * rank + g : 4);
#pragma unroll
          for (int k = 0; k < 32; ++k) x[k] = fmaf(f[5 * k], s[k], x[k]);
        }
      } else {
        ok = wait(a, &a->s_full[n & 1], (n >> 1) & 1, err) && ok;
        tc_fence_after();
        tmem_ld_sync(lane_base + kColS + 64 * (n & 1) + 32 * h, x);
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&a->s_empty[n & 1]);
      }
    };
    // O of this row (128 of the columns) times f, once the tile before has been added.
    auto rescale = [&](int n, float f) {
      ok = wait(a, &a->pv_done[(n - 1) & 1], ((n - 1) >> 1) & 1, err) && ok;
      tc_fence_after();
#pragma unroll 1
      for (int c = 0; c < 128; c += 16) {
        float o[16];
        tmem_ld_sync(lane_base + kColO + 128 * h + c, o);
        uint32_t v[16];
#pragma unroll
        for (int k = 0; k < 16; ++k) v[k] = __float_as_uint(o[k] * f);
        tmem_st16(lane_base + kColO + 128 * h + c, v);
      }
      tmem_wait_st();
    };

    for (int i = 0; get_item(p, pl, a, i, it); ++i) {
      const int row_lo = it.rt * kRows;
      const int64_t at = (int64_t)it.seq * rows + row_lo;  // the item's first row in out and lse
      const int nrows = min(kRows, rows - row_lo);
      if (it.t0 >= it.t1) {  // nothing to see: padding nodes, or an empty sequence
        if (rank == 0) {
          const int st = tid - 128;
          for (int k = st; k < nrows * (kDv / 8); k += 256)
            reinterpret_cast<uint4*>(p.out + at * kDv)[k] = make_uint4(0u, 0u, 0u, 0u);
          if (p.lse && st < nrows) p.lse[at + st] = -INFINITY;
        }
        continue;
      }
      // the query's rows: 128 of this CTA's 256 value columns into tensor memory, half of its 32 rotary
      // columns into shared memory (the previous item's products are done: its epilogue waited for them)
      {
        const uint4* src = reinterpret_cast<const uint4*>(p.q + (at + (row < nrows ? row : 0)) * kDqk);
        const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
        uint4 r[2];
#pragma unroll
        for (int k = 0; k < 2; ++k) r[k] = row < nrows ? __ldg(src + 64 + 4 * rank + 2 * h + k) : zero;
#pragma unroll
        for (int g = 0; g < 4; ++g) {
          uint32_t v[16];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const uint4 u = row < nrows ? __ldg(src + 32 * rank + 16 * h + 4 * g + k) : zero;
            v[4 * k] = u.x, v[4 * k + 1] = u.y, v[4 * k + 2] = u.z, v[4 * k + 3] = u.w;
          }
          tmem_st16(lane_base + kColQ + 64 * h + 16 * g, v);
        }
#pragma unroll
        for (int k = 0; k < 2; ++k)
          *reinterpret_cast<uint4*>(qr_s + row * 128 + (((4 * rank + 2 * h + k) ^ (row & 7)) << 4)) = r[k];
        tmem_wait_st();
        tc_fence_before();
        fence_proxy_async_smem();
        mbar_arrive(&a->q_full);
      }
      float l = 0.f;
      if (own) {
        // ======== softmax of our rows
        const int node = min((row_lo + row) / p.H, p.q_per_seq - 1);
        float m = -INFINITY;
        for (int t = it.t0; t < it.t1; ++t, ++tile) {
          const int xb = tile & 1, pb = tile % C::PB;
          const bool tail = (t + 1) * kKeys > it.ctx;
          const float* sc = sc_s + (tile % C::SC_DEPTH) * kKeys * C::NSC + 32 * h * C::NSC;
          float x[32];
          partial(tile, x);
          ok = wait_cluster(a, &a->x_full[xb], (tile >> 1) & 1, err) && ok;
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const float4 v = my_x[xb * (C::X_BYTES / 16) + j * 32];
            x[4 * j] += v.x, x[4 * j + 1] += v.y, x[4 * j + 2] += v.z, x[4 * j + 3] += v.w;
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(&a->x_read[xb]);
          // ---- scale, mask
          if constexpr (FMT == kFp8Row) {
            ok = wait(a, &a->sc_full[tile % C::SC_DEPTH], (tile / C::SC_DEPTH) & 1, err) && ok;
#pragma unroll
            for (int k = 0; k < 32; k += 4) {
              const float4 f = *reinterpret_cast<const float4*>(sc + k);
              x[k] *= f.x * p.scale_log2, x[k + 1] *= f.y * p.scale_log2;
              x[k + 2] *= f.z * p.scale_log2, x[k + 3] *= f.w * p.scale_log2;
            }
          } else {
#pragma unroll
            for (int k = 0; k < 32; ++k) x[k] *= p.scale_log2;
          }
          const bool bad = p.pages.table && a->tile_bad[tile & 3];
          uint32_t clear = 0;
          if (tail || bad) {
            const uint32_t see = bad ? 0u : (uint32_t)(seen_bits(p, it, node, t) >> (32 * h));
#pragma unroll
            for (int k = 0; k < 32; ++k) {
              if (!((see >> k) & 1)) {
                // a hidden position that may hold infinities or NaN (its logit is not finite, or it lies past
                // the end): its values are cleared in the tile, so that 0 * value is 0
                if (!C::FP8 && (!(fabsf(x[k]) < INFINITY) || t * kKeys + 32 * h + k >= it.len)) clear |= 1u << k;
                x[k] = -INFINITY;
              }
            }
            clear = __reduce_or_sync(0xffffffffu, clear);
          }
          // ---- the reference maximum moves when a position exceeds it by more than kLazy
          float mx = x[0];
#pragma unroll
          for (int k = 1; k < 32; ++k) mx = fmaxf(mx, x[k]);
          a->red[h][r64] = mx;
          float f = 1.f;
          if (pair_any(bar_id, mx > m + kLazy)) {
            mx = fmaxf(a->red[0][r64], a->red[1][r64]);
            if (mx > m + kLazy) {  // (m = -inf: nothing summed yet, the factor is 0)
              f = ex2(m - mx);
              m = mx;
              l *= f;
            }
            if (t > it.t0) rescale(tile, f);
            pair_bar(bar_id);  // red is read before the next tile's maxima are written
          }
          // ---- weights
          const float mu = m == -INFINITY ? 0.f : m;
#pragma unroll
          for (int k = 0; k < 32; ++k) {
            x[k] = ex2(x[k] - mu);
            l += x[k];
          }
          // the tile that used this P buffer has been added, here and at the peer
          if (tile >= C::PB) ok = wait(a, &a->pv_done[(tile - C::PB) & 1], ((tile - C::PB) >> 1) & 1, err) && ok;
          ok = wait_cluster(a, &a->p_free[pb], ((tile / C::PB) & 1) ^ 1, err) && ok;
          if (C::TILED) {
            if (h == 0 && lane == 0) copy_wait_read();  // the staged copies of the tile before have left
            pair_bar(bar_id);
          }
          const uint32_t msg = peer_msg + 8 * pb;
#pragma unroll
          for (int pc = 0; pc < C::PC; ++pc) {
            const int off = (pb * C::PC + pc) * C::P_BYTES;
#pragma unroll
            for (int j = 0; j < 4; ++j) {  // 16-byte chunks of eight positions
              uint32_t v[4];
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                const int e = 8 * j + 2 * k;
                float y0 = x[e], y1 = x[e + 1];
                if constexpr (C::FP8) {
                  // the weight carries the position's scale (of the values' tile, here of this CTA's columns: the
                  // peer's copy is made below); a hidden position's weight is 0 whatever its scale holds
                  const float f0 = sc[e * C::NSC + (C::TILED ? 2 * rank + pc : 0)];
                  const float f1 = sc[(e + 1) * C::NSC + (C::TILED ? 2 * rank + pc : 0)];
                  y0 = y0 == 0.f ? 0.f : y0 * f0;
                  y1 = y1 == 0.f ? 0.f : y1 * f1;
                }
                v[k] = pack_bf16(y0, y1);
              }
              const int sw = ((4 * h + j) ^ (row & 7)) << 4;
              *reinterpret_cast<uint4*>(p_s + off + row * 128 + sw) = make_uint4(v[0], v[1], v[2], v[3]);
              if constexpr (C::TILED) {  // the peer's copy carries the scales of its value tiles
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                  const int e = 8 * j + 2 * k;
                  const float f0 = sc[e * 5 + 2 * (rank ^ 1) + pc], f1 = sc[(e + 1) * 5 + 2 * (rank ^ 1) + pc];
                  v[k] = pack_bf16(x[e] == 0.f ? 0.f : x[e] * f0, x[e + 1] == 0.f ? 0.f : x[e + 1] * f1);
                }
                *reinterpret_cast<uint4*>(pp_s + pc * (C::P_BYTES / 2) + r64 * 128 + sw) = make_uint4(v[0], v[1], v[2], v[3]);
              }
            }
          }
          if (h == 0) a->fac_own[pb][r64] = f;
          fence_proxy_async_smem();
          pair_bar(bar_id);  // both halves of the 32 rows are written
          if (ok && lane == 0) {
            if (h == 0) {
#pragma unroll
              for (int pc = 0; pc < C::PC; ++pc)
                copy_remote(peer_p + (pb * C::PC + pc) * C::P_BYTES,
                            C::TILED ? pp_s + pc * (C::P_BYTES / 2) + 32 * (quarter & 1) * 128
                                     : p_s + (pb * C::PC + pc) * C::P_BYTES + 32 * quarter * 128,
                            4096, msg);
              copy_remote(peer_fac + 256 * pb, &a->fac_own[pb][32 * (quarter & 1)], 128, msg);
              copy_commit();
            }
            st_async4(peer_clear + 16 * pb, clear, msg);
          }
          if (!C::FP8 && tail) {
            if (lane == 0) a->clear_own[tile & 1][2 * (quarter & 1) + h] = clear;
            row_bar();  // the other four warps clear the tile
          }
          tc_fence_before();
          __syncwarp();
          if (lane == 0) {
            if constexpr (C::FP8) mbar_arrive(&a->sc_empty[tile % C::SC_DEPTH]);
            mbar_arrive(&a->p_full[tile & 1]);
          }
        }
        // ---- the item's sums, to the peer as well
        pair_bar(bar_id);
        a->red[h][r64] = l;
        pair_bar(bar_id);
        l = a->red[0][r64] + a->red[1][r64];
        pair_bar(bar_id);
        if (h == 0) {
          if (ok) st_async4(dsmem_addr(&a->stat[r64], rank ^ 1), __float_as_uint(l), dsmem_addr(&a->stat_full, rank ^ 1));
          const bool live = row < nrows && (row_lo + row) / p.H < it.fresh;
          if (it.slot >= 0) pl.part_ml[(int64_t)it.slot * kRows + row] = make_float2(m, l);
          else if (p.lse && row < nrows) p.lse[at + row] = !live || l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
        }
      } else {
        // ======== the peer's rows: send it our partial logits a tile ahead, take in its P
        auto send = [&](int n) {
          float x[32];
          partial(n, x);
          if constexpr (C::TILED) {
            __syncwarp();
            if (lane == 0) mbar_arrive(&a->sc_empty[n % C::SC_DEPTH]);
          }
          ok = wait_cluster(a, &a->x_free[n & 1], ((n >> 1) & 1) ^ 1, err) && ok;
          if (lane == 0) copy_wait_read();  // the tile before has left
          __syncwarp();
          float4* o = reinterpret_cast<float4*>(out_s + unit * 4096) + lane;
#pragma unroll
          for (int j = 0; j < 8; ++j) o[32 * j] = make_float4(x[4 * j], x[4 * j + 1], x[4 * j + 2], x[4 * j + 3]);
          fence_proxy_async_smem();
          __syncwarp();
          if (ok && lane == 0) {
            copy_remote(peer_x + (n & 1) * C::X_BYTES, out_s + unit * 4096, 4096, peer_xf + 8 * (n & 1));
            copy_commit();
          }
        };
        send(tile);
        for (int t = it.t0; t < it.t1; ++t, ++tile) {
          const int pb = tile % C::PB;
          if (t + 1 < it.t1) send(tile + 1);
          ok = wait_cluster(a, &a->p_msg[pb], (tile / C::PB) & 1, err) && ok;
          const float f = a->fac[pb][r64];
          uint32_t clear[2] = {a->clear[pb][0] | a->clear[pb][2], a->clear[pb][1] | a->clear[pb][3]};
          if (t > it.t0 && __any_sync(0xffffffffu, f != 1.f)) rescale(tile, f);
          if (!C::FP8 && (t + 1) * kKeys > it.ctx) {
            row_bar();
            // zero the value columns of the positions to clear (the tile's first product is done): a position
            // past the end always, another one only if it holds something that is not finite
            const uint32_t* mine = a->clear_own[tile & 1];
            clear[0] |= mine[0] | mine[2];
            clear[1] |= mine[1] | mine[3];
            const int st = (h * 2 + (quarter & 1)) * 32 + lane, key = st >> 1;  // a position, two of its four boxes
            if ((clear[key >> 5] >> (key & 31)) & 1) {
              for (int b = 2 * (st & 1); b < 2 * (st & 1) + 2; ++b) {
                uint8_t* line = tiles_s + (tile % C::STAGES) * kTile + b * kBox + key * 128;
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
                }
              }
            }
          }
          fence_proxy_async_smem();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) {
            if (warp == (rank ? 4 : 6)) mbar_arrive_expect_tx(&a->p_msg[pb], C::MSG_BYTES);  // for this buffer's next use
            mbar_arrive(&a->p_full[tile & 1]);
          }
        }
        ok = wait_cluster(a, &a->stat_full, items & 1, err) && ok;
        l = a->stat[r64];
        row_bar();
      }
      // ---- the item's outputs
      if (own) row_bar();
      if (!own && lane == 0 && warp == (rank ? 4 : 6)) mbar_arrive_expect_tx(&a->stat_full, 64 * 4);
      const bool live = row < nrows && (row_lo + row) / p.H < it.fresh;
      const float inv = live && l != 0.f ? 1.f / l : 0.f;
      ok = wait(a, &a->o_done, items & 1, err) && ok;
      tc_fence_after();
      const int v0 = 256 * rank + 128 * h;
#pragma unroll 1
      for (int c = 0; c < 128; c += 32) {
        float o[32];
        tmem_ld_sync(lane_base + kColO + 128 * h + c, o);
        if (row < nrows && it.slot >= 0) {
          float4* dst = pl.part_o + ((int64_t)it.slot * (kDv / 4) + (v0 + c) / 4) * kRows + row;
#pragma unroll
          for (int k = 0; k < 8; ++k) dst[k * kRows] = make_float4(o[4 * k], o[4 * k + 1], o[4 * k + 2], o[4 * k + 3]);
        } else if (row < nrows) {
          uint4* dst = reinterpret_cast<uint4*>(p.out + (at + row) * kDv + v0 + c);
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            uint32_t y[4];
#pragma unroll
            for (int q = 0; q < 4; ++q)
              y[q] = live ? pack_bf16(o[8 * k + 2 * q] * inv, o[8 * k + 2 * q + 1] * inv) : 0u;
            dst[k] = make_uint4(y[0], y[1], y[2], y[3]);
          }
        }
        __syncwarp();
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&a->o_free);
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
  const cuuint32_t box[3] = {64, (cuuint32_t)kKeys, 1};
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
