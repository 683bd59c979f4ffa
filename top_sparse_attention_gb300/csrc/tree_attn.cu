// Attention of drafted tokens over the latent cache (dsa_tree_attn): query node i of sequence s sees
// the n_ctx[s] cached positions and the drafted positions n_ctx[s] + j whose bit j is set in its row
// of the tree mask,
//   logit[p] = sm_scale * q[i, h] . Kv[p],  out[i, h] = sum_p softmax(logit)[p] * Kv[p, :512].
//
// A "row" is one head of one node; the rows of a sequence are consecutive in q and share its cache.
// A CTA takes NR rows (16, 32 or 64) and walks tiles of 64 positions, each loaded once and used for
// both products on the 5th-generation tensor cores:
//   * S[64 x 64] = Q K^T: A = the rows (M = 64), B = the tile's 64 positions (K-major), 36 steps of
//     K = 16, into tensor memory (for 128-column scales: one accumulator per scale tile, each added with
//     its positions' scales in fp32);
//   * one pass over the positions keeps a reference maximum m and a sum l per row,
//       l' = l 2^(m - m') + sum_p 2^(x_p - m'),   o' = o 2^(m - m') + sum_p 2^(x_p - m') v_p,
//     where m is moved only when a tile's maximum exceeds it by more than 2^8 (weights stay below 2^8,
//     fp32 sums and bf16 weights lose nothing by it), so o in tensor memory is rescaled rarely;
//   * O^T[512 x NR] += V^T P^T: A = the same tile in shared memory read MN-major (values along M, four
//     blocks of 128), B = P (bf16) [NR rows x 64 positions], 4 steps of K = 16 each.
// O transposed: 512 values x NR fp32 columns take 4 NR of the 512 tensor-memory columns, which leaves
// room for S beside it; with the rows along M they would take all of it.
//
// Weights are rounded to bf16 for the second product (as the bf16 cache is); sums, maxima, logits and
// outputs are fp32.  E4M3 rows are widened to bf16 exactly, and their scales are applied in fp32 to the
// logit and to the weight.
//
// Warp roles: producer (TMA, or for E4M3 eight warps that load, widen and store), MMA issuer, scale
// loader, query loader, four softmax warps (also the rescale and the epilogue).
//
// Work split: items (sequence, chunk of its tiles, row tile), in this order, so that CTAs that run
// together read the same positions and the cache comes from HBM once.  The lengths are on the device:
// every CTA evaluates the same cost model over them and picks the chunk length (plan_items); partial
// results are merged by tree_combine_kernel.
#include <string.h>

#include "dsa_internal.h"

namespace dsa {
namespace {

constexpr float kLn2 = 0.6931471805599453f;
constexpr int kDqk = 576, kDv = 512;
constexpr int kKeys = 64;                 // positions per tile
constexpr int kBox = kKeys * 128;         // one 64-column box of a tile: 64 rows x 128 bytes
constexpr int kSlot = 2 * kBox;           // 128 columns
constexpr int kSmemMax = 227 * 1024;
constexpr float kLazy = 8.f;              // log2 growth of a row's maximum that is left unscaled
constexpr int kItemsMax = 8;              // items per CTA in a split launch
constexpr int kItemsPerCta = 3;           // split launches are cut into at most this many items per CTA

enum { kBf16 = 0, kFp8Row = 1, kFp8Tile = 2 };

template <int NR, int FMT>
struct Cfg {
  static constexpr bool FP8 = FMT != kBf16;
  static constexpr int NSC = FMT == kFp8Tile ? 5 : FMT == kFp8Row ? 1 : 0;
  static constexpr int SACC = FMT == kFp8Tile ? 5 : 1;   // S accumulators per tile
  static constexpr int PC = FMT == kFp8Tile ? 4 : 1;     // copies of P (one per 128 values)
  static constexpr int THREADS = FP8 ? 512 : 256;
  static constexpr int Q_BOX = NR * 128, Q_BYTES = 9 * Q_BOX;
  static constexpr int P_BYTES = NR * 128;
  static constexpr int SC_DEPTH = 2;
  static constexpr int SC_BYTES = NSC * kKeys * 4;
  static constexpr int ROPE_SLOTS = 2;
  static constexpr int AUX = 1536;                        // barriers, row statistics, item list, flags
  static constexpr int FIXED = Q_BYTES + PC * P_BYTES + SC_DEPTH * SC_BYTES + ROPE_SLOTS * kBox + AUX + 1024;
  static constexpr int SLOTS_FIT = (kSmemMax - FIXED) / kSlot;
  static constexpr int SLOTS = SLOTS_FIT > 12 ? 12 : SLOTS_FIT;
  // with fewer than two tiles of slots the two products of neighbouring tiles take turns by halves
  static constexpr bool HALVES = SLOTS < 8;
  static constexpr int NSB = 4;                           // S buffers of 64 columns
  static constexpr int OFF_SLOT = Q_BYTES;
  static constexpr int OFF_ROPE = OFF_SLOT + SLOTS * kSlot;
  static constexpr int OFF_P = OFF_ROPE + ROPE_SLOTS * kBox;
  static constexpr int OFF_SC = OFF_P + PC * P_BYTES;
  static constexpr int OFF_AUX = OFF_SC + SC_DEPTH * SC_BYTES;
  static constexpr int SMEM = OFF_AUX + AUX + 1024;
  static constexpr int S_COL = 256;
  static_assert(SLOTS >= 6, "shared memory");
  static_assert(4 * NR <= S_COL, "tensor memory");
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
  int grid;
  int* head;               // [0]: chunk length in tiles (0: not split), [1 + s]: first item of sequence s
  float* part_o;           // [cap][NR][512]
  float2* part_ml;         // [cap][NR]
};

__device__ __forceinline__ void seq_facts(const TreeAttnParams& p, int seq, int& ctx, int& fresh, int& len) {
  ctx = min(max(p.n_ctx[seq], 0), p.L);
  fresh = p.n_new ? min(max(p.n_new[seq], 0), p.q_per_seq) : p.q_per_seq;
  len = min(ctx + fresh, p.L);
}

__device__ __forceinline__ int live_row_tiles(const TreeAttnParams& p, int fresh, int nr) {
  return (fresh * p.H + nr - 1) / nr;  // row tiles that hold a node below `fresh`
}

struct Aux {
  uint64_t full[12], empty[12], rfull[2], rempty[2];
  uint64_t s_full[4], s_empty[4];
  uint64_t p_full, p_empty, o_done, o_free, q_full, q_empty, sc_full[4], sc_empty[4], drain;
  uint32_t tmem;
  int abort;
  int n_items;
  float fac[64], linv[64];
  int kbad[kKeys];
  int tile_bad[4];
  int items[kItemsPerCta][8];
};
static_assert(sizeof(Aux) <= 1536, "Aux");

// A bounded wait that gives up at once when another wait of this CTA already has.
__device__ __forceinline__ bool wait(Aux* a, uint64_t* bar, uint32_t parity, int* err) {
  if (mbar_try_wait(bar, parity)) return true;
  if (*reinterpret_cast<volatile int*>(&a->abort)) return false;
  if (mbar_wait(bar, parity, err)) return true;
  *reinterpret_cast<volatile int*>(&a->abort) = 1;
  return false;
}

__device__ __forceinline__ void softmax_bar() { asm volatile("bar.sync 1, 128;" ::: "memory"); }
__device__ __forceinline__ bool softmax_any(bool pred) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.u32 p, %1, 0;\n\t"
      "bar.red.or.pred q, 2, 128, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"((uint32_t)pred)
      : "memory");
  return r != 0;
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
// box apart.  Adding bytes / 16 moves the start address.
constexpr uint32_t kDescHi = (1024u >> 4) | (1u << 14) | (2u << 29);
__device__ __forceinline__ uint32_t kmajor_lo(uint32_t saddr) { return ((saddr & 0x3FFFFu) >> 4) | (1u << 16); }
__device__ __forceinline__ uint32_t mnmajor_lo(uint32_t saddr) {
  return ((saddr & 0x3FFFFu) >> 4) | ((uint32_t)(kBox >> 4) << 16);
}

__device__ __forceinline__ void mma_f16_lo(uint32_t d, uint32_t a_lo, uint32_t b_lo, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 da, db;\n\t"
      "mov.b64 da, {%1, %5};\n\t"
      "mov.b64 db, {%2, %5};\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %3, p;\n\t}" ::"r"(d),
      "r"(a_lo), "r"(b_lo), "r"(idesc), "r"(acc), "r"(kDescHi)
      : "memory");
}

// 16 rows (tensor-memory lanes) x 64 fp32 columns: v[4 j + {0, 1}] is row lane / 4, columns
// 8 j + 2 (lane % 4) + {0, 1}; v[4 j + {2, 3}] the same columns of row lane / 4 + 8.
__device__ __forceinline__ void tmem_ld_16x64(uint32_t taddr, float (&v)[32]) {
  uint32_t r[32];
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, "
      "%12, %13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, "
      "%30, %31}, [%32];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]),
        "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]),
        "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr)
      : "memory");
#pragma unroll
  for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(r[i]);
}

__device__ __forceinline__ void tmem_st16(uint32_t taddr, const float (&v)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
      "%15, %16};" ::"r"(taddr),
      "r"(__float_as_uint(v[0])), "r"(__float_as_uint(v[1])), "r"(__float_as_uint(v[2])), "r"(__float_as_uint(v[3])),
      "r"(__float_as_uint(v[4])), "r"(__float_as_uint(v[5])), "r"(__float_as_uint(v[6])), "r"(__float_as_uint(v[7])),
      "r"(__float_as_uint(v[8])), "r"(__float_as_uint(v[9])), "r"(__float_as_uint(v[10])), "r"(__float_as_uint(v[11])),
      "r"(__float_as_uint(v[12])), "r"(__float_as_uint(v[13])), "r"(__float_as_uint(v[14])), "r"(__float_as_uint(v[15]))
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
// tiles plus the fill and drain of its pipeline, and for a split the merge.  Fills this CTA's list;
// CTA 0 leaves the plan for the merge.  Scratch: 3 n_seq + 160 ints of shared memory.
template <int NR>
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
    live[s] = live_row_tiles(p, fresh, NR);
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
    // this CTA's items: blockIdx.x, blockIdx.x + grid, ...
    const int mine = (int)blockIdx.x + tid * pl.grid;
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
    if (tid == 0) a->n_items = (int)blockIdx.x < run ? (run - (int)blockIdx.x + pl.grid - 1) / pl.grid : 0;
    if (blockIdx.x == 0) {
      if (tid == 0) pl.head[0] = ch;
      for (int s = tid; s < n; s += 32) pl.head[1 + s] = base[s];
    }
  }
  __syncthreads();
}

// Item i of this CTA: from the list of a split launch, or unit blockIdx.x + i * grid whole.
template <int NR>
__device__ __forceinline__ bool get_item(const TreeAttnParams& p, const TreePlan& pl, const Aux* a, int i, Item& it) {
  if (pl.cap) {
    if (i >= a->n_items) return false;
    memcpy(&it, a->items[i], sizeof(it));
    return true;
  }
  const int u = (int)blockIdx.x + i * pl.grid;
  if (u >= pl.units) return false;
  it.seq = u / pl.row_tiles;
  it.rt = u - it.seq * pl.row_tiles;
  seq_facts(p, it.seq, it.ctx, it.fresh, it.len);
  it.t0 = 0;
  it.t1 = it.rt < live_row_tiles(p, it.fresh, NR) ? (it.len + kKeys - 1) / kKeys : 0;
  it.slot = -1;
  return true;
}

template <int NR, int FMT>
__global__ void __launch_bounds__(Cfg<NR, FMT>::THREADS, 1)
    tree_attn_kernel(const __grid_constant__ CUtensorMap tm, const TreeAttnParams p, const TreePlan pl) {
  using C = Cfg<NR, FMT>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* q_s = smem;
  uint8_t* slots = smem + C::OFF_SLOT;
  uint8_t* rope_s = smem + C::OFF_ROPE;
  uint8_t* p_s = smem + C::OFF_P;
  float* sc_s = reinterpret_cast<float*>(smem + C::OFF_SC);
  Aux* a = reinterpret_cast<Aux*>(smem + C::OFF_AUX);
  const int tid = threadIdx.x, lane = tid & 31, warp = uniform(tid >> 5);
  int* err = p.err;

  if (warp == 0) {
    tmem_alloc(&a->tmem, 512);
    tmem_relinquish();
  }
  if (tid == 32) {
    const int fillers = C::FP8 ? 8 : 1;  // arrivals that fill a slot: converter warps, or the TMA's thread
    for (int i = 0; i < C::SLOTS; ++i) mbar_init(&a->full[i], fillers), mbar_init(&a->empty[i], 1);
    for (int i = 0; i < C::ROPE_SLOTS; ++i) mbar_init(&a->rfull[i], fillers), mbar_init(&a->rempty[i], 1);
    for (int i = 0; i < C::NSB; ++i) mbar_init(&a->s_full[i], 1), mbar_init(&a->s_empty[i], NR / 16);
    for (int i = 0; i < C::SC_DEPTH; ++i) mbar_init(&a->sc_full[i], 32), mbar_init(&a->sc_empty[i], NR / 16);
    mbar_init(&a->p_full, 128);
    mbar_init(&a->p_empty, 1);
    mbar_init(&a->o_done, 1);
    mbar_init(&a->o_free, 128);
    mbar_init(&a->q_full, 32);
    mbar_init(&a->q_empty, 1);
    mbar_init(&a->drain, 1);
    a->abort = 0;
    fence_mbar_init();
  }
  if (tid < kKeys) a->kbad[tid] = 0;
  if (pl.cap) plan_items<NR>(p, pl, a, reinterpret_cast<int*>(slots));
  fence_proxy_async_smem();  // the plan's scratch is a slot that the copies write
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = a->tmem;
  pdl_launch_dependents();

  Item it;
  if (warp == 0 && !C::FP8) {
    // ---- producer: tiles by TMA, 64-column boxes of 64 positions
    if (lane == 0) {
      prefetch_tmap(&tm);
      int sl = 0, ph = 0, rs = 0, rph = 0, tiles = 0;
      bool ok = true;
      for (int i = 0; ok && get_item<NR>(p, pl, a, i, it); ++i) {
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
          for (int b = 0; ok && b < 4; ++b) {
            ok = wait(a, &a->empty[sl], ph ^ 1, err);
            if (!ok) break;
            if (b == 0) a->tile_bad[tiles & 3] = bad;
            mbar_arrive_expect_tx(&a->full[sl], kSlot);
            uint8_t* dst = slots + sl * kSlot;
            tma_load_3d(dst, &tm, &a->full[sl], 128 * b, row, z);
            tma_load_3d(dst + kBox, &tm, &a->full[sl], 128 * b + 64, row, z);
            if (++sl == C::SLOTS) sl = 0, ph ^= 1;
          }
          ok = ok && wait(a, &a->rempty[rs], rph ^ 1, err);
          if (!ok) break;
          mbar_arrive_expect_tx(&a->rfull[rs], kBox);
          tma_load_3d(rope_s + rs * kBox, &tm, &a->rfull[rs], 512, row, z);
          if (++rs == C::ROPE_SLOTS) rs = 0, rph ^= 1;
        }
      }
      if (*reinterpret_cast<volatile int*>(&a->abort)) {
        // wind down: the copies in flight land before this CTA leaves
        for (int s = 0; s < C::SLOTS; ++s) mbar_wait(&a->full[s], s < sl ? ph : ph ^ 1, err);
        for (int s = 0; s < C::ROPE_SLOTS; ++s) mbar_wait(&a->rfull[s], s < rs ? rph : rph ^ 1, err);
      }
    }
    __syncwarp();
  } else if (warp == 1) {
    // ---- MMA issuer.  The warp stays converged and one elected lane issues; descriptors are sums of
    // 32-bit words (their upper words are one constant), so that issuing an instruction costs less than
    // the tensor cores take for it
    constexpr uint32_t idesc_qk = make_idesc(1, 1, 64, kKeys);
    constexpr uint32_t idesc_pv = make_idesc(1, 1, 128, NR) | (1u << 15);  // A (the tile) MN-major
    const uint32_t tm_base = (uint32_t)uniform((int)tmem);
    const uint32_t q_lo = kmajor_lo(smem_u32(q_s)), k_lo = kmajor_lo(smem_u32(slots)), r_lo = kmajor_lo(smem_u32(rope_s));
    const uint32_t v_lo = mnmajor_lo(smem_u32(slots)), p_lo = kmajor_lo(smem_u32(p_s));
    int qsl = 0, qph = 0, rs = 0, rph = 0;  // slots of the first product
    int psl = 0;                            // slots of the second
    uint32_t su = 0;                        // S buffers used
    int tile = 0, items = 0;
    bool ok = true;
    auto all = [&](uint64_t* bar, uint32_t parity) { ok = ok && __all_sync(0xffffffffu, wait(a, bar, parity, err)); };
    auto s_acquire = [&]() { all(&a->s_empty[su & (C::NSB - 1)], ((su / C::NSB) & 1) ^ 1); };
    // part h of a tile's first product: blocks 2 h, 2 h + 1 (and the rotary columns with the second)
    auto qk_part = [&](int h) {
#pragma unroll 1
      for (int b = 2 * h; b < 2 * h + 2; ++b) {
        if (C::SACC > 1 || b == 0) s_acquire();
        all(&a->full[qsl], qph);
        if (!ok) return;
        tc_fence_after();
        const uint32_t d = tm_base + C::S_COL + 64 * (su & (C::NSB - 1));
        const uint32_t A = q_lo + b * (2 * C::Q_BOX >> 4), B = k_lo + qsl * (kSlot >> 4);
        const uint32_t acc0 = C::SACC == 1 && b > 0;
        if (elect_one()) {
#pragma unroll
          for (int k = 0; k < 8; ++k)
            mma_f16_lo(d, A + ((k >> 2) * C::Q_BOX + 32 * (k & 3)) / 16, B + ((k >> 2) * kBox + 32 * (k & 3)) / 16, idesc_qk,
                       k ? 1u : acc0);
          if (C::SACC > 1) tc_commit(&a->s_full[su & (C::NSB - 1)]);
        }
        __syncwarp();
        if (C::SACC > 1) ++su;
        if (++qsl == C::SLOTS) qsl = 0, qph ^= 1;
      }
      if (h == 1) {
        if (C::SACC > 1) s_acquire();
        all(&a->rfull[rs], rph);
        if (!ok) return;
        tc_fence_after();
        const uint32_t d = tm_base + C::S_COL + 64 * (su & (C::NSB - 1));
        const uint32_t A = q_lo + (8 * C::Q_BOX >> 4), B = r_lo + rs * (kBox >> 4);
        if (elect_one()) {
#pragma unroll
          for (int k = 0; k < 4; ++k) mma_f16_lo(d, A + 2 * k, B + 2 * k, idesc_qk, k || C::SACC == 1 ? 1u : 0u);
          tc_commit(&a->s_full[su & (C::NSB - 1)]);
          tc_commit(&a->rempty[rs]);
        }
        __syncwarp();
        ++su;
        if (++rs == C::ROPE_SLOTS) rs = 0, rph ^= 1;
      }
    };
    auto pv_part = [&](int h, bool first) {
      const uint32_t acc0 = first ? 0u : 1u;
#pragma unroll 1
      for (int b = 2 * h; b < 2 * h + 2; ++b) {
        const uint32_t A = v_lo + psl * (kSlot >> 4), B = p_lo + (C::PC > 1 ? b : 0) * (C::P_BYTES >> 4);
        const uint32_t d = tm_base + NR * b;
        if (elect_one()) {
#pragma unroll
          for (int ks = 0; ks < 4; ++ks) mma_f16_lo(d, A + ks * (2048 >> 4), B + 2 * ks, idesc_pv, ks ? 1u : acc0);
          tc_commit(&a->empty[psl]);
        }
        __syncwarp();
        if (++psl == C::SLOTS) psl = 0;
      }
    };
    auto commit = [&](uint64_t* bar) {
      if (elect_one()) tc_commit(bar);
      __syncwarp();
    };
    for (int i = 0; ok && uniform(get_item<NR>(p, pl, a, i, it)); ++i) {
      const int t0 = uniform(it.t0), t1 = uniform(it.t1);
      if (t0 >= t1) continue;
      all(&a->q_full, items & 1);
      tc_fence_after();
      if (ok) qk_part(0);
      if (ok) qk_part(1);
      for (int t = t0; ok && t < t1; ++t, ++tile) {
        const bool next = t + 1 < t1, first = t == t0;
        if (next) {
          qk_part(0);
          if (ok && !C::HALVES) qk_part(1);
        } else {
          commit(&a->q_empty);
        }
        all(&a->p_full, tile & 1);
        if (first) all(&a->o_free, (items & 1) ^ 1);
        if (!ok) break;
        tc_fence_after();
        pv_part(0, first);
        if (next && C::HALVES) qk_part(1);
        if (!ok) break;
        pv_part(1, first);
        commit(&a->p_empty);
        if (!next) commit(&a->o_done);
      }
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
    for (int i = 0; ok && get_item<NR>(p, pl, a, i, it); ++i) {
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
        if (lane == 0) a->tile_bad[tiles & 3] = bad;
        __syncwarp();
        mbar_arrive(&a->sc_full[d]);
        if (bad && lane == 0) record_error(err, DSA_DEVERR_INDEX_RANGE);
      }
    }
  } else if (warp == 3) {
    // ---- queries: the item's NR rows into 128-byte-swizzled K-major boxes (rows past the end: zeros)
    int items = 0;
    bool ok = true;
    const int rows = p.q_per_seq * p.H;
    for (int i = 0; ok && get_item<NR>(p, pl, a, i, it); ++i) {
      if (it.t0 >= it.t1) continue;
      ok = __all_sync(0xffffffffu, wait(a, &a->q_empty, (items & 1) ^ 1, err));
      if (!ok) break;
      const int n = min(NR, rows - it.rt * NR);
      const __nv_bfloat16* q = p.q + ((int64_t)it.seq * rows + it.rt * NR) * kDqk;
#pragma unroll 4
      for (int k = lane; k < NR * 72; k += 32) {
        const int r = k / 72, c = k - r * 72;
        cp_async16(q_s + (c >> 3) * C::Q_BOX + r * 128 + (((c & 7) ^ (r & 7)) << 4), q + (int64_t)(r < n ? r : 0) * kDqk + 8 * c,
                   r < n);
      }
      cp_async_commit();
      cp_async_wait<0>();
      fence_proxy_async_smem();
      mbar_arrive(&a->q_full);
      ++items;
    }
  } else if (warp >= 8) {
    // ---- converters (E4M3): thread = position ct / 4 and, of every 64 columns, codes 16 (ct % 4) ...
    const int ct = tid - 256, key = ct >> 2, c4 = ct & 3;
    int sl = 0, ph = 0, rs = 0, rph = 0;
    bool ok = true;
    uint4 raw[9];
    auto row_ptr = [&](const Item& x, int t) -> const uint8_t* {
      const int pos = t * kKeys + key;
      if (t >= x.t1 || pos >= x.len) return nullptr;
      const int64_t row = tree_row(p, x.seq, pos);
      if (row < 0) return nullptr;
      return p.kv + (p.pages.table ? 0 : (int64_t)x.seq * p.kv_seq_stride) + row * p.kv_row_stride + 16 * c4;
    };
    auto fetch = [&](const uint8_t* r, int j) {
      raw[j] = r ? __ldg(reinterpret_cast<const uint4*>(r + 64 * j)) : make_uint4(0u, 0u, 0u, 0u);
    };
    auto store = [&](uint8_t* box, const uint4& v) {
      uint8_t* d = box + key * 128;
      const int c0 = 2 * c4, x = key & 7;
      *reinterpret_cast<uint4*>(d + ((c0 ^ x) << 4)) =
          make_uint4(e4m3x2_to_bf16x2(v.x, 0x1404), e4m3x2_to_bf16x2(v.x, 0x3424), e4m3x2_to_bf16x2(v.y, 0x1404),
                     e4m3x2_to_bf16x2(v.y, 0x3424));
      *reinterpret_cast<uint4*>(d + (((c0 + 1) ^ x) << 4)) =
          make_uint4(e4m3x2_to_bf16x2(v.z, 0x1404), e4m3x2_to_bf16x2(v.z, 0x3424), e4m3x2_to_bf16x2(v.w, 0x1404),
                     e4m3x2_to_bf16x2(v.w, 0x3424));
    };
    for (int i = 0; ok && get_item<NR>(p, pl, a, i, it); ++i) {
      const uint8_t* r = row_ptr(it, it.t0);
#pragma unroll
      for (int j = 0; j < 9; ++j) fetch(r, j);
      for (int t = it.t0; ok && t < it.t1; ++t) {
        r = row_ptr(it, t + 1);
#pragma unroll
        for (int b = 0; b < 4; ++b) {
          ok = ok && __all_sync(0xffffffffu, wait(a, &a->empty[sl], ph ^ 1, err));
          if (ok) {
            uint8_t* dst = slots + sl * kSlot;
            store(dst, raw[2 * b]);
            store(dst + kBox, raw[2 * b + 1]);
            fetch(r, 2 * b);
            fetch(r, 2 * b + 1);
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(&a->full[sl]);
            if (++sl == C::SLOTS) sl = 0, ph ^= 1;
          }
        }
        ok = ok && __all_sync(0xffffffffu, wait(a, &a->rempty[rs], rph ^ 1, err));
        if (!ok) break;
        store(rope_s + rs * kBox, raw[8]);
        fetch(r, 8);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&a->rfull[rs]);
        if (++rs == C::ROPE_SLOTS) rs = 0, rph ^= 1;
      }
    }
  } else if (warp >= 4 && warp < 8) {
    // ---- softmax, rescale, epilogue.  Softmax: warp w < NR / 16 has rows 16 w ..., a thread the rows
    // r0 and r0 + 8 and 16 of the 64 positions; rescale and epilogue: thread = value 32 w + lane of a block
    const int w = warp - 4, st = tid - 128;
    const bool mine = w < NR / 16;
    const int r0 = 16 * w + (lane >> 2), cq = lane & 3;
    const uint32_t lane_base = tmem + ((uint32_t)(32 * w) << 16);
    uint32_t su = 0;
    int tile = 0, items = 0;
    bool ok = true;
    const int rows = p.q_per_seq * p.H;
    for (int i = 0; get_item<NR>(p, pl, a, i, it); ++i) {
      const int row_lo = it.rt * NR;
      const int64_t at = (int64_t)it.seq * rows + row_lo;  // the item's first row in out and lse
      const int nrows = min(NR, rows - row_lo);
      if (it.t0 >= it.t1) {  // nothing to see: padding nodes, or an empty sequence
        for (int k = st; k < nrows * (kDv / 8); k += 128)
          reinterpret_cast<uint4*>(p.out + at * kDv)[k] = make_uint4(0u, 0u, 0u, 0u);
        if (p.lse && st < nrows) p.lse[at + st] = -INFINITY;
        continue;
      }
      const int node[2] = {min((row_lo + r0) / p.H, p.q_per_seq - 1), min((row_lo + r0 + 8) / p.H, p.q_per_seq - 1)};
      float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
      bool dead = false;  // (the same for all four warps, unlike ok)
      for (int t = it.t0; t < it.t1; ++t, ++tile) {
        float x[32];
        const bool tail = (t + 1) * kKeys > it.ctx;
        bool hidden_bad = false;
        if (mine) {
          const float* sc = sc_s + (tile % C::SC_DEPTH) * kKeys * C::NSC;
          if constexpr (FMT == kFp8Tile) {
            ok = ok && wait(a, &a->sc_full[tile % C::SC_DEPTH], (tile / C::SC_DEPTH) & 1, err);
#pragma unroll
            for (int k = 0; k < 32; ++k) x[k] = 0.f;
            for (int g = 0; g < 5; ++g, ++su) {
              ok = ok && wait(a, &a->s_full[su & (C::NSB - 1)], (su / C::NSB) & 1, err);
              tc_fence_after();
              float s[32];
              tmem_ld_16x64(lane_base + C::S_COL + 64 * (su & (C::NSB - 1)), s);
              tc_fence_before();
              __syncwarp();
              if (lane == 0) mbar_arrive(&a->s_empty[su & (C::NSB - 1)]);
#pragma unroll
              for (int j = 0; j < 8; ++j) {
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                  const float f = sc[(8 * j + 2 * cq + e) * 5 + g];
                  x[4 * j + e] = fmaf(f, s[4 * j + e], x[4 * j + e]);
                  x[4 * j + 2 + e] = fmaf(f, s[4 * j + 2 + e], x[4 * j + 2 + e]);
                }
              }
            }
#pragma unroll
            for (int k = 0; k < 32; ++k) x[k] *= p.scale_log2;
          } else {
            ok = ok && wait(a, &a->s_full[su & (C::NSB - 1)], (su / C::NSB) & 1, err);
            tc_fence_after();
            tmem_ld_16x64(lane_base + C::S_COL + 64 * (su & (C::NSB - 1)), x);
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&a->s_empty[su & (C::NSB - 1)]);
            ++su;
            if constexpr (FMT == kFp8Row) {
              ok = ok && wait(a, &a->sc_full[tile % C::SC_DEPTH], (tile / C::SC_DEPTH) & 1, err);
#pragma unroll
              for (int j = 0; j < 8; ++j) {
                const float2 f = *reinterpret_cast<const float2*>(sc + 8 * j + 2 * cq);
                const float f0 = f.x * p.scale_log2, f1 = f.y * p.scale_log2;
                x[4 * j] *= f0, x[4 * j + 1] *= f1, x[4 * j + 2] *= f0, x[4 * j + 3] *= f1;
              }
            } else {
#pragma unroll
              for (int k = 0; k < 32; ++k) x[k] *= p.scale_log2;
            }
          }
          const bool bad = p.pages.table && a->tile_bad[tile & 3];
          if (tail || bad) {
#pragma unroll
            for (int hh = 0; hh < 2; ++hh) {
              const uint64_t see = bad ? 0ull : seen_bits(p, it, node[hh], t);
#pragma unroll
              for (int j = 0; j < 8; ++j) {
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                  const int k = 8 * j + 2 * cq + e;
                  float& v = x[4 * j + 2 * hh + e];
                  if (!((see >> k) & 1)) {
                    // a hidden row that may hold infinities or NaN (its logit would not be finite, or it lies
                    // past the end): its values are cleared below, so that 0 * value is 0
                    if (!C::FP8 && (!(fabsf(v) < INFINITY) || t * kKeys + k >= it.len)) {
                      a->kbad[k] = 1;
                      hidden_bad = true;
                    }
                    v = -INFINITY;
                  }
                }
              }
            }
          }
        }
        if (!C::FP8 && tail) {
          if (softmax_any(hidden_bad)) {
            // zero the cleared positions' value columns in the tile (its first product is done): a position
            // past the end always, another one only if it holds something that is not finite
            for (int k = st >> 3; k < kKeys; k += 16) {
              const int b = st & 7;  // box of 64 columns
              uint8_t* line = slots + ((4 * tile + (b >> 1)) % C::SLOTS) * kSlot + (b & 1) * kBox + k * 128;
              if (a->kbad[k]) {
                bool clear = t * kKeys + k >= it.len;
                if (!clear) {
#pragma unroll
                  for (int c = 0; c < 8; ++c) {
                    const uint4 u = *reinterpret_cast<const uint4*>(line + 16 * c);
                    const uint32_t ws[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
                    for (int q = 0; q < 4; ++q)
                      clear |= (ws[q] & 0x7F80u) == 0x7F80u || (ws[q] & 0x7F800000u) == 0x7F800000u;
                  }
                }
                if (clear) {
#pragma unroll
                  for (int c = 0; c < 8; ++c) *reinterpret_cast<uint4*>(line + 16 * c) = make_uint4(0u, 0u, 0u, 0u);
                }
              }
            }
            softmax_bar();
            if (st < kKeys) a->kbad[st] = 0;
          }
        }
        // the tile's maxima; the reference moves when one exceeds it by more than kLazy
        bool need = false;
        float mx[2] = {-INFINITY, -INFINITY};
        if (mine) {
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            mx[0] = fmaxf(mx[0], fmaxf(x[4 * j], x[4 * j + 1]));
            mx[1] = fmaxf(mx[1], fmaxf(x[4 * j + 2], x[4 * j + 3]));
          }
#pragma unroll
          for (int hh = 0; hh < 2; ++hh) {
            mx[hh] = fmaxf(mx[hh], __shfl_xor_sync(0xffffffffu, mx[hh], 1));
            mx[hh] = fmaxf(mx[hh], __shfl_xor_sync(0xffffffffu, mx[hh], 2));
            if (m[hh] == -INFINITY) m[hh] = mx[hh];  // nothing summed yet
            need |= mx[hh] > m[hh] + kLazy;
          }
        }
        const bool any = softmax_any(need || !ok);
        if (any) {
          if (softmax_any(!ok)) {
            dead = true;
            break;
          }
          if (mine) {
#pragma unroll
            for (int hh = 0; hh < 2; ++hh) {
              float f = 1.f;
              if (mx[hh] > m[hh] + kLazy) {
                f = ex2(m[hh] - mx[hh]);
                m[hh] = mx[hh];
                l[hh] *= f;
              }
              if (cq == 0) a->fac[r0 + 8 * hh] = f;
            }
          }
        }
        // the previous tile's second product is done: its P may be overwritten, O may be rescaled
        ok = wait(a, &a->p_empty, (tile & 1) ^ 1, err);
        if (any) {
          softmax_bar();
          tc_fence_after();
          if (t > it.t0) {
#pragma unroll 1
            for (int c = 0; c < 4 * NR; c += 16) {
              float o[16];
              tmem_ld_sync(lane_base + c, o);
              const float* f = a->fac + (c & (NR - 1));
#pragma unroll
              for (int k = 0; k < 16; ++k) o[k] *= f[k];
              tmem_st16(lane_base + c, o);
            }
            tmem_wait_st();
          }
          tc_fence_before();
        }
        if (mine) {
          const float mu[2] = {m[0] == -INFINITY ? 0.f : m[0], m[1] == -INFINITY ? 0.f : m[1]};
#pragma unroll
          for (int j = 0; j < 8; ++j) {
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              x[4 * j + e] = ex2(x[4 * j + e] - mu[0]);
              x[4 * j + 2 + e] = ex2(x[4 * j + 2 + e] - mu[1]);
              l[0] += x[4 * j + e];
              l[1] += x[4 * j + 2 + e];
            }
          }
          const float* sc = sc_s + (tile % C::SC_DEPTH) * kKeys * C::NSC;
#pragma unroll
          for (int pc = 0; pc < C::PC; ++pc) {
            uint8_t* d = p_s + pc * C::P_BYTES + r0 * 128 + cq * 4;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              float f0 = 1.f, f1 = 1.f;
              if constexpr (C::FP8) {
                f0 = sc[(8 * j + 2 * cq) * C::NSC + pc];
                f1 = sc[(8 * j + 2 * cq + 1) * C::NSC + pc];
              }
              // a hidden position's weight is 0 whatever its scale holds
              auto w8 = [](float pr, float f) { return C::FP8 ? (pr == 0.f ? 0.f : pr * f) : pr; };
              const int sw = (j ^ (r0 & 7)) << 4;  // (r0 + 8) % 8 == r0 % 8
              *reinterpret_cast<uint32_t*>(d + sw) = pack_bf16(w8(x[4 * j], f0), w8(x[4 * j + 1], f1));
              *reinterpret_cast<uint32_t*>(d + 1024 + sw) = pack_bf16(w8(x[4 * j + 2], f0), w8(x[4 * j + 3], f1));
            }
          }
          if constexpr (C::FP8) {
            __syncwarp();
            if (lane == 0) mbar_arrive(&a->sc_empty[tile % C::SC_DEPTH]);
          }
        }
        fence_proxy_async_smem();
        mbar_arrive(&a->p_full);
      }
      if (dead) break;
      // ---- the item's sums, then its outputs
      if (mine) {
#pragma unroll
        for (int hh = 0; hh < 2; ++hh) {
          l[hh] += __shfl_xor_sync(0xffffffffu, l[hh], 1);
          l[hh] += __shfl_xor_sync(0xffffffffu, l[hh], 2);
          const int r = r0 + 8 * hh;
          const bool live = r < nrows && (row_lo + r) / p.H < it.fresh;
          if (cq == 0) {
            if (it.slot >= 0) {
              pl.part_ml[(int64_t)it.slot * NR + r] = make_float2(m[hh], l[hh]);
            } else {
              a->linv[r] = live ? (l[hh] == 0.f ? 0.f : 1.f / l[hh]) : 0.f;
              if (p.lse && r < nrows) p.lse[at + r] = !live || l[hh] == 0.f ? -INFINITY : (m[hh] + log2f(l[hh])) * kLn2;
            }
          }
        }
      }
      softmax_bar();
      ok = ok && wait(a, &a->o_done, items & 1, err);
      if (softmax_any(!ok)) break;
      tc_fence_after();
      const int live_rows = min(nrows, it.fresh * p.H - row_lo);  // the others are written as zeros
#pragma unroll 1
      for (int c = 0; c < 4 * NR; c += 16) {
        float o[16];
        tmem_ld_sync(lane_base + c, o);
        const int v = 128 * (c / NR) + 32 * w + lane, rr = c & (NR - 1);
        if (it.slot >= 0) {
          float* dst = pl.part_o + ((int64_t)it.slot * NR + rr) * kDv + v;
#pragma unroll
          for (int k = 0; k < 16; ++k)
            if (rr + k < nrows) dst[k * kDv] = o[k];
        } else {
          // two rows at a time: even lanes write the first one's pair of values, odd lanes the second's
          const bool odd = lane & 1;
#pragma unroll
          for (int k = 0; k < 16; k += 2) {
            const float y0 = rr + k < live_rows ? o[k] * a->linv[rr + k] : 0.f;
            const float y1 = rr + k + 1 < live_rows ? o[k + 1] * a->linv[rr + k + 1] : 0.f;
            const float got = __shfl_xor_sync(0xffffffffu, odd ? y0 : y1, 1);
            const int r = rr + k + odd;
            if (r < nrows)
              *reinterpret_cast<uint32_t*>(p.out + (at + r) * kDv + (v & ~1)) = odd ? pack_bf16(got, y1) : pack_bf16(y0, got);
          }
        }
      }
      tc_fence_before();
      mbar_arrive(&a->o_free);
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

// Merges the chunks of each split row: out = sum_j 2^(m_j - M) o_j / sum_j 2^(m_j - M) l_j.  One CTA per
// row, four values per thread, eight chunks' loads in flight.
template <int NR>
__global__ void __launch_bounds__(128) tree_combine_kernel(const TreeAttnParams p, const TreePlan pl) {
  pdl_wait();
  const int rows = p.q_per_seq * p.H;
  const int seq = blockIdx.y, row = blockIdx.x;
  int ctx, fresh, len;
  seq_facts(p, seq, ctx, fresh, len);
  const int live = live_row_tiles(p, fresh, NR);
  const int rt = row / NR, r = row - rt * NR;
  const int ch = pl.head[0], nt = (len + kKeys - 1) / kKeys;
  int chunks = nt ? (nt + ch - 1) / ch : 1;
  if (rt >= live || chunks == 1) return;  // written by the attention kernel
  if (row / p.H >= fresh) chunks = 0;     // a padding node beside live ones: zeros
  const int item0 = pl.head[1 + seq] + rt;
  const int c = 4 * threadIdx.x;
  float M = -INFINITY, l = 0.f;
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
  constexpr int B = 8;
  for (int j0 = 0; j0 < chunks; j0 += B) {
    float2 ml[B];
    float4 v[B];
#pragma unroll
    for (int k = 0; k < B; ++k) {
      const int64_t s = (int64_t)(item0 + (j0 + k) * live) * NR + r;
      const bool in = j0 + k < chunks;
      ml[k] = in ? pl.part_ml[s] : make_float2(-INFINITY, 0.f);
      v[k] = in ? *reinterpret_cast<const float4*>(pl.part_o + s * kDv + c) : make_float4(0.f, 0.f, 0.f, 0.f);
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
  *reinterpret_cast<uint2*>(p.out + at * kDv + c) =
      make_uint2(pack_bf16(o.x * inv, o.y * inv), pack_bf16(o.z * inv, o.w * inv));
  if (p.lse && threadIdx.x == 0) p.lse[at] = l == 0.f ? -INFINITY : (M + log2f(l)) * kLn2;
}

__global__ void tree_nothing_kernel(const TreeAttnParams p, int64_t rows) {
  const int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
  if (i < rows * (kDv / 8)) reinterpret_cast<uint4*>(p.out)[i] = make_uint4(0u, 0u, 0u, 0u);
  if (p.lse && i < rows) p.lse[i] = -INFINITY;
}

int rows_per_cta(const TreeAttnParams& p) {
  const int rows = p.q_per_seq * p.H;
  return rows <= 16 ? 16 : rows <= 32 ? 32 : 64;
}

// A launch with many units needs no split: its rounds of the grid are full enough.
TreePlan plan_of(const TreeAttnParams& p, int sms) {
  TreePlan pl = {};
  const int nr = rows_per_cta(p);
  pl.row_tiles = (p.q_per_seq * p.H + nr - 1) / nr;
  pl.units = p.n_seq * pl.row_tiles;
  pl.cap = pl.units <= kItemsPerCta * sms ? kItemsPerCta * sms : 0;
  pl.grid = pl.cap ? sms : (pl.units < sms ? pl.units : sms);
  return pl;
}

size_t head_bytes(const TreeAttnParams& p) { return align_up((size_t)(1 + p.n_seq) * sizeof(int), 256); }

constexpr int kSms = 152;

template <int NR, int FMT>
cudaError_t launch_cfg(const TreeAttnParams& p, TreePlan pl, void* ws, cudaStream_t stream) {
  using C = Cfg<NR, FMT>;
  CUtensorMap tm;
  memset(&tm, 0, sizeof(tm));
  if (!C::FP8) {
    const bool paged = p.pages.table != nullptr;
    const cuuint64_t n = paged ? (cuuint64_t)p.pages.num_blocks * p.pages.block_size : (cuuint64_t)p.L;
    const cuuint64_t dims[3] = {(cuuint64_t)kDqk, n, paged ? 1 : (cuuint64_t)p.n_seq};
    const cuuint64_t strides[2] = {(cuuint64_t)p.kv_row_stride,
                                   paged || p.n_seq == 1 ? n * (cuuint64_t)p.kv_row_stride : (cuuint64_t)p.kv_seq_stride};
    const cuuint32_t box[3] = {64, (cuuint32_t)kKeys, 1};
    if (encode_tensor_map(&tm, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<uint8_t*>(p.kv), dims, strides, box,
                          CU_TENSOR_MAP_SWIZZLE_128B) != CUDA_SUCCESS)
      return cudaErrorInvalidValue;
  }
  if (pl.cap) {
    uint8_t* w = reinterpret_cast<uint8_t*>(ws);
    pl.head = reinterpret_cast<int*>(w);
    w += head_bytes(p);
    pl.part_ml = reinterpret_cast<float2*>(w);
    w += align_up((size_t)pl.cap * NR * sizeof(float2), 256);
    pl.part_o = reinterpret_cast<float*>(w);
  }
  auto kern = tree_attn_kernel<NR, FMT>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
  if (e != cudaSuccess) return e;
  e = launch_kernel(kern, dim3(pl.grid), dim3(C::THREADS), C::SMEM, stream, false, tm, p, pl);
  if (e != cudaSuccess || !pl.cap) return e;
  return launch_kernel(tree_combine_kernel<NR>, dim3(p.q_per_seq * p.H, p.n_seq), dim3(128), 0, stream, true, p, pl);
}

template <int NR>
cudaError_t launch_nr(const TreeAttnParams& p, const TreePlan& pl, void* ws, cudaStream_t stream) {
  if (!p.kv_fp8) return launch_cfg<NR, kBf16>(p, pl, ws, stream);
  return p.nsc == 1 ? launch_cfg<NR, kFp8Row>(p, pl, ws, stream) : launch_cfg<NR, kFp8Tile>(p, pl, ws, stream);
}

}  // namespace

size_t tree_attn_ws_bytes(const TreeAttnParams& p) {
  const TreePlan pl = plan_of(p, kSms);
  if (!pl.cap || p.L == 0) return 0;
  const int nr = rows_per_cta(p);
  return head_bytes(p) + align_up((size_t)pl.cap * nr * sizeof(float2), 256) + (size_t)pl.cap * nr * kDv * sizeof(float);
}

cudaError_t launch_tree_attn(const TreeAttnParams& p, void* ws, cudaStream_t stream) {
  const int64_t rows = (int64_t)p.n_seq * p.q_per_seq * p.H;
  if (p.L == 0) {
    const int64_t n = rows * (kDv / 8);
    return launch_kernel(tree_nothing_kernel, dim3((unsigned)((n + 255) / 256)), dim3(256), 0, stream, false, p, rows);
  }
  const TreePlan pl = plan_of(p, kSms);
  switch (rows_per_cta(p)) {
    case 16: return launch_nr<16>(p, pl, ws, stream);
    case 32: return launch_nr<32>(p, pl, ws, stream);
    default: return launch_nr<64>(p, pl, ws, stream);
  }
}

}  // namespace dsa
