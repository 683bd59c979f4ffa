// Cached latent rows expanded to every head's key and value (dsa_latent_expand):
//   out[r, h, j] = sum_c row[r, c] * w[h, j, c]   (c < 512, j < 256: 128 key columns, then 128 value columns)
// for the packed positions r of ragged sequences, whose rows are found through kv_start (and the block table); the rows' 64
// rotary columns, which all heads share, are copied beside them.
//
// A matrix product [rows x 512] x [512 x 256 H].  A pair of CTAs (cta_group::2) takes 256 rows: each CTA gathers 128 of
// them once, for all of K, into shared memory as bf16 (eight swizzled boxes of 64 columns, 128 KB), and both walk the
// heads' columns in units of NT: per unit each CTA loads half of the weights' rows by TMA (the tensor cores read the
// other half from the partner), so that 256 rows share one pass over W; a CTA alone would take twice the bytes from L2
// per product, more than L2 gives.  Accumulators of two units in tensor memory: one is read out while the next is summed.
//
// Formats: E4M3 codes are widened to bf16 exactly; a scale per row multiplies the fp32 sums, a scale per 128 columns the
// codes, whose product is rounded to bf16, 2^-8 of it at most, as much as a bf16 cache has lost: the scales differ along K, so
// that exact ones would want a sum of its own for each of the four tiles, and tensor memory holds two sums per row.  An output over
// normal values is 1.4 times as far from 64 bits as one of unrounded products (0.0024 against 0.0017 of the output's size).
//
// Measured (36864 rows x 16 heads: 155 GFLOP, 302 MB written): E4M3 codes with row scales 123 us, 1260 TFLOP/s and 2.5 TB/s (tile
// scales 120, bf16 128; 36900 rows, whose last tile is partial, 125).  Without the
// output's copies the same kernel takes 95, without reading the sums out 87 (1780 TFLOP/s); writing alone costs as much (torch
// fills 316 MB in 81 us), and the two do not overlap as they should: the products wait for the read-out, which waits for its
// boxes to leave.  Tried: stores of 32 bytes straight from registers 129 (140 with eight warps), whole lines by plain stores 128,
// eight warps with a box each 126, boxes of consecutive lines (another layout) 117.  364 rows of short prompts: 11.6, latency.
//
// Warp roles: 0 weights (TMA), 1 MMA issuer (the even CTA's), 4 to 11 gather rows, 12 to 15 read out, scale and store.
#include <limits.h>
#include <string.h>

#include "tc_common.cuh"

namespace dsa {
namespace {

constexpr int kLat = 512, kRope = 64, kOut = 256;  // latent and rotary columns of a row, expanded columns of a head
constexpr int kRowsCta = 128, kBoxes = kLat / 64, kBoxA = kRowsCta * 128;
constexpr int kThreads = 512, kLoaders = 256;
constexpr int kPairs = 76;
enum { kBf16 = 0, kFp8Row = 1, kFp8Tile = 2 };

struct ExpandParams {
  const uint8_t* kv;
  const float* kv_scale;   // per row, or five per row, or null (bf16)
  int64_t kv_row_stride, kv_seq_stride;
  int L;                   // positions per sequence
  const int32_t* kv_start; // [n_seq + 1]
  int n_seq, rows, H;
  __nv_bfloat16* out;      // [rows, H, 256]
  __nv_bfloat16* rope_out; // [rows, 64] or null
  PagedCache pages;        // table null: contiguous per sequence
  int* err;                // device error word
};

struct Aux {
  uint64_t b_full[8], b_empty[8], a_full[kBoxes], a_empty, acc_full[2], acc_empty[2], drain;
  uint32_t tmem;
  int abort;
  int64_t src[kRowsCta];  // source row of each row of the tile, -1: none
};

template <int NT>
struct Cfg {
  static constexpr int BOX_B = NT / 2 * 128;       // half of a unit's weight rows, 64 columns
  static constexpr int STAGES = NT == 256 ? 4 : 8;
  static constexpr int OFF_B = kBoxes * kBoxA;
  static constexpr int OFF_ST = OFF_B + STAGES * BOX_B;  // two boxes of 32 rows x 64 columns per storing warp
  static constexpr int OFF_AUX = OFF_ST + 4 * 2 * 4096;
  static constexpr int SMEM = OFF_AUX + (int)sizeof(Aux) + 1024;
  static_assert(SMEM <= 227 * 1024, "shared memory");
};

// ---- waits.  Bounded; once one has run out the CTA's others return at once and the roles leave (as in tc_common.cuh).
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
__device__ __noinline__ bool wait_pair_slow(Aux* a, uint64_t* bar, uint32_t parity, int* err) {
  const unsigned long long t0 = globaltimer_ns();
  for (uint32_t i = 0;; ++i) {
    if (try_wait_cluster(bar, parity)) return true;
    if ((i & 15u) != 15u) continue;
    if (*reinterpret_cast<volatile int*>(&a->abort)) return false;
    if (globaltimer_ns() - t0 > kWaitLimitNs) {
      record_error(err, DSA_DEVERR_WAIT_TIMEOUT);
      *reinterpret_cast<volatile int*>(&a->abort) = 1;
      return false;
    }
  }
}
__device__ __forceinline__ bool wait_pair(Aux* a, uint64_t* bar, uint32_t parity, int* err) {
  return try_wait_cluster(bar, parity) || wait_pair_slow(a, bar, parity, err);
}

// The eight loading warps' barrier, and whether all of them are still well (so that all leave together).
__device__ __forceinline__ bool loaders_ok(bool ok) {
  uint32_t all;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.b32 p, %1, 0;\n\t"
      "barrier.cta.red.and.pred q, 1, 256, p;\n\t"
      "selp.b32 %0, 1, 0, q;\n\t}"
      : "=r"(all)
      : "r"((uint32_t)ok)
      : "memory");
  return all != 0;
}

// Arrives on the even CTA's barrier of this address.
__device__ __forceinline__ void arrive_even(uint64_t* bar) {
  asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(dsmem_addr(bar, 0)) : "memory");
}
// All MMAs issued so far: arrive on both CTAs' barriers of this address.
__device__ __forceinline__ void commit_both(uint64_t* bar) {
  asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(smem_u32(bar)),
               "h"((uint16_t)3)
               : "memory");
}
__device__ __forceinline__ void mma2(uint32_t d, uint64_t adesc, uint64_t bdesc, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(acc)
      : "memory");
}
// A box of weights into this CTA, counted on the even CTA's barrier.
__device__ __forceinline__ void tma_load_pair(void* dst, const CUtensorMap* tm, uint32_t bar_even, int x, int y) {
  asm volatile(
      "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(
          smem_u32(dst)),
      "l"(tm), "r"(x), "r"(y), "r"(bar_even)
      : "memory");
}

// The source row of packed row r: in the pool when paged, else seq * L + position; -1 for a row of no sequence.  A
// position or a block outside the cache is recorded; its row reads as zeros (`there` false).
__device__ __forceinline__ int64_t source_row(const ExpandParams& p, int r, bool& there) {
  there = false;
  if (r >= min(p.rows, p.kv_start[p.n_seq]) || r < p.kv_start[0]) return -1;
  int lo = 0, hi = p.n_seq - 1;  // the last sequence that starts at or before r
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (p.kv_start[mid] <= r) lo = mid;
    else hi = mid - 1;
  }
  const int pos = r - p.kv_start[lo];
  if (pos < 0 || pos >= p.L) {
    record_error(p.err, DSA_DEVERR_INDEX_RANGE);
    return 0;
  }
  if (!p.pages.table) {
    there = true;
    return (int64_t)lo * p.L + pos;
  }
  const int32_t b = p.pages.table[(int64_t)lo * p.pages.max_blocks + pos / p.pages.block_size];
  if ((unsigned)b >= (unsigned)p.pages.num_blocks) {
    record_error(p.err, DSA_DEVERR_INDEX_RANGE);
    return 0;
  }
  there = true;
  return (int64_t)b * p.pages.block_size + pos % p.pages.block_size;
}
__device__ __forceinline__ const uint8_t* row_at(const ExpandParams& p, int64_t row) {
  if (p.pages.table) return p.kv + row * p.kv_row_stride;
  const int64_t seq = row / p.L;
  return p.kv + seq * p.kv_seq_stride + (row - seq * p.L) * p.kv_row_stride;
}

// A load that stays where it is written (an ordinary one sinks behind the wait that it is to be in flight during).
__device__ __forceinline__ uint4 load_now(const uint8_t* p) {
  uint4 v;
  asm volatile("ld.global.nc.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
  return v;
}

__device__ __forceinline__ uint32_t bf16x2(float lo, float hi) {
  const __nv_bfloat162 b = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&b);
}
__device__ __forceinline__ float lo_bf16(uint32_t x) { return __uint_as_float(x << 16); }
__device__ __forceinline__ float hi_bf16(uint32_t x) { return __uint_as_float(x & 0xFFFF0000u); }
// Four codes as bf16, times s.
__device__ __forceinline__ uint2 widen4(uint32_t x) { return make_uint2(e4m3x2_to_bf16x2(x, 0x1404), e4m3x2_to_bf16x2(x, 0x3424)); }
__device__ __forceinline__ uint32_t scaled(uint32_t x, float s) { return bf16x2(lo_bf16(x) * s, hi_bf16(x) * s); }

template <int FMT, int NT>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    expand_kernel(const __grid_constant__ CUtensorMap tm, const __grid_constant__ CUtensorMap tm_out, const ExpandParams p) {
  using C = Cfg<NT>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* a_s = smem;
  uint8_t* b_s = smem + C::OFF_B;
  Aux* a = reinterpret_cast<Aux*>(smem + C::OFF_AUX);
  const int tid = threadIdx.x, lane = tid & 31, warp = __reduce_max_sync(0xffffffffu, tid >> 5);
  const int rank = (int)cluster_rank();
  int* err = p.err;

  if (warp == 0) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&a->tmem)), "r"(2 * NT) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  }
  if (tid == 32) {
    for (int i = 0; i < C::STAGES; ++i) mbar_init(&a->b_full[i], 1), mbar_init(&a->b_empty[i], 1);
    for (int i = 0; i < kBoxes; ++i) mbar_init(&a->a_full[i], 2 * kLoaders / 32);
    mbar_init(&a->a_empty, 1);
    for (int i = 0; i < 2; ++i) mbar_init(&a->acc_full[i], 1), mbar_init(&a->acc_empty[i], 2 * 4);
    mbar_init(&a->drain, 1);
    a->abort = 0;
    fence_mbar_init();
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();
  tc_fence_after();
  const uint32_t tmem = a->tmem;

  // this pair's units: u = row tile * per + unit of columns
  const int rows = min(p.rows, max(p.kv_start[p.n_seq], 0));
  const int per = p.H * kOut / NT;
  const int64_t units = (int64_t)((rows + 2 * kRowsCta - 1) / (2 * kRowsCta)) * per;
  const int pairs = (int)(gridDim.x >> 1), pair = (int)(blockIdx.x >> 1);
  const int64_t u0 = units * pair / pairs, u1 = units * (pair + 1) / pairs;

  if (warp == 0) {
    // ---- weights
    if (lane == 0) {
      prefetch_tmap(&tm);
      int s = 0, ph = 0;
      bool ok = true;
      for (int64_t u = u0; ok && u < u1; ++u) {
        const int y = (int)(u % per) * NT + rank * (NT / 2);
        for (int k = 0; k < kBoxes; ++k) {
          ok = wait_pair(a, &a->b_empty[s], ph ^ 1, err);
          if (!ok) break;
          if (rank == 0) mbar_arrive_expect_tx(&a->b_full[s], 2 * C::BOX_B);
          tma_load_pair(b_s + s * C::BOX_B, &tm, dsmem_addr(&a->b_full[s], 0), 64 * k, y);
          if (++s == C::STAGES) s = 0, ph ^= 1;
        }
      }
      for (int i = 0; ok && i < C::STAGES; ++i) {  // the even CTA's last arrivals here have landed
        ok = wait_pair(a, &a->b_empty[s], ph ^ 1, err);
        if (++s == C::STAGES) s = 0, ph ^= 1;
      }
      if (*reinterpret_cast<volatile int*>(&a->abort) && rank == 0)  // wind down: copies in flight land first
        for (int i = 0; i < C::STAGES; ++i) mbar_wait(&a->b_full[i], i < s ? ph : ph ^ 1, err);
    }
    __syncwarp();
  } else if (warp == 1) {
    // ---- MMA issuer
    if (rank == 0) {
      constexpr uint32_t idesc = make_idesc(1, 1, 2 * kRowsCta, NT);
      const uint64_t a_desc = smem_desc_sw128(smem_u32(a_s)), b_desc = smem_desc_sw128(smem_u32(b_s));
      int s = 0, ph = 0, tiles = 0, unit = 0;
      bool ok = true;
      auto all = [&](uint64_t* bar, uint32_t parity) { ok = __all_sync(0xffffffffu, wait_pair(a, bar, parity, err)) && ok; };
      for (int64_t u = u0; ok && u < u1; ++u, ++unit) {
        const bool first = u == u0 || u % per == 0, last = u + 1 == u1 || (u + 1) % per == 0;  // of its row tile
        const uint32_t d = tmem + (unit & 1) * NT;
        all(&a->acc_empty[unit & 1], ((unit >> 1) & 1) ^ 1);
        for (int k = 0; ok && k < kBoxes; ++k) {
          if (first) all(&a->a_full[k], tiles & 1);
          all(&a->b_full[s], ph);
          if (!ok) break;
          tc_fence_after();
          if (elect_one()) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
              mma2(d, a_desc + k * (kBoxA >> 4) + 2 * i, b_desc + s * (C::BOX_B >> 4) + 2 * i, idesc, k || i ? 1u : 0u);
            commit_both(&a->b_empty[s]);
            if (k == kBoxes - 1) {
              if (last) commit_both(&a->a_empty);
              commit_both(&a->acc_full[unit & 1]);
            }
          }
          __syncwarp();
          if (++s == C::STAGES) s = 0, ph ^= 1;
        }
        if (last) ++tiles;
      }
      if (__any_sync(0xffffffffu, *reinterpret_cast<volatile int*>(&a->abort))) {  // wind down: what was issued ends first
        if (elect_one()) commit_both(&a->drain);
        __syncwarp();
        mbar_wait(&a->drain, 0, err);
      }
    }
  } else if (warp >= 4 && warp < 12) {
    // ---- rows
    const int t = tid - 128;
    int tiles = 0;
    bool ok = true;
    for (int64_t u = u0; ok && u < u1; u += per - u % per, ++tiles) {
      const int64_t base = (u / per) * (2 * kRowsCta) + rank * kRowsCta;
      if (t < kRowsCta) {
        bool there;
        const int64_t src = source_row(p, (int)min(base + t, (int64_t)INT_MAX), there);
        a->src[t] = there ? src : src < 0 ? -1 : -2;  // -2: zeros
      }
      loaders_ok(true);
      if constexpr (FMT == kBf16) {
        const int r = t >> 3, c = t & 7;  // 8 lanes a row's 128 bytes of a box
        const uint8_t* from[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int64_t src = a->src[r + 32 * i];
          from[i] = src < 0 ? nullptr : row_at(p, src) + 16 * c;
        }
#pragma unroll
        for (int k0 = 0; k0 < kBoxes; k0 += 4) {
          uint4 v[4][4];
#pragma unroll
          for (int k = 0; k < 4; ++k)
#pragma unroll
            for (int i = 0; i < 4; ++i)
              v[k][i] = from[i] ? load_now(from[i] + 128 * (k0 + k)) : make_uint4(0u, 0u, 0u, 0u);
          if (k0 == 0) ok = __all_sync(0xffffffffu, wait_pair(a, &a->a_empty, (tiles & 1) ^ 1, err));
          if (!ok) break;  // (to the barrier below)
#pragma unroll
          for (int k = 0; k < 4; ++k) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const int row = r + 32 * i;
              *reinterpret_cast<uint4*>(a_s + (k0 + k) * kBoxA + row * 128 + ((c ^ (row & 7)) << 4)) = v[k][i];
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) arrive_even(&a->a_full[k0 + k]);
          }
        }
        if (ok && p.rope_out && u % per == 0) {
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (a->src[r + 32 * i] != -1)
              *reinterpret_cast<uint4*>(p.rope_out + (base + r + 32 * i) * kRope + 8 * c) =
                  from[i] ? __ldg(reinterpret_cast<const uint4*>(from[i] + 2 * kLat)) : make_uint4(0u, 0u, 0u, 0u);
        }
      } else {
        const int r = t >> 2, c = t & 3;  // 4 lanes a row's 64 codes of a box
        const uint8_t* from[2];
        const float* sc[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int64_t src = a->src[r + 64 * i];
          from[i] = src < 0 ? nullptr : row_at(p, src) + 16 * c;
          sc[i] = p.kv_scale + (src < 0 ? 0 : src) * (FMT == kFp8Tile ? 5 : 1);
        }
        uint4 v[kBoxes][2];
        float f[2][5];
#pragma unroll
        for (int k = 0; k < kBoxes; ++k)
#pragma unroll
          for (int i = 0; i < 2; ++i) v[k][i] = from[i] ? load_now(from[i] + 64 * k) : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int k = 0; k < 5; ++k) f[i][k] = FMT == kFp8Tile && from[i] ? __ldg(sc[i] + k) : 1.f;
        ok = __all_sync(0xffffffffu, wait_pair(a, &a->a_empty, (tiles & 1) ^ 1, err));
#pragma unroll
        for (int k = 0; ok && k < kBoxes; ++k) {
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const int row = r + 64 * i;
            uint2 w[4] = {widen4(v[k][i].x), widen4(v[k][i].y), widen4(v[k][i].z), widen4(v[k][i].w)};
            if constexpr (FMT == kFp8Tile) {
#pragma unroll
              for (int q = 0; q < 4; ++q) w[q] = make_uint2(scaled(w[q].x, f[i][k >> 1]), scaled(w[q].y, f[i][k >> 1]));
            }
            uint8_t* d = a_s + k * kBoxA + row * 128;
            *reinterpret_cast<uint4*>(d + (((2 * c) ^ (row & 7)) << 4)) = make_uint4(w[0].x, w[0].y, w[1].x, w[1].y);
            *reinterpret_cast<uint4*>(d + (((2 * c + 1) ^ (row & 7)) << 4)) = make_uint4(w[2].x, w[2].y, w[3].x, w[3].y);
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) arrive_even(&a->a_full[k]);
        }
        if (ok && p.rope_out && u % per == 0) {
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            if (a->src[r + 64 * i] == -1) continue;
            const uint4 x = from[i] ? __ldg(reinterpret_cast<const uint4*>(from[i] + kLat)) : make_uint4(0u, 0u, 0u, 0u);
            const float s = FMT == kFp8Tile ? f[i][4] : from[i] ? __ldg(sc[i]) : 1.f;
            const uint2 w[4] = {widen4(x.x), widen4(x.y), widen4(x.z), widen4(x.w)};
            uint4* d = reinterpret_cast<uint4*>(p.rope_out + (base + r + 64 * i) * kRope + 16 * c);
            d[0] = make_uint4(scaled(w[0].x, s), scaled(w[0].y, s), scaled(w[1].x, s), scaled(w[1].y, s));
            d[1] = make_uint4(scaled(w[2].x, s), scaled(w[2].y, s), scaled(w[3].x, s), scaled(w[3].y, s));
          }
        }
      }
      ok = loaders_ok(ok);  // and the rows' places have been read
    }
    if (ok && u0 < u1) wait_pair(a, &a->a_empty, (tiles & 1) ^ 1, err);  // the even CTA's last arrival here has landed
  } else if (warp >= 12) {
    // ---- read out: thread = row = tensor-memory lane.  64 columns at a time go through shared memory, from where a TMA
    // copy takes them, or, where some of the warp's rows are no sequence's, plain stores
    const int quarter = warp & 3;
    uint8_t* stage = smem + C::OFF_ST + quarter * 2 * 4096;
    const uint32_t lane_base = tmem + ((uint32_t)(32 * quarter) << 16);
    int unit = 0, piece = 0;
    bool ok = true;
    float s = 1.f;
    uint32_t live = 0;  // rows of this warp that are a sequence's
    if (lane == 0) prefetch_tmap(&tm_out);
    for (int64_t u = u0; ok && u < u1; ++u, ++unit) {
      const int64_t base = (u / per) * (2 * kRowsCta) + rank * kRowsCta + 32 * quarter;
      if (u == u0 || u % per == 0) {
        bool there;
        const int64_t src = source_row(p, (int)min(base + lane, (int64_t)INT_MAX), there);
        live = __ballot_sync(0xffffffffu, src >= 0);
        if (FMT == kFp8Row) s = there ? __ldg(p.kv_scale + src) : 1.f;
      }
      ok = __all_sync(0xffffffffu, wait_pair(a, &a->acc_full[unit & 1], (unit >> 1) & 1, err));
      if (!ok) break;
      tc_fence_after();
      const uint32_t acc = lane_base + (unit & 1) * NT;
      const int col = (int)(u % per) * NT;
      float v[2][32];
      tmem_ld_issue(acc, v[0]);
#pragma unroll 1
      for (int c0 = 0; c0 < NT; c0 += 64, ++piece) {
        uint8_t* box = stage + (piece & 1) * 4096;
        // the copy out of this box two pieces ago has read it: a piece commits one group (below), so all but the last one's have
        if (lane == 0) asm volatile("cp.async.bulk.wait_group.read 1;" ::: "memory");
        __syncwarp();
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          tmem_ld_wait(v[h]);
          if (c0 + 32 * h + 32 < NT) {
            tmem_ld_issue(acc + c0 + 32 * h + 32, v[h ^ 1]);
          } else {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) arrive_even(&a->acc_empty[unit & 1]);
          }
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const float* x = &v[h][8 * k];
            const float f = FMT == kFp8Row ? s : 1.f;
            *reinterpret_cast<uint4*>(box + lane * 128 + (((4 * h + k) ^ (lane & 7)) << 4)) =
                make_uint4(bf16x2(x[0] * f, x[1] * f), bf16x2(x[2] * f, x[3] * f), bf16x2(x[4] * f, x[5] * f), bf16x2(x[6] * f, x[7] * f));
          }
        }
        if (live == 0xffffffffu) {
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0)
            asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.bulk_group [%0, {%1, %2}], [%3];" ::"l"(&tm_out), "r"(col + c0),
                         "r"((int)base), "r"(smem_u32(box))
                         : "memory");
        } else {
          __syncwarp();
          __nv_bfloat16* out = p.out + base * ((int64_t)p.H * kOut) + col + c0;
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            const int r = 4 * k + (lane >> 3), c = lane & 7;
            const uint4 x = *reinterpret_cast<const uint4*>(box + r * 128 + ((c ^ (r & 7)) << 4));
            if ((live >> r) & 1) *reinterpret_cast<uint4*>(out + r * ((int64_t)p.H * kOut) + 8 * c) = x;
          }
        }
        // (of a piece that went by plain stores an empty group: without one the wait of the piece behind would leave the copy
        // before this one in flight, whose box that piece writes)
        if (lane == 0) asm volatile("cp.async.bulk.commit_group;" ::: "memory");
      }
    }
    if (lane == 0) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
    __syncwarp();
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();  // the partner's MMAs have read this CTA's memory, its arrivals have landed
  if (warp == 0) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(2 * NT) : "memory");
  }
}

template <int FMT, int NT>
cudaError_t launch_form(const ExpandParams& p, const void* w, cudaStream_t stream) {
  using C = Cfg<NT>;
  const cuuint64_t dims[2] = {(cuuint64_t)kLat, (cuuint64_t)p.H * kOut};
  const cuuint64_t strides[1] = {(cuuint64_t)kLat * 2};
  const cuuint32_t box[2] = {64, NT / 2};
  CUtensorMap tm;
  memset(&tm, 0, sizeof(tm));
  if (encode_tensor_map(&tm, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(w), dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B) !=
      CUDA_SUCCESS)
    return cudaErrorInvalidValue;
  CUtensorMap tm_out;
  const cuuint64_t out_dims[2] = {(cuuint64_t)p.H * kOut, (cuuint64_t)p.rows};
  const cuuint64_t out_strides[1] = {(cuuint64_t)p.H * kOut * 2};
  const cuuint32_t out_box[2] = {64, 32};
  memset(&tm_out, 0, sizeof(tm_out));
  if (encode_tensor_map(&tm_out, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, p.out, out_dims, out_strides, out_box, CU_TENSOR_MAP_SWIZZLE_128B) !=
      CUDA_SUCCESS)
    return cudaErrorInvalidValue;
  auto kern = expand_kernel<FMT, NT>;
  static std::atomic<uint64_t> allowed{0};
  cudaError_t e = allow_smem_once(&allowed, reinterpret_cast<const void*>(kern), C::SMEM);
  if (e != cudaSuccess) return e;
  const int64_t units = (int64_t)((p.rows + 2 * kRowsCta - 1) / (2 * kRowsCta)) * (p.H * kOut / NT);
  const unsigned pairs = (unsigned)(units < kPairs ? units : kPairs);
  return launch_kernel(kern, dim3(2 * pairs), dim3(kThreads), C::SMEM, stream, false, tm, tm_out, p);
}

template <int FMT>
cudaError_t launch_fmt(const ExpandParams& p, const void* w, cudaStream_t stream) {
  // units of a head, or of half a head where those would leave pairs of CTAs idle
  const int64_t heads = (int64_t)((p.rows + 2 * kRowsCta - 1) / (2 * kRowsCta)) * p.H;
  return heads >= 2 * kPairs ? launch_form<FMT, 256>(p, w, stream) : launch_form<FMT, 128>(p, w, stream);
}

dsa_status check_expand(const dsa_expand_args* a) {
  if (!a || a->n_seq < 0 || a->rows < 0 || a->L < 0 || a->H < 1) return DSA_ERR_INVALID_ARG;
  if (a->kv_dtype != DSA_BF16 && a->kv_dtype != DSA_FP8_E4M3 && a->kv_dtype != DSA_FP8_E4M3_T128) return DSA_ERR_UNSUPPORTED;
  if (a->H > 128 || a->n_seq > 4096 || a->L > INT32_MAX - 4096 || a->rows > INT32_MAX - 4096) return DSA_ERR_UNSUPPORTED;
  if (a->block_table) {
    if (a->block_size <= 0 || a->block_size % 64 != 0 || a->num_blocks <= 0 || a->max_blocks < 0) return DSA_ERR_INVALID_ARG;
    if ((int64_t)a->max_blocks * a->block_size < a->L) return DSA_ERR_INVALID_ARG;
    if ((int64_t)a->num_blocks * a->block_size >= (1ll << 31)) return DSA_ERR_UNSUPPORTED;
  }
  if (a->n_seq == 0 || a->rows == 0) return DSA_OK;
  auto ok16 = [](const void* p) { return p && (reinterpret_cast<uintptr_t>(p) & 15) == 0; };
  if (((reinterpret_cast<uintptr_t>(a->kv_start) | reinterpret_cast<uintptr_t>(a->block_table)) & 3) != 0) return DSA_ERR_INVALID_ARG;
  if (!a->kv_start || !ok16(a->w) || !ok16(a->out) || (a->rope_out && !ok16(a->rope_out))) return DSA_ERR_INVALID_ARG;
  if (!ok16(a->kv) || a->kv_row_stride % 16 != 0 || a->kv_row_stride < kLat + kRope) return DSA_ERR_INVALID_ARG;
  if (a->kv_dtype == DSA_BF16 && a->kv_row_stride < 2 * (kLat + kRope)) return DSA_ERR_INVALID_ARG;
  if (!a->block_table && a->n_seq > 1 && (a->kv_seq_stride % 16 != 0 || a->kv_seq_stride < (int64_t)a->L * a->kv_row_stride))
    return DSA_ERR_INVALID_ARG;
  if (a->kv_dtype != DSA_BF16 && (!a->kv_scale || (reinterpret_cast<uintptr_t>(a->kv_scale) & 3) != 0)) return DSA_ERR_INVALID_ARG;
  return DSA_OK;
}

}  // namespace
}  // namespace dsa

using namespace dsa;

extern "C" dsa_status dsa_latent_expand(const dsa_expand_args* a, void* stream) {
  dsa_status s = check_expand(a);
  if (s != DSA_OK || a->n_seq == 0 || a->rows == 0) return s;
  if ((s = check_device_arch()) != DSA_OK) return s;
  ExpandParams p = {};
  p.kv = reinterpret_cast<const uint8_t*>(a->kv);
  p.kv_scale = a->kv_scale;
  p.kv_row_stride = a->kv_row_stride;
  p.kv_seq_stride = a->n_seq > 1 ? a->kv_seq_stride : 0;
  p.L = a->L;
  p.kv_start = a->kv_start;
  p.n_seq = a->n_seq;
  p.rows = a->rows;
  p.H = a->H;
  p.out = reinterpret_cast<__nv_bfloat16*>(a->out);
  p.rope_out = reinterpret_cast<__nv_bfloat16*>(a->rope_out);
  if (a->block_table) {
    p.pages.table = a->block_table;
    p.pages.block_size = a->block_size;
    p.pages.max_blocks = a->max_blocks;
    p.pages.num_blocks = a->num_blocks;
  }
  p.err = device_error_word();
  const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const cudaError_t e = a->kv_dtype == DSA_BF16       ? launch_fmt<kBf16>(p, a->w, st)
                        : a->kv_dtype == DSA_FP8_E4M3 ? launch_fmt<kFp8Row>(p, a->w, st)
                                                      : launch_fmt<kFp8Tile>(p, a->w, st);
  return e == cudaSuccess ? DSA_OK : DSA_ERR_CUDA;
}
