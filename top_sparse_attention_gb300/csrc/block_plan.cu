// Cache blocks and destination rows of one serving step, from request lengths (dsa_block_plan):
// which free blocks each sequence takes, the block-table entries they fill, and the pool row of
// every token the step appends.
//
// With c_s cached and m_s new tokens, block size b, have_s = ceil(c_s / b) and
// need_s = ceil((c_s + m_s) / b) - have_s, the whole plan follows from two prefix sums over the
// sequences: of m_s (where a sequence's rows start) and of need_s (where its blocks start in the
// free list).
//
// One kernel.  The lengths are a few KB in L2, so every CTA takes both prefix sums itself (1024
// threads, shuffles) and keeps them in shared memory; no CTA waits for another, and the rows are
// then independent: a row finds its sequence by bisection (packed) or division (padded).  A new
// block starts with a new token (its first position p has p % b == 0 and c_s <= p), so the row of
// that token writes the block-table entry: no second pass over the table.
// Bound: launch and memory latency; the whole step reads and writes well under 3 MB for 128K rows.  4096 sequences take
// 8.3 us on the device, 256 take 3.4: each CTA loads the lengths and divides by the block size twice, once for the sums and
// once behind them, since a thread's run of sequences does not stay in registers.
#include "dsa_internal.h"

namespace dsa {
namespace {

constexpr int kThreads = 1024;
constexpr int kRowsPerThread = 2;

__device__ __forceinline__ int64_t warp_incl_scan(int64_t v) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t u = __shfl_up_sync(0xffffffffu, v, o);
    if ((threadIdx.x & 31) >= o) v += u;
  }
  return v;
}

struct SeqNeed {
  int c, m;        // cached and new tokens
  int need;        // blocks to take
  bool fits;       // the sequence's block-table row holds all its blocks
};

__device__ __forceinline__ SeqNeed need_of(const BlockPlanParams& p, int s) {
  SeqNeed n;
  n.c = max(p.n_ctx[s], 0);
  n.m = max(p.n_new[s], 0);
  if (p.q_per_seq > 0) n.m = min(n.m, p.q_per_seq);
  // (both sums stay below 2^32: each term is at most 2^31 - 1)
  const uint32_t b = (uint32_t)p.block_size, last = b - 1;
  const uint32_t have = ((uint32_t)n.c + last) / b;
  n.fits = (int64_t)n.c + n.m <= (int64_t)p.max_blocks * p.block_size;
  n.need = n.fits ? (int)(((uint32_t)n.c + (uint32_t)n.m + last) / b - have) : 0;
  return n;
}

__global__ void __launch_bounds__(kThreads) block_plan_kernel(const BlockPlanParams p) {
  extern __shared__ int32_t plan_smem[];
  int32_t* row_off = plan_smem;                    // [n_seq + 1] first row of each sequence
  int32_t* blk_off = plan_smem + p.n_seq + 1;      // [n_seq] first free-list entry; -1: not placed
  __shared__ int64_t warp_rows[kThreads / 32], warp_blocks[kThreads / 32];
  __shared__ int64_t warp_taken[kThreads / 32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int nwarp = blockDim.x >> 5;
  const bool padded = p.q_per_seq > 0;
  const bool first = blockIdx.x == 0;

  // ---- both prefix sums; each thread takes a run of consecutive sequences
  const int per = (p.n_seq + blockDim.x - 1) / blockDim.x;
  const int s0 = min(tid * per, p.n_seq), s1 = min(s0 + per, p.n_seq);
  int64_t rows = 0, blocks = 0;
  for (int s = s0; s < s1; ++s) {
    const SeqNeed n = need_of(p, s);
    rows += n.m;
    blocks += n.need;
  }
  const int64_t rows_in = warp_incl_scan(rows), blocks_in = warp_incl_scan(blocks);
  if (lane == 31) warp_rows[warp] = rows_in, warp_blocks[warp] = blocks_in;
  __syncthreads();
  if (warp == 0) {
    const int64_t r = lane < nwarp ? warp_rows[lane] : 0, b = lane < nwarp ? warp_blocks[lane] : 0;
    const int64_t ri = warp_incl_scan(r), bi = warp_incl_scan(b);
    if (lane < nwarp) warp_rows[lane] = ri - r, warp_blocks[lane] = bi - b;
  }
  __syncthreads();
  int64_t row = warp_rows[warp] + rows_in - rows, blk = warp_blocks[warp] + blocks_in - blocks;
  const int n_free = min(max(p.n_free ? *p.n_free : p.num_free, 0), p.num_free);
  int64_t taken = 0;
  bool failed = false;
  for (int s = s0; s < s1; ++s) {
    const SeqNeed n = need_of(p, s);
    // in order: once the list (or the rows) run out, only sequences that need none are still placed
    const bool placed = n.fits && (n.need == 0 || blk + n.need <= n_free) && (padded || n.m == 0 || row + n.m <= p.rows);
    const int start = padded ? (int)min((int64_t)s * p.q_per_seq, (int64_t)INT32_MAX) : (int)min(row, (int64_t)INT32_MAX);
    row_off[s] = start;
    blk_off[s] = placed ? (n.need ? (int)blk : 0) : -1;
    if (placed) taken += n.need;
    failed |= !placed && n.m > 0;
    if (first) {
      if (p.row_start) p.row_start[s] = start;
      if (p.n_placed) p.n_placed[s] = placed ? n.m : 0;
    }
    row += n.m;
    blk += n.need;
    if (s == p.n_seq - 1) {
      const int64_t end = padded ? (int64_t)p.n_seq * p.q_per_seq : row;
      row_off[p.n_seq] = (int)min(end, (int64_t)INT32_MAX);
      if (first && p.row_start) p.row_start[p.n_seq] = row_off[p.n_seq];
    }
  }
  if (p.n_seq == 0 && tid == 0) {
    row_off[0] = 0;
    if (first && p.row_start) p.row_start[0] = 0;
  }
  if (first) {
    if (failed) record_error(p.err, DSA_DEVERR_BLOCKS);
    const int64_t in_warp = warp_incl_scan(taken);
    if (lane == 31) warp_taken[warp] = in_warp;
  }
  __syncthreads();
  if (first && tid == 0 && p.taken) {
    int64_t t = 0;
    for (int w = 0; w < nwarp; ++w) t += warp_taken[w];
    *p.taken = (int)t;
  }

  // ---- rows
  const int64_t stride = (int64_t)gridDim.x * blockDim.x;
  for (int64_t r = (int64_t)blockIdx.x * blockDim.x + tid; r < p.rows; r += stride) {
    int s, i;
    if (padded) {
      s = (int)((uint32_t)r / (uint32_t)p.q_per_seq);
      i = (int)r - s * p.q_per_seq;
    } else {
      int lo = 0, hi = p.n_seq;  // the last sequence (n_seq: none) whose rows start at or before r
      while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (row_off[mid] <= r) lo = mid;
        else hi = mid - 1;
      }
      s = lo;
      i = (int)(r - row_off[s]);
    }
    int64_t dst = -1;
    int pos = -1;
    if (s < p.n_seq && blk_off[s] >= 0) {
      const int c = max(p.n_ctx[s], 0);
      const int m = padded ? min(max(p.n_new[s], 0), p.q_per_seq) : max(p.n_new[s], 0);
      if (i < m) {
        const int at = c + i;  // fits: below max_blocks * block_size
        const int j = (int)((uint32_t)at / (uint32_t)p.block_size), in = at - j * p.block_size;
        const int have = (int)(((uint32_t)c + (uint32_t)p.block_size - 1) / (uint32_t)p.block_size);
        int32_t* entry = p.block_table + (int64_t)s * p.max_blocks + j;
        const int id = j < have ? *entry : p.free_blocks[blk_off[s] + j - have];
        if ((unsigned)id < (unsigned)p.num_blocks) {
          if (in == 0) *entry = id;  // (in == 0 implies j >= have: a new block's first token)
          dst = (int64_t)id * p.block_size + in;
          pos = at;
        } else {
          record_error(p.err, DSA_DEVERR_INDEX_RANGE);
        }
      }
    }
    p.dst_rows[r] = dst;
    if (p.pos) p.pos[r] = pos;
    if (p.seq) p.seq[r] = pos >= 0 ? s : -1;
  }
}

}  // namespace
}  // namespace dsa

using namespace dsa;

extern "C" dsa_status dsa_block_plan(const int32_t* n_ctx, const int32_t* n_new, int n_seq, int q_per_seq,
                                     int block_size, const int32_t* free_blocks, const int32_t* n_free, int num_free,
                                     int num_blocks, int32_t* block_table, int max_blocks, int rows, int64_t* dst_rows,
                                     int32_t* pos, int32_t* seq, int32_t* row_start, int32_t* n_placed, int32_t* taken,
                                     void* stream) {
  if (n_seq < 0 || q_per_seq < 0 || block_size < 1 || num_free < 0 || num_blocks < 0 || max_blocks < 0 || rows < 0)
    return DSA_ERR_INVALID_ARG;
  if ((int64_t)n_seq * q_per_seq > rows) return DSA_ERR_INVALID_ARG;
  if (n_seq > DSA_BLOCK_PLAN_MAX_SEQ || (int64_t)max_blocks * block_size > INT32_MAX) return DSA_ERR_UNSUPPORTED;
  if (n_seq > 0 && (!n_ctx || !n_new || (max_blocks > 0 && !block_table))) return DSA_ERR_INVALID_ARG;
  if ((rows > 0 && !dst_rows) || (num_free > 0 && !free_blocks)) return DSA_ERR_INVALID_ARG;
  if (n_seq == 0 && rows == 0 && !row_start && !taken) return DSA_OK;
  dsa_status s = check_device_arch();
  if (s != DSA_OK) return s;
  BlockPlanParams p = {};
  p.n_ctx = n_ctx;
  p.n_new = n_new;
  p.n_seq = n_seq;
  p.q_per_seq = q_per_seq;
  p.block_size = block_size;
  p.free_blocks = free_blocks;
  p.n_free = n_free;
  p.num_free = num_free;
  p.num_blocks = num_blocks;
  p.block_table = block_table;
  p.max_blocks = max_blocks;
  p.rows = rows;
  p.dst_rows = dst_rows;
  p.pos = pos;
  p.seq = seq;
  p.row_start = row_start;
  p.n_placed = n_placed;
  p.taken = taken;
  p.err = device_error_word();
  // small batches: fewer threads, so that the two block-wide sums have fewer steps
  const int most = n_seq > rows ? n_seq : rows;
  const int threads = most >= kThreads ? kThreads : (most + 31) / 32 * 32 < 64 ? 64 : (most + 31) / 32 * 32;
  const int64_t want = ((int64_t)rows + (int64_t)threads * kRowsPerThread - 1) / ((int64_t)threads * kRowsPerThread);
  const int grid = (int)(want < 1 ? 1 : want > 304 ? 304 : want);
  const size_t smem = ((size_t)2 * n_seq + 1) * sizeof(int32_t);
  static std::atomic<uint64_t> allowed{0};
  if (allow_smem_once(&allowed, reinterpret_cast<const void*>(block_plan_kernel),
                      (2 * DSA_BLOCK_PLAN_MAX_SEQ + 1) * (int)sizeof(int32_t)) != cudaSuccess)
    return DSA_ERR_CUDA;
  block_plan_kernel<<<grid, threads, smem, reinterpret_cast<cudaStream_t>(stream)>>>(p);
  return cudaGetLastError() == cudaSuccess ? DSA_OK : DSA_ERR_CUDA;
}
