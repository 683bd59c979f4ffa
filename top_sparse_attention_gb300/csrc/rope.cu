// Rotary positions with one or several axes, on queries (dsa_rope) and on the rows that the cache
// writer stores (dsa_rope_append).
//
// Pair i of a row turns by theta = pos[row, axis(i)] * inv_freq[i]:
//   y0 = x0 cos(theta) - x1 sin(theta),   y1 = x1 cos(theta) + x0 sin(theta),
// the pair being elements (i, i + rot_dim / 2) of the rotated columns or (2i, 2i + 1).
//
// The angle.  A position of a million times a frequency of one loses the angle in fp32 (an ulp of
// 10^6 is 0.06 rad).  Here inv_freq / 2 pi, in turns, becomes a 64-bit fixed-point fraction (its
// significand times 128 bits of 1 / 2 pi, in integers, once per pair and CTA; fp64 took 0.2 us longer);
// position times fraction modulo 2^64 is then exact integer arithmetic that drops the whole turns by
// itself, and it is theta in half turns, in [-1, 1), for sincospif: rounded to fp32 from all 64 bits, so
// that small angles keep their digits.  The fraction is cut off, by less than 2^-64 (for |inv_freq| <=
// 2^40, where 1 / 2 pi has bits enough), so the angle is off by at most 2^-33 turns at the farthest
// position.
//
// A warp takes one row (append; half a warp for many rows with tile or MXFP8 scales) or 16 heads of a row (rope) after
// another: the lanes take the sines of the row's pairs once and share them through shared memory; 16-byte loads and
// stores.  Rotated values enter the cache format's rounding in fp32 (one rounding, not two).
// Bound, and measured: bf16 rows by HBM (131072 rows of 576, 302 MB: 54 us, 5.6 TB/s); E4M3 rows by instructions (tile
// scales 77 us, row scales 65, MXFP8 50); rope into 128-byte pieces of wider rows by no single unit (32768 x 16 heads,
// 134 MB: 34 us, with issue slots 53 % busy, DRAM 33 %, and a third of the waits for loads); small calls by the launch (3
// us).
#include "rope_common.cuh"

namespace dsa {
namespace {

constexpr int kHeadsPerWarp = 16;
constexpr int kSms = 152;
constexpr int kCtasPerSm = 3;  // resident CTAs (registers); a large launch has this many per SM

// ---------------------------------------------------------------------------------------------
// dsa_rope: x [rows, heads, width] -> out, columns [rot_off, rot_off + 2 pairs) turned, the others
// copied when out is another buffer.

// 16-byte chunks.  A warp's items (16 heads of a row) are software-pipelined: the next item's loads, and its
// position, are in flight while one is turned and stored.
__global__ void __launch_bounds__(32 * kWarps, kCtasPerSm) rope_vec_kernel(const RopeParams p) {
  __shared__ RopeSmem sm;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int hblocks = (p.heads + kHeadsPerWarp - 1) / kHeadsPerWarp;
  const int64_t items = (int64_t)p.rows * hblocks, step = (int64_t)gridDim.x * kWarps;
  fill_freq(p, sm);
  float2* cs = sm.turns[warp];
  const int per = p.half ? p.pairs / 8 : p.pairs / 4;  // loads of one head: a chunk and its other half, or a chunk
  constexpr int U = 2;                                 // chunk pairs per lane and batch
  const uint64_t f0 = lane < p.pairs ? sm.freq[lane] : 0;
  const int ax0 = lane < p.pairs ? sm.axis[lane] : 0;
  uint4 a[U], b[U];
  int pos0 = 0;
  // batch of chunks [base, base + 64) of an item: chunk i is head i / per, columns 8 (i % per) (and the same of
  // the other half); neighbouring pairs take two chunks per step
  auto chunk = [&](int i, int& h, int& c) {
    h = i / per;
    c = i - h * per;
  };
  auto fetch = [&](int64_t item, int base) {
    const int64_t row = hblocks == 1 ? item : item / hblocks;
    const int h0 = (int)(item - row * hblocks) * kHeadsPerWarp, n = min(kHeadsPerWarp, p.heads - h0) * per;
    const __nv_bfloat16* x = p.x + row * p.x_row_stride + h0 * p.x_head_stride + p.rot_off;
    if (base == 0) pos0 = p.pos[row * p.pos_stride + ax0];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      int h, c;
      const int i = base + (p.half ? 32 * u : 64 * u) + lane;
      if (i < n) {
        chunk(i, h, c);
        const __nv_bfloat16* src = x + h * p.x_head_stride + 8 * c;
        a[u] = *reinterpret_cast<const uint4*>(src);
        if (p.half) b[u] = *reinterpret_cast<const uint4*>(src + p.pairs);
      }
      if (!p.half && i + 32 < n) {
        chunk(i + 32, h, c);
        b[u] = *reinterpret_cast<const uint4*>(x + h * p.x_head_stride + 8 * c);
      }
    }
  };
  const int width = p.half ? 32 * U : 64 * U;  // chunks per batch
  int64_t item = (int64_t)blockIdx.x * kWarps + warp;
  if (item < items) fetch(item, 0);
#pragma unroll 1
  for (; item < items; item += step) {
    const int64_t row = hblocks == 1 ? item : item / hblocks;
    const int h0 = (int)(item - row * hblocks) * kHeadsPerWarp, nh = min(kHeadsPerWarp, p.heads - h0), n = nh * per;
    __nv_bfloat16* out = p.out + row * p.out_row_stride + h0 * p.out_head_stride;
    __syncwarp();
    if (lane < p.pairs) cs[lane] = pair_turn(p, f0, pos0);
    for (int i = lane + 32; i < p.pairs; i += 32)
      cs[i] = pair_turn(p, sm.freq[i], p.pos[row * p.pos_stride + sm.axis[i]]);
    __syncwarp();
    for (int base = 0; base < n; base += width) {
      uint4 va[U], vb[U];
#pragma unroll
      for (int u = 0; u < U; ++u) va[u] = a[u], vb[u] = b[u];
      if (base + width < n) fetch(item, base + width);
      else if (item + step < items) fetch(item + step, 0);
#pragma unroll
      for (int u = 0; u < U; ++u) {
        int h, c;
        const int i = base + (p.half ? 32 * u : 64 * u) + lane;
        float x0[8], x1[8];
        unpack8(va[u], x0);
        unpack8(vb[u], x1);
        if (p.half) {
          if (i < n) {
            chunk(i, h, c);
            __nv_bfloat16* dst = out + h * p.out_head_stride + p.rot_off + 8 * c;
#pragma unroll
            for (int k = 0; k < 8; ++k) turn(x0[k], x1[k], cs[8 * c + k]);
            *reinterpret_cast<uint4*>(dst) = pack8(x0);
            *reinterpret_cast<uint4*>(dst + p.pairs) = pack8(x1);
          }
        } else {
          if (i < n) {
            chunk(i, h, c);
#pragma unroll
            for (int k = 0; k < 4; ++k) turn(x0[2 * k], x0[2 * k + 1], cs[4 * c + k]);
            *reinterpret_cast<uint4*>(out + h * p.out_head_stride + p.rot_off + 8 * c) = pack8(x0);
          }
          if (i + 32 < n) {
            chunk(i + 32, h, c);
#pragma unroll
            for (int k = 0; k < 4; ++k) turn(x1[2 * k], x1[2 * k + 1], cs[4 * c + k]);
            *reinterpret_cast<uint4*>(out + h * p.out_head_stride + p.rot_off + 8 * c) = pack8(x1);
          }
        }
      }
    }
    if (p.copy) {
      const __nv_bfloat16* x = p.x + row * p.x_row_stride + h0 * p.x_head_stride;
      const int rest = (p.width - 2 * p.pairs) / 8;
      for (int i = lane; i < nh * rest; i += 32) {
        const int h = i / rest;
        int c = 8 * (i - h * rest);
        if (c >= p.rot_off) c += 2 * p.pairs;
        *reinterpret_cast<uint4*>(out + h * p.out_head_stride + c) =
            *reinterpret_cast<const uint4*>(x + h * p.x_head_stride + c);
      }
    }
  }
}

// Any offset, pitch and alignment: one pair per lane and step.
__global__ void __launch_bounds__(32 * kWarps) rope_kernel(const RopeParams p) {
  __shared__ RopeSmem sm;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int hblocks = (p.heads + kHeadsPerWarp - 1) / kHeadsPerWarp;
  const int64_t items = (int64_t)p.rows * hblocks;
  fill_freq(p, sm);
  float2* cs = sm.turns[warp];
#pragma unroll 1
  for (int64_t item = (int64_t)blockIdx.x * kWarps + warp; item < items; item += (int64_t)gridDim.x * kWarps) {
    const int64_t row = item / hblocks;
    const int h0 = (int)(item - row * hblocks) * kHeadsPerWarp, nh = min(kHeadsPerWarp, p.heads - h0);
    const __nv_bfloat16* x = p.x + row * p.x_row_stride + h0 * p.x_head_stride;
    __nv_bfloat16* out = p.out + row * p.out_row_stride + h0 * p.out_head_stride;
    fill_turns(p, row, sm, cs);
    for (int i = lane; i < nh * p.pairs; i += 32) {
      const int h = i / p.pairs, k = i - h * p.pairs;
      const int c0 = p.rot_off + (p.half ? k : 2 * k), c1 = p.half ? c0 + p.pairs : c0 + 1;
      float a = __bfloat162float(x[h * p.x_head_stride + c0]), b = __bfloat162float(x[h * p.x_head_stride + c1]);
      turn(a, b, cs[k]);
      out[h * p.out_head_stride + c0] = __float2bfloat16_rn(a);
      out[h * p.out_head_stride + c1] = __float2bfloat16_rn(b);
    }
    if (p.copy) {
      const int rest = p.width - 2 * p.pairs;
      for (int i = lane; i < nh * rest; i += 32) {
        const int h = i / rest;
        int c = i - h * rest;
        if (c >= p.rot_off) c += 2 * p.pairs;
        out[h * p.out_head_stride + c] = x[h * p.x_head_stride + c];
      }
    }
  }
}

// ---------------------------------------------------------------------------------------------
// dsa_rope_append: x [rows, width], turned, encoded as FMT and written to destination rows.

enum { kFmtBf16 = 0, kFmtRow = 1, kFmtTile = 2, kFmtMx = 3 };

constexpr int kMaxChunks = 4;  // 8-element chunks per lane: rows up to 1024 elements
// The form with half a warp per row: tiles per row, resident CTAs (registers), and the rows from which it pays (tile
// scales, us: 8192 rows 9.0 against 7.8 of a warp per row, 65536 41.1 against 43.3, 131072 76.5 against 84.8; MX 6.0
// against 6.2, 27.4 against 32.3, 49.7 against 61.2; row scales and bf16 gain nothing or lose).
constexpr int kHalfTiles = 5, kHalfCtasPerSm = 2, kHalfRows = 32768;

// Rows of up to 128 NT columns with up to 32 pairs (the latent row): half a warp takes a row, lane j of it the
// 8-element chunks j, j + 16, ..., so that a slot of the 16 lanes is a tile of 128.  (A warp per row leaves a
// quarter of the lanes idle at 576 columns and spends the row's other instructions on one row: 562 per row instead
// of 427.)  The rotary columns are turned pair by pair, two pairs per
// lane, into fp32 in shared memory, from where the lanes that hold their chunks take them.  The next row's loads (its
// chunks, pairs, position and destination) are in flight while a row is encoded.
template <int FMT, int NT>
__global__ void __launch_bounds__(32 * kWarps, kHalfCtasPerSm) rope_append_half_kernel(const RopeParams p) {
  __shared__ RopeSmem sm;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, half = lane >> 4, hl = lane & 15;
  const int nch = p.width / 8;
  const int64_t step = (int64_t)gridDim.x * kWarps * 2;
  fill_freq(p, sm);
  float* turned = reinterpret_cast<float*>(sm.turns[warp]) + 64 * half;  // the row's rotary columns
  uint64_t freq[2];
  int axis[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int k = hl + 16 * i;
    freq[i] = k < p.pairs ? sm.freq[k] : 0;
    axis[i] = k < p.pairs ? sm.axis[k] : 0;
  }
  // the rotary columns' first chunk from this lane's chunk 0 on (at most one of its chunks is among them)
  const int rot0 = hl - p.rot_off / 8, rots = p.pairs / 4;
  uint4 raw[NT];
  __nv_bfloat16 x0[2], x1[2];
  int pos[2] = {0, 0};
  int64_t dst = -1;
  auto fetch = [&](int64_t row) {
    dst = -1;
    if (row >= p.rows) return;
    const __nv_bfloat16* x = p.x + row * p.x_row_stride;
    dst = p.dst_rows ? p.dst_rows[row] : row;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int k = hl + 16 * i;
      if (k < p.pairs) {
        pos[i] = p.pos[row * p.pos_stride + axis[i]];
        const int c0 = p.rot_off + (p.half ? k : 2 * k);
        x0[i] = x[c0];
        x1[i] = x[p.half ? c0 + p.pairs : c0 + 1];
      }
    }
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      const int c = hl + 16 * j;
      raw[j] = c < nch ? *reinterpret_cast<const uint4*>(x + 8 * c) : make_uint4(0u, 0u, 0u, 0u);
    }
  };
  int64_t row0 = ((int64_t)blockIdx.x * kWarps + warp) * 2;  // the warp's pair of rows
#pragma unroll
  for (int j = 0; j < NT; ++j) raw[j] = make_uint4(0u, 0u, 0u, 0u);
  x0[0] = x0[1] = x1[0] = x1[1] = __float2bfloat16_rn(0.f);
  if (row0 < p.rows) fetch(row0 + half);
#pragma unroll 1
  for (; row0 < p.rows; row0 += step) {
    const int64_t at_row = dst;
    const bool keep = at_row >= 0 && at_row < p.dst_count;
    if (at_row >= p.dst_count && hl == 0) record_error(p.err, DSA_DEVERR_INDEX_RANGE);
    __syncwarp();
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int k = hl + 16 * i;
      float a = __bfloat162float(x0[i]), b = __bfloat162float(x1[i]);
      turn(a, b, pair_turn(p, freq[i], pos[i]));
      if (k < p.pairs) {
        turned[p.half ? k : 2 * k] = a;
        turned[p.half ? k + p.pairs : 2 * k + 1] = b;
      }
    }
    __syncwarp();
    float v[NT][8];
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      unpack8(raw[j], v[j]);
      const int at = rot0 + 16 * j;
      if (at >= 0 && at < rots) {
        const float4 t0 = *reinterpret_cast<const float4*>(turned + 8 * at), t1 = *reinterpret_cast<const float4*>(turned + 8 * at + 4);
        v[j][0] = t0.x, v[j][1] = t0.y, v[j][2] = t0.z, v[j][3] = t0.w;
        v[j][4] = t1.x, v[j][5] = t1.y, v[j][6] = t1.z, v[j][7] = t1.w;
      }
    }
    if (row0 + step < p.rows) fetch(row0 + step + half);
    uint8_t* out = p.dst + at_row * p.dst_row_stride;
    auto across = [](float a, int lanes) {
#pragma unroll
      for (int o = 1; o < 16; o <<= 1)
        if (o < lanes) a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, o));
      return a;
    };
    if constexpr (FMT == kFmtTile) {
      // lane j of each half takes tile j's scale and reciprocal (a division each, once instead of NT times)
      float own = 0.f;
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        const float a = across(amax8(v[j]), 16);
        if (hl == j) own = a;
      }
      const Quotient div(own > 0.f ? __fdiv_rn(own, 448.f) : 1.f);
      const int tiles = (nch + 15) / 16;
      if (keep && hl < tiles) reinterpret_cast<float*>(p.scale)[at_row * tiles + hl] = div.s;
      const uint32_t fast = __ballot_sync(0xffffffffu, div.fast);
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        const int c = hl + 16 * j, from = (lane & 16) + j;
        const float s = __shfl_sync(0xffffffffu, div.s, from), r = __shfl_sync(0xffffffffu, div.r, from);
        if (keep && c < nch)
          *reinterpret_cast<uint2*>(out + 8 * c) = encode8(v[j], s, r * kBelow, r * kAbove, (fast >> from) & 1);
      }
    } else {
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        const int c = hl + 16 * j;
        const float a = across(amax8(v[j]), 4);
        if (keep && c < nch) {
          const int e = mx_exponent(a);
          const float inv = ldexpf(1.f, -e);  // a power of two: exact
          *reinterpret_cast<uint2*>(out + 8 * c) =
              make_uint2(e4m3x4(v[j][0] * inv, v[j][1] * inv, v[j][2] * inv, v[j][3] * inv),
                         e4m3x4(v[j][4] * inv, v[j][5] * inv, v[j][6] * inv, v[j][7] * inv));
          if ((lane & 3) == 0) p.scale[at_row * (p.width / 32) + c / 4] = (uint8_t)(e + 127);
        }
      }
    }
  }
}

// Vector form: a warp takes a row, lane j the 8-element chunks j, j + 32, ... of the row, so 4 consecutive lanes hold
// a group of 32 and 16 lanes a tile of 128.  The rotary columns are turned pair by pair, a pair per lane (PP
// per lane), into fp32 in shared memory, from where the lanes that hold their chunks take them.  The next
// row's loads (its chunks, pairs, position and destination) are in flight while a row is encoded.
template <int FMT, int NCH, int PP>
__global__ void __launch_bounds__(32 * kWarps, NCH == 3 ? kCtasPerSm : 1) rope_append_vec_kernel(const RopeParams p) {
  __shared__ RopeSmem sm;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int nch = p.width / 8;
  const int64_t step = (int64_t)gridDim.x * kWarps;
  fill_freq(p, sm);
  float* turned = reinterpret_cast<float*>(sm.turns[warp]);  // [2 pairs] the row's rotary columns
  uint64_t freq[PP];
  int axis[PP];
#pragma unroll
  for (int i = 0; i < PP; ++i) {
    const int k = lane + 32 * i;
    freq[i] = k < p.pairs ? sm.freq[k] : 0;
    axis[i] = k < p.pairs ? sm.axis[k] : 0;
  }
  uint4 raw[NCH];
  __nv_bfloat16 x0[PP], x1[PP];
  int pos[PP];
  int64_t dst = -1;
  auto fetch = [&](int64_t row) {
    const __nv_bfloat16* x = p.x + row * p.x_row_stride;
    dst = p.dst_rows ? p.dst_rows[row] : row;
#pragma unroll
    for (int i = 0; i < PP; ++i) {
      const int k = lane + 32 * i;
      if (k < p.pairs) {
        pos[i] = p.pos[row * p.pos_stride + axis[i]];
        const int c0 = p.rot_off + (p.half ? k : 2 * k);
        x0[i] = x[c0];
        x1[i] = x[p.half ? c0 + p.pairs : c0 + 1];
      }
    }
#pragma unroll
    for (int j = 0; j < NCH; ++j) {
      const int c = lane + 32 * j;
      raw[j] = c < nch ? *reinterpret_cast<const uint4*>(x + 8 * c) : make_uint4(0u, 0u, 0u, 0u);
    }
  };
  int64_t row = (int64_t)blockIdx.x * kWarps + warp;
  if (row < p.rows) fetch(row);
#pragma unroll 1
  for (; row < p.rows;) {
    const int64_t at_row = dst;
    const bool drop = at_row < 0 || at_row >= p.dst_count;  // the same for the whole warp
    if (at_row >= p.dst_count && lane == 0) record_error(p.err, DSA_DEVERR_INDEX_RANGE);
    __syncwarp();
#pragma unroll
    for (int i = 0; i < PP; ++i) {
      const int k = lane + 32 * i;
      if (k < p.pairs) {
        float a = __bfloat162float(x0[i]), b = __bfloat162float(x1[i]);
        turn(a, b, pair_turn(p, freq[i], pos[i]));
        turned[p.half ? k : 2 * k] = a;
        turned[p.half ? k + p.pairs : 2 * k + 1] = b;
      }
    }
    __syncwarp();
    float v[NCH][8];
#pragma unroll
    for (int j = 0; j < NCH; ++j) {
      unpack8(raw[j], v[j]);
      const int at = 8 * (lane + 32 * j) - p.rot_off;
      if (at >= 0 && at < 2 * p.pairs) {
        const float4 t0 = *reinterpret_cast<const float4*>(turned + at), t1 = *reinterpret_cast<const float4*>(turned + at + 4);
        v[j][0] = t0.x, v[j][1] = t0.y, v[j][2] = t0.z, v[j][3] = t0.w;
        v[j][4] = t1.x, v[j][5] = t1.y, v[j][6] = t1.z, v[j][7] = t1.w;
      }
    }
    row += step;
    if (row < p.rows) fetch(row);
    if (drop) continue;
    uint8_t* out = p.dst + at_row * p.dst_row_stride;
    if constexpr (FMT == kFmtBf16) {
#pragma unroll
      for (int j = 0; j < NCH; ++j) {
        const int c = lane + 32 * j;
        if (c < nch) *reinterpret_cast<uint4*>(out + 16 * c) = pack8(v[j]);
      }
    } else if constexpr (FMT == kFmtRow) {
      float a = 0.f;
#pragma unroll
      for (int j = 0; j < NCH; ++j) a = fmaxf(a, amax8(v[j]));
      const float amax = warp_amax(a);
      const float s = amax > 0.f ? __fdiv_rn(amax, 448.f) : 1.f;
      const Quotient div(s);
#pragma unroll
      for (int j = 0; j < NCH; ++j) {
        const int c = lane + 32 * j;
        if (c < nch) *reinterpret_cast<uint2*>(out + 8 * c) = encode8(v[j], s, div.r * kBelow, div.r * kAbove, div.fast);
      }
      if (lane == 0) reinterpret_cast<float*>(p.scale)[at_row] = s;
    } else if constexpr (FMT == kFmtTile) {
      const int tiles = (p.width + 127) / 128;
      // the tiles' maxima, one per 16 lanes and j; then lane j of each 16 takes tile j's scale and reciprocal
      // (a division each, once instead of NCH times)
      float own = 0.f;
#pragma unroll
      for (int j = 0; j < NCH; ++j) {
        float a = amax8(v[j]);
#pragma unroll
        for (int o = 1; o < 16; o <<= 1) a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, o));
        if ((lane & 15) == j) own = a;
      }
      Quotient div(own > 0.f ? __fdiv_rn(own, 448.f) : 1.f);
      const float s_own = div.s, r_own = div.r;
      const uint32_t fast = __ballot_sync(0xffffffffu, div.fast);
#pragma unroll
      for (int j = 0; j < NCH; ++j) {
        const int c = lane + 32 * j, from = (lane & 16) + j;
        div.s = __shfl_sync(0xffffffffu, s_own, from);
        div.r = __shfl_sync(0xffffffffu, r_own, from);
        div.fast = (fast >> from) & 1;
        if (c < nch) {
          *reinterpret_cast<uint2*>(out + 8 * c) = encode8(v[j], div.s, div.r * kBelow, div.r * kAbove, div.fast);
          if ((lane & 15) == 0) reinterpret_cast<float*>(p.scale)[at_row * tiles + c / 16] = div.s;
        }
      }
    } else {
#pragma unroll
      for (int j = 0; j < NCH; ++j) {
        if (32 * j >= nch) break;
        const int c = lane + 32 * j;
        float a = amax8(v[j]);
        a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, 1));
        a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, 2));
        if (c < nch) {
          const int e = mx_exponent(a);
          const float inv = ldexpf(1.f, -e);  // a power of two: exact
          *reinterpret_cast<uint2*>(out + 8 * c) =
              make_uint2(e4m3x4(v[j][0] * inv, v[j][1] * inv, v[j][2] * inv, v[j][3] * inv),
                         e4m3x4(v[j][4] * inv, v[j][5] * inv, v[j][6] * inv, v[j][7] * inv));
          if ((lane & 3) == 0) p.scale[at_row * (p.width / 32) + c / 4] = (uint8_t)(e + 127);
        }
      }
    }
  }
}

// Any width, pitch and alignment: the same arithmetic, one element per lane and step; each scale
// group (the row, 128 or 32 elements) is taken in two passes, its maximum and its codes.
template <int FMT>
__global__ void __launch_bounds__(32 * kWarps) rope_append_kernel(const RopeParams p) {
  __shared__ RopeSmem sm;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  fill_freq(p, sm);
  const int64_t row = (int64_t)blockIdx.x * kWarps + warp;
  if (row >= p.rows) return;
  const int64_t dst = p.dst_rows ? p.dst_rows[row] : row;
  if (dst < 0) return;
  if (dst >= p.dst_count) {
    if (lane == 0) record_error(p.err, DSA_DEVERR_INDEX_RANGE);
    return;
  }
  const __nv_bfloat16* x = p.x + row * p.x_row_stride;
  float2* cs = sm.turns[warp];
  fill_turns(p, row, sm, cs);
  auto value = [&](int c) {
    const float v = __bfloat162float(x[c]);
    const int at = c - p.rot_off;
    if (at < 0 || at >= 2 * p.pairs) return v;
    const bool low = p.half ? at < p.pairs : (at & 1) == 0;
    const int k = p.half ? (low ? at : at - p.pairs) : at >> 1;
    const float w = __bfloat162float(x[c + (p.half ? (low ? p.pairs : -p.pairs) : (low ? 1 : -1))]);
    return fmaf(v, cs[k].x, __fmul_rn(w, low ? -cs[k].y : cs[k].y));
  };
  uint8_t* out = p.dst + dst * p.dst_row_stride;
  if constexpr (FMT == kFmtBf16) {
    for (int c = lane; c < p.width; c += 32)
      *reinterpret_cast<__nv_bfloat16*>(out + 2 * c) = __float2bfloat16_rn(value(c));
  } else {
    const int group = FMT == kFmtRow ? p.width : FMT == kFmtTile ? 128 : 32;
    const int groups = (p.width + group - 1) / group;
    for (int g = 0; g < groups; ++g) {
      const int lo = g * group, hi = min(lo + group, p.width);
      float a = 0.f;
      for (int c = lo + lane; c < hi; c += 32) a = fmaxf(a, fabsf(value(c)));
      const float amax = warp_amax(a);
      if constexpr (FMT == kFmtMx) {
        const int e = mx_exponent(amax);
        const float inv = ldexpf(1.f, -e);
        for (int c = lo + lane; c < hi; c += 32) out[c] = to_e4m3(value(c) * inv);
        if (lane == 0) p.scale[dst * groups + g] = (uint8_t)(e + 127);
      } else {
        const float s = amax > 0.f ? __fdiv_rn(amax, 448.f) : 1.f;
        const Quotient div(s);
        for (int c = lo + lane; c < hi; c += 32) out[c] = to_e4m3(div(value(c)));
        if (lane == 0) reinterpret_cast<float*>(p.scale)[dst * groups + g] = s;
      }
    }
  }
}

using AppendKernel = void (*)(const RopeParams);
template <int FMT>
AppendKernel append_vec(bool small, bool half) {
  if constexpr (FMT == kFmtTile || FMT == kFmtMx)
    if (half) return rope_append_half_kernel<FMT, kHalfTiles>;
  return small ? rope_append_vec_kernel<FMT, 3, 1> : rope_append_vec_kernel<FMT, kMaxChunks, 4>;
}

}  // namespace
}  // namespace dsa

using namespace dsa;

extern "C" {

dsa_status dsa_rope(const void* x, int64_t x_row_stride, int64_t x_head_stride, int rows, int heads, int width,
                    int rot_off, int rot_dim, const int32_t* pos, int n_axes, const uint8_t* pair_axis,
                    const float* inv_freq, int style, int inverse, void* out, int64_t out_row_stride,
                    int64_t out_head_stride, void* stream) {
  RopeParams p = {};
  if (rows < 0 || heads < 1) return DSA_ERR_INVALID_ARG;
  dsa_status s = rope_args(&p, width, rot_off, rot_dim, pos, n_axes, pair_axis, inv_freq, style, rows > 0);
  if (s != DSA_OK) return s;
  if (heads > 1 && (x_head_stride < width || out_head_stride < width)) return DSA_ERR_INVALID_ARG;
  if (rows > 1 && (x_row_stride < width || out_row_stride < width)) return DSA_ERR_INVALID_ARG;
  if (rows == 0) return DSA_OK;
  if (!x || !out || !aligned2(x) || !aligned2(out)) return DSA_ERR_INVALID_ARG;
  // in place means the same elements: another layout over the same memory would race
  if (x == out && ((rows > 1 && x_row_stride != out_row_stride) || (heads > 1 && x_head_stride != out_head_stride)))
    return DSA_ERR_INVALID_ARG;
  if ((s = check_device_arch()) != DSA_OK) return s;
  p.x = reinterpret_cast<const __nv_bfloat16*>(x);
  p.out = reinterpret_cast<__nv_bfloat16*>(out);
  p.x_row_stride = x_row_stride;
  p.x_head_stride = heads > 1 ? x_head_stride : 0;
  p.out_row_stride = out_row_stride;
  p.out_head_stride = heads > 1 ? out_head_stride : 0;
  p.rows = rows;
  p.heads = heads;
  p.inverse = inverse != 0;
  p.copy = x != out && width > rot_dim;
  const bool vec = rot_off % 8 == 0 && p.pairs % 8 == 0 && (!p.copy || width % 8 == 0) && aligned(x, 16) &&
                   aligned(out, 16) && (rows == 1 || (x_row_stride % 8 == 0 && out_row_stride % 8 == 0)) &&
                   p.x_head_stride % 8 == 0 && p.out_head_stride % 8 == 0;
  const int64_t items = (int64_t)rows * ((heads + kHeadsPerWarp - 1) / kHeadsPerWarp);
  const int64_t want = (items + kWarps - 1) / kWarps;
  const int64_t most = vec ? kSms * kCtasPerSm : 8 * kSms;
  const int64_t grid = want < most ? want : most;
  auto kern = vec ? rope_vec_kernel : rope_kernel;
  kern<<<(unsigned)grid, 32 * kWarps, 0, reinterpret_cast<cudaStream_t>(stream)>>>(p);
  return cudaGetLastError() == cudaSuccess ? DSA_OK : DSA_ERR_CUDA;
}

dsa_status dsa_rope_append(const void* x, int64_t x_row_stride, int rows, int width, int rot_off, int rot_dim,
                           const int32_t* pos, int n_axes, const uint8_t* pair_axis, const float* inv_freq, int style,
                           dsa_dtype dtype, void* dst, int64_t dst_row_stride, int64_t dst_count, void* scale,
                           const int64_t* dst_rows, void* stream) {
  RopeParams p = {};
  if (rows < 0 || dst_count < 0) return DSA_ERR_INVALID_ARG;
  dsa_status s = rope_args(&p, width, rot_off, rot_dim, pos, n_axes, pair_axis, inv_freq, style, rows > 0);
  if (s != DSA_OK) return s;
  if (dtype != DSA_BF16 && dtype != DSA_FP8_E4M3 && dtype != DSA_FP8_E4M3_T128 && dtype != DSA_MXFP8_E4M3)
    return DSA_ERR_UNSUPPORTED;
  const int64_t elem = dtype == DSA_BF16 ? 2 : 1;
  if (dst_row_stride < width * elem || dst_row_stride % elem != 0 || (rows > 1 && x_row_stride < width))
    return DSA_ERR_INVALID_ARG;
  if (dtype == DSA_MXFP8_E4M3 && width % 32 != 0) return DSA_ERR_INVALID_ARG;
  if (!dst_rows && rows > dst_count) return DSA_ERR_INVALID_ARG;
  if (rows == 0) return DSA_OK;
  if (!x || !dst || !aligned2(x) || (elem == 2 && !aligned2(dst)) || !aligned(dst_rows, 8)) return DSA_ERR_INVALID_ARG;
  if (dtype != DSA_BF16 && !scale) return DSA_ERR_INVALID_ARG;
  if ((dtype == DSA_FP8_E4M3 || dtype == DSA_FP8_E4M3_T128) && !aligned(scale, 4)) return DSA_ERR_INVALID_ARG;
  if ((s = check_device_arch()) != DSA_OK) return s;
  p.x = reinterpret_cast<const __nv_bfloat16*>(x);
  p.x_row_stride = x_row_stride;
  p.rows = rows;
  p.dst = reinterpret_cast<uint8_t*>(dst);
  p.dst_row_stride = dst_row_stride;
  p.dst_count = dst_count;
  p.scale = reinterpret_cast<uint8_t*>(scale);
  p.dst_rows = dst_rows;
  p.err = device_error_word();
  const uintptr_t out_align = elem == 2 ? 16 : 8;
  const bool vec = width % 8 == 0 && width <= 256 * kMaxChunks && rot_off % 8 == 0 &&
                   (2 * p.pairs) % 8 == 0 && aligned(x, 16) && (rows == 1 || x_row_stride % 8 == 0) &&
                   aligned(dst, out_align) && dst_row_stride % (int64_t)out_align == 0;
  // rows of up to 768 columns with up to 32 pairs (the latent row) take the form with fewer registers; many of up to
  // 640 with scales per 128 or 32 columns half a warp each
  const bool small = width <= 768 && p.pairs <= 32;
  const bool half = vec && p.pairs <= 32 && width <= 128 * kHalfTiles && rows >= kHalfRows &&
                    (dtype == DSA_FP8_E4M3_T128 || dtype == DSA_MXFP8_E4M3);
  AppendKernel kern = nullptr;
  switch (dtype) {
    case DSA_BF16: kern = vec ? append_vec<kFmtBf16>(small, half) : rope_append_kernel<kFmtBf16>; break;
    case DSA_FP8_E4M3: kern = vec ? append_vec<kFmtRow>(small, half) : rope_append_kernel<kFmtRow>; break;
    case DSA_FP8_E4M3_T128: kern = vec ? append_vec<kFmtTile>(small, half) : rope_append_kernel<kFmtTile>; break;
    default: kern = vec ? append_vec<kFmtMx>(small, half) : rope_append_kernel<kFmtMx>; break;
  }
  int grid = half ? (rows + 2 * kWarps - 1) / (2 * kWarps) : (rows + kWarps - 1) / kWarps;
  const int most = kSms * (half ? kHalfCtasPerSm : small ? kCtasPerSm : 1);
  if (vec && grid > most) grid = most;
  kern<<<grid, 32 * kWarps, 0, reinterpret_cast<cudaStream_t>(stream)>>>(p);
  return cudaGetLastError() == cudaSuccess ? DSA_OK : DSA_ERR_CUDA;
}

}  // extern "C"
