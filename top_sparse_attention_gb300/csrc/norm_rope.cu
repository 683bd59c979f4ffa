// Norm of each head's query or key, or of a latent row, with the rotary positions in the same pass (dsa_norm_rope,
// dsa_norm_rope_append): per vector (a head of a row, or a row)
//   y_c = (x_c - mu) r w_c + b_c over the normed columns, r = 1 / sqrt(var + eps),
// with mu = 0 and var = mean x^2 (RMS), or the mean and the variance (layer norm, the variance from the centred values);
// then the rotary columns turn (rope.cu), and the result is rounded once, to bf16 or to the cache's format.
//
// G lanes (8, 16 or 32) take a vector, lane j of them the 8-element chunks j, j + G, ..., so that the sums are G-wide shuffles
// and everything between the load and the store stays in registers; a warp takes 32 / G heads of a row at a time (rows,
// where there is one head) and the next ones' loads are in flight meanwhile.  The sines of a row are taken once for
// all of its heads.  Columns i and i + rot_dim / 2 of a pair lie in different lanes: the rotary columns pass through
// shared memory.  Norms, sums and angles are fp32.
//
// Lanes: 8 with up to four chunks each for heads of up to 256 columns (32 with a chunk each, the first form: 16384 x 16 heads
// of 192 columns 142 us instead of 37), 16 with five for the latent row (32 with three: 65536 rows, tile scales 78 instead of 67).
// Measured: those heads 37 us (201 MB, 5.4 TB/s, 0.80 of the copy rate; 0.70 instructions per cycle and scheduler); 65536
// latent rows into tile scales 45 us (2.6 TB/s): instructions, 464 per row at 0.59 per cycle, of which the sines, the norm and the
// codes take about a third each (row scales 42, bf16 34, MXFP8 46; keys of 128 columns 18 in bf16 and 19 in MXFP8); layer norm of
// those heads 54; 129 rows 4.1, 64 x 64 heads of 128 columns 3.6: latency of a launch.  The form for any columns is for those that
// are not whole chunks: 16384 x 16 heads of 190 columns 184.
#include "rope_common.cuh"

namespace dsa {
namespace {

struct NormParams {
  const float* weight;  // [dim] or null (ones)
  const float* bias;    // [dim] or null
  int off, dim;
  float eps, inv_dim;
  bool layer;
  int heads_per_item;   // vector form: heads of a row that a warp takes in turn
};

constexpr int kMaxWidth = 1024;
constexpr int kSms = 152;
enum { kFmtBf16 = 0, kFmtRow = 1, kFmtTile = 2, kFmtMx = 3 };

template <int G>
__device__ __forceinline__ float sum_across(float a) {
#pragma unroll
  for (int o = 1; o < G; o <<= 1) a += __shfl_xor_sync(0xffffffffu, a, o);
  return a;
}
template <int G>
__device__ __forceinline__ float max_across(float a) {
#pragma unroll
  for (int o = 1; o < G; o <<= 1) a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, o));
  return a;
}

// encode8 (rope_common.cuh) of four pairs, two products per instruction: the codes of the IEEE quotients v / s, from the
// products that enclose them where those agree.
__device__ __forceinline__ uint32_t e4m3_pairs(float2 a, float2 b) {
  return (uint32_t)__nv_cvt_float2_to_fp8x2(a, __NV_SATFINITE, __NV_E4M3) | (uint32_t)__nv_cvt_float2_to_fp8x2(b, __NV_SATFINITE, __NV_E4M3) << 16;
}
__device__ __forceinline__ uint2 encode_pairs(const float2 (&v)[4], float s, float r, bool fast) {
  const float2 lo = make_float2(r * kBelow, r * kBelow), hi = make_float2(r * kAbove, r * kAbove);
  const uint2 a = make_uint2(e4m3_pairs(fmul2(v[0], lo), fmul2(v[1], lo)), e4m3_pairs(fmul2(v[2], lo), fmul2(v[3], lo)));
  const uint2 b = make_uint2(e4m3_pairs(fmul2(v[0], hi), fmul2(v[1], hi)), e4m3_pairs(fmul2(v[2], hi), fmul2(v[3], hi)));
  if (fast && a.x == b.x && a.y == b.y) return a;
  float2 q[4];
#pragma unroll
  for (int k = 0; k < 4; ++k)
    q[k] = make_float2(v[k].x == 0.f ? v[k].x : __fdiv_rn(v[k].x, s), v[k].y == 0.f ? v[k].y : __fdiv_rn(v[k].y, s));
  return make_uint2(e4m3_pairs(q[0], q[1]), e4m3_pairs(q[2], q[3]));
}

template <int FMT, int G, int NCH, int CTAS>
__global__ void __launch_bounds__(32 * kWarps, CTAS) norm_rope_vec_kernel(const RopeParams p, const NormParams n) {
  constexpr int VEC = 32 / G;  // vectors per step of a warp
  __shared__ RopeSmem sm;
  __shared__ alignas(16) float stage_s[kWarps][VEC * 8 * G * NCH < 256 * VEC ? VEC * 8 * G * NCH : 256 * VEC];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane / G, gl = lane % G;
  const int nch = p.width / 8;
  const bool one = p.heads == 1;  // then the vectors of a step are rows
  const int hblocks = one ? 1 : (p.heads + n.heads_per_item - 1) / n.heads_per_item;
  // weights and biases by column, in shared memory (in registers they would spill)
  __shared__ alignas(16) float w_s[8 * G * NCH], b_s[8 * G * NCH];
  for (int c = threadIdx.x; c < n.dim; c += 32 * kWarps) {
    w_s[c] = n.weight ? n.weight[c] : 1.f;
    b_s[c] = n.bias ? n.bias[c] : 0.f;
  }
  fill_freq(p, sm);  // (with the barrier)
  float2* cs = sm.turns[warp];
  float* stage = stage_s[warp] + g * 2 * p.pairs;
  const int entries = one ? VEC * p.pairs : p.pairs;  // of the table: pairs of the step's rows, or of the row

  // this lane's entries of the table, lane + 32 e: of row `row` of the step, pair `pair` (divisions once, not per step)
  constexpr int E = kRopeMaxPairs / 32, EP = 2;  // entries of a lane at most, those whose positions are loaded ahead
  int entry[E];                 // row | pair << 8 | axis << 16, -1: none
#pragma unroll
  for (int e = 0; e < E; ++e) {
    const int i = lane + 32 * e, v = one ? i / p.pairs : 0, k = i - v * p.pairs;
    entry[e] = i < entries ? v | k << 8 | sm.axis[k] << 16 : -1;
  }

  uint4 raw[NCH];
  int64_t dst = 0;
  int pos[EP] = {};
  // a step: vectors g of `row` and heads [h0 + VEC pass, ...), or of rows [row, row + VEC)
  struct Step {
    int64_t row;
    int hb, pass;
  };
  auto head_of = [&](const Step& s) { return one ? 0 : s.hb * n.heads_per_item + s.pass * VEC + g; };
  auto row_of = [&](const Step& s) { return one ? s.row + g : s.row; };
  auto mine_of = [&](const Step& s) {
    return one ? s.row + g < p.rows : s.pass * VEC + g < n.heads_per_item && head_of(s) < p.heads;
  };
  auto fetch = [&](const Step& s) {
    const bool live = mine_of(s);
    const int64_t row = row_of(s);
    const __nv_bfloat16* x = p.x + row * p.x_row_stride + head_of(s) * p.x_head_stride + 8 * gl;
    if (p.dst) dst = !live ? -1 : p.dst_rows ? p.dst_rows[row] : row;
#pragma unroll
    for (int j = 0; j < NCH; ++j)
      raw[j] = live && gl + G * j < nch ? *reinterpret_cast<const uint4*>(x + 8 * G * j) : make_uint4(0u, 0u, 0u, 0u);
    if (s.pass == 0) {
#pragma unroll
      for (int e = 0; e < EP; ++e) {
        const int64_t r = s.row + (entry[e] & 255);
        if (entry[e] >= 0 && r < p.rows) pos[e] = p.pos[r * p.pos_stride + (entry[e] >> 16)];
      }
    }
  };
  const int64_t item0 = (int64_t)blockIdx.x * kWarps + warp, stride = (int64_t)gridDim.x * kWarps;
  Step at = {one ? item0 * VEC : item0 / hblocks, one ? 0 : (int)(item0 % hblocks), 0};
  const int64_t row_step = one ? stride * VEC : stride / hblocks;
  const int hb_step = one ? 0 : (int)(stride % hblocks);
  if (at.row < p.rows) fetch(at);
#pragma unroll 1
  while (at.row < p.rows) {
    const int64_t to = dst, row = row_of(at);
    const bool mine = mine_of(at);
    const int head = head_of(at);
    if (at.pass == 0) {
      __syncwarp();  // the table's last row has been used
#pragma unroll
      for (int e = 0; e < E; ++e) {
        if (entry[e] < 0) continue;
        const int64_t r = at.row + (entry[e] & 255);
        const int where = e < EP ? pos[e < EP ? e : 0] : r < p.rows ? p.pos[r * p.pos_stride + (entry[e] >> 16)] : 0;
        cs[lane + 32 * e] = pair_turn(p, sm.freq[entry[e] >> 8 & 255], where);
      }
      __syncwarp();
    }
    float2 v[NCH][4];
#pragma unroll
    for (int j = 0; j < NCH; ++j) {
      const uint32_t u[4] = {raw[j].x, raw[j].y, raw[j].z, raw[j].w};
#pragma unroll
      for (int k = 0; k < 4; ++k) v[j][k] = make_float2(__uint_as_float(u[k] << 16), __uint_as_float(u[k] & 0xFFFF0000u));
    }
    // the next step's loads
    ++at.pass;
    if (one || at.pass * VEC >= min(n.heads_per_item, p.heads - at.hb * n.heads_per_item)) {
      at.pass = 0;
      at.row += row_step;
      at.hb += hb_step;
      if (at.hb >= hblocks) at.hb -= hblocks, ++at.row;
    }
    if (at.row < p.rows) fetch(at);

    // ---- the norm
    float mean = 0.f;
    if (n.layer) {
      float2 s = make_float2(0.f, 0.f);
#pragma unroll
      for (int j = 0; j < NCH; ++j) {
        const int c = 8 * (gl + G * j) - n.off;
        if (c >= 0 && c < n.dim)
#pragma unroll
          for (int k = 0; k < 4; ++k) s.x += v[j][k].x, s.y += v[j][k].y;
      }
      mean = sum_across<G>(s.x + s.y) * n.inv_dim;
    }
    float2 ss = make_float2(0.f, 0.f);
#pragma unroll
    for (int j = 0; j < NCH; ++j) {
      const int c = 8 * (gl + G * j) - n.off;
      if (c >= 0 && c < n.dim) {
        if (n.layer)
#pragma unroll
          for (int k = 0; k < 4; ++k) v[j][k].x -= mean, v[j][k].y -= mean;
#pragma unroll
        for (int k = 0; k < 4; ++k) ss = ffma2(v[j][k], v[j][k], ss);
      }
    }
    const float r = __frsqrt_rn(fmaf(sum_across<G>(ss.x + ss.y), n.inv_dim, n.eps));
#pragma unroll
    for (int j = 0; j < NCH; ++j) {
      const int c = 8 * (gl + G * j) - n.off;
      if (c < 0 || c >= n.dim) continue;
#pragma unroll
      for (int k = 0; k < 4; k += 2) {
        const float4 w = *reinterpret_cast<const float4*>(w_s + c + 2 * k);
        v[j][k] = fmul2(fmul2(v[j][k], make_float2(r, r)), make_float2(w.x, w.y));
        v[j][k + 1] = fmul2(fmul2(v[j][k + 1], make_float2(r, r)), make_float2(w.z, w.w));
        if (n.bias) {
          const float4 b = *reinterpret_cast<const float4*>(b_s + c + 2 * k);
          v[j][k].x += b.x, v[j][k].y += b.y, v[j][k + 1].x += b.z, v[j][k + 1].y += b.w;
        }
      }
    }
    // ---- the rotary columns
    const float2* turns = cs + (one ? g * p.pairs : 0);
    if (p.half) {
      __syncwarp();
#pragma unroll
      for (int j = 0; j < NCH; ++j) {
        const int c = 8 * (gl + G * j) - p.rot_off;
        if (c >= 0 && c < 2 * p.pairs) {
          *reinterpret_cast<float4*>(stage + c) = make_float4(v[j][0].x, v[j][0].y, v[j][1].x, v[j][1].y);
          *reinterpret_cast<float4*>(stage + c + 4) = make_float4(v[j][2].x, v[j][2].y, v[j][3].x, v[j][3].y);
        }
      }
      __syncwarp();
    }
#pragma unroll
    for (int j = 0; j < NCH; ++j) {
      const int c = 8 * (gl + G * j) - p.rot_off;
      if (c < 0 || c >= 2 * p.pairs) continue;
      if (p.half) {
        const bool low = c < p.pairs;
        const float2* other = reinterpret_cast<const float2*>(stage + (low ? c + p.pairs : c - p.pairs));
        const float4* t = reinterpret_cast<const float4*>(turns + (low ? c : c - p.pairs));
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const float4 t2 = t[k];  // (cos, sin) of two pairs
          const float2 o = other[k];
          float a0 = low ? v[j][k].x : o.x, b0 = low ? o.x : v[j][k].x, a1 = low ? v[j][k].y : o.y, b1 = low ? o.y : v[j][k].y;
          turn(a0, b0, make_float2(t2.x, t2.y));
          turn(a1, b1, make_float2(t2.z, t2.w));
          v[j][k] = low ? make_float2(a0, a1) : make_float2(b0, b1);
        }
      } else {
#pragma unroll
        for (int k = 0; k < 4; ++k) turn(v[j][k].x, v[j][k].y, turns[c / 2 + k]);
      }
    }
    // ---- out
    const bool keep = mine && (!p.dst || (to >= 0 && to < p.dst_count));
    if (p.dst && mine && to >= p.dst_count && gl == 0) record_error(p.err, DSA_DEVERR_INDEX_RANGE);
    auto amax_of = [&](int j) {
      float a = 0.f;
#pragma unroll
      for (int k = 0; k < 4; ++k) a = fmaxf(a, fmaxf(fabsf(v[j][k].x), fabsf(v[j][k].y)));
      return a;
    };
    if constexpr (FMT == kFmtBf16) {
      __nv_bfloat16* out = p.dst ? reinterpret_cast<__nv_bfloat16*>(p.dst + to * p.dst_row_stride)
                                 : p.out + row * p.out_row_stride + head * p.out_head_stride;
#pragma unroll
      for (int j = 0; j < NCH; ++j) {
        const int c = gl + G * j;
        uint32_t u[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const __nv_bfloat162 b = __floats2bfloat162_rn(v[j][k].x, v[j][k].y);
          u[k] = *reinterpret_cast<const uint32_t*>(&b);
        }
        if (keep && c < nch) *reinterpret_cast<uint4*>(out + 8 * c) = make_uint4(u[0], u[1], u[2], u[3]);
      }
    } else if constexpr (FMT == kFmtRow) {
      float a = 0.f;
#pragma unroll
      for (int j = 0; j < NCH; ++j) a = fmaxf(a, amax_of(j));
      a = max_across<G>(a);
      const Quotient div(a > 0.f ? __fdiv_rn(a, 448.f) : 1.f);
#pragma unroll
      for (int j = 0; j < NCH; ++j) {
        const int c = gl + G * j;
        if (keep && c < nch)
          *reinterpret_cast<uint2*>(p.dst + to * p.dst_row_stride + 8 * c) = encode_pairs(v[j], div.s, div.r, div.fast);
      }
      if (keep && gl == 0) reinterpret_cast<float*>(p.scale)[to] = div.s;
    } else if constexpr (FMT == kFmtTile) {
      // A tile is a slot of 16 lanes, or two slots of 8.  Lane j of its lanes takes slot j's scale and its reciprocal, once
      // instead of NCH times
      constexpr int T = G < 16 ? G : 16;
      const int tiles = (nch + 15) / 16;
      float own = 0.f;
#pragma unroll
      for (int j = 0; j < NCH; ++j) {
        float a = amax_of(j);
        if (G == 8 && (j ^ 1) < NCH) a = fmaxf(a, amax_of(j ^ 1));
        a = max_across<T>(a);
        if (lane % T == j) own = a;
      }
      const Quotient div(own > 0.f ? __fdiv_rn(own, 448.f) : 1.f);
      const uint32_t fast = __ballot_sync(0xffffffffu, div.fast);
#pragma unroll
      for (int j = 0; j < NCH; ++j) {
        const int c = gl + G * j, from = lane / T * T + j;
        const float s = __shfl_sync(0xffffffffu, div.s, from), rs = __shfl_sync(0xffffffffu, div.r, from);
        if (!keep || c >= nch) continue;
        *reinterpret_cast<uint2*>(p.dst + to * p.dst_row_stride + 8 * c) = encode_pairs(v[j], s, rs, (fast >> from) & 1);
        if (c % 16 == 0) reinterpret_cast<float*>(p.scale)[to * tiles + c / 16] = s;
      }
    } else {
#pragma unroll
      for (int j = 0; j < NCH; ++j) {
        const int c = gl + G * j;
        const float a = max_across<4>(amax_of(j));
        if (!keep || c >= nch) continue;
        const int e = mx_exponent(a);
        const float inv = ldexpf(1.f, -e);  // a power of two: exact
        const float2* y = v[j];
        *reinterpret_cast<uint2*>(p.dst + to * p.dst_row_stride + 8 * c) =
            make_uint2(e4m3x4(y[0].x * inv, y[0].y * inv, y[1].x * inv, y[1].y * inv),
                       e4m3x4(y[2].x * inv, y[2].y * inv, y[3].x * inv, y[3].y * inv));
        if (c % 4 == 0) p.scale[to * (p.width / 32) + c / 4] = (uint8_t)(e + 127);
      }
    }
  }
}

// Any width up to 1024, offset, pitch and alignment: a warp per vector, which it holds in shared memory.
constexpr int kPlainWarps = 4;
template <int FMT>
__global__ void __launch_bounds__(32 * kPlainWarps) norm_rope_kernel(const RopeParams p, const NormParams n) {
  __shared__ RopeSmem sm;
  __shared__ float rows_s[kPlainWarps][kMaxWidth];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  fill_freq(p, sm);
  float2* cs = sm.turns[warp];
  float* v = rows_s[warp];
  const int64_t vectors = (int64_t)p.rows * p.heads, step = (int64_t)gridDim.x * kPlainWarps;
#pragma unroll 1
  for (int64_t at = (int64_t)blockIdx.x * kPlainWarps + warp; at < vectors; at += step) {
    const int64_t row = at / p.heads;
    const int head = (int)(at - row * p.heads);
    const __nv_bfloat16* x = p.x + row * p.x_row_stride + head * p.x_head_stride;
    fill_turns(p, row, sm, cs);
    for (int c = lane; c < p.width; c += 32) v[c] = __bfloat162float(x[c]);
    __syncwarp();
    float mean = 0.f;
    if (n.layer) {
      for (int c = lane; c < n.dim; c += 32) mean += v[n.off + c];
      mean = sum_across<32>(mean) * n.inv_dim;
    }
    float ss = 0.f;
    for (int c = lane; c < n.dim; c += 32) {
      const float d = v[n.off + c] - mean;
      ss = fmaf(d, d, ss);
    }
    const float r = __frsqrt_rn(fmaf(sum_across<32>(ss), n.inv_dim, n.eps));
    for (int c = lane; c < n.dim; c += 32)
      v[n.off + c] = fmaf((v[n.off + c] - mean) * r, n.weight ? n.weight[c] : 1.f, n.bias ? n.bias[c] : 0.f);
    __syncwarp();
    for (int k = lane; k < p.pairs; k += 32) {
      const int c0 = p.rot_off + (p.half ? k : 2 * k), c1 = p.half ? c0 + p.pairs : c0 + 1;
      turn(v[c0], v[c1], cs[k]);
    }
    __syncwarp();
    if (!p.dst) {
      __nv_bfloat16* out = p.out + row * p.out_row_stride + head * p.out_head_stride;
      for (int c = lane; c < p.width; c += 32) out[c] = __float2bfloat16_rn(v[c]);
      continue;
    }
    const int64_t to = p.dst_rows ? p.dst_rows[row] : row;
    if (to >= p.dst_count && lane == 0) record_error(p.err, DSA_DEVERR_INDEX_RANGE);
    if (to < 0 || to >= p.dst_count) continue;
    uint8_t* out = p.dst + to * p.dst_row_stride;
    if constexpr (FMT == kFmtBf16) {
      for (int c = lane; c < p.width; c += 32) *reinterpret_cast<__nv_bfloat16*>(out + 2 * c) = __float2bfloat16_rn(v[c]);
    } else {
      const int group = FMT == kFmtRow ? p.width : FMT == kFmtTile ? 128 : 32;
      const int groups = (p.width + group - 1) / group;
      for (int i = 0; i < groups; ++i) {
        const int lo = i * group, hi = min(lo + group, p.width);
        float a = 0.f;
        for (int c = lo + lane; c < hi; c += 32) a = fmaxf(a, fabsf(v[c]));
        a = max_across<32>(a);
        if constexpr (FMT == kFmtMx) {
          const int e = mx_exponent(a);
          const float inv = ldexpf(1.f, -e);
          for (int c = lo + lane; c < hi; c += 32) out[c] = to_e4m3(v[c] * inv);
          if (lane == 0) p.scale[to * groups + i] = (uint8_t)(e + 127);
        } else {
          const Quotient div(a > 0.f ? __fdiv_rn(a, 448.f) : 1.f);
          for (int c = lo + lane; c < hi; c += 32) out[c] = to_e4m3(div(v[c]));
          if (lane == 0) reinterpret_cast<float*>(p.scale)[to * groups + i] = div.s;
        }
      }
    }
  }
}

using NormKernel = void (*)(const RopeParams, const NormParams);

// The vector form for a width: the lanes of a vector, and resident CTAs.  `whole`: a warp per vector.
template <int FMT>
NormKernel vec_form(int width, bool few, bool whole, int* lanes, int* ctas) {
  *lanes = whole ? 32 : width <= 256 ? 8 : width <= 640 && !few ? 16 : 32;
  *ctas = width <= 256 ? 3 : 2;
  if (whole && width <= 256) return norm_rope_vec_kernel<FMT, 32, 1, 3>;
  if (width <= 64) return norm_rope_vec_kernel<FMT, 8, 1, 3>;
  if (width <= 128) return norm_rope_vec_kernel<FMT, 8, 2, 3>;
  if (width <= 192) return norm_rope_vec_kernel<FMT, 8, 3, 3>;
  if (width <= 256) return norm_rope_vec_kernel<FMT, 8, 4, 3>;
  if (width <= 640 && !few && !whole) return norm_rope_vec_kernel<FMT, 16, 5, 2>;
  if (width <= 768) return norm_rope_vec_kernel<FMT, 32, 3, 2>;
  return norm_rope_vec_kernel<FMT, 32, 4, 2>;
}

dsa_status norm_args(NormParams* n, const dsa_norm* norm, int width) {
  if (!norm || (norm->kind != DSA_NORM_RMS && norm->kind != DSA_NORM_LAYER)) return DSA_ERR_INVALID_ARG;
  if (norm->off < 0 || norm->dim < 1 || (int64_t)norm->off + norm->dim > width) return DSA_ERR_INVALID_ARG;
  if (!(norm->eps >= 0.f) || !(norm->eps < INFINITY)) return DSA_ERR_INVALID_ARG;
  if (!aligned(norm->weight, 4) || !aligned(norm->bias, 4)) return DSA_ERR_INVALID_ARG;
  if (width > kMaxWidth) return DSA_ERR_UNSUPPORTED;
  n->weight = norm->weight;
  n->bias = norm->bias;
  n->off = norm->off;
  n->dim = norm->dim;
  n->eps = norm->eps;
  n->inv_dim = 1.f / (float)norm->dim;
  n->layer = norm->kind == DSA_NORM_LAYER;
  return DSA_OK;
}

// The columns that need whole 16-byte chunks, for the vector form.  (Weights and biases do not: it reads them one by one, once per CTA.)
bool whole_chunks(const RopeParams& p, const NormParams& n) {
  return p.width % 8 == 0 && p.rot_off % 8 == 0 && (2 * p.pairs) % 8 == 0 && (!p.half || p.pairs % 8 == 0) && n.off % 8 == 0 &&
         n.dim % 8 == 0 && aligned(p.x, 16) && (p.rows == 1 || p.x_row_stride % 8 == 0) && p.x_head_stride % 8 == 0;
}

template <int FMT>
dsa_status launch_norm(const RopeParams& p, NormParams n, bool vec, cudaStream_t stream) {
  if (!vec) {
    const int64_t want = ((int64_t)p.rows * p.heads + kPlainWarps - 1) / kPlainWarps;
    norm_rope_kernel<FMT><<<(unsigned)(want < 8 * kSms ? want : 8 * kSms), 32 * kPlainWarps, 0, stream>>>(p, n);
  } else {
    int lanes, ctas;
    // a warp per vector where every warp has one at most (latent rows, us: 129 rows 3.6 and 4.2 with half a warp, 4800 5.7 and 5.3)
    const bool few = (int64_t)p.rows * p.heads <= 2 * kSms * kWarps;
    // (a step's rows have a table of turns each: of all the pairs that a warp's table holds at most)
    const bool whole = p.heads == 1 && (p.width <= 256 ? 4 : 2) * p.pairs > kRopeMaxPairs;
    const NormKernel kern = vec_form<FMT>(p.width, few, whole, &lanes, &ctas);
    const int per = 32 / lanes, most = ctas * kSms;
    // heads of a row for a warp: all of up to 16, or as few as leave no warp idle
    n.heads_per_item = 16;
    while (n.heads_per_item > per && (int64_t)p.rows * ((p.heads + n.heads_per_item - 1) / n.heads_per_item) < (int64_t)most * kWarps)
      n.heads_per_item /= 2;
    const int64_t items = p.heads == 1 ? ((int64_t)p.rows + per - 1) / per
                                       : (int64_t)p.rows * ((p.heads + n.heads_per_item - 1) / n.heads_per_item);
    const int64_t want = (items + kWarps - 1) / kWarps;
    kern<<<(unsigned)(want < most ? want : most), 32 * kWarps, 0, stream>>>(p, n);
  }
  return cudaGetLastError() == cudaSuccess ? DSA_OK : DSA_ERR_CUDA;
}

}  // namespace
}  // namespace dsa

using namespace dsa;

extern "C" {

dsa_status dsa_norm_rope(const void* x, int64_t x_row_stride, int64_t x_head_stride, int rows, int heads, int width,
                         const dsa_norm* norm, int rot_off, int rot_dim, const int32_t* pos, int n_axes, const uint8_t* pair_axis,
                         const float* inv_freq, int style, void* out, int64_t out_row_stride, int64_t out_head_stride, void* stream) {
  RopeParams p = {};
  NormParams n = {};
  if (rows < 0 || heads < 1) return DSA_ERR_INVALID_ARG;
  dsa_status s = rope_args(&p, width, rot_off, rot_dim, pos, n_axes, pair_axis, inv_freq, style, rows > 0);
  if (s != DSA_OK || (s = norm_args(&n, norm, width)) != DSA_OK) return s;
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
  const bool vec = whole_chunks(p, n) && aligned(out, 16) && (rows == 1 || out_row_stride % 8 == 0) && p.out_head_stride % 8 == 0;
  return launch_norm<kFmtBf16>(p, n, vec, reinterpret_cast<cudaStream_t>(stream));
}

dsa_status dsa_norm_rope_append(const void* x, int64_t x_row_stride, int rows, int width, const dsa_norm* norm, int rot_off,
                                int rot_dim, const int32_t* pos, int n_axes, const uint8_t* pair_axis, const float* inv_freq,
                                int style, dsa_dtype dtype, void* dst, int64_t dst_row_stride, int64_t dst_count, void* scale,
                                const int64_t* dst_rows, void* stream) {
  RopeParams p = {};
  NormParams n = {};
  if (rows < 0 || dst_count < 0) return DSA_ERR_INVALID_ARG;
  dsa_status s = rope_args(&p, width, rot_off, rot_dim, pos, n_axes, pair_axis, inv_freq, style, rows > 0);
  if (s != DSA_OK || (s = norm_args(&n, norm, width)) != DSA_OK) return s;
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
  p.heads = 1;
  p.dst = reinterpret_cast<uint8_t*>(dst);
  p.dst_row_stride = dst_row_stride;
  p.dst_count = dst_count;
  p.scale = reinterpret_cast<uint8_t*>(scale);
  p.dst_rows = dst_rows;
  p.err = device_error_word();
  const uintptr_t out_align = elem == 2 ? 16 : 8;
  const bool vec = whole_chunks(p, n) && aligned(dst, out_align) && dst_row_stride % (int64_t)out_align == 0;
  const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  switch (dtype) {
    case DSA_BF16: return launch_norm<kFmtBf16>(p, n, vec, st);
    case DSA_FP8_E4M3: return launch_norm<kFmtRow>(p, n, vec, st);
    case DSA_FP8_E4M3_T128: return launch_norm<kFmtTile>(p, n, vec, st);
    default: return launch_norm<kFmtMx>(p, n, vec, st);
  }
}

}  // extern "C"
