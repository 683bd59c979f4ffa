// Rotation by positions and the encoding of rows, shared by the kernels that turn rows (rope.cu) and that norm and turn
// them (norm_rope.cu).  The angles are described in rope.cu.
#pragma once

#include <math.h>

#include "quant_common.cuh"

namespace dsa {
namespace {

constexpr int kWarps = 8;

// What a CTA keeps in shared memory: the pairs' frequencies as fixed-point turns, and per warp the (cos,
// sin) of the row in hand.
struct RopeSmem {
  uint64_t freq[kRopeMaxPairs];
  alignas(16) float2 turns[kWarps][kRopeMaxPairs];  // (the append kernels read turned columns from here as float4)
  uint8_t axis[kRopeMaxPairs];  // (a copy: lanes read different entries, which parameters serve one by one)
};
static_assert(alignof(RopeSmem) >= 16 && offsetof(RopeSmem, turns) % 16 == 0, "float4 reads");

// f / 2 pi modulo 1, times 2^64.  With f = m 2^e and C = 2^130 / 2 pi it is m C 2^(e - 66), of which the low 64 bits of
// the whole part are kept.
__device__ __forceinline__ uint64_t turn_fraction(float f) {
  constexpr uint64_t kHi = 0xa2f9836e4e441529ull, kLo = 0xfc2757d1f534ddc0ull;  // C
  const uint32_t bits = __float_as_uint(f), ex = bits >> 23 & 255;
  const uint32_t m = (bits & 0x7FFFFFu) | (ex ? 0x800000u : 0u);
  const int down = min(max(66 + 150 - (int)max(ex, 1u), 1), 64 + 127);
  const uint64_t low = kLo * m;
  const unsigned __int128 high = (unsigned __int128)kHi * m + __umul64hi(kLo, m);  // m C = high 2^64 + low
  const uint64_t r = down < 64 ? (uint64_t)(high << (64 - down)) | low >> down : (uint64_t)(high >> (down - 64));
  return (int32_t)bits < 0 ? 0 - r : r;
}

// The pairs' fractions (once per CTA).
__device__ __forceinline__ void fill_freq(const RopeParams& p, RopeSmem& s) {
  for (int i = threadIdx.x; i < p.pairs; i += blockDim.x) {
    s.freq[i] = turn_fraction(p.inv_freq[i]);
    s.axis[i] = p.axis[i];
  }
  __syncthreads();
}

// (cos, sin) of a pair at a position.
__device__ __forceinline__ float2 pair_turn(const RopeParams& p, uint64_t freq, int pos) {
  const uint64_t phase = (uint64_t)(int64_t)pos * freq;
  float s, c;
  sincospif(__ll2float_rn((int64_t)phase) * 0x1p-63f, &s, &c);
  return make_float2(c, p.inverse ? -s : s);
}

// The row's (cos, sin) for every pair, into this warp's shared table.
__device__ __forceinline__ void fill_turns(const RopeParams& p, int64_t row, const RopeSmem& sm, float2* cs) {
  const int lane = threadIdx.x & 31;
  const int32_t* pos = p.pos + row * p.pos_stride;
  __syncwarp();  // the table's last row has been used
  for (int i = lane; i < p.pairs; i += 32) cs[i] = pair_turn(p, sm.freq[i], pos[sm.axis[i]]);
  __syncwarp();
}

// (The roundings are spelled out, so that every kernel of this file turns a pair to the same bits.)
__device__ __forceinline__ void turn(float& a, float& b, float2 cs) {
  const float y0 = fmaf(a, cs.x, -__fmul_rn(b, cs.y)), y1 = fmaf(b, cs.x, __fmul_rn(a, cs.y));
  a = y0;
  b = y1;
}

__device__ __forceinline__ void unpack8(uint4 u, float (&v)[8]) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&w[i]));
    v[2 * i] = f.x, v[2 * i + 1] = f.y;
  }
}

__device__ __forceinline__ uint4 pack8(const float (&v)[8]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 b = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t*>(&b);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

__device__ __forceinline__ int mx_exponent(float amax) {
  return amax > 0.f ? min(max(ilogbf(amax) - 8, -127), 127) : 0;
}

__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d) {
  return (uint32_t)__nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3) |
         (uint32_t)__nv_cvt_float2_to_fp8x2(make_float2(c, d), __NV_SATFINITE, __NV_E4M3) << 16;
}

// Eight codes of the IEEE quotients v / s.  The products with r (1 + 2^-21) and r (1 - 2^-21), r = 1 / s to half an
// ulp, have the quotient between them, and E4M3's rounding is monotone: where both give the same codes, those are
// the quotient's.  Otherwise (a rounding midpoint within 2^-21; r or s not normal) the divisions are made.
__device__ __forceinline__ uint2 encode8(const float (&v)[8], float s, float lo, float hi, bool fast) {
  const uint2 a = make_uint2(e4m3x4(v[0] * lo, v[1] * lo, v[2] * lo, v[3] * lo), e4m3x4(v[4] * lo, v[5] * lo, v[6] * lo, v[7] * lo));
  const uint2 b = make_uint2(e4m3x4(v[0] * hi, v[1] * hi, v[2] * hi, v[3] * hi), e4m3x4(v[4] * hi, v[5] * hi, v[6] * hi, v[7] * hi));
  if (fast && a.x == b.x && a.y == b.y) return a;
  float q[8];
#pragma unroll
  for (int k = 0; k < 8; ++k) q[k] = v[k] == 0.f ? v[k] : __fdiv_rn(v[k], s);
  return make_uint2(e4m3x4(q[0], q[1], q[2], q[3]), e4m3x4(q[4], q[5], q[6], q[7]));
}
constexpr float kAbove = 1.f + 0x1p-21f, kBelow = 1.f - 0x1p-21f;

__device__ __forceinline__ float amax8(const float (&v)[8]) {
  float a = 0.f;
#pragma unroll
  for (int k = 0; k < 8; ++k) a = fmaxf(a, fabsf(v[k]));
  return a;
}

// What both entries check of the rotation itself; fills the pair -> axis table.
dsa_status rope_args(RopeParams* p, int width, int rot_off, int rot_dim, const int32_t* pos, int n_axes,
                     const uint8_t* pair_axis, const float* inv_freq, int style, bool any_rows) {
  if (width < 1 || rot_off < 0 || rot_dim < 2 || rot_dim % 2 != 0 || (int64_t)rot_off + rot_dim > width || n_axes < 1)
    return DSA_ERR_INVALID_ARG;
  if (style != DSA_ROPE_HALF && style != DSA_ROPE_PAIRS) return DSA_ERR_INVALID_ARG;
  if (rot_dim > 2 * kRopeMaxPairs || n_axes > 4) return DSA_ERR_UNSUPPORTED;
  if (n_axes > 1 && !pair_axis) return DSA_ERR_INVALID_ARG;
  if (any_rows && (!pos || !inv_freq)) return DSA_ERR_INVALID_ARG;
  if (!aligned(pos, 4) || !aligned(inv_freq, 4)) return DSA_ERR_INVALID_ARG;
  p->pairs = rot_dim / 2;
  for (int i = 0; i < p->pairs; ++i) {
    const int a = pair_axis ? pair_axis[i] : 0;
    if (a >= n_axes) return DSA_ERR_INVALID_ARG;
    p->axis[i] = (uint8_t)a;
  }
  p->width = width;
  p->rot_off = rot_off;
  p->pos = pos;
  p->pos_stride = n_axes;
  p->inv_freq = inv_freq;
  p->half = style == DSA_ROPE_HALF;
  return DSA_OK;
}

}  // namespace
}  // namespace dsa
