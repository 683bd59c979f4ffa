// What the cache writers share: E4M3 encoding, the exact quotient without a division per element,
// warp maxima, vector loads and host alignment checks.
#pragma once

#include "dsa_internal.h"

namespace dsa {
namespace {

__device__ __forceinline__ uint8_t to_e4m3(float v) {
  return (uint8_t)__nv_cvt_float_to_fp8(v, __NV_SATFINITE, __NV_E4M3);
}

// |v| of finite floats orders like the bit patterns, so the warp max runs on integers.
__device__ __forceinline__ float warp_amax(float a) {
  return __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(fabsf(a))));
}

// The E4M3 code of the IEEE quotient x / s (fp32, round to nearest), without a division per
// element.  Per row: r = 1/s correctly rounded, usable when s and r are normal floats.  Per element:
// q0 = x * r lies within 2.5 fp32 ulps of x / s rounded, and E4M3 rounding is monotone, so the two
// give the same code unless an E4M3 rounding midpoint lies that close to q0.  A midpoint of two
// normal E4M3 values (those two a binade apart included) has fp32 mantissa bit 19 set and bits
// 18..0 clear, so a q0 whose low 20 bits are within 4 of 0x80000 takes the division, and so does
// a q0 in E4M3's subnormal range (below 2^-6), whose midpoints sit elsewhere.
struct Quotient {
  float s, r;
  bool fast;
  __device__ explicit Quotient(float s_) : s(s_) {
    r = __frcp_rn(s_);
    fast = s_ >= 0x1p-126f && r >= 0x1p-126f && r <= 0x1p126f;
  }
  // q0, and whether it gives the code of the IEEE quotient
  __device__ __forceinline__ float fast_part(float x, bool* exact) const {
    const float q0 = x * r;
    const uint32_t low = __float_as_uint(q0) & 0xFFFFFu;
    *exact = fast && !(low - 0x7FFFCu <= 8u || fabsf(q0) < 0x1p-6f);
    return q0;
  }
  __device__ __forceinline__ float operator()(float x) const {
    bool exact;
    const float q0 = fast_part(x, &exact);
    return exact ? q0 : __fdiv_rn(x, s);
  }
};

__device__ __forceinline__ uint32_t pack4(uint8_t a, uint8_t b, uint8_t c, uint8_t d) {
  return (uint32_t)a | (uint32_t)b << 8 | (uint32_t)c << 16 | (uint32_t)d << 24;
}

__device__ __forceinline__ void load8(const __nv_bfloat16* p, float (&v)[8]) {
  const uint4 u = *reinterpret_cast<const uint4*>(p);
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&w[i]));
    v[2 * i] = f.x, v[2 * i + 1] = f.y;
  }
}

inline bool aligned2(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 1u) == 0; }
inline bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

}  // namespace
}  // namespace dsa
