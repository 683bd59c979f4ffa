// Attention of drafted tokens over the latent cache (dsa_tree_attn): query node i of sequence s sees
// the n_ctx[s] cached positions and the drafted positions n_ctx[s] + j whose bit j is set in its row
// of the tree mask,
//   logit[p] = sm_scale * q[i, h] . Kv[p],  out[i, h] = sum_p softmax(logit)[p] * Kv[p, :512],
// with one pass over the positions that keeps the running maximum m and sum l of each row:
//   m' = max(m, max_p x_p), l' = l 2^(m - m') + sum_p 2^(x_p - m'), o' = o 2^(m - m') + sum_p 2^(x_p - m') v_p.
#include "dsa_internal.h"

namespace dsa {
namespace {

constexpr float kLn2 = 0.6931471805599453f;
constexpr int kDqk = 576, kDv = 512;

__device__ __forceinline__ float e4m3_f32(uint8_t c) {
  const __half_raw h = __nv_cvt_fp8_to_halfraw(c, __NV_E4M3);
  return __half2float(*reinterpret_cast<const __half*>(&h));
}

// One CTA per (16 rows, sequence), a row being one head of one node; 32 positions at a time in fp32.
constexpr int kRowsS = 16, kKeysS = 32, kThreadsS = 256;

__global__ void __launch_bounds__(kThreadsS) tree_attn_simple_kernel(const TreeAttnParams p) {
  extern __shared__ float sm[];
  float* qs = sm;                          // [16][576]
  float* ks = qs + kRowsS * kDqk;          // [32][577]
  float* xs = ks + kKeysS * (kDqk + 1);    // [16][33]
  float* ms = xs + kRowsS * (kKeysS + 1);  // [16] m, l, factor
  const int tid = threadIdx.x, seq = blockIdx.y, r0 = blockIdx.x * kRowsS;
  const int rows = p.q_per_seq * p.H;
  const int ctx = min(max(p.n_ctx[seq], 0), p.L);
  const int fresh = p.n_new ? min(max(p.n_new[seq], 0), p.q_per_seq) : p.q_per_seq;
  const int len = (int)min((int64_t)ctx + fresh, (int64_t)p.L);
  const int nsc = p.nsc;
  for (int i = tid; i < kRowsS * kDqk; i += kThreadsS) {
    const int r = r0 + i / kDqk;
    qs[i] = r < rows ? __bfloat162float(p.q[((int64_t)seq * rows + r) * kDqk + i % kDqk]) * p.scale_log2 : 0.f;
  }
  if (tid < kRowsS) ms[tid] = -INFINITY, ms[kRowsS + tid] = 0.f;
  float o[kRowsS * kDv / kThreadsS];
#pragma unroll
  for (int i = 0; i < kRowsS * kDv / kThreadsS; ++i) o[i] = 0.f;
  for (int k0 = 0; k0 < len; k0 += kKeysS) {
    __syncthreads();
    bool bad = false;
    for (int i = tid; i < kKeysS * kDqk; i += kThreadsS) {
      const int k = i / kDqk, c = i % kDqk, pos = k0 + k;
      float v = 0.f;
      if (pos < len) {
        const int64_t row = tree_row(p, seq, pos);
        if (row >= 0) {
          if (p.kv_fp8) v = e4m3_f32(p.kv[row * p.kv_row_stride + (p.pages.table ? 0 : seq * p.kv_seq_stride) + c]) *
                            p.kv_scale[((p.pages.table ? 0 : (int64_t)seq * p.L) + row) * nsc + (nsc > 1 ? c / 128 : 0)];
          else v = __bfloat162float(*reinterpret_cast<const __nv_bfloat16*>(
                   p.kv + row * p.kv_row_stride + (p.pages.table ? 0 : seq * p.kv_seq_stride) + 2 * c));
        } else {
          bad = true;
        }
      }
      ks[k * (kDqk + 1) + c] = v;
    }
    if (bad) record_error(p.err, DSA_DEVERR_INDEX_RANGE);
    __syncthreads();
    for (int i = tid; i < kRowsS * kKeysS; i += kThreadsS) {
      const int r = i / kKeysS, k = i % kKeysS, pos = k0 + k, node = (r0 + r) / p.H;
      float x = -INFINITY;
      if (r0 + r < rows && node < fresh && pos < len && tree_sees(p, seq, node, pos, ctx) && tree_row(p, seq, pos) >= 0) {
        x = 0.f;
        for (int c = 0; c < kDqk; ++c) x = fmaf(qs[r * kDqk + c], ks[k * (kDqk + 1) + c], x);
      }
      xs[r * (kKeysS + 1) + k] = x;
    }
    __syncthreads();
    if (tid < kRowsS) {
      float* x = xs + tid * (kKeysS + 1);
      float m = ms[tid], l = ms[kRowsS + tid];
      float mx = m;
      for (int k = 0; k < kKeysS; ++k) mx = fmaxf(mx, x[k]);
      const float mu = mx == -INFINITY ? 0.f : mx;
      const float f = exp2f(m - mu);
      l *= f;
      for (int k = 0; k < kKeysS; ++k) {
        x[k] = exp2f(x[k] - mu);
        l += x[k];
      }
      ms[tid] = mx, ms[kRowsS + tid] = l, ms[2 * kRowsS + tid] = f;
    }
    __syncthreads();
#pragma unroll 1
    for (int r = 0; r < kRowsS; ++r) {
#pragma unroll
      for (int j = 0; j < kDv / kThreadsS; ++j) {
        // (o is indexed statically per row below)
        const int c = tid + j * kThreadsS;
        float a = 0.f;
        for (int k = 0; k < kKeysS; ++k) {
          const float w = xs[r * (kKeysS + 1) + k];
          if (w != 0.f) a = fmaf(w, ks[k * (kDqk + 1) + c], a);  // a hidden row's contents do not matter
        }
#pragma unroll
        for (int q = 0; q < kRowsS; ++q)
          if (q == r) o[q * (kDv / kThreadsS) + j] = o[q * (kDv / kThreadsS) + j] * ms[2 * kRowsS + r] + a;
      }
    }
  }
  __syncthreads();
#pragma unroll
  for (int r = 0; r < kRowsS; ++r) {
    if (r0 + r >= rows) break;
    const float l = ms[kRowsS + r], inv = l > 0.f ? 1.f / l : l == l ? 0.f : l;
    const int64_t at = (int64_t)seq * rows + r0 + r;
#pragma unroll
    for (int j = 0; j < kDv / kThreadsS; ++j)
      p.out[at * kDv + tid + j * kThreadsS] = __float2bfloat16_rn(o[r * (kDv / kThreadsS) + j] * inv);
    if (tid == 0 && p.lse) p.lse[at] = l == 0.f ? -INFINITY : (ms[r] + log2f(l)) * kLn2;
  }
}

}  // namespace

size_t tree_attn_ws_bytes(const TreeAttnParams&) { return 0; }

cudaError_t launch_tree_attn(const TreeAttnParams& p, void* ws, cudaStream_t stream) {
  (void)ws;
  const int smem = (kRowsS * kDqk + kKeysS * (kDqk + 1) + kRowsS * (kKeysS + 1) + 3 * kRowsS) * 4;
  cudaError_t e = cudaFuncSetAttribute(tree_attn_simple_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  const dim3 grid((p.q_per_seq * p.H + kRowsS - 1) / kRowsS, p.n_seq);
  return launch_kernel(tree_attn_simple_kernel, grid, dim3(kThreadsS), smem, stream, false, p);
}

}  // namespace dsa
