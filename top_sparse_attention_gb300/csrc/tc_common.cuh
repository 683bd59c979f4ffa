// What the attention kernels on tcgen05 share (tree_kernel.cuh, expanded_attn.cu; expand.cu takes parts): bounded waits of roles, packed fp32
// arithmetic, matrix instructions by 32-bit descriptor words, copies to tensor memory.
#pragma once

#include <limits.h>

#include "dsa_internal.h"

namespace dsa {
namespace {

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
template <int SLEEP, class Aux>
__device__ __noinline__ bool wait_slow(Aux* a, uint64_t* bar, uint32_t parity, int* err);
template <class Aux>
__device__ __forceinline__ bool wait(Aux* a, uint64_t* bar, uint32_t parity, int* err) {
  return mbar_test(bar, parity) || wait_slow<0>(a, bar, parity, err);
}
// The same for the roles that run ahead of the others (producer, scale loader, converters): they look again after 50
// ns, since warps that poll take issue slots from the others (8 x 64 nodes at 32K, E4M3 rows: 603 -> 590 us).
template <class Aux>
__device__ __forceinline__ bool wait_ahead(Aux* a, uint64_t* bar, uint32_t parity, int* err) {
  return mbar_test(bar, parity) || wait_slow<50>(a, bar, parity, err);
}
template <int SLEEP, class Aux>
__device__ __forceinline__ bool wait_loop(Aux* a, uint64_t* bar, uint32_t parity, int* err) {
  const unsigned long long t0 = globaltimer_ns();
  for (uint32_t i = 0;; ++i) {
    if (mbar_try_wait(bar, parity)) return true;
    if (SLEEP) __nanosleep(SLEEP);
    if ((i & 15u) != 15u) continue;
    if (*reinterpret_cast<volatile int*>(&a->abort)) return false;
    if (globaltimer_ns() - t0 > kWaitLimitNs) {
      record_error(err, DSA_DEVERR_WAIT_TIMEOUT);
      *reinterpret_cast<volatile int*>(&a->abort) = 1;
      return false;
    }
  }
}

template <int SLEEP, class Aux>
__device__ __noinline__ bool wait_slow(Aux* a, uint64_t* bar, uint32_t parity, int* err) {
  return wait_loop<SLEEP>(a, bar, parity, err);
}
// The same without a call, for kernels that move registers between their warps (a called function would need the
// registers that a caller may not have).
template <int SLEEP = 0, class Aux>
__device__ __forceinline__ bool wait_here(Aux* a, uint64_t* bar, uint32_t parity, int* err) {
  return mbar_test(bar, parity) || wait_loop<SLEEP>(a, bar, parity, err);
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

// Two fp32 operations per instruction.  (8 x 64 nodes at 32K, E4M3 rows with row scales: 625 -> 597 us; with tile
// scales, where the waits between the accumulations bind, they measured slower, 196 against 185 us, and are not used.)
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  float2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(reinterpret_cast<uint64_t&>(r)) : "l"(reinterpret_cast<uint64_t&>(a)), "l"(reinterpret_cast<uint64_t&>(b)));
  return r;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(reinterpret_cast<uint64_t&>(r)) : "l"(reinterpret_cast<uint64_t&>(a)), "l"(reinterpret_cast<uint64_t&>(b)));
  return r;
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 b = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&b);
}

// Low words of shared-memory descriptors with 128-byte swizzle (the upper word, kDescHi, holds the 1024-byte
// stride, the version and the swizzle): K-major operands, and MN-major ones whose 64-element atoms are one
// box (of `box` bytes) apart.  Adding bytes / 16 moves the start address.  Boxes of codes have rows of 64 bytes, with 64-byte
// swizzle (kDescHi64: 8 rows are 512 bytes; 16-byte chunk c of row r lies at chunk c ^ (r / 2 % 4)).
constexpr uint32_t kDescHi = (1024u >> 4) | (1u << 14) | (2u << 29);
constexpr uint32_t kDescHi64 = (512u >> 4) | (1u << 14) | (4u << 29);
__device__ __forceinline__ uint32_t kmajor_lo(uint32_t saddr) { return ((saddr & 0x3FFFFu) >> 4) | (1u << 16); }
__device__ __forceinline__ uint32_t mnmajor_lo(uint32_t saddr, int box) {
  return ((saddr & 0x3FFFFu) >> 4) | ((uint32_t)(box >> 4) << 16);
}

// D += A B^T with A in shared memory, or in tensor memory (lane = row, two bf16 or four 8-bit elements per
// column); F8: 8-bit operands, B's rows 64 bytes.
template <bool F8 = false>
__device__ __forceinline__ void mma_ss(uint32_t d, uint32_t a_lo, uint32_t b_lo, uint32_t idesc, uint32_t acc) {
  if constexpr (F8)
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 da, db;\n\t"
        "mov.b64 da, {%1, %5};\n\t"
        "mov.b64 db, {%2, %6};\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], da, db, %3, p;\n\t}" ::"r"(d),
        "r"(a_lo), "r"(b_lo), "r"(idesc), "r"(acc), "r"(kDescHi), "r"(kDescHi64)
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 da, db;\n\t"
        "mov.b64 da, {%1, %5};\n\t"
        "mov.b64 db, {%2, %5};\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %3, p;\n\t}" ::"r"(d),
        "r"(a_lo), "r"(b_lo), "r"(idesc), "r"(acc), "r"(kDescHi)
        : "memory");
}
template <bool F8 = false>
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a_tmem, uint32_t b_lo, uint32_t idesc, uint32_t acc) {
  if constexpr (F8)
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 db;\n\t"
        "mov.b64 db, {%2, %5};\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], [%1], db, %3, p;\n\t}" ::"r"(d),
        "r"(a_tmem), "r"(b_lo), "r"(idesc), "r"(acc), "r"(kDescHi64)
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 db;\n\t"
        "mov.b64 db, {%2, %5};\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], db, %3, p;\n\t}" ::"r"(d),
        "r"(a_tmem), "r"(b_lo), "r"(idesc), "r"(acc), "r"(kDescHi)
        : "memory");
}

// `bytes` (a multiple of 16) on their way to L2.
__device__ __forceinline__ void prefetch_l2(const void* p, uint32_t bytes) {
  asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(p), "r"(bytes) : "memory");
}
__device__ __forceinline__ void tma_prefetch_3d(const CUtensorMap* tm, int x, int y, int z) {
  asm volatile("cp.async.bulk.prefetch.tensor.3d.L2.global.tile [%0, {%1, %2, %3}];" ::"l"(tm), "r"(x), "r"(y), "r"(z)
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

// Tensor memory -> registers in two parts, so that the latency of a load can be spent on the values before it: `issue`
// starts a load of 32 columns, `wait` ends all loads in flight.  `v` may be used after a wait that names it.
__device__ __forceinline__ void tmem_ld_issue(uint32_t taddr, float (&v)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, "
      "%12, %13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, "
      "%30, %31}, [%32];"
      : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7]), "=f"(v[8]), "=f"(v[9]),
        "=f"(v[10]), "=f"(v[11]), "=f"(v[12]), "=f"(v[13]), "=f"(v[14]), "=f"(v[15]), "=f"(v[16]), "=f"(v[17]), "=f"(v[18]),
        "=f"(v[19]), "=f"(v[20]), "=f"(v[21]), "=f"(v[22]), "=f"(v[23]), "=f"(v[24]), "=f"(v[25]), "=f"(v[26]), "=f"(v[27]),
        "=f"(v[28]), "=f"(v[29]), "=f"(v[30]), "=f"(v[31])
      : "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tmem_ld_wait(float (&v)[32]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+f"(v[0]), "+f"(v[1]), "+f"(v[2]), "+f"(v[3]), "+f"(v[4]), "+f"(v[5]), "+f"(v[6]), "+f"(v[7]), "+f"(v[8]), "+f"(v[9]),
                 "+f"(v[10]), "+f"(v[11]), "+f"(v[12]), "+f"(v[13]), "+f"(v[14]), "+f"(v[15]), "+f"(v[16]), "+f"(v[17]), "+f"(v[18]),
                 "+f"(v[19]), "+f"(v[20]), "+f"(v[21]), "+f"(v[22]), "+f"(v[23]), "+f"(v[24]), "+f"(v[25]), "+f"(v[26]), "+f"(v[27]),
                 "+f"(v[28]), "+f"(v[29]), "+f"(v[30]), "+f"(v[31])
               :
               : "memory");
}

}  // namespace
}  // namespace dsa
