// Asynchronous page copies (cp.async.bulk tracked by mbarriers with bounded waits), packed fp32
// pairs and arrival counters, shared by the kernels that attend over the paged cache.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace kvq {

constexpr uint32_t kSpinLimit = 1u << 22;

__device__ __forceinline__ uint32_t smem_u32(const void* p) { return (uint32_t)__cvta_generic_to_shared(p); }

__device__ __forceinline__ void mbar_init(uint64_t* bar, uint32_t count) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(smem_u32(bar)), "r"(count) : "memory");
}
__device__ __forceinline__ void mbar_expect_tx(uint64_t* bar, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(smem_u32(bar)), "r"(bytes) : "memory");
}
__device__ __forceinline__ void mbar_arrive(uint64_t* bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_u32(bar)) : "memory");
}
__device__ __forceinline__ void bulk_g2s(void* dst, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                   smem_u32(dst)),
               "l"(src), "r"(bytes), "r"(smem_u32(bar))
               : "memory");
}
// Bounded wait on an mbarrier phase: false if the phase did not complete within `limit` tries.
__device__ __forceinline__ bool mbar_wait(uint64_t* bar, uint32_t phase, uint32_t limit = kSpinLimit) {
  const uint32_t addr = smem_u32(bar);
  for (uint32_t it = 0; it < limit; ++it) {
    uint32_t ok;
    asm volatile(
        "{\n .reg .pred p;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n selp.u32 %0, 1, 0, p;\n}\n"
        : "=r"(ok)
        : "r"(addr), "r"(phase)
        : "memory");
    if (ok) return true;
  }
  return false;
}

// The arrival counters of a workspace: its first kCounterBytes, zero between calls.  No call keeps anything else there,
// whatever the shape, so that one workspace serves calls of different shapes in turn.  1, 2, 4 or 8 groups share a word (2 to
// the power returned here), for up to 64, 128, 256 and 512 groups; more have no counters (-1).
constexpr int kCounterBytes = 256;
inline int counter_sharing(int64_t groups) { return groups <= 64 ? 0 : groups <= 128 ? 1 : groups <= 256 ? 2 : groups <= 512 ? 3 : -1; }
inline int64_t most_arrivals(int sharing) { return sharing < 0 ? 1 : (INT64_C(1) << (32 >> sharing)) - 1; }
// One arrival of the n <= most_arrivals of group grp: true for the last, which leaves the counter at zero.
__device__ __forceinline__ bool arrive_last(unsigned* counters, int grp, int sharing, unsigned n) {
  const int bits = 32 >> sharing, shift = (grp & ((1 << sharing) - 1)) * bits;
  unsigned* word = counters + (grp >> sharing);
  const bool last = (atomicAdd(word, 1u << shift) >> shift & (0xffffffffu >> (32 - bits))) == n - 1u;
  if (last) atomicSub(word, n << shift);
  return last;
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Packed fp32 pairs (sm_100a f32x2 instructions).
__device__ __forceinline__ unsigned long long pk(float a, float b) {
  unsigned long long r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ void upk(unsigned long long r, float& a, float& b) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(r));
}
__device__ __forceinline__ unsigned long long mul2(unsigned long long a, unsigned long long b) {
  unsigned long long r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ unsigned long long add2(unsigned long long a, unsigned long long b) {
  unsigned long long r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ unsigned long long fma2(unsigned long long a, unsigned long long b, unsigned long long c) {
  unsigned long long r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}

}  // namespace kvq
