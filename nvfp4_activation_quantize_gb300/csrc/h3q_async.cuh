// h3q_async.cuh -- mbarriers and bulk copies (sm_100+ asynchronous copies into
// shared memory), shared by the kernels that stage their inputs with them.
//
// Every wait in the library's kernels is bounded in time: wait_or_abort gives up
// after kWaitNs of the global timer, so a copy that never lands cannot keep a
// kernel (and the GPU) waiting forever; the caller decides what to do then.
// wait_bounded is for what is under way when a role has given up, and has its own limit.
//
// A test compiles the attention kernels with H3Q_SHORT_WAITS, a limit in nanoseconds that ordinary
// waits pass (polls do not suspend then, and each looks at the clock), to see what they leave.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

namespace h3q {

constexpr uint64_t kDrainNs = 2000000000ull;  // 2 s
#ifdef H3Q_SHORT_WAITS
constexpr uint64_t kWaitNs = H3Q_SHORT_WAITS;
constexpr uint32_t kPolls = 1;
#define H3Q_POLL "mbarrier.test_wait"
#else
constexpr uint64_t kWaitNs = 2000000000ull;
constexpr uint32_t kPolls = 256;              // between two looks at the clock (a power of two)
#define H3Q_POLL "mbarrier.try_wait"
#endif

__device__ __forceinline__ uint32_t smem_u32(const void* p) {
  return static_cast<uint32_t>(__cvta_generic_to_shared(p));
}

__device__ __forceinline__ void mbar_init(uint32_t bar, uint32_t count) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(count) : "memory");
}

// Makes mbarrier initialisations visible to the asynchronous proxy (the copy
// engine) and to the other CTAs of a cluster; call before the barrier that
// precedes the first copy.
__device__ __forceinline__ void mbar_init_fence() {
  asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
}

__device__ __forceinline__ void mbar_expect_tx(uint32_t bar, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes)
               : "memory");
}

__device__ __forceinline__ void mbar_arrive(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}

__device__ __forceinline__ bool mbar_try_wait(uint32_t bar, uint32_t parity) {
  uint32_t done;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      H3Q_POLL ".parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(done)
      : "r"(bar), "r"(parity)
      : "memory");
  return done != 0;
}

__device__ __forceinline__ uint64_t now_ns() {
  uint64_t t;
  asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
  return t;
}

// Wait for the phase of parity `parity` of the barrier to complete; false if
// kDrainNs went by first.
// The timer is read only once the first poll has failed: reading it costs more
// than a poll, and most waits find the phase complete.
__device__ __forceinline__ bool wait_bounded(uint32_t bar, uint32_t parity) {
  if (mbar_try_wait(bar, parity)) return true;
  const uint64_t start = now_ns();
  for (uint32_t i = 1; !mbar_try_wait(bar, parity); ++i)
    if ((i & 255u) == 0 && now_ns() - start > kDrainNs) return false;
  return true;
}

// The same for a role among others of a CTA: gives up too when another has raised *abort; one
// that runs out of time raises it, and *fault.
__device__ __forceinline__ bool wait_or_abort(uint32_t bar, uint32_t parity, volatile int* abort, int* fault) {
  if (mbar_try_wait(bar, parity)) return true;
  const uint64_t start = now_ns();
  for (uint32_t i = 1;; ++i) {
    if (mbar_try_wait(bar, parity)) return true;
    if ((i & (kPolls - 1)) == 0) {
      if (*abort) return false;
      if (now_ns() - start >= kWaitNs) break;
    }
  }
  *abort = 1;
  atomicExch(fault, 1);
  return false;
}

// 1-D bulk copy of `bytes` (a multiple of 16; both addresses 16-byte aligned)
// from global to shared memory, completing on the barrier.
__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
      "l"(src), "r"(bytes), "r"(bar)
      : "memory");
}

}  // namespace h3q
