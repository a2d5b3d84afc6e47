// sv_bulk.cuh -- mbarriers and one-dimensional bulk asynchronous copies (TMA)
// between global memory and the shared memory of a CTA.
#pragma once

#include <stdint.h>

namespace sv {

// ---------------------------------------------------------------------------
// mbarrier and bulk-copy primitives (shared memory of this CTA)
// ---------------------------------------------------------------------------
__device__ __forceinline__ unsigned smem_addr(const void* p) { return (unsigned)__cvta_generic_to_shared(p); }

__device__ __forceinline__ void mbar_init(unsigned long long* bar, unsigned count) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(smem_addr(bar)), "r"(count) : "memory");
}
__device__ __forceinline__ void mbar_arrive(unsigned long long* bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_addr(bar)) : "memory");
}
// arrive and add `bytes` to the transaction count the phase waits for
__device__ __forceinline__ void mbar_arrive_tx(unsigned long long* bar, unsigned bytes) {
  asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(smem_addr(bar)), "r"(bytes)
               : "memory");
}
// Has the phase with this parity completed?  Acquire: the completing arrivals
// and copies are visible afterwards.
__device__ __forceinline__ bool mbar_test(unsigned long long* bar, unsigned parity) {
  unsigned ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(smem_addr(bar)), "r"(parity)
      : "memory");
  return ok != 0;
}
// The same, but the thread is suspended while the phase is still open, until it
// completes or for about 4 us (no instructions issue meanwhile; a GB300 takes
// 3.9 to 4.0 us before it gives up on a phase that stays open, although the
// hint says 128 ns).
constexpr unsigned kSuspendNs = 128;
__device__ __forceinline__ bool mbar_try(unsigned long long* bar, unsigned parity) {
  unsigned ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(smem_addr(bar)), "r"(parity), "r"(kSuspendNs)
      : "memory");
  return ok != 0;
}
// Tries that last as long as `polls` polls of the other waits, which nap for
// 128 ns each (4 us = 32 of them): the limit on polls bounds the time of both.
__host__ __device__ constexpr unsigned mbar_tries(unsigned polls) { return polls / 32u; }
// One bulk copy global -> shared, completing `bytes` on the mbarrier.  Both
// addresses and the size are multiples of 16 bytes.
__device__ __forceinline__ void bulk_load(void* dst, const void* src, unsigned bytes, unsigned long long* bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
          smem_addr(dst)),
      "l"(src), "r"(bytes), "r"(smem_addr(bar))
      : "memory");
}
// Warp-uniform bounded wait: every lane looks, and the warp leaves together
// once all lanes have seen the phase; false after a look and `tries` tries
// (each suspends for at most about 4 us).
__device__ __forceinline__ bool warp_wait(unsigned long long* bar, unsigned parity, unsigned tries) {
  if (__all_sync(0xffffffffu, mbar_test(bar, parity))) return true;
  for (unsigned it = 0; it < tries; ++it)
    if (__all_sync(0xffffffffu, mbar_try(bar, parity))) return true;
  return false;
}

// This thread's generic writes to shared memory come before later bulk copies.
__device__ __forceinline__ void fence_async() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

// Asks the hardware for a CTA of this grid that has not started: it then never
// starts, and its index comes to `slot` (16 bytes on a 16-byte boundary of
// shared memory), completing 16 bytes on the mbarrier.
__device__ __forceinline__ void cta_request(void* slot, unsigned long long* bar) {
  mbar_arrive_tx(bar, 16u);
  asm volatile("clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128 [%0], [%1];" ::"r"(
                   smem_addr(slot)),
               "r"(smem_addr(bar))
               : "memory");
}
// The answer once it has come: blockIdx.x of that CTA, -1 when none is left
// (after which none may be asked for).
__device__ __forceinline__ int cta_answer(const void* slot) {
  int x;
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b128 r;\n\t.reg .b32 y, z, w;\n\t"
      "ld.shared.b128 r, [%1];\n\t"
      "mov.b32 %0, -1;\n\t"
      "clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, r;\n\t"
      "@p clusterlaunchcontrol.query_cancel.get_first_ctaid.v4.b32.b128 {%0, y, z, w}, r;\n\t}"
      : "=r"(x)
      : "r"(smem_addr(slot))
      : "memory");
  return x;
}

}  // namespace sv
