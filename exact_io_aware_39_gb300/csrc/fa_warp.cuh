// Bounded waits of little code and warp-wide copy steps, for the kernels over
// packed sequences and paged caches.
#pragma once

#include "fa_ptx.cuh"

namespace fa {

// Bounded waits of little code: these kernels wait at some thirty places, and
// one that inlines the report of a timeout at each of them no longer fits the
// instruction cache. A wait that runs out leaves its site in the abort word;
// report_aborted, once at the end of the kernel, records it.
__device__ __forceinline__ bool bar_wait(uint32_t bar, uint32_t parity, const Ctl& c, uint32_t site) {
  if (mbar_try(bar, parity)) return true;
  const uint64_t t0 = globaltimer();
  do {
    if (mbar_try(bar, parity)) return true;
    if (globaltimer() - t0 > 1000ull * c.abort[2] && *c.abort == 0u) *c.abort = site;
  } while (*c.abort == 0u);
  return false;
}
__device__ __forceinline__ bool bar_wait_warp(uint32_t bar, uint32_t parity, const Ctl& c, uint32_t site) {
  const bool ok = bar_wait(bar, parity, c, site);
  return __all_sync(0xFFFFFFFFu, ok);
}
// by one thread that has seen a wait fail, or behind a barrier of the whole CTA
__device__ __forceinline__ void report_aborted(const Ctl& c) {
  const uint32_t site = *c.abort;
  if (site != 0u) report_error(c, kErrTimeout, site);
}

// Warp-wide forms of the producers' steps (as for the MMAs: every lane runs the
// call, elect.sync picks the one that issues), so that the producers run without
// a lane-dependent branch and their operands stay in uniform registers.
__device__ __forceinline__ void tma_load_3d_w(uint32_t dst, const CUtensorMap* m, uint32_t bar, int c0, int c1, int c2) {
  asm volatile(
      "{\n\t.reg .pred e;\n\t"
      "elect.sync _|e, 0xffffffff;\n\t"
      "@e cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5}], [%2];\n\t}"
      :: "r"(dst), "l"(reinterpret_cast<uint64_t>(m)), "r"(bar), "r"(c0), "r"(c1), "r"(c2) : "memory");
}
__device__ __forceinline__ void mbar_arrive_expect_tx_w(uint32_t bar, uint32_t bytes) {
  asm volatile(
      "{\n\t.reg .pred e;\n\t"
      "elect.sync _|e, 0xffffffff;\n\t"
      "@e mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;\n\t}"
      :: "r"(bar), "r"(bytes) : "memory");
}
__device__ __forceinline__ void bulk_load_w(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
  asm volatile(
      "{\n\t.reg .pred e;\n\t"
      "elect.sync _|e, 0xffffffff;\n\t"
      "@e cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];\n\t}"
      :: "r"(dst), "l"(reinterpret_cast<uint64_t>(src)), "r"(bytes), "r"(bar) : "memory");
}
// Brings a tile box into L2 (same coordinates as the load).
__device__ __forceinline__ void tma_prefetch_3d_w(const CUtensorMap* m, int c0, int c1, int c2) {
  asm volatile(
      "{\n\t.reg .pred e;\n\t"
      "elect.sync _|e, 0xffffffff;\n\t"
      "@e cp.async.bulk.prefetch.tensor.3d.L2.global.tile [%0, {%1, %2, %3}];\n\t}"
      :: "l"(reinterpret_cast<uint64_t>(m)), "r"(c0), "r"(c1), "r"(c2) : "memory");
}

}  // namespace fa
