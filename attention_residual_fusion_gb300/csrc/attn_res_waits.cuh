// attn_res_waits.cuh -- the bounded waits of the microscaled and 8-bit kernels.
#pragma once

#include "attn_res_common.cuh"

namespace attn_res_dev {

// The bounded waits of these kernels: as wait_or_flag, with the clock (whose
// reading takes longer than a stage's wait) looked at only from the 256th try
// on.  PEERS: the barrier is arrived on by other CTAs of the cluster too.
template <bool PEERS = false>
__device__ __forceinline__ bool phase_done(uint32_t bar, uint32_t parity) {
  if constexpr (!PEERS) return mbar_try_wait(bar, parity);
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0;
}
template <bool PEERS = false>
__device__ __forceinline__ bool phase_wait(uint32_t bar, uint32_t parity, uint64_t limit_ns = kWaitLimitNs) {
  uint64_t t0 = 0;
  for (uint32_t it = 1;; ++it) {
    if (phase_done<PEERS>(bar, parity)) return true;
    if ((it & 255u) == 0) {
      const uint64_t now = global_timer_ns();
      if (t0 == 0) t0 = now;
      if (now - t0 > limit_ns) return false;
    }
  }
}
template <bool PEERS = false>
__device__ __forceinline__ void phase_or_flag(uint32_t bar, uint32_t parity, bool& failed, unsigned* err,
                                              unsigned bit, uint64_t limit_ns = kWaitLimitNs) {
  if (failed || phase_wait<PEERS>(bar, parity, limit_ns)) return;
  failed = true;
  atomicOr(err, bit);
}

}  // namespace attn_res_dev
