// Issuing tensor-core products from a converged warp, and loads with a cache policy.
#pragma once

#include "tc_common.cuh"

namespace llatte {
namespace tc {

// One lane of a converged warp, and a wait that the warp agrees on.
__device__ __forceinline__ bool elect_one() {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok));
  return ok != 0;
}
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity,
                                          volatile int* abort_flag, int32_t* status,
                                          uint64_t limit_ns = kWaitTimeoutNs) {
  return __all_sync(0xffffffffu, mbar_wait(bar, parity, abort_flag, status, limit_ns));
}
// Limit of the wait that an injected timeout makes run out.
constexpr uint64_t kInjectTimeoutNs = 20000;

// tma_load_2d whose lines are the first to leave L2 when they are read only once in a
// call: they would push out everything else, the kernel's own code included.
__device__ __forceinline__ uint64_t policy_stream(bool once) {
  uint64_t p;
  if (once) asm volatile("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(p));
  else asm volatile("createpolicy.fractional.L2::evict_normal.b64 %0, 1.0;" : "=l"(p));
  return p;
}
__device__ __forceinline__ void tma_load_2d_hint(const CUtensorMap* map, uint64_t* bar, void* smem,
                                                 int32_t x, int32_t y, uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint"
      " [%0], [%1, {%3, %4}], [%2], %5;" ::"r"(smem_u32(smem)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(x), "r"(y), "l"(policy)
      : "memory");
}

}  // namespace tc
}  // namespace llatte
