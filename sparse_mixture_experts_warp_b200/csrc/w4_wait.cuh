// Barrier steps of the 4-bit products' kernels (inline PTX, sm_100a), on shared-memory addresses.
#pragma once

#include <cuda.h>
#include <stdint.h>

#include "mbar.cuh"
#include "tc_ops.cuh"

namespace moe {

constexpr uint64_t kWaitNs = 2000000000ull;     // 2 s per wait
constexpr uint64_t kDrainNs = 200000000ull;     // 0.2 s to drain after an abort
constexpr unsigned kFullWarp = 0xffffffffu;

// Every role runs as a whole warp with one elected lane issuing, and waits are inline and taken by
// all lanes together: no call and no divergence stands between a role's loop counters and the
// uniform registers that its descriptors come from.
__device__ __forceinline__ bool bar_try(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0;
}
struct BarWait {
  volatile int* abort_flag;
  int* err;
  // Whole warp; false when it gave up: after its time limit (which records `code` and raises the
  // CTA's abort flag) or, with kHonor, once another role has.
  template <bool kHonor = true>
  __device__ __forceinline__ bool operator()(uint32_t bar, uint32_t parity, int code,
                                             uint64_t limit = kWaitNs) const {
    if (__all_sync(kFullWarp, bar_try(bar, parity))) return true;
    const uint64_t t0 = gtimer();
#pragma unroll 1
    while (!__all_sync(kFullWarp, bar_try(bar, parity))) {
      if (kHonor && __any_sync(kFullWarp, *abort_flag)) return false;
      if (__any_sync(kFullWarp, gtimer() - t0 > limit)) {
        *abort_flag = 1;
        atomicCAS(err, 0, code);
        return false;
      }
    }
    return true;
  }
  // Copies or MMAs in flight, before the CTA exits.
  __device__ __forceinline__ void drain(uint32_t bar, uint32_t parity, int code,
                                        uint64_t limit) const {
    (void)operator()<false>(bar, parity, code, limit);
  }
};
__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(r));
  return r != 0;
}
__device__ __forceinline__ void bar_arrive(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void bar_expect(uint32_t bar, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes)
               : "memory");
}
__device__ __forceinline__ void bar_commit(uint32_t bar) {
  asm volatile(
      "tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar)
      : "memory");
}
__device__ __forceinline__ void bar_load(uint32_t dst, const CUtensorMap* map, uint32_t bar, int x,
                                         int y) {
  tma_load_2d(dst, map, static_cast<uint64_t*>(__cvta_shared_to_generic(bar)), x, y);
}

__device__ __forceinline__ void bar_load_3d(uint32_t dst, const CUtensorMap* map, uint32_t bar,
                                            int x, int y, int z) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(x), "r"(y), "r"(z)
      : "memory");
}

}  // namespace moe
