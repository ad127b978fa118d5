// tensor.cuh -- what the kernels on the tensor cores (tcgen05) share: operand
// descriptors, and waits on barriers that end when a block gives up.
#pragma once

#include "tma.cuh"

namespace echo {

__device__ __forceinline__ uint64_t smem_desc(uint32_t addr) {
  // K-major, 128-byte swizzle: rows of 128 bytes in groups of eight, 1024 bytes apart
  return (uint64_t)((addr >> 4) & 0x3FFF) | (1ull << 16) | (64ull << 32) | (1ull << 46) | (2ull << 61);
}

__device__ __forceinline__ bool wait_on(uint32_t bar, uint32_t parity, volatile int* give_up) {
  uint64_t began = 0;
  for (;;) {
    uint32_t done;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(done) : "r"(bar), "r"(parity) : "memory");
    if (done) return true;
    if (*give_up) return false;
    const uint64_t t = global_ns();
    if (began == 0) began = t;
    else if (t - began > kWaitLimitNs) {
      *give_up = 1;
      return false;
    }
  }
}

// Arrives on a barrier of this block.
__device__ __forceinline__ void arrive_here(uint32_t bar) {
  asm volatile("mbarrier.arrive.release.cta.shared::cta.b64 _, [%0];" :: "r"(bar) : "memory");
}

__device__ __forceinline__ bool elect_one() {
  uint32_t is;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xFFFFFFFF;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(is));
  return is != 0;
}

}  // namespace echo
