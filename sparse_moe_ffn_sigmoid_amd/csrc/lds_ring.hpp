// Copies from global memory straight into LDS, the waits and the barrier that
// order them.
#pragma once

#include "common.hpp"

namespace moe {

// A block barrier that the compiler moves no memory access across, without the
// wait for loads in flight that __syncthreads() brings.
__device__ __forceinline__ void ring_barrier() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

// 16 bytes per lane from each lane's own address to lds + 16 * lane (the base
// is wave-uniform and goes through M0).  Inline assembly, so that the compiler
// does not wait for every copy in flight before any LDS read; the callers wait
// with ring_wait() and a barrier.
__device__ __forceinline__ void copy16_to_lds(const void* g, void* lds) {
#if defined(__HIP_DEVICE_COMPILE__)
  const uint32_t m =
      __builtin_amdgcn_readfirstlane(static_cast<uint32_t>(reinterpret_cast<uintptr_t>(lds)));
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"
  asm volatile("s_mov_b32 m0, %1\n\tglobal_load_lds_dwordx4 %0, off" ::"v"(g), "s"(m)
               : "memory", "m0");
#pragma clang diagnostic pop
#endif
}

// Wait until at most N of this wave's vector memory operations are in flight.
template <int N>
__device__ __forceinline__ void ring_wait() {
  static_assert(N >= 0 && N < 64, "vmcnt range");
  __builtin_amdgcn_s_waitcnt((N & 15) | (7 << 4) | (15 << 8) | ((N >> 4) << 14));
  asm volatile("" ::: "memory");
}

}  // namespace moe
