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

// The LDS address of a shared object, in a scalar register.
__device__ __forceinline__ uint32_t lds_address(const void* p) {
  return __builtin_amdgcn_readfirstlane(static_cast<uint32_t>(reinterpret_cast<uintptr_t>(p)));
}

// 16 bytes per lane from each lane's own address to LDS address lds + 16 * lane
// (lds is wave-uniform and goes through M0).  Inline assembly, so that the
// compiler does not wait for every copy in flight before any LDS read; the
// callers wait with ring_wait() and a barrier.
__device__ __forceinline__ void copy16_to_lds(const void* g, uint32_t lds) {
#if defined(__HIP_DEVICE_COMPILE__)
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"
  asm volatile("s_mov_b32 m0, %1\n\tglobal_load_lds_dwordx4 %0, off" ::"v"(g), "s"(lds)
               : "memory", "m0");
#pragma clang diagnostic pop
#endif
}

// The same from a wave-uniform base plus each lane's own offset.
__device__ __forceinline__ void copy16_to_lds(const void* base, uint32_t off, uint32_t lds) {
#if defined(__HIP_DEVICE_COMPILE__)
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"
  asm volatile("s_mov_b32 m0, %2\n\tglobal_load_lds_dwordx4 %0, %1" ::"v"(off), "s"(base), "s"(lds)
               : "memory", "m0");
#pragma clang diagnostic pop
#endif
}

// A pointer that is the same in every lane, in scalar registers.
__device__ __forceinline__ const uint8_t* uniform_ptr(const uint8_t* p) {
  const uint64_t v = reinterpret_cast<uint64_t>(p);
  const uint32_t lo = __builtin_amdgcn_readfirstlane(static_cast<uint32_t>(v));
  const uint32_t hi = __builtin_amdgcn_readfirstlane(static_cast<uint32_t>(v >> 32));
  return reinterpret_cast<const uint8_t*>(static_cast<uint64_t>(hi) << 32 | lo);
}

// Wait until at most N of this wave's vector memory operations are in flight.
template <int N>
__device__ __forceinline__ void ring_wait() {
  static_assert(N >= 0 && N < 64, "vmcnt range");
  __builtin_amdgcn_s_waitcnt((N & 15) | (7 << 4) | (15 << 8) | ((N >> 4) << 14));
  asm volatile("" ::: "memory");
}

// Wait for this wave's LDS accesses.
__device__ __forceinline__ void lds_wait() {
  __builtin_amdgcn_s_waitcnt(0xC07F);  // lgkmcnt(0)
  asm volatile("" ::: "memory");
}

}  // namespace moe
