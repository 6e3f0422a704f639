// Loads from global memory straight into LDS.
#pragma once

#include "common.h"

namespace staple {

// 16-byte-per-lane global -> LDS load (lane l writes LDS bytes [dst + 16 l,
// +16), dst wave-uniform, passed in M0).  Issued from inline asm, like the
// loads of gemm.hip and for their reason: the compiler would wait for every
// outstanding LDS read while it knew of one.  No register outputs; completion
// is waited for by hand (vmcnt) before the barrier that publishes the data.
__device__ __forceinline__ void dma16(const void* src, lds_void* dst) {
  const uint32_t m0 = __builtin_amdgcn_readfirstlane(static_cast<uint32_t>(reinterpret_cast<uintptr_t>(dst)));
  asm volatile("s_nop 0\n\tglobal_load_lds_dwordx4 %0, off" ::"v"(src), "{m0}"(m0) : "memory");
}

// The same load through a buffer descriptor: the lane reads 16 bytes at
// `offset` of the buffer, zeros where that is past its end.  The compiler does
// not look into the asm, and a scalar register that a vector instruction has
// written (a descriptor word that was spilled to a lane and read back) may be
// read by a memory instruction only five wait states later: hence s_nop 4.
__device__ __forceinline__ void dma16(const u32x4_t& buffer, uint32_t offset, lds_void* dst) {
  const uint32_t m0 = __builtin_amdgcn_readfirstlane(static_cast<uint32_t>(reinterpret_cast<uintptr_t>(dst)));
  asm volatile("s_nop 4\n\tbuffer_load_dwordx4 %0, %1, 0 offen lds" ::"v"(offset), "s"(buffer), "{m0}"(m0) : "memory");
}
// Descriptor of `bytes` bytes at `base` (both uniform over the wave): no
// stride, no swizzle, 32-bit data format.
__device__ __forceinline__ u32x4_t make_buffer(const void* base, uint32_t bytes) {
  const uint64_t a = reinterpret_cast<uint64_t>(base);
  return u32x4_t{static_cast<uint32_t>(__builtin_amdgcn_readfirstlane(static_cast<uint32_t>(a))),
                 static_cast<uint32_t>(__builtin_amdgcn_readfirstlane(static_cast<uint32_t>(a >> 32) & 0xffffu)),
                 static_cast<uint32_t>(__builtin_amdgcn_readfirstlane(bytes)), 0x00027000u};
}

// One 4-byte-per-lane global -> LDS load (lane l writes LDS bytes [dst + 4 l, +4)).
__device__ __forceinline__ void dma4(const void* src, lds_void* dst) {
  const uint32_t m0 = __builtin_amdgcn_readfirstlane(static_cast<uint32_t>(reinterpret_cast<uintptr_t>(dst)));
  asm volatile("s_nop 0\n\tglobal_load_lds_dword %0, off" ::"v"(src), "{m0}"(m0) : "memory");
}

}  // namespace staple
