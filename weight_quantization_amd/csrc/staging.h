// staging.h — loads from memory straight to LDS, with the waits that the compiler,
// which does not see them, cannot add.
#pragma once

#include "kv_common.h"

namespace hlwq_kv {

// A buffer resource over `bytes` bytes at p (uniform): reads past them give 0.
__device__ __forceinline__ u32x4 buffer_of(const void* p, int64_t bytes) {
  const uint64_t u = reinterpret_cast<uint64_t>(p);
  return u32x4{static_cast<uint32_t>(__builtin_amdgcn_readfirstlane(static_cast<uint32_t>(u))),
               static_cast<uint32_t>(__builtin_amdgcn_readfirstlane(static_cast<uint32_t>(u >> 32) & 0xffffu)),
               static_cast<uint32_t>(__builtin_amdgcn_readfirstlane(static_cast<uint32_t>(min(bytes, int64_t{0x7fffffff})))),
               0x00020000u};
}

// 16 bytes a lane from memory straight to LDS: lane l's land at lds + 16 l.
// The compiler does not see these loads; a wait on the vector-memory counter
// stands before the barrier that publishes them (wait_staged).  M0, which
// holds the LDS address, is used by nothing else in these kernels.  (Nor does it
// see what the load reads: five wait states after a VALU write of the buffer's
// scalar registers, one after M0's, are the block's own.)
__device__ __forceinline__ void stage16(u32x4 buffer, uint32_t offset, uint32_t lds) {
  lds = __builtin_amdgcn_readfirstlane(lds);
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 3\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds" ::"s"(lds), "v"(offset), "s"(buffer)
               : "memory");
}
__device__ __forceinline__ void stage16(const void* p, uint32_t lds) {
  lds = __builtin_amdgcn_readfirstlane(lds);
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, off" ::"s"(lds), "v"(p) : "memory");
}
__device__ __forceinline__ void stage4(u32x4 buffer, uint32_t offset, uint32_t lds) {
  lds = __builtin_amdgcn_readfirstlane(lds);
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 3\n\tbuffer_load_dword %1, %2, 0 offen lds" ::"s"(lds), "v"(offset), "s"(buffer)
               : "memory");
}
// 4 bytes, or 2 and two of zeroes: lane l's land at lds + 4 l.
__device__ __forceinline__ void stage4(const void* p, uint32_t lds) {
  lds = __builtin_amdgcn_readfirstlane(lds);
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dword %1, off" ::"s"(lds), "v"(p) : "memory");
}
__device__ __forceinline__ void stage2(const void* p, uint32_t lds) {
  lds = __builtin_amdgcn_readfirstlane(lds);
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_ushort %1, off" ::"s"(lds), "v"(p) : "memory");
}
__device__ __forceinline__ void wait_staged() { asm volatile("s_waitcnt vmcnt(0)" ::: "memory"); }
__device__ __forceinline__ void wait_lds() { asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory"); }
__device__ __forceinline__ void barrier() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

template <class T>
__device__ __forceinline__ T lds_at(uint32_t at) {
  return *reinterpret_cast<const __attribute__((address_space(3))) T*>(static_cast<uintptr_t>(at));
}
template <class T>
__device__ __forceinline__ void lds_put(uint32_t at, T v) {
  *reinterpret_cast<__attribute__((address_space(3))) T*>(static_cast<uintptr_t>(at)) = v;
}

}  // namespace hlwq_kv
