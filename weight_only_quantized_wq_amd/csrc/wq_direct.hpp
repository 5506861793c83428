// Direct loads from global memory to LDS (global_load_lds) and the waits for them.
#pragma once

#include <stdint.h>

#include <hip/hip_runtime.h>

namespace wq {

// Offset in LDS of a __shared__ object.
__device__ __forceinline__ uint32_t lds_offset(const void* p) {
  return (uint32_t)(uintptr_t)(const __attribute__((address_space(3))) void*)p;
}

// Lane l's 16 (4) bytes at `from` to LDS at `to` + 16 (4) l.  In assembly so that
// no wait is placed for it but those below; `to` is an operand in m0, so that the
// compiler itself writes that register (one wait state before its use).
__device__ __forceinline__ void request16(const void* from, uint32_t to) {
  asm volatile("s_nop 0\n\tglobal_load_lds_dwordx4 %1, off" ::"{m0}"(to), "v"(from) : "memory");
}
// The same from lane offsets to a uniform address, which scalar additions make: a
// vector write of `base` would need five wait states before the load (a test reads the
// listing for that; with them in place one token takes 12.4 us instead of 12.3, wide
// trees 103 instead of 102).
__device__ __forceinline__ void request16(const void* base, uint32_t off, uint32_t to) {
  asm volatile("s_nop 0\n\tglobal_load_lds_dwordx4 %1, %2" ::"{m0}"(to), "v"(off), "s"(base) : "memory");
}
__device__ __forceinline__ void request4(const void* from, uint32_t to) {
  asm volatile("s_nop 0\n\tglobal_load_lds_dword %1, off" ::"{m0}"(to), "v"(from) : "memory");
}
__device__ __forceinline__ void request4(const void* base, uint32_t off, uint32_t to) {
  asm volatile("s_nop 0\n\tglobal_load_lds_dword %1, %2" ::"{m0}"(to), "v"(off), "s"(base) : "memory");
}
// With the five wait states that a base written by a vector instruction (a value read
// off a lane) needs.
__device__ __forceinline__ void request16_late(const void* base, uint32_t off, uint32_t to) {
  asm volatile("s_nop 4\n\tglobal_load_lds_dwordx4 %1, %2" ::"{m0}"(to), "v"(off), "s"(base) : "memory");
}
__device__ __forceinline__ void request4_late(const void* base, uint32_t off, uint32_t to) {
  asm volatile("s_nop 4\n\tglobal_load_lds_dword %1, %2" ::"{m0}"(to), "v"(off), "s"(base) : "memory");
}
// All but the N newest requests of this wave are done, its LDS accesses too.
template <int N>
__device__ __forceinline__ void wait_requests() {
  asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" ::"n"(N) : "memory");
}
// LDS accesses of this wave are done: what they read may be overwritten.
__device__ __forceinline__ void wait_lds() { asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory"); }
__device__ __forceinline__ void meet() { asm volatile("s_barrier" ::: "memory"); }

}  // namespace wq
