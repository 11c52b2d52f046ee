// Loads from memory to LDS without registers between, and their waits.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "device_common.hpp"

namespace arcs {

typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));

#define ARCS_LDS __attribute__((address_space(3)))

constexpr uint32_t kNoLoad = 0x80000000u;       // an offset past every buffer: the load gives zeros
constexpr uint32_t kBufMost = 0x7FFFFFF0u;

// A buffer descriptor of `bytes` bytes from p (raw, bounds checked).
__device__ __forceinline__ u32x4 buffer_of(const void* p, int64_t bytes) {
  const uint64_t b = (uint64_t)p;
  u32x4 d;
  d[0] = (uint32_t)b;
  d[1] = (uint32_t)(b >> 32) & 0xFFFFu;
  d[2] = bytes < 0 ? 0u : bytes > (int64_t)kBufMost ? kBufMost : (uint32_t)bytes;
  d[3] = 0x00020000u;
  return d;
}

// 16 bytes a lane from descriptor + offset to LDS at `to` + 16 * lane.  The
// wait is the caller's (vmcnt).  m0 takes one wait state, a descriptor that a
// vector instruction has just written five: the first load of a descriptor has them.
template <bool FIRST = true>
__device__ __forceinline__ void load_to_lds(uint32_t to, uint32_t off, u32x4 from) {
  to = __builtin_amdgcn_readfirstlane(to);
  if (FIRST)
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 4\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds" ::"s"(to), "v"(off), "s"(from)
                 : "memory", "m0");
  else
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds" ::"s"(to), "v"(off), "s"(from)
                 : "memory", "m0");
}

template <int N>
__device__ __forceinline__ void wait_loads() {
  asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
}
__device__ __forceinline__ void wait_lds() { asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory"); }

}  // namespace arcs
