// Loads from global memory straight to LDS (gfx950), shared by the kernels that
// stage their tiles with them.
#ifndef SSMSCAN_LDS_LOAD_H
#define SSMSCAN_LDS_LOAD_H

#include "device.h"

namespace ssm {
namespace {

// A wavefront's load of 64 x 16 bytes to LDS: lane l's come from base + off and go
// to `to` + 16 l.  (Of lanes that are off, nothing is written.)  Completion is the
// wavefront's to wait for: loaded<0>(), then a barrier.  Written as an
// instruction: of the compiler's own form every later LDS read waits, which
// would serialise a chunk's loads with the arithmetic of the one before.
__device__ __forceinline__ void load_lds(const char* base, uint32_t off, void* to) {
  const uint32_t lds = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) char*)static_cast<char*>(to);
  asm volatile(
      "s_mov_b32 m0, %0\n\t"
      "s_nop 0\n\t"
      "global_load_lds_dwordx4 %1, %2"
      :
      : "s"(__builtin_amdgcn_readfirstlane(lds)), "v"(off), "s"(base)
      : "memory");   // (m0 is a scratch register: whoever needs it sets it)
}
// The same through a buffer descriptor: lane l's 16 bytes come from byte `off` of the
// buffer, and a lane whose offset lies past its end leaves zeros; `to` is an LDS address.
typedef int i32x4_t __attribute__((ext_vector_type(4)));
__device__ __forceinline__ void load_lds(i32x4_t buffer, uint32_t off, uint32_t to) {
  asm volatile(
      "s_mov_b32 m0, %0\n\t"
      "s_nop 0\n\t"
      "buffer_load_dwordx4 %1, %2, 0 offen lds"
      :
      : "s"(__builtin_amdgcn_readfirstlane(to)), "v"(off), "s"(buffer)
      : "memory");
}
__device__ __forceinline__ uint32_t lds_address(const void* p) {
  return (uint32_t)(uintptr_t)(__attribute__((address_space(3))) const char*)static_cast<const char*>(p);
}
// Waits until at most N of the wavefront's loads and stores, the youngest, are
// still under way.
template <int N>
__device__ __forceinline__ void loaded() {
  asm volatile("s_waitcnt vmcnt(%0)" ::"i"(N) : "memory");
}
// ... and for the wavefront's own reads of LDS.
template <int N>
__device__ __forceinline__ void loaded_and_read() {
  asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" ::"i"(N) : "memory");
}

}  // namespace
}  // namespace ssm

#endif  // SSMSCAN_LDS_LOAD_H
