// LDS DMA on gfx950: loads that go from memory to LDS without registers, the
// explicit waits for them, and a barrier that waits for nothing else.
#pragma once

#include "internal.h"

namespace fp8lin {

// s_waitcnt with only vmcnt constrained (gfx9 encoding: vmcnt bits [3:0] and
// [15:14], expcnt [6:4] = 7 and lgkmcnt [11:8] = 15 mean "no wait").
template <int N>
__device__ __forceinline__ void wait_vmcnt() {
  static_assert(N >= 0 && N < 64, "vmcnt range");
  __builtin_amdgcn_s_waitcnt((N & 15) | ((N >> 4) << 14) | (7 << 4) | (15 << 8));
}

// Wait until at most `younger` stages of this wave's DMA (D instructions per
// stage) are still in flight.
template <int D>
__device__ __forceinline__ void wait_stages(int younger) {
  if (younger >= 2) wait_vmcnt<2 * D>();
  else if (younger == 1) wait_vmcnt<D>();
  else wait_vmcnt<0>();
}

// A bare barrier: no memory access may move across it (asm "memory" clobber),
// and it waits for nothing the explicit waits did not.
__device__ __forceinline__ void bare_barrier() { asm volatile("s_barrier" ::: "memory"); }

// LDS byte address of a __shared__ object.
__device__ __forceinline__ uint32_t lds_addr(const void* p) {
  return (uint32_t)(uintptr_t)((__attribute__((address_space(3))) const void*)p);
}

// One LDS-DMA load: 16 bytes per lane from `src` into LDS at
// `lds_kb + 16 * lane` (lds_kb: the wave-uniform LDS byte address of the
// destination KB).  Issued from inline assembly so that the compiler does not
// treat it as a write it must wait for before every later LDS read: the ring
// protocol waits for it explicitly (wait_vmcnt + barrier).  Vector memory
// operations complete in issue order, so the compiler's own vmcnt waits stay
// correct (they can only wait longer).
__device__ __forceinline__ void dma16(const uint8_t* src, uint32_t lds_kb) {
  asm volatile(
      "s_mov_b32 m0, %1\n\t"
      "global_load_lds_dwordx4 %0, off"
      :
      : "v"(src), "s"(__builtin_amdgcn_readfirstlane(lds_kb))
      : "memory", "m0");
}

// The same from a wave-uniform base and a 32-bit byte offset per lane.
__device__ __forceinline__ void dma16(const uint8_t* base, uint32_t offset, uint32_t lds_kb) {
  asm volatile(
      "s_mov_b32 m0, %2\n\t"
      "global_load_lds_dwordx4 %0, %1"
      :
      : "v"(offset), "s"(base), "s"(__builtin_amdgcn_readfirstlane(lds_kb))
      : "memory", "m0");
}

}  // namespace fp8lin
