// Copies from global memory straight into LDS (gfx950).
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

namespace fp4k {

// LDS byte address of a pointer into a __shared__ array (a generic pointer to LDS keeps the
// LDS offset in its low 32 bits).
__device__ __forceinline__ uint32_t lds_offset(const void* p) { return (uint32_t)reinterpret_cast<uintptr_t>(p); }

// One global_load_lds_dwordx4 for the wave: lane i copies the 16 bytes at sbase + voff(i)
// to LDS bytes [dst + 16 i, dst + 16 i + 16) (dst is wave-uniform and goes in M0). Between the
// start of the block and the load stand five wait states: the M0 write needs one, and sbase may
// come from a v_readlane just before (a spilled address), which a vector memory instruction may
// read five states later at the earliest; the compiler puts no waits into a block that it cannot
// look into. Written as inline assembly so
// that the compiler's wait-count insertion does not treat the copy as an LDS write that may
// alias later LDS reads of the other buffer: the kernels wait for these copies themselves
// (vmcnt, and a barrier where other waves read the buffer).
__device__ __forceinline__ void lds_dma16(const void* sbase, uint32_t voff, uint32_t dst) {
  asm volatile(
      "s_mov_b32 m0, %2\n\t"
      "s_nop 3\n\t"
      "global_load_lds_dwordx4 %0, %1"
      :
      : "v"(voff), "s"(sbase), "s"(dst)
      : "memory", "m0");
}

// The same for one dword, or for one byte (zero-extended to a dword), per lane: LDS bytes
// [dst + 4 i, dst + 4 i + 4).
__device__ __forceinline__ void lds_dma4(const void* sbase, uint32_t voff, uint32_t dst) {
  asm volatile(
      "s_mov_b32 m0, %2\n\t"
      "s_nop 3\n\t"
      "global_load_lds_dword %0, %1"
      :
      : "v"(voff), "s"(sbase), "s"(dst)
      : "memory", "m0");
}
__device__ __forceinline__ void lds_dma1(const void* sbase, uint32_t voff, uint32_t dst) {
  asm volatile(
      "s_mov_b32 m0, %2\n\t"
      "s_nop 3\n\t"
      "global_load_lds_ubyte %0, %1"
      :
      : "v"(voff), "s"(sbase), "s"(dst)
      : "memory", "m0");
}

}  // namespace fp4k
