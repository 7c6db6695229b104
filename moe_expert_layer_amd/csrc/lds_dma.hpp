// Direct global -> LDS loads, their waits, and the LDS chunk swizzle of the GEMM kernels (gfx950).
#pragma once
#include <hip/hip_runtime.h>
#include <cstdint>

namespace moe {

// ---------------------------------------------------------------------------------------
// direct global -> LDS loads (the wave writes 64 lanes x 16 bytes at m0, lane order)

// the source is a uniform 64-bit base plus a 32-bit per-lane offset (the saddr form); the base
// is passed through readfirstlane so it sits in SGPRs even where the compiler cannot prove it
// uniform.  A VMEM instruction that reads an SGPR written by a VALU instruction (readfirstlane,
// an SGPR spill reload) needs 5 wait states in between; the compiler inserts them before its
// own loads but not inside inline asm, so the asm provides them: s_mov + s_nop 3 (this also
// covers the 1 wait state between writing m0 and the LDS DMA that reads it)
__device__ __forceinline__ const void* sbase(const void* p) {
  const uint64_t v = reinterpret_cast<uint64_t>(p);
  const uint32_t lo = __builtin_amdgcn_readfirstlane((uint32_t)v), hi = __builtin_amdgcn_readfirstlane((uint32_t)(v >> 32));
  return reinterpret_cast<const void*>(((uint64_t)hi << 32) | lo);
}
__device__ __forceinline__ void dma16(const void* base, uint32_t off, uint32_t lds) {
  base = sbase(base);
  asm volatile("s_mov_b32 m0, %2\n\ts_nop 3\n\tglobal_load_lds_dwordx4 %0, %1" ::"v"(off), "s"(base), "s"(lds)
               : "memory", "m0");
}
__device__ __forceinline__ void dma4(const void* base, uint32_t off, uint32_t lds) {
  base = sbase(base);
  asm volatile("s_mov_b32 m0, %2\n\ts_nop 3\n\tglobal_load_lds_dword %0, %1" ::"v"(off), "s"(base), "s"(lds)
               : "memory", "m0");
}
// the same from a buffer: its base and length sit in a four-dword descriptor in SGPRs, soff is a
// uniform byte offset, and a lane whose voff + soff reaches past the length reads nothing there (the
// hardware checks every load: voff >= length - soff is out of range, so soff is kept within the
// length).  The length is cut to 2^31 - 1, past which no caller's offsets reach.
typedef int v4i_srd __attribute__((ext_vector_type(4)));
__device__ __forceinline__ v4i_srd buffer_srd(const void* base, long long bytes) {
  const uint64_t b = reinterpret_cast<uint64_t>(base);
  const uint32_t len = bytes < 0x7fffffffLL ? (uint32_t)bytes : 0x7fffffffu;
  return v4i_srd{(int)__builtin_amdgcn_readfirstlane((uint32_t)b),
                 (int)(__builtin_amdgcn_readfirstlane((uint32_t)(b >> 32)) & 0xffffu),
                 (int)__builtin_amdgcn_readfirstlane(len), 0x00020000};  // raw buffer, 32-bit format
}
__device__ __forceinline__ void dma16_buffer(v4i_srd srd, uint32_t voff, uint32_t soff, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %3\n\ts_nop 3\n\tbuffer_load_dwordx4 %0, %1, %2 offen lds" ::"v"(voff), "s"(srd),
               "s"(soff), "s"(lds)
               : "memory", "m0");
}
__device__ __forceinline__ void dma4_buffer(v4i_srd srd, uint32_t voff, uint32_t soff, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %3\n\ts_nop 3\n\tbuffer_load_dword %0, %1, %2 offen lds" ::"v"(voff), "s"(srd),
               "s"(soff), "s"(lds)
               : "memory", "m0");
}
template <int N>
__device__ __forceinline__ void wait_vm_barrier() {
  asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(N) : "memory");
}
__device__ __forceinline__ uint32_t lds_addr(const void* p) { return (uint32_t)(uintptr_t)p; }
__device__ __forceinline__ uint32_t uniform(uint32_t v) { return __builtin_amdgcn_readfirstlane(v); }

// XOR swizzles of 16-byte chunks, conflict-free when 8 (or 16) consecutive rows are read at
// one logical chunk: rows of 128, 64 and 32 bytes.
template <int CPR>
__device__ __forceinline__ int swz(int r) {
  if (CPR == 8) return (r ^ (r >> 3)) & 7;
  if (CPR == 4) return ((r >> 1) ^ (r >> 3)) & 3;
  return ((r >> 2) ^ (r >> 3)) & 1;
}

__device__ __forceinline__ uint4 lds16(const uint8_t* p) { return *reinterpret_cast<const uint4*>(p); }

}  // namespace moe
