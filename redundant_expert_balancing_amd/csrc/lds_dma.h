// Buffer descriptors, direct global -> LDS DMA and the waits around it, shared by the GEMM
// kernels.
#pragma once

#include "common.h"

namespace moonep {

typedef int v4i_t __attribute__((ext_vector_type(4)));
constexpr int kRsrcFlags = 0x00020000;      // raw (unswizzled) 32-bit data, gfx9 family
constexpr uint32_t kOffNone = 0x80000000u;  // an offset past every range used here

__device__ inline __amdgpu_buffer_rsrc_t make_rsrc(const void* base, uint32_t bytes) {
  // the range is uniform; readfirstlane keeps it (and the descriptor) in scalar
  // registers even where it was computed with 64-bit vector compares
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(base), (short)0,
                                           __builtin_amdgcn_readfirstlane((int)bytes), kRsrcFlags);
}

__device__ inline uint32_t clamp_bytes(int64_t b) {
  return b <= 0 ? 0u : (b >= int64_t(kOffNone) ? kOffNone : uint32_t(b));
}

// One 16-byte-per-lane DMA into LDS at byte address lds (uniform). Issued as
// inline assembly so that the compiler's wait-count pass does not wait for all
// outstanding DMAs at every LDS read; the k-loop waits for exactly the steps it
// needs (wait_vm).
__device__ inline void dma16(__amdgpu_buffer_rsrc_t r, uint32_t voff, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %2\n\tbuffer_load_dwordx4 %0, %1, 0 offen lds"
               :
               : "v"(voff), "s"(r), "s"(__builtin_amdgcn_readfirstlane(lds))
               : "memory");
}

// The same with a uniform byte offset added to every lane's.
__device__ inline void dma16(__amdgpu_buffer_rsrc_t r, uint32_t voff, uint32_t soff, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %2\n\tbuffer_load_dwordx4 %0, %1, %3 offen lds"
               :
               : "v"(voff), "s"(r), "s"(__builtin_amdgcn_readfirstlane(lds)),
                 "s"(__builtin_amdgcn_readfirstlane(soff))
               : "memory");
}

// Wait until at most n of this wavefront's vector memory operations are pending.
template <int n>
__device__ inline void wait_vm() {
  static_assert(n >= 0 && n < 64, "vmcnt range");
  // s_waitcnt simm16: vmcnt[3:0] in bits 3:0, vmcnt[5:4] in bits 15:14, expcnt and
  // lgkmcnt left at their maxima (no wait)
  __builtin_amdgcn_s_waitcnt((n & 15) | ((n >> 4) << 14) | (7 << 4) | (15 << 8));
}

// Chunk swizzle of a 128-byte LDS row of 16-byte chunks: chunk c of row r is stored at
// c ^ swz_k(r).
__device__ inline int swz_k(int r) { return (r >> 1) & 7; }

typedef __attribute__((address_space(3))) char lds_char;

// LDS byte address of a pointer into __shared__ memory (address-space cast).
__device__ inline uint32_t lds_addr(const void* p) {
  return uint32_t(reinterpret_cast<uintptr_t>((const lds_char*)p));
}

}  // namespace moonep
