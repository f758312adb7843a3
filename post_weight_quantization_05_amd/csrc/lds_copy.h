// Copies from memory into LDS, for kernels that stream tiles through it: the order of an LDS row, the
// copy of a wavefront, and the join of a workgroup's wavefronts.
#pragma once

#include "qz_internal.h"

namespace qz {

// Chunk c (16 bytes) of row r lies at chunk c ^ swz(r), stepping once per 256 bytes of rows of RB
// bytes: sixteen rows at the same column touch all 64 banks.  The copies keep LDS linear and permute
// their global sources instead.
template <int RB>
__device__ __forceinline__ int swz(int row) {
  return (row / (256 / RB)) & (RB / 16 - 1);
}

typedef __attribute__((address_space(3))) uint8_t lds_u8;

// One copy of a wavefront, lane i of it to LDS at dst + BYTES i: scalar base, 32-bit offsets.
// Inline asm, so that the compiler does not wait for it before every LDS read; it has no
// register result, and the stages are synchronised by explicit waits.  The s_nop is the wait state
// that a copy needs after the write of m0; the five after a vector write of its base are not needed,
// since the bases are scalar results (a test reads both distances off the built library; waiting for
// five here took 1% longer).
template <int BYTES>
__device__ __forceinline__ void copy_lds(lds_u8* dst, const uint8_t* base, uint32_t voff) {
  const uint32_t at = __builtin_amdgcn_readfirstlane(static_cast<uint32_t>(reinterpret_cast<uintptr_t>(dst)));
  const uint64_t b = reinterpret_cast<uint64_t>(base);
  const uint32_t lo = static_cast<uint32_t>(__builtin_amdgcn_readfirstlane(static_cast<uint32_t>(b)));
  const uint32_t hi = static_cast<uint32_t>(__builtin_amdgcn_readfirstlane(static_cast<uint32_t>(b >> 32)));
  const uint64_t su = (static_cast<uint64_t>(hi) << 32) | lo;
  if constexpr (BYTES == 16)
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2"
                 :: "s"(at), "v"(voff), "s"(su) : "memory", "m0");
  else
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dword %1, %2"
                 :: "s"(at), "v"(voff), "s"(su) : "memory", "m0");
}

// Waits until at most N copies of this wavefront are in flight (vmcnt = N) and its LDS accesses
// are done (lgkmcnt = 0), then for the other wavefronts.
template <int N>
__device__ __forceinline__ void wait_and_join() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_waitcnt((N & 15) | ((N >> 4) << 14) | (7 << 4));
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

}  // namespace qz
