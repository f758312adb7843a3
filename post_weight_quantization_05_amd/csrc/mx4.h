// Microscaled 4-bit storage shared by the MX4 kernels (layout: include/qz.h).
//
// A block is 32 consecutive columns of one row: 16 bytes of E2M1 codes (even column in the
// low nibble) and one E8M0 byte E for the factor 2^(E - 127).  The gfx950 conversions and
// matrix instructions take the factor as the exponent field of an fp32 word, so E << 23 is
// all the decoding there is: E = 0 means 2^-127 (not zero) and E = 255 gives NaN, as stored.
#pragma once

#include "qz_internal.h"

namespace qz {

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef int i32x8 __attribute__((ext_vector_type(8)));

constexpr int kMxBlock = 32;
constexpr uint32_t kMxOne = 127;   // E of the factor 1

__host__ __device__ inline int64_t mx_blocks(int64_t cols) { return ceil_div(cols, kMxBlock); }

__device__ __forceinline__ float mx_factor(uint32_t e) { return __uint_as_float(e << 23); }

// Eight codes (one 32-bit word) as bf16: exact, an E2M1 value has two significant bits and
// bf16 the exponent range of E8M0.
__device__ __forceinline__ bf16x8 mx_word_bf16(uint32_t w, float factor) {
  const bf16x2 a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, factor, 0);
  const bf16x2 b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, factor, 1);
  const bf16x2 c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, factor, 2);
  const bf16x2 d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, factor, 3);
  bf16x8 r;
  r[0] = a[0]; r[1] = a[1]; r[2] = b[0]; r[3] = b[1];
  r[4] = c[0]; r[5] = c[1]; r[6] = d[0]; r[7] = d[1];
  return r;
}

__device__ __forceinline__ i32x8 mx_operand(uint4 c) {   // fp4 operands use the low four words
  i32x8 v = {static_cast<int>(c.x), static_cast<int>(c.y), static_cast<int>(c.z),
             static_cast<int>(c.w), 0, 0, 0, 0};
  return v;
}

// bf16 bits of v, nearest even (a NaN stays a NaN).
__device__ __forceinline__ uint16_t f32_to_bf16(float v) {
  return __builtin_bit_cast(uint16_t, static_cast<__bf16>(v));
}

}  // namespace qz
