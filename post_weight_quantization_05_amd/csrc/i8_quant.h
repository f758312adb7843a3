// One row onto int8 codes with a scale: the pieces shared by the quantisation kernel and by the
// few-token kernels, which quantize their rows themselves.
#pragma once

#include "qz_internal.h"

namespace qz {

// What a row's codes are found with.  Small rows are moved up by a power of two, exactly, so that
// 1 / s is a number.
struct RowScale {
  float s;         // as stored: NaN for a row that is not finite
  float up, su, r; // 2^80 or 1; s up; 1 / (s up) to 32 bits
  bool codes;      // whether the row has codes other than zero
};
// top: the largest magnitude's bits (magnitudes compare as integers, and a NaN is above every number).
__device__ __forceinline__ RowScale row_scale(uint32_t top) {
  RowScale c;
  const bool finite = top < 0x7f800000u;
  c.s = finite ? __uint_as_float(top) * (1.f / 127.f) : __uint_as_float(0x7fc00000u);
  c.up = c.s < 0x1p-60f ? 0x1p80f : 1.f;
  c.su = c.s * c.up;
  c.r = 1.f / c.su;
  c.codes = finite && c.s > 0.f;
  return c;
}

// The whole number nearest to v / s (the quotient itself), ties to the even one, within +-127.
// v r is off by less than 2^-14 of a code (127 codes, three roundings), so only a quotient that near
// to a half needs the remainder v - q s, which one fused step gives exactly: it is a multiple of the
// smaller of both numbers' last bits, and at most s / 2 or so.
__device__ __forceinline__ float nearest_code(float v, const RowScale& c) {
  v *= c.up;
  const float t = v * c.r;
  float q = __builtin_rintf(t);
  if (fabsf(t - q) > 0.5f - 0x1p-13f) {
    const float rest = fmaf(-q, c.su, v), half = 0.5f * c.su;
    if (fabsf(rest) > half || (fabsf(rest) == half && (static_cast<int>(q) & 1)))
      q += rest > 0.f ? 1.f : -1.f;
  }
  return fminf(fmaxf(q, -127.f), 127.f);
}

// Eight neighbouring elements of a row, columns past `left` as zeros.  VEC: all eight or none are
// there, on a 16-byte boundary.
template <int WT, bool VEC>
__device__ __forceinline__ void load8(const void* p, int64_t at, int64_t left, float (&v)[8]) {
  if constexpr (VEC) {
    if (left <= 0) {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = 0.f;
    } else if constexpr (WT == QZ_BF16) {
      const uint4 x = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p) + at);
      const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        v[2 * i] = __uint_as_float(w[i] << 16);
        v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
      }
    } else {
      const float4* f = reinterpret_cast<const float4*>(static_cast<const float*>(p) + at);
      const float4 a = f[0], b = f[1];
      v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
      v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = i < left ? load_w<WT>(p, at + i) : 0.f;
  }
}

__device__ __forceinline__ uint32_t top8(const float (&v)[8], uint32_t top) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint32_t b = __float_as_uint(v[i]) & 0x7fffffffu;
    top = b > top ? b : top;
  }
  return top;
}

// Codes of eight elements (two words), and their values' whole numbers.
__device__ __forceinline__ uint2 codes8(const float (&v)[8], const RowScale& c, float (&q)[8]) {
  uint32_t w[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    uint32_t b[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      q[4 * h + i] = c.codes ? nearest_code(v[4 * h + i], c) : 0.f;
      b[i] = static_cast<uint32_t>(static_cast<int>(q[4 * h + i])) & 255u;
    }
    w[h] = b[0] | b[1] << 8 | b[2] << 16 | b[3] << 24;
  }
  return make_uint2(w[0], w[1]);
}

__device__ __forceinline__ uint32_t bf16_pair(float a, float b) {
  return __builtin_bit_cast(uint16_t, static_cast<__bf16>(a)) |
         static_cast<uint32_t>(__builtin_bit_cast(uint16_t, static_cast<__bf16>(b))) << 16;
}

// Whole number sums of four codes a word, in integers.
__device__ __forceinline__ int add_codes(uint32_t w, int sum) {
  return __builtin_amdgcn_sdot4(static_cast<int>(w), 0x01010101, sum, false);
}

__device__ __forceinline__ uint32_t wave_top(uint32_t v) {
  for (int o = 32; o; o >>= 1) {
    const uint32_t u = static_cast<uint32_t>(__shfl_xor(static_cast<int>(v), o));
    v = u > v ? u : v;
  }
  return v;
}
__device__ __forceinline__ int wave_sum(int v) {
  for (int o = 32; o; o >>= 1) v += __shfl_xor(v, o);
  return v;
}

}  // namespace qz
