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
//
// s is a product with the rounded 1 / 127, not a quotient: that is what PyTorch makes of max / 127 on this GPU, so
// whoever quantizes there gets the same scales and codes, bit for bit.  The factor is 2^-28 of itself off, and
// in 4.5% of the rows s is a last bit off the quotient's rounding; the largest value's quotient stays within 127 (1 +- 2^-23),
// and codes are those of s as it is stored.
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

// Code of v: the whole number nearest to v / s (the quotient itself), ties to the even one, within
// +-127, from the remainder v - q s, which one fused step gives exactly: it is a multiple of the smaller
// of both numbers' last bits, and at most s / 2 or so.  q: at most one off.
__device__ __forceinline__ float settled_code(float v, float q, const RowScale& c) {
  const float rest = fmaf(-q, c.su, v), half = 0.5f * c.su;
  if (fabsf(rest) > half || (fabsf(rest) == half && (static_cast<int>(q) & 1))) q += rest > 0.f ? 1.f : -1.f;
  return fminf(fmaxf(q, -127.f), 127.f);
}

// Eight neighbouring elements of a row as they lie in memory, and as numbers; columns past `left` are
// zeros.  VEC: all eight or none are there, on a 16-byte boundary.
template <int WT>
struct Raw8 {
  uint4 w[WT == QZ_BF16 ? 1 : 2];
};
template <int WT, bool VEC>
__device__ __forceinline__ Raw8<WT> load8(const void* p, int64_t at, int64_t left) {
  Raw8<WT> r;
  if constexpr (VEC) {
    constexpr int n = WT == QZ_BF16 ? 1 : 2;
    const uint4* src = reinterpret_cast<const uint4*>(static_cast<const char*>(p) + at * (2 * n));
#pragma unroll
    for (int i = 0; i < n; ++i) r.w[i] = left > 0 ? src[i] : make_uint4(0, 0, 0, 0);
  } else if constexpr (WT == QZ_BF16) {
    uint32_t w[4];
    const uint16_t* src = static_cast<const uint16_t*>(p) + at;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      w[i] = (2 * i < left ? static_cast<uint32_t>(src[2 * i]) : 0u) | (2 * i + 1 < left ? static_cast<uint32_t>(src[2 * i + 1]) << 16 : 0u);
    r.w[0] = make_uint4(w[0], w[1], w[2], w[3]);
  } else {
    uint32_t w[8];
    const uint32_t* src = static_cast<const uint32_t*>(p) + at;
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = i < left ? src[i] : 0u;
    r.w[0] = make_uint4(w[0], w[1], w[2], w[3]);
    r.w[1] = make_uint4(w[4], w[5], w[6], w[7]);
  }
  return r;
}
template <int WT>
__device__ __forceinline__ void numbers8(const Raw8<WT>& r, float (&v)[8]) {
  if constexpr (WT == QZ_BF16) {
    const uint32_t w[4] = {r.w[0].x, r.w[0].y, r.w[0].z, r.w[0].w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float(w[i] << 16);
      v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  } else {
    const uint32_t w[8] = {r.w[0].x, r.w[0].y, r.w[0].z, r.w[0].w, r.w[1].x, r.w[1].y, r.w[1].z, r.w[1].w};
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(w[i]);
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
//
// v r is off by less than 2^-16 of a code (127 codes, two roundings of 2^-24 each), so only quotients that
// near to a half need their remainder.  Adding 1.5 2^23 rounds to a whole number, nearest even, and leaves its low
// byte in the sum's.
__device__ __forceinline__ uint2 codes8(const float (&v)[8], const RowScale& c, float (&q)[8]) {
  constexpr float kWhole = 12582912.f;
  float u[8], m[8];
  bool near = c.up != 1.f;   // small rows: all by their remainders
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    u[i] = v[i] * c.r;
    m[i] = u[i] + kWhole;
    q[i] = m[i] - kWhole;
    near = near || fabsf(u[i] - q[i]) > 0.5f - 0x1p-15f;
  }
  if (near) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float w = v[i] * c.up;
      q[i] = settled_code(w, fminf(fmaxf(__builtin_rintf(w * c.r), -127.f), 127.f), c);
      m[i] = q[i] + kWhole;
    }
  }
  if (!c.codes) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      q[i] = 0.f;
      m[i] = kWhole;
    }
  }
  uint32_t w[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const uint32_t lo = __builtin_amdgcn_perm(__float_as_uint(m[4 * h + 1]), __float_as_uint(m[4 * h]), 0x0c0c0400);
    const uint32_t hi = __builtin_amdgcn_perm(__float_as_uint(m[4 * h + 3]), __float_as_uint(m[4 * h + 2]), 0x04000c0c);
    w[h] = lo | hi;
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

// Sum over the wavefront, in every lane; the largest below.  By moves inside the vector unit: through LDS each
// of the six steps would wait a hundred cycles.
__device__ __forceinline__ int wave_sum(int v) {
  v += __builtin_amdgcn_mov_dpp(v, 0xB1, 0xf, 0xf, true);    // lane ^ 1
  v += __builtin_amdgcn_mov_dpp(v, 0x4E, 0xf, 0xf, true);    // lane ^ 2
  v += __builtin_amdgcn_mov_dpp(v, 0x141, 0xf, 0xf, true);   // mirrored in eight
  v += __builtin_amdgcn_mov_dpp(v, 0x140, 0xf, 0xf, true);   // mirrored in sixteen
  const auto a = __builtin_amdgcn_permlane16_swap(v, v, false, false);
  v = static_cast<int>(a[0]) + static_cast<int>(a[1]);
  const auto b = __builtin_amdgcn_permlane32_swap(v, v, false, false);
  return static_cast<int>(b[0]) + static_cast<int>(b[1]);
}
__device__ __forceinline__ uint32_t wave_top(uint32_t v) {
  const auto up = [](uint32_t a, uint32_t b) { return a > b ? a : b; };
  v = up(v, __builtin_amdgcn_mov_dpp(v, 0xB1, 0xf, 0xf, true));
  v = up(v, __builtin_amdgcn_mov_dpp(v, 0x4E, 0xf, 0xf, true));
  v = up(v, __builtin_amdgcn_mov_dpp(v, 0x141, 0xf, 0xf, true));
  v = up(v, __builtin_amdgcn_mov_dpp(v, 0x140, 0xf, 0xf, true));
  const auto a = __builtin_amdgcn_permlane16_swap(v, v, false, false);
  v = up(a[0], a[1]);
  const auto b = __builtin_amdgcn_permlane32_swap(v, v, false, false);
  return up(b[0], b[1]);
}

}  // namespace qz
