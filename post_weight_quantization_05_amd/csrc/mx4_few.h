// Products of a few rows of W with a few tokens, for one wavefront: the inner loop of the
// few-token product and of the expert layer.
//
// A tile is 16 rows of W by 16 tokens.  The wavefront goes along d_i a unit of 256 columns at a
// time: whole 128-byte lines of codes, straight from global memory to the matrix cores, since
// every code is used once.  Of each 128 columns lane l loads row l % 16, block l / 16: 16 bytes of
// codes.  AHEAD: the next unit's loads are issued before the current one's products (for one
// workgroup a compute unit; with several of them the registers are better spent on more).
//
// bf16 X: a load of 16 bytes a lane covers 64 contiguous bytes of each row, so product j of the
// four takes the columns 32 j + 8 (l / 16) + 0..7 of X, and the codes have to follow: a 4 x 4
// transpose of words between the four lanes of a row (two pairs of lane swaps) turns word i of
// block l / 16 into word l / 16 of block i.  (With X read in the shape of whole blocks instead,
// each of the four loads touches the same two lines of every row, and a compute unit looks up a
// line in about four clocks: at 13 tokens that cost more than the codes did.)
#pragma once

#include "mx4.h"

namespace qz {

struct __attribute__((packed)) Bytes8 {
  uint32_t lo, hi;
};

// Eight factors of a row from block b0 on, at any alignment (1 past the row's end).
__device__ __forceinline__ uint2 eight_factors(const uint8_t* row, int b0, int G, bool whole) {
  if (whole) {
    const Bytes8 v = *reinterpret_cast<const Bytes8*>(row + b0);
    return make_uint2(v.lo, v.hi);
  }
  uint32_t lo = 0, hi = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    lo |= (b0 + i < G ? static_cast<uint32_t>(row[b0 + i]) : kMxOne) << (8 * i);
    hi |= (b0 + 4 + i < G ? static_cast<uint32_t>(row[b0 + 4 + i]) : kMxOne) << (8 * i);
  }
  return make_uint2(lo, hi);
}

// Word i of lane group g (16 lanes each) <-> word g of lane group i.
__device__ __forceinline__ void transpose_words(uint32_t (&w)[4]) {
  const auto a = __builtin_amdgcn_permlane32_swap(w[0], w[2], false, false);
  const auto b = __builtin_amdgcn_permlane32_swap(w[1], w[3], false, false);
  const auto c = __builtin_amdgcn_permlane16_swap(a[0], b[0], false, false);
  const auto d = __builtin_amdgcn_permlane16_swap(a[1], b[1], false, false);
  w[0] = c[0];
  w[1] = c[1];
  w[2] = d[0];
  w[3] = d[1];
}

// What the tokens come as: MX4 codes, bf16, or bf16 twice (value and remainder).
enum class Few { kMx4, kBf16, kBf16Twice };

template <Few X, int RT, int NT>
struct FewUnit {
  uint4 c[2][RT];
  uint2 e[RT];
  uint4 x[2][NT][X == Few::kMx4 ? 1 : X == Few::kBf16 ? 4 : 8];
  uint2 f[NT];
};

// A lane's pointers: wc at its row's codes + 16 q bytes, ws at its row's factors, xc at its
// token's codes or values + 16 q bytes (xl: the remainders), xs at its token's factors, for
// q = lane / 16; have: whether the lane has a token.
template <Few X, int RT, int NT>
struct FewRows {
  const uint8_t* wc[RT];
  const uint8_t* ws[RT];
  const uint8_t* xc[NT];
  const uint8_t* xl[NT];
  const uint8_t* xs[NT];
  bool have[NT];
};

// acc += the products over the units first, first + step, ... of G blocks.
template <bool AHEAD, Few X, int RT, int NT>
__device__ __forceinline__ void few_products(const FewRows<X, RT, NT>& p, int G, int first, int step,
                                             f32x4 (&acc)[RT][NT]) {
  constexpr bool X4 = X == Few::kMx4;
  constexpr int kX = X4 ? 1 : X == Few::kBf16 ? 4 : 8;
  const int q = (threadIdx.x & 63) >> 4;
  using Unit = FewUnit<X, RT, NT>;
  const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
  auto load = [&](int b0, Unit& v) {
    const bool whole = b0 + 8 <= G;
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int blk = b0 + 4 * u;
#pragma unroll
      for (int a = 0; a < RT; ++a) {
        v.c[u][a] = zero;
        if (whole || blk + q < G) v.c[u][a] = *reinterpret_cast<const uint4*>(p.wc[a] + blk * 16);
      }
#pragma unroll
      for (int b = 0; b < NT; ++b)
#pragma unroll
        for (int j = 0; j < kX; ++j) {
          v.x[u][b][j] = zero;
          if (p.have[b] && (whole || blk + (X4 ? q : j % 4) < G))
            v.x[u][b][j] = *reinterpret_cast<const uint4*>(
                (j < 4 ? p.xc[b] : p.xl[b]) + blk * (X4 ? 16 : 64) + 64 * (j % 4));
        }
    }
#pragma unroll
    for (int a = 0; a < RT; ++a) v.e[a] = eight_factors(p.ws[a], b0, G, whole);
    if constexpr (X4) {
#pragma unroll
      for (int b = 0; b < NT; ++b) v.f[b] = eight_factors(p.xs[b], b0, G, whole);
    }
  };
  auto multiply = [&](const Unit& v) {
#pragma unroll
    for (int u = 0; u < 2; ++u) {
#pragma unroll
      for (int a = 0; a < RT; ++a) {
        const uint32_t e = u ? v.e[a].y : v.e[a].x;
        if constexpr (X4) {
#pragma unroll
          for (int b = 0; b < NT; ++b)
            acc[a][b] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
                mx_operand(v.c[u][a]), mx_operand(v.x[u][b][0]), acc[a][b], 4, 4, 0,
                static_cast<int>(e >> (8 * q)), 0, static_cast<int>((u ? v.f[b].y : v.f[b].x) >> (8 * q)));
        } else {
          uint32_t w[4] = {v.c[u][a].x, v.c[u][a].y, v.c[u][a].z, v.c[u][a].w};
          transpose_words(w);
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const bf16x8 wv = mx_word_bf16(w[j], mx_factor((e >> (8 * j)) & 255u));
#pragma unroll
            for (int b = 0; b < NT; ++b) {
              acc[a][b] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                  wv, __builtin_bit_cast(bf16x8, v.x[u][b][j]), acc[a][b], 0, 0, 0);
              if constexpr (kX == 8)
                acc[a][b] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                    wv, __builtin_bit_cast(bf16x8, v.x[u][b][4 + j]), acc[a][b], 0, 0, 0);
            }
          }
        }
      }
    }
  };
  int b0 = first * 8;
  const int ahead = step * 8;
  if constexpr (!AHEAD) {
    for (; b0 < G; b0 += ahead) {
      Unit u;
      load(b0, u);
      multiply(u);
    }
    return;
  }
  Unit u0, u1;
  if (b0 < G) load(b0, u0);
  while (b0 < G) {
    if (b0 + ahead < G) load(b0 + ahead, u1);
    multiply(u0);
    b0 += ahead;
    if (b0 >= G) break;
    if (b0 + ahead < G) load(b0 + ahead, u0);
    multiply(u1);
    b0 += ahead;
  }
}

}  // namespace qz

