// Products of a few rows of W with a few tokens, for one wavefront: the inner loop of the
// few-token product and of the expert layer.
//
// A tile is 16 rows of W by 16 tokens.  The wavefront goes along d_i a unit of 256 columns at a
// time: whole 128-byte lines of codes.  Of each 128 columns lane l has row l % 16, block l / 16:
// 16 bytes of codes.
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

struct __attribute__((packed)) Bytes16 {
  uint32_t w[4];
};

// Sixteen factors of a row from block b on, at any alignment.  Past the row's end they are 0 (any
// factor but the NaN will do, the codes there are zeros): the row's last sixteen bytes, moved down.
__device__ __forceinline__ uint4 sixteen_factors(const uint8_t* row, int b, int G) {
  uint32_t w[4] = {0, 0, 0, 0};
  if (b < G) {
    const int past = b + 16 - G;
    if (past <= 0 || G >= 16) {
      const Bytes16 v = *reinterpret_cast<const Bytes16*>(row + (past > 0 ? G - 16 : b));
      uint64_t lo = static_cast<uint64_t>(v.w[1]) << 32 | v.w[0], hi = static_cast<uint64_t>(v.w[3]) << 32 | v.w[2];
      if (past >= 8) {
        lo = hi;
        hi = 0;
      }
      if (past > 0 && past % 8) {
        lo = lo >> (8 * (past % 8)) | hi << (64 - 8 * (past % 8));
        hi >>= 8 * (past % 8);
      }
      w[0] = static_cast<uint32_t>(lo);
      w[1] = static_cast<uint32_t>(lo >> 32);
      w[2] = static_cast<uint32_t>(hi);
      w[3] = static_cast<uint32_t>(hi >> 32);
    } else {
#pragma unroll
      for (int i = 0; i < 16; ++i)
        if (b + i < G) w[i / 4] |= static_cast<uint32_t>(row[b + i]) << (8 * (i % 4));
    }
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
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

// RT tiles of 16 rows of W and a lane's tokens.  codes, scales: at a tile's first row (uniform);
// last: its last row inside the matrix, counted from the first (rows past it are read as that one).
// x: codes or values of the tokens lane / 8 and lane / 8 + 8 of a tile, or, where the lanes of the
// operand load them (not SHARED), of token lane % 16 at [0]; xs: factors of token lane % 16.
// Places without a token take another's (their columns are not stored).
template <bool X4, int RT, int NT>
struct FewRows {
  const uint8_t* codes[RT];
  const uint8_t* scales[RT];
  int last[RT];
  const uint8_t* x[NT][2];
  const uint8_t* xs[NT];
};

// LDS of a wavefront, bytes: its codes of a unit, and where the tokens pass through it (SHARED),
// half a unit of 16 of them in bf16.
template <bool SHARED, bool X4, int RT, int NT>
constexpr int kFewLds = !SHARED ? 2048 * RT : X4 ? 2048 * (RT > NT ? RT : NT) : RT > 2 ? 2048 * RT : 4096;

// acc += the products over the units [unit, end) of G blocks.
//
// Factors come 64 blocks (eight units) of a row at a time, 16 bytes to each of the row's four
// lanes, and go from there to the lanes that need them: fetched a unit at a time they would be a
// third of all the row segments that a wavefront asks for.
//
// lds: kFewLds bytes of the wavefront's own.  A load that the lanes of an operand made for
// themselves would have 16 rows in each run of 16 lanes, and the memory pipeline takes four lanes
// at a time: 64 accesses of 16 bytes.  So eight lanes load 128 bytes of a row, of W and (SHARED) of
// X, and the lanes of the operand read their parts back from LDS: codes first, then the tokens, half
// a unit at a time, through the same bytes (a wavefront's LDS instructions stay in order).
// 13 tokens, 12288 -> 4096, before the codes were loaded ahead: 10.2 us with X SHARED, 12.3 without;
// in the expert layer, where a tile has a token or two and the other lanes repeat them, 143 and 129
// us (7 tokens, 2 of 8 x 12288).
//
// AHEAD: the codes of the next unit are asked for before the products of the current one, its
// tokens before them: results come back in the order of the requests, so waiting for the tokens
// leaves the codes in flight.  Every lane always loads, at clamped places: behind a branch the
// compiler does not know how many loads are in flight and waits for all.  Where the tile needs so
// many registers that this costs wavefronts, those hide the latency better (us, with and without:
// 13 tokens 12288 -> 4096, 1 x 1 tiles, 8.9 and 10.1; 256 tokens 4096 -> 4096, 4 x 2 tiles, 23.5
// and 18.2; the same in MX4, 2 x 2, 11.1 and 13.0).
template <bool AHEAD, bool SHARED, bool X4, int RT, int NT>
__device__ __forceinline__ void few_products(const FewRows<X4, RT, NT>& p, uint8_t* lds, int G,
                                             int unit, int end, f32x4 (&acc)[RT][NT]) {
  static_assert(SHARED || !X4, "tokens in MX4 pass through LDS");
  constexpr int kX = X4 ? 1 : 4;   // 128-byte pieces of a token's unit
  if (unit >= end) return;
  const int lane = threadIdx.x & 63, q = lane >> 4;
  uint4 fw[RT], fx[NT];
  auto load_factors = [&](int first) {
#pragma unroll
    for (int a = 0; a < RT; ++a)
      fw[a] = sixteen_factors(p.scales[a] + static_cast<int64_t>(lane / 4 < p.last[a] ? lane / 4 : p.last[a]) * G,
                              first * 8 + 16 * (lane % 4), G);
    if constexpr (X4) {
#pragma unroll
      for (int b = 0; b < NT; ++b) fx[b] = sixteen_factors(p.xs[b], first * 8 + 16 * q, G);
    }
  };
  // factors of the four blocks of step s (of the sixteen that a fetch serves), held by lane `from`
  auto four = [&](const uint4& f, int s, int from) {
    const uint32_t even = s & 2 ? f.z : f.x, odd = s & 2 ? f.w : f.y;
    return static_cast<uint32_t>(__builtin_amdgcn_ds_bpermute(4 * from, static_cast<int>(s & 1 ? odd : even)));
  };
  struct Codes {
    uint4 c[2][RT];
  };
  // SHARED: [tile][rows 0 to 7, 8 to 15][piece of 128 bytes], else [tile][half of the unit][product]
  uint4 x[NT][2][kX];
  auto load_codes = [&](int u0, Codes& v) {   // eight lanes a row; rows 8 u to 8 u + 7
    const int blk = u0 * 8 + lane % 8 < G ? u0 * 8 + lane % 8 : G - 1;
#pragma unroll
    for (int u = 0; u < 2; ++u)
#pragma unroll
      for (int a = 0; a < RT; ++a) {
        const int row = 8 * u + lane / 8;
        v.c[u][a] = *reinterpret_cast<const uint4*>(
            p.codes[a] + (static_cast<uint32_t>(row < p.last[a] ? row : p.last[a]) * (16u * G) + 16 * blk));
      }
  };
  auto load_tokens = [&](int u0) {
    if constexpr (!SHARED) {
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int want = u0 * 8 + 4 * u + j;   // block
          const int blk = want < G ? want : G - 1;
#pragma unroll
          for (int b = 0; b < NT; ++b)
            x[b][u][j] = *reinterpret_cast<const uint4*>(p.x[b][0] + 64 * blk + 16 * q);
        }
      return;
    }
#pragma unroll
    for (int j = 0; j < kX; ++j) {
      const int want = 8 * (kX * u0 + j) + lane % 8;   // chunk of 16 bytes
      const int chunk = want < kX * G ? want : kX * G - 1;
#pragma unroll
      for (int b = 0; b < NT; ++b)
#pragma unroll
        for (int h = 0; h < 2; ++h)
          x[b][h][j] = *reinterpret_cast<const uint4*>(p.x[b][h] + 16 * chunk);
    }
  };
  // Rows of 128 bytes: chunk c of a row lies at chunk c ^ (row / 2 % 8), off its neighbours' banks.
  // Rows of 256: at c ^ a permutation of the sixteen rows that puts neighbours into other halves.
  const auto at = [](int row, int chunk) { return row * 128 + 16 * (chunk ^ (row >> 1 & 7)); };
  const auto at256 = [](int row, int chunk) { return row * 256 + 16 * (chunk ^ ((row >> 1 & 7) | (row & 1) << 3)); };
  const auto put = [&](int place, const uint4& v) { *reinterpret_cast<uint4*>(lds + place) = v; };
  const auto get = [&](int place) { return *reinterpret_cast<const uint4*>(lds + place); };
  auto multiply = [&](Codes& v, int u0, int of_fetch) {
    const int r8 = lane / 8, c8 = lane % 8, m = lane & 15;
    if (u0 * 8 + 8 > G) {   // blocks past the end: zeros on both sides
      const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
      for (int h = 0; h < 2; ++h) {
#pragma unroll
        for (int a = 0; a < RT; ++a)
          if (u0 * 8 + c8 >= G) v.c[h][a] = zero;
#pragma unroll
        for (int b = 0; b < NT; ++b)
#pragma unroll
          for (int j = 0; j < kX; ++j)
            if (SHARED ? 8 * (kX * u0 + j) + c8 >= kX * G : u0 * 8 + 4 * h + j >= G) x[b][h][j] = zero;
      }
    }
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int a = 0; a < RT; ++a) put(2048 * a + at(8 * h + r8, c8), v.c[h][a]);
    uint4 c[2][RT];
#pragma unroll
    for (int u = 0; u < 2; ++u)
#pragma unroll
      for (int a = 0; a < RT; ++a) c[u][a] = get(2048 * a + at(m, 4 * u + q));
    if constexpr (X4) {
#pragma unroll
      for (int b = 0; b < NT; ++b)
#pragma unroll
        for (int h = 0; h < 2; ++h) put(2048 * b + at(8 * h + r8, c8), x[b][h][0]);
    }
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int step = 2 * of_fetch + u;
      uint32_t e[RT];
#pragma unroll
      for (int a = 0; a < RT; ++a) e[a] = four(fw[a], step, 4 * m + (step >> 2));
      if constexpr (X4) {
#pragma unroll
        for (int b = 0; b < NT; ++b) {
          const uint32_t f = four(fx[b], step, m + 16 * (step >> 2)) >> (8 * q);
          const uint4 t = get(2048 * b + at(m, 4 * u + q));
#pragma unroll
          for (int a = 0; a < RT; ++a)
            acc[a][b] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
                mx_operand(c[u][a]), mx_operand(t), acc[a][b], 4, 4, 0,
                static_cast<int>(e[a] >> (8 * q)), 0, static_cast<int>(f));
        }
      } else {
        uint4 t[NT][4];
#pragma unroll
        for (int b = 0; b < NT; ++b) {
          if constexpr (!SHARED) {
#pragma unroll
            for (int j = 0; j < 4; ++j) t[b][j] = x[b][u][j];
            continue;
          }
#pragma unroll
          for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int j = 0; j < 2; ++j) put(at256(8 * h + r8, 8 * j + c8), x[b][h][(2 * u + j) % kX]);
#pragma unroll
          for (int j = 0; j < 4; ++j) t[b][j] = get(at256(m, 4 * j + q));
        }
#pragma unroll
        for (int a = 0; a < RT; ++a) {
          uint32_t w[4] = {c[u][a].x, c[u][a].y, c[u][a].z, c[u][a].w};
          transpose_words(w);
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const bf16x8 wv = mx_word_bf16(w[j], mx_factor((e[a] >> (8 * j)) & 255u));
#pragma unroll
            for (int b = 0; b < NT; ++b)
              acc[a][b] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                  wv, __builtin_bit_cast(bf16x8, t[b][j]), acc[a][b], 0, 0, 0);
          }
        }
      }
    }
  };
  const int begin = unit;
  if constexpr (!AHEAD) {
    for (; unit < end; ++unit) {
      Codes c;
      load_codes(unit, c);
      load_tokens(unit);
      if (((unit - begin) & 7) == 0) load_factors(unit);
      multiply(c, unit, (unit - begin) & 7);
    }
    return;
  }
  Codes c, next;
  load_factors(unit);
  load_codes(unit, c);
  for (; unit + 1 < end; ++unit) {
    load_tokens(unit);
    load_codes(unit + 1, next);
    multiply(c, unit, (unit - begin) & 7);
    c = next;
    if (((unit + 1 - begin) & 7) == 0) load_factors(unit + 1);
  }
  load_tokens(unit);
  multiply(c, unit, (unit - begin) & 7);
}

}  // namespace qz

