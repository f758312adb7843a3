// Products with MX4 weights: Y = X W^T + b, W [d_o x d_i] in MX4, X in bf16 or MX4.
#include <atomic>

#include "mx4.h"

namespace qz {

namespace {

// Four results of token t, rows r .. r + 3: the output with its bias, or the partial sums of a
// split (fp32 [split][n][d_o]).
__device__ __forceinline__ void store4(const Mx4Product& p, int split, int64_t t, int64_t r, f32x4 v) {
  if (r >= p.d_o) return;
  if (p.partial) {
    float* o = p.partial + (split * p.n + t) * p.d_o + r;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (r + i < p.d_o) o[i] = v[i];
    return;
  }
  const bool whole = r + 4 <= p.d_o;
  if (p.bias) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (r + i < p.d_o) v[i] += p.bias[r + i];
  }
  const int64_t at = t * p.ldy + r;
  if (p.yt == QZ_BF16) {
    uint16_t* o = static_cast<uint16_t*>(p.Y) + at;
    if (whole && p.y_vec) {
      const uint32_t lo = f32_to_bf16(v[0]) | (static_cast<uint32_t>(f32_to_bf16(v[1])) << 16);
      const uint32_t hi = f32_to_bf16(v[2]) | (static_cast<uint32_t>(f32_to_bf16(v[3])) << 16);
      *reinterpret_cast<uint2*>(o) = make_uint2(lo, hi);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (r + i < p.d_o) o[i] = f32_to_bf16(v[i]);
    }
  } else {
    float* o = static_cast<float*>(p.Y) + at;
    if (whole && p.y_vec) {
      *reinterpret_cast<f32x4*>(o) = v;
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (r + i < p.d_o) o[i] = v[i];
    }
  }
}

// ------------------------------------------------------------------------------ few tokens
// Workgroup of 16 RT rows of W by 16 NT tokens; its wavefronts take turns along d_i, a unit of 256
// columns at a time: whole 128-byte lines of codes, straight from global memory to the matrix
// cores, since every code is used once.  Of each 128 columns lane l loads row l % 16, block
// l / 16: 16 bytes of codes.  Sums in fp32; the wavefronts' sums are added in their order.
//
// bf16 X: a load of 16 bytes a lane covers 64 contiguous bytes of each row, so product j of the
// four takes the columns 32 j + 8 (l / 16) + 0..7 of X, and the codes have to follow: a 4 x 4
// transpose of words between the four lanes of a row (two pairs of lane swaps) turns word i of
// block l / 16 into word l / 16 of block i.  (With X read in the shape of whole blocks instead,
// each of the four loads touches the same two lines of every row, and a compute unit looks up a
// line in about four clocks: at 13 tokens that cost more than the codes did.)
//
// The next unit's loads are issued before the current one's products.
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

template <bool X4, int RT, int NT>
struct SkinnyUnit {
  uint4 c[2][RT];
  uint2 e[RT];
  uint4 x[2][NT][X4 ? 1 : 4];
  uint2 f[NT];
};

constexpr int kSkinnyWaves = 8;

template <bool X4, int RT, int NT>
__global__ __launch_bounds__(kSkinnyWaves * 64) void mx4_skinny_kernel(const Mx4Product p) {
  __shared__ f32x4 part[kSkinnyWaves][RT * NT][64];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), waves = blockDim.x >> 6;
  const int m = lane & 15, q = lane >> 4;
  const int64_t r0 = blockIdx.x * (int64_t)(16 * RT), t0 = blockIdx.y * (int64_t)(16 * NT);
  const int G = static_cast<int>(p.G);
  const uint8_t* wc[RT];
  const uint8_t* ws[RT];
  const uint8_t* xc[NT];
  const uint8_t* xs[NT];
  bool have[NT];   // lanes without a token read nothing
#pragma unroll
  for (int a = 0; a < RT; ++a) {
    const int64_t r = r0 + 16 * a + m < p.d_o ? r0 + 16 * a + m : p.d_o - 1;
    wc[a] = p.codes + r * G * 16 + 16 * q;
    ws[a] = p.scales + r * G;
  }
#pragma unroll
  for (int b = 0; b < NT; ++b) {
    have[b] = t0 + 16 * b + m < p.n;
    const int64_t t = have[b] ? t0 + 16 * b + m : p.n - 1;
    xc[b] = (X4 ? p.xcodes + t * G * 16 : reinterpret_cast<const uint8_t*>(p.X + t * p.ldx)) + 16 * q;
    xs[b] = X4 ? p.xscales + t * G : nullptr;
  }
  f32x4 acc[RT][NT];
#pragma unroll
  for (int a = 0; a < RT; ++a)
#pragma unroll
    for (int b = 0; b < NT; ++b) acc[a][b] = f32x4{0.f, 0.f, 0.f, 0.f};

  using Unit = SkinnyUnit<X4, RT, NT>;
  const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
  auto load = [&](int b0, Unit& v) {
    const bool whole = b0 + 8 <= G;
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int blk = b0 + 4 * u;
#pragma unroll
      for (int a = 0; a < RT; ++a) {
        v.c[u][a] = zero;
        if (whole || blk + q < G) v.c[u][a] = *reinterpret_cast<const uint4*>(wc[a] + blk * 16);
      }
#pragma unroll
      for (int b = 0; b < NT; ++b)
#pragma unroll
        for (int j = 0; j < (X4 ? 1 : 4); ++j) {
          v.x[u][b][j] = zero;
          if (have[b] && (whole || blk + (X4 ? q : j) < G))
            v.x[u][b][j] = *reinterpret_cast<const uint4*>(xc[b] + blk * (X4 ? 16 : 64) + 64 * j);
        }
    }
#pragma unroll
    for (int a = 0; a < RT; ++a) v.e[a] = eight_factors(ws[a], b0, G, whole);
    if constexpr (X4) {
#pragma unroll
      for (int b = 0; b < NT; ++b) v.f[b] = eight_factors(xs[b], b0, G, whole);
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
            for (int b = 0; b < NT; ++b)
              acc[a][b] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                  wv, __builtin_bit_cast(bf16x8, v.x[u][b][j]), acc[a][b], 0, 0, 0);
          }
        }
      }
    }
  };
  {
    Unit u0, u1;
    const int step = waves * 8;
    int b0 = wave * 8;
    if (b0 < G) load(b0, u0);
    while (b0 < G) {
      if (b0 + step < G) load(b0 + step, u1);
      multiply(u0);
      b0 += step;
      if (b0 >= G) break;
      if (b0 + step < G) load(b0 + step, u0);
      multiply(u1);
      b0 += step;
    }
  }

#pragma unroll
  for (int a = 0; a < RT; ++a)
#pragma unroll
    for (int b = 0; b < NT; ++b) part[wave][a * NT + b][lane] = acc[a][b];
  __syncthreads();
  for (int i = wave; i < RT * NT; i += waves) {   // the sums of RT NT tiles, a wavefront each
    f32x4 v = part[0][i][lane];
    for (int w = 1; w < waves; ++w) v += part[w][i][lane];
    const int64_t t = t0 + 16 * (i % NT) + m;
    if (t < p.n) store4(p, 0, t, r0 + 16 * (i / NT) + 4 * q, v);
  }
}

template <bool X4, int RT, int NT>
int launch_skinny(const Mx4Product& p, int waves, hipStream_t s) {
  const dim3 g(static_cast<unsigned>(ceil_div(p.d_o, 16 * RT)), static_cast<unsigned>(ceil_div(p.n, 16 * NT)));
  hipLaunchKernelGGL((mx4_skinny_kernel<X4, RT, NT>), g, dim3(64 * waves), 0, s, p);
  return check_launch("mx4_skinny");
}

// ---------------------------------------------------------------------------- large products
// Workgroup tile of BM rows of W by BN rows of X (tokens), BM = 32 MT WM, BN = 32 NT WN, in
// WM x WN wavefronts of 32 MT x 32 NT each.  Codes (and bf16 X) stream into LDS by
// global_load_lds, `kBlocks` blocks of every row a stage, `kRing` stages deep; weights are
// widened in registers on the way from LDS to the matrix cores.  In a stage lane l holds row
// (or token) l % 32 of a 32-row tile and, of each pair of blocks, block l / 32, so a lane's
// operand is one 16-byte read with one factor; the order of the contraction is free as long
// as both operands agree on it.
//
// LDS rows hold kBlocks 16-byte chunks (codes) or 8 (bf16 X of two blocks).  Chunk c of row r
// lies at chunk c ^ swz(r), with swz stepping once per 256 bytes of rows, so that 16 rows at the
// same column touch all 64 banks (stepping once per 128 bytes cost half of the LDS cycles in
// conflicts).  The copies keep LDS linear and permute their global sources instead.
//
// Factors come 16 blocks of a row at a time, by 4-byte copies where rows of factors are
// 4-byte aligned (G % 4 == 0 and the base), through registers otherwise.
template <bool X4>
struct TileGeom;
template <>
struct TileGeom<true> {    // 128 columns a stage: 64 bytes of codes a row on both sides
  static constexpr int kBlocks = 4, kRing = 4, kWRow = 64, kXRow = 64;
};
template <>
struct TileGeom<false> {   // 64 columns a stage: 32 bytes of codes, 128 bytes of X a row
  static constexpr int kBlocks = 2, kRing = 3, kWRow = 32, kXRow = 128;
};

template <int RB>
__device__ __forceinline__ int swz(int row) {
  return (row / (256 / RB)) & (RB / 16 - 1);
}

typedef __attribute__((address_space(3))) uint8_t lds_u8;

// One copy of a wavefront, lane i of it to LDS at dst + BYTES i: scalar base, 32-bit offsets.
// Inline asm, so that the compiler does not wait for it before every LDS read; it has no
// register result, and the stages are synchronised by explicit waits.
template <int BYTES>
__device__ __forceinline__ void copy_lds(lds_u8* dst, const uint8_t* base, uint32_t voff) {
  const uint32_t at = __builtin_amdgcn_readfirstlane(static_cast<uint32_t>(reinterpret_cast<uintptr_t>(dst)));
  const uint64_t b = reinterpret_cast<uint64_t>(base);
  const uint32_t lo = static_cast<uint32_t>(__builtin_amdgcn_readfirstlane(static_cast<uint32_t>(b)));
  const uint32_t hi = static_cast<uint32_t>(__builtin_amdgcn_readfirstlane(static_cast<uint32_t>(b >> 32)));
  const uint64_t su = (static_cast<uint64_t>(hi) << 32) | lo;
  if constexpr (BYTES == 16)
    asm volatile("s_mov_b32 m0, %0\n\tglobal_load_lds_dwordx4 %1, %2"
                 :: "s"(at), "v"(voff), "s"(su) : "memory", "m0");
  else
    asm volatile("s_mov_b32 m0, %0\n\tglobal_load_lds_dword %1, %2"
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

template <bool X4, int WM, int WN, int MT, int NT>
struct TileShape {
  using G = TileGeom<X4>;
  static constexpr int kThreads = WM * WN * 64;
  static constexpr int BM = 32 * MT * WM, BN = 32 * NT * WN;
  static constexpr int kStage = BM * G::kWRow + BN * G::kXRow;          // bytes of a stage
  static constexpr int kFRows = BM + (X4 ? BN : 0);                     // rows of factors
  static constexpr int kFactors = kFRows * 16;
  static constexpr int kLds = G::kRing * kStage + 2 * kFactors;
  static constexpr int kWPieces = BM * G::kWRow / 1024, kXPieces = BN * G::kXRow / 1024;
  static constexpr int kPieces = kWPieces + kXPieces;                   // copies of a stage
  static constexpr int kCopies = kPieces / (WM * WN);                   // of a wavefront; the first
  static constexpr int kExtra = kPieces % (WM * WN);                    // kExtra have one more
  static_assert(kLds <= 160 * 1024, "LDS of a compute unit");
};

template <bool X4, int WM, int WN, int MT, int NT>
__global__ __launch_bounds__(WM * WN * 64) void mx4_tile_kernel(const Mx4Product p, int tiles_w,
                                                                int tiles_x, int stages_per_split) {
  using T = TileShape<X4, WM, WN, MT, NT>;
  using Geo = TileGeom<X4>;
  constexpr int kWaves = WM * WN, kRing = Geo::kRing, kBlocks = Geo::kBlocks;
  constexpr int kPer = 16 / kBlocks;   // stages that one fetch of factors serves
  extern __shared__ __align__(1024) uint8_t smem[];
  lds_u8* const lds = (lds_u8*)smem;
  lds_u8* const fac = lds + kRing * T::kStage;

  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave / WN, wn = wave % WN;

  // The hardware deals workgroups to the 8 XCDs in turn.  Each XCD gets a run of consecutive
  // tiles, and runs go through 8 rows of W tiles by all X tiles, so the tiles that are
  // resident on an XCD share panels in its L2.
  const int split = blockIdx.y;
  int pid = blockIdx.x;
  {
    const int nb = gridDim.x, per = nb / 8, extra = nb % 8, x = pid % 8;
    pid = x * per + (x < extra ? x : extra) + pid / 8;
  }
  constexpr int kGroup = 8;
  const int in_group = kGroup * tiles_x;
  const int g0 = pid / in_group * kGroup;
  const int gh = tiles_w - g0 < kGroup ? tiles_w - g0 : kGroup;
  const int64_t r0 = static_cast<int64_t>(g0 + pid % in_group % gh) * T::BM;
  const int64_t t0 = static_cast<int64_t>(pid % in_group / gh) * T::BN;

  const int64_t Gb = p.G;
  const int all = static_cast<int>(ceil_div(Gb, kBlocks));
  const int st0 = split * stages_per_split;
  const int nst = all - st0 < stages_per_split ? all - st0 : stages_per_split;   // >= 1
  const int full = static_cast<int>(Gb / kBlocks);   // stages before the ragged one

  // Copy roles: wavefront w makes the copies w, w + kWaves, ... of a stage, 1024 bytes of LDS
  // each, whole rows.  Rows past the matrix read its last row again; their results are not
  // stored.
  constexpr int kMine = T::kCopies + (T::kExtra ? 1 : 0);
  uint32_t off[kMine];
  constexpr int wl = Geo::kWRow / 16, xl = Geo::kXRow / 16;
  const int wchunk = (lane % wl) ^ swz<Geo::kWRow>(lane / wl);   // swz repeats after 16 rows
  auto xchunk = [&](int piece) {   // a copy of bf16 X is only 8 rows
    return (lane % xl) ^ swz<Geo::kXRow>((piece - T::kWPieces) * (64 / xl) + lane / xl);
  };
  {
    const int64_t xp = X4 ? Gb * 16 : p.ldx * 2;
#pragma unroll
    for (int j = 0; j < kMine; ++j) {
      const int piece = wave + j * kWaves;
      if (piece < T::kWPieces) {
        const int row = piece * (64 / wl) + lane / wl;
        const int64_t r = r0 + row < p.d_o ? row : p.d_o - 1 - r0;
        off[j] = static_cast<uint32_t>(r * Gb * 16 + 16 * wchunk);
      } else {
        const int row = (piece - T::kWPieces) * (64 / xl) + lane / xl;
        const int64_t t = t0 + row < p.n ? row : p.n - 1 - t0;
        off[j] = static_cast<uint32_t>(t * xp + 16 * xchunk(piece));
      }
    }
  }
  const uint8_t* const wbase = p.codes + r0 * Gb * 16;
  const uint8_t* const xbase = X4 ? p.xcodes + t0 * Gb * 16
                                  : reinterpret_cast<const uint8_t*>(p.X) + t0 * p.ldx * 2;
  const bool dword_factors = Gb % 4 == 0 && p.factors_aligned;

  // Factors of 16 blocks from block b0 on, to buffer `buf`: row i at 16 i.
  auto fetch_factors = [&](int64_t b0, int buf) {
    lds_u8* const dst = fac + buf * T::kFactors;
    if (dword_factors) {
#pragma unroll
      for (int j = 0; j < (T::kFRows / 16 + kWaves - 1) / kWaves; ++j) {
        const int piece = wave + j * kWaves;      // 16 rows of four words
        if (piece * 16 >= T::kFRows) break;
        const int row = piece * 16 + lane / 4;
        const int64_t b = b0 + 4 * (lane % 4);
        lds_u8* const at = dst + piece * 256;
        if (b < Gb) {
          if (!X4 || piece * 16 < T::BM) {
            const int64_t r = r0 + row < p.d_o ? row : p.d_o - 1 - r0;
            copy_lds<4>(at, p.scales + r0 * Gb, static_cast<uint32_t>(r * Gb + b));
          } else {
            const int64_t t = t0 + row - T::BM < p.n ? row - T::BM : p.n - 1 - t0;
            copy_lds<4>(at, p.xscales + t0 * Gb, static_cast<uint32_t>(t * Gb + b));
          }
        } else {
          *(__attribute__((address_space(3))) uint32_t*)(at + 4 * lane) = 0x7f7f7f7fu;
        }
      }
    } else {
      for (int row = tid; row < T::kFRows; row += T::kThreads) {
        const uint8_t* src;
        if (!X4 || row < T::BM)
          src = p.scales + (r0 + row < p.d_o ? r0 + row : p.d_o - 1) * Gb;
        else
          src = p.xscales + (t0 + row - T::BM < p.n ? t0 + row - T::BM : p.n - 1) * Gb;
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          w[i] = 0;
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const int64_t b = b0 + 4 * i + k;
            w[i] |= (b < Gb ? static_cast<uint32_t>(src[b]) : kMxOne) << (8 * k);
          }
        }
        *(__attribute__((address_space(3))) i32x4*)(dst + 16 * row) =
            i32x4{static_cast<int>(w[0]), static_cast<int>(w[1]), static_cast<int>(w[2]), static_cast<int>(w[3])};
      }
    }
  };

  auto issue = [&](int st) {   // stage st (counted from st0) into its ring slot
    const int64_t b0 = static_cast<int64_t>(st0 + st) * kBlocks;
    if (st % kPer == 0) fetch_factors(b0, (st / kPer) & 1);
    lds_u8* const dst = lds + (st % kRing) * T::kStage;
    const bool whole = st0 + st < full;
#pragma unroll
    for (int j = 0; j < kMine; ++j) {
      const int piece = wave + j * kWaves;
      if (piece >= T::kPieces) break;
      lds_u8* const at = dst + piece * 1024;
      const bool w = piece < T::kWPieces;
      if (whole || b0 + (w ? wchunk : X4 ? xchunk(piece) : xchunk(piece) / 4) < Gb)
        copy_lds<16>(at, w ? wbase + b0 * 16 : xbase + b0 * (X4 ? 16 : 64), off[j]);
      else
        *(__attribute__((address_space(3))) i32x4*)(at + 16 * lane) = i32x4{0, 0, 0, 0};
    }
  };

  f32x16 acc[MT][NT];
#pragma unroll
  for (int a = 0; a < MT; ++a)
#pragma unroll
    for (int b = 0; b < NT; ++b)
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[a][b][r] = 0.f;

  // Stage st + 1 has landed: everything but the copies of the kRing - 2 stages after it, which
  // may be in flight where those stages are whole (a wavefront then has issued exactly its
  // number of copies for each; a fetch of factors only makes the wait longer).
  auto landed = [&](int st) {
    if (st + kRing - 1 >= nst || st0 + st + kRing - 1 >= full)
      wait_and_join<0>();
    else if (wave < T::kExtra)
      wait_and_join<(kRing - 2) * (T::kCopies + 1)>();
    else
      wait_and_join<(kRing - 2) * T::kCopies>();
  };

#pragma unroll
  for (int i = 0; i < kRing - 1; ++i)
    if (i < nst) issue(i);
  landed(-1);

  const int row = lane & 31, half = lane >> 5;
  for (int st = 0; st < nst; ++st) {
    if (st + kRing - 1 < nst) issue(st + kRing - 1);
    lds_u8* const ws = lds + (st % kRing) * T::kStage + (wm * 32 * MT + row) * Geo::kWRow;
    lds_u8* const xs = lds + (st % kRing) * T::kStage + T::BM * Geo::kWRow +
                       (wn * 32 * NT + row) * Geo::kXRow;
    lds_u8* const fw = fac + ((st / kPer) & 1) * T::kFactors + (wm * 32 * MT + row) * 16 +
                       (st % kPer) * kBlocks;
    auto rd16 = [](lds_u8* q) {
      return *(__attribute__((address_space(3))) i32x4*)q;
    };
    if constexpr (X4) {
      lds_u8* const fx = fw + (T::BM + wn * 32 * NT - wm * 32 * MT) * 16;
      int ew[MT], ex[NT];
#pragma unroll
      for (int a = 0; a < MT; ++a)
        ew[a] = static_cast<int>(*(__attribute__((address_space(3))) uint32_t*)(fw + a * 512) >> (8 * half));
#pragma unroll
      for (int b = 0; b < NT; ++b)
        ex[b] = static_cast<int>(*(__attribute__((address_space(3))) uint32_t*)(fx + b * 512) >> (8 * half));
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        i32x8 wv[MT], xv[NT];
        const int cw = 16 * ((2 * s + half) ^ swz<Geo::kWRow>(row));
#pragma unroll
        for (int a = 0; a < MT; ++a) {
          const i32x4 c = rd16(ws + a * 32 * Geo::kWRow + cw);
          wv[a] = i32x8{c[0], c[1], c[2], c[3], 0, 0, 0, 0};
        }
#pragma unroll
        for (int b = 0; b < NT; ++b) {
          const i32x4 c = rd16(xs + b * 32 * Geo::kXRow + cw);
          xv[b] = i32x8{c[0], c[1], c[2], c[3], 0, 0, 0, 0};
        }
#pragma unroll
        for (int a = 0; a < MT; ++a)
#pragma unroll
          for (int b = 0; b < NT; ++b) {
            if (s == 0)
              acc[a][b] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(wv[a], xv[b], acc[a][b], 4, 4,
                                                                         0, ew[a], 0, ex[b]);
            else
              acc[a][b] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(wv[a], xv[b], acc[a][b], 4, 4,
                                                                         2, ew[a], 2, ex[b]);
          }
      }
    } else {
      const int cw = 16 * (half ^ swz<Geo::kWRow>(row));
      i32x4 c[MT];
      float f[MT];
#pragma unroll
      for (int a = 0; a < MT; ++a) {
        c[a] = rd16(ws + a * 32 * Geo::kWRow + cw);
        f[a] = mx_factor(fw[a * 512 + half]);
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        bf16x8 xv[NT];
#pragma unroll
        for (int b = 0; b < NT; ++b)
          xv[b] = __builtin_bit_cast(bf16x8, rd16(xs + b * 32 * Geo::kXRow + 16 * ((4 * half + j) ^ swz<Geo::kXRow>(row))));
#pragma unroll
        for (int a = 0; a < MT; ++a) {
          const bf16x8 wv = mx_word_bf16(static_cast<uint32_t>(c[a][j]), f[a]);
#pragma unroll
          for (int b = 0; b < NT; ++b)
            acc[a][b] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(wv, xv[b], acc[a][b], 0, 0, 0);
        }
      }
    }
    if (st + 1 < nst) landed(st);
  }

  // Register r of lane l: row 8 (r / 4) + 4 (l / 32) + r % 4 of a tile, token l % 32.
#pragma unroll
  for (int b = 0; b < NT; ++b) {
    const int64_t t = t0 + (wn * NT + b) * 32 + row;
    if (t >= p.n) continue;
#pragma unroll
    for (int a = 0; a < MT; ++a)
#pragma unroll
      for (int r4 = 0; r4 < 4; ++r4) {
        const int64_t r = r0 + (wm * MT + a) * 32 + 8 * r4 + 4 * half;
        f32x4 v = {acc[a][b][4 * r4], acc[a][b][4 * r4 + 1], acc[a][b][4 * r4 + 2], acc[a][b][4 * r4 + 3]};
        store4(p, split, t, r, v);
      }
  }
}

template <bool X4, int WM, int WN, int MT, int NT>
int launch_tile(const Mx4Product& p, int splits, hipStream_t s) {
  using T = TileShape<X4, WM, WN, MT, NT>;
  const auto kernel = mx4_tile_kernel<X4, WM, WN, MT, NT>;
  static std::atomic<uint64_t> allowed{0};   // devices on which the kernel may use its LDS
  int dev = 0;
  QZ_HIP(hipGetDevice(&dev));
  if (dev > 63 || !(allowed.load(std::memory_order_relaxed) >> dev & 1)) {
    QZ_HIP(hipFuncSetAttribute(reinterpret_cast<const void*>(kernel),
                               hipFuncAttributeMaxDynamicSharedMemorySize, T::kLds));
    if (dev <= 63) allowed.fetch_or(uint64_t{1} << dev, std::memory_order_relaxed);
  }
  const int tw = static_cast<int>(ceil_div(p.d_o, T::BM)), tx = static_cast<int>(ceil_div(p.n, T::BN));
  const int all = static_cast<int>(ceil_div(p.G, TileGeom<X4>::kBlocks));
  const int per = static_cast<int>(ceil_div(all, splits));
  hipLaunchKernelGGL(kernel, dim3(static_cast<unsigned>(tw) * tx, static_cast<unsigned>(ceil_div(all, per))),
                     dim3(T::kThreads), T::kLds, s, p, tw, tx, per);
  return check_launch("mx4_tile");
}

// Rows of X copied to rows of whole blocks, zero beyond d_i.
__global__ __launch_bounds__(256) void mx4_pad_kernel(const uint16_t* __restrict__ X, int64_t n,
                                                      int64_t d_i, int64_t ldx,
                                                      uint16_t* __restrict__ out, int64_t ldo) {
  for (int64_t t = blockIdx.x * (int64_t)256 + threadIdx.x; t < n * ldo;
       t += (int64_t)gridDim.x * 256) {
    const int64_t r = t / ldo, c = t % ldo;
    out[t] = c < d_i ? X[r * ldx + c] : static_cast<uint16_t>(0);
  }
}

}  // namespace

int launch_mx4_pad(const uint16_t* X, int64_t n, int64_t d_i, int64_t ldx, uint16_t* out,
                   int64_t ldo, hipStream_t s) {
  const int64_t b = ceil_div(n * ldo, 256);
  hipLaunchKernelGGL(mx4_pad_kernel, dim3(static_cast<unsigned>(b < 65536 ? b : 65536)), dim3(256),
                     0, s, X, n, d_i, ldx, out, ldo);
  return check_launch("mx4_pad");
}

int mx4_product_splits(bool, int64_t, int64_t, int64_t) { return 1; }

namespace {

template <bool X4>
int launch_product(const Mx4Product& p, hipStream_t s) {
  if (p.n > 64) return launch_tile<X4, 2, 4, 4, 2>(p, 1, s);
  return launch_skinny<X4, 1, 1>(p, 8, s);
}

}  // namespace

int launch_mx4_product(const Mx4Product& p, hipStream_t s) {
  return p.X ? launch_product<false>(p, s) : launch_product<true>(p, s);
}

}  // namespace qz
