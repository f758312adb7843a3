// Products with MX4 weights: Y = X W^T + b, W [d_o x d_i] in MX4, X in bf16 or MX4.
#include <atomic>
#include <cmath>

#include "lds_copy.h"
#include "mx4_few.h"

namespace qz {

namespace {

// Four results of token t, rows r .. r + 3, with their bias.
__device__ __forceinline__ void store4(const Mx4Product& p, int64_t t, int64_t r, f32x4 v) {
  if (r >= p.d_o) return;
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
// Workgroup of 16 RT rows of W by 16 NT tokens; each of its wavefronts has a part of d_i (mx4_few.h).
// Sums in fp32; the wavefronts' sums are added in their order.
//
// Bound by reading W, and below about 10 MB by the launch (3 us): 13 tokens 12288 -> 4096 bf16 8.9
// us (26.7 MB; 4.3 at 6.2 TB/s), one token 4096 -> 1024 4.7, one token 5120 -> 25600 17.0 (2 x 1; 69.6
// MB, 4.1 TB/s).  More rows a workgroup (RT) load the tokens less often, more tokens (NT) the rows.
template <int RT, int NT>
constexpr int kSkinnyWaves = RT * NT == 1 ? 8 : 4;

template <bool X4, int RT, int NT>
__global__ __launch_bounds__((kSkinnyWaves<RT, NT>) * 64) void mx4_skinny_kernel(const Mx4Product p) {
  __shared__ f32x4 part[kSkinnyWaves<RT, NT>][RT * NT][64];
  __shared__ __align__(16) uint8_t lds[kSkinnyWaves<RT, NT>][kFewLds<true, X4, RT, NT>];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), waves = blockDim.x >> 6;
  const int m = lane & 15, q = lane >> 4;
  const int64_t r0 = blockIdx.x * (int64_t)(16 * RT), t0 = blockIdx.y * (int64_t)(16 * NT);
  const int G = static_cast<int>(p.G);
  FewRows<X4, RT, NT> rows;
#pragma unroll
  for (int a = 0; a < RT; ++a) {
    const int64_t r = r0 + 16 * a < p.d_o ? r0 + 16 * a : p.d_o - 1;
    rows.codes[a] = p.codes + r * G * 16;
    rows.scales[a] = p.scales + r * G;
    rows.last[a] = static_cast<int>(p.d_o - 1 - r < 15 ? p.d_o - 1 - r : 15);
  }
#pragma unroll
  for (int b = 0; b < NT; ++b) {
    const auto token = [&](int i) { return t0 + 16 * b + i < p.n ? t0 + 16 * b + i : p.n - 1; };
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int64_t t = token(8 * h + lane / 8);
      rows.x[b][h] = X4 ? p.xcodes + t * G * 16 : reinterpret_cast<const uint8_t*>(p.X + t * p.ldx);
    }
    rows.xs[b] = X4 ? p.xscales + token(m) * G : nullptr;
  }
  f32x4 acc[RT][NT];
#pragma unroll
  for (int a = 0; a < RT; ++a)
#pragma unroll
    for (int b = 0; b < NT; ++b) acc[a][b] = f32x4{0.f, 0.f, 0.f, 0.f};
  const int units = (G + 7) / 8, mine = (units + waves - 1) / waves;
  const int u0 = wave * mine, u1 = u0 + mine < units ? u0 + mine : units;
  few_products<X4 || RT * NT == 1, true>(rows, lds[wave], G, u0, u1, acc);

#pragma unroll
  for (int a = 0; a < RT; ++a)
#pragma unroll
    for (int b = 0; b < NT; ++b) part[wave][a * NT + b][lane] = acc[a][b];
  __syncthreads();
  for (int i = wave; i < RT * NT; i += waves) {   // the sums of RT NT tiles, a wavefront each
    f32x4 v = part[0][i][lane];
    for (int w = 1; w < waves; ++w) v += part[w][i][lane];
    const int64_t t = t0 + 16 * (i % NT) + m;
    if (t < p.n) store4(p, t, r0 + 16 * (i / NT) + 4 * q, v);
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
// global_load_lds; weights are widened in registers between LDS and the matrix cores.  Of a pair
// of blocks, lane l holds row (or token) l % 32 of a 32-row tile and block l / 32 of the pair, so
// an operand is one 16-byte read with one factor; the order of the contraction is free as long as
// both operands agree on it.
//
// What sets the shapes: a compute unit takes about one row segment (up to a 128-byte line) from
// L2 in 3.5 clocks, whatever its length (measured on the copies alone: 14 B/clk in 64-byte pieces,
// 23 with mostly 128-byte ones), and 32 x 32 products of 64 columns take 32 clocks of a SIMD.  So:
//   X in MX4: stages of 256 columns, 128 bytes of a row on both sides, two of them in LDS;
//   X in bf16: stages of 64 columns of X (128 bytes a row), three in LDS, and W in pairs of
//   stages (64 bytes a row), two pairs in LDS, half the rows of a pair copied with each stage;
//   factors: 64 of a row at a time (a fetch costs a request a row, like a stage).
// LDS rows are swizzled in 16-byte chunks: chunk c of row r lies at chunk c ^ swz(r), stepping
// once per 256 bytes of rows, so that 16 rows at the same column touch all 64 banks (stepping
// once per 128 bytes cost half of the LDS cycles in conflicts).  The copies keep LDS linear and
// permute their global sources instead.
//
// Measured: 8192 tokens 5120 -> 25600 bf16 1.85 to 1.89 ms, 1.14 to 1.16 PFLOP/s (the library's bf16
// product of the same sizes, on widened weights, 1.63 ms; both draw the card's 1400 W; matrix cores
// busy 51% at 2.13 GHz; of the kernel's parts alone the products take 1.38 to 1.57 ms, the copies
// 0.74); 2048 tokens 4096 -> 4096 71 to 72 us (0.96 PFLOP/s; the library 55 to 58; busy 37%); MX4 X,
// 4096 tokens 4096 -> 12288 123 to 133 us (3.1 to 3.35 PFLOP/s; busy 35% at 2.26 GHz, 1329 W):
// products alone 85% of that, copies 67%, the epilogue 12%.
template <bool X4, int WM, int WN, int MT, int NT>
__global__ __launch_bounds__(WM * WN * 64, 2) void mx4_tile_kernel(const Mx4Product p, int tiles_w,
                                                                int tiles_x, int stages_per_split) {
  using T = TileShape<X4, WM, WN, MT, NT>;
  using Geo = TileGeom<X4>;
  constexpr int kRing = Geo::kRing, kBlocks = Geo::kBlocks, kParts = Geo::kWParts;
  constexpr int kPer = kFetch / kBlocks;   // stages that one fetch of factors serves
  extern __shared__ __align__(1024) uint8_t smem[];
  lds_u8* const lds_w = (lds_u8*)smem;
  lds_u8* const lds_x = lds_w + T::kWBuffers * T::kWBytes;
  lds_u8* const lds_f = lds_x + kRing * T::kXBytes;

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
  // (the divisions leave the uniform tile in vector registers, and with it every address)
  const int64_t r0 = static_cast<int64_t>(__builtin_amdgcn_readfirstlane(g0 + pid % in_group % gh)) * T::BM;
  const int64_t t0 = static_cast<int64_t>(__builtin_amdgcn_readfirstlane(pid % in_group / gh)) * T::BN;
  // last rows inside the matrices, counted in the tile: rows past them read these again
  const int last_r = static_cast<int>(p.d_o - 1 - r0 < T::BM ? p.d_o - 1 - r0 : T::BM);
  const int last_t = static_cast<int>(p.n - 1 - t0 < T::BN ? p.n - 1 - t0 : T::BN);

  const int Gb = static_cast<int>(p.G);
  const int all = (Gb + kBlocks - 1) / kBlocks;
  const int st0 = split * stages_per_split;
  const int nst = all - st0 < stages_per_split ? all - st0 : stages_per_split;   // >= 1
  const int whole = Gb / kBlocks - st0;     // stages of this split before the ragged one
  const int first = st0 * kBlocks;          // its first block

  const uint32_t w_pitch = static_cast<uint32_t>(Gb) * 16;
  const uint32_t x_pitch = X4 ? w_pitch : static_cast<uint32_t>(p.ldx) * 2;
  const uint8_t* const wbase = p.codes + r0 * w_pitch + static_cast<int64_t>(first) * 16;
  const uint8_t* const xbase = X4 ? p.xcodes + t0 * w_pitch + static_cast<int64_t>(first) * 16
                                  : reinterpret_cast<const uint8_t*>(p.X + t0 * p.ldx) + static_cast<int64_t>(first) * 64;

  // Stage st (of this split) into its buffers: wavefront w makes the copies w, w + waves, ...
  // of whole LDS rows.  The lanes' offsets are formed anew each time: kept in registers they
  // would push the accumulators out.
  auto zero16 = [&](lds_u8* at) {
    *(__attribute__((address_space(3))) i32x4*)(at + 16 * lane) = i32x4{0, 0, 0, 0};
  };
  auto copy_w = [&](int st, int piece, int ln, bool full) {
    constexpr int per = Geo::kWRow / 16;
    const int wp = piece + (st % kParts) * T::kWPieces;
    const int r = wp * (64 / per) + ln / per, chunk = (ln % per) ^ swz<Geo::kWRow>(r);
    const int b = st / kParts * (kParts * kBlocks);     // first block of the buffer
    lds_u8* const at = lds_w + (st / kParts % T::kWBuffers) * T::kWBytes + wp * 1024;
    if (full || first + b + chunk < Gb)
      copy_lds<16>(at, wbase + static_cast<int64_t>(b) * 16,
                   static_cast<uint32_t>(r < last_r ? r : last_r) * w_pitch + 16 * chunk);
    else
      zero16(at);
  };
  auto copy_x = [&](int st, int piece, int ln, bool full) {
    constexpr int per = Geo::kXRow / 16;
    const int r = piece * (64 / per) + ln / per, chunk = (ln % per) ^ swz<Geo::kXRow>(r);
    lds_u8* const at = lds_x + (st % kRing) * T::kXBytes + piece * 1024;
    if (full || first + st * kBlocks + (X4 ? chunk : chunk / 4) < Gb)
      copy_lds<16>(at, xbase + static_cast<int64_t>(st) * (kBlocks * (X4 ? 16 : 64)),
                   static_cast<uint32_t>(r < last_t ? r : last_t) * x_pitch + 16 * chunk);
    else
      zero16(at);
  };
  auto copies = [&](int st, bool full) {
    int ln = lane;
    asm volatile("" : "+v"(ln));
#pragma unroll
    for (int j = 0; j < T::kCopies + (T::kExtra ? 1 : 0); ++j) {
      const int piece = wave + j * T::kWaves;
      if ((j + 1) * T::kWaves <= T::kWPieces) {
        copy_w(st, piece, ln, full);
      } else if (j * T::kWaves >= T::kWPieces) {
        if (piece < T::kPieces && st < nst) copy_x(st, piece - T::kWPieces, ln, full);
      } else if (piece < T::kWPieces) {
        copy_w(st, piece, ln, full);
      } else if (piece < T::kPieces && st < nst) {
        copy_x(st, piece - T::kWPieces, ln, full);
      }
    }
  };
  const int issues = static_cast<int>(round_up(nst, kParts));   // the last one may be W's alone
  auto issue = [&](int st) {
    if (st / kParts * kParts + kParts <= whole)
      copies(st, true);
    else
      copies(st, false);
  };

  // kFetch factors of every row from block b0 on (counted from `first`).  Word k of row r lies at
  // word k ^ (r % 16) of its 64 bytes, off the banks of its neighbours.
  const bool word_factors = Gb % 4 == 0 && p.factors_aligned;
  auto fetch_factors = [&](int b0) {
    if (word_factors) {
      int ln = lane;
      asm volatile("" : "+v"(ln));
      for (int piece = wave; piece < T::kFRows / 4; piece += T::kWaves) {   // four rows each
        const int row = piece * 4 + ln / 16;
        const int b = first + b0 + 4 * ((ln % 16) ^ (row % 16));
        lds_u8* const at = lds_f + piece * 256;
        if (b < Gb) {
          if (!X4 || piece < T::BM / 4)
            copy_lds<4>(at, p.scales + r0 * Gb, static_cast<uint32_t>((row < last_r ? row : last_r) * Gb + b));
          else
            copy_lds<4>(at, p.xscales + t0 * Gb,
                        static_cast<uint32_t>((row - T::BM < last_t ? row - T::BM : last_t) * Gb + b));
        }
        else
          *(__attribute__((address_space(3))) uint32_t*)(at + 4 * lane) = 0x7f7f7f7fu;
      }
    } else {
      for (int i = tid; i < T::kFRows * 16; i += T::kThreads) {
        const int row = i / 16, k = i % 16;
        const bool w = !X4 || row < T::BM;
        const int r = w ? (row < last_r ? row : last_r) : (row - T::BM < last_t ? row - T::BM : last_t);
        const uint8_t* src = (w ? p.scales + r0 * Gb : p.xscales + t0 * Gb) + static_cast<int64_t>(r) * Gb;
        uint32_t v = 0;
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const int b = first + b0 + 4 * k + c;
          v |= (b < Gb ? static_cast<uint32_t>(src[b]) : kMxOne) << (8 * c);
        }
        *(__attribute__((address_space(3))) uint32_t*)(lds_f + row * kFetch + 4 * (k ^ (row % 16))) = v;
      }
    }
  };

  f32x16 acc[MT][NT];
#pragma unroll
  for (int a = 0; a < MT; ++a)
#pragma unroll
    for (int b = 0; b < NT; ++b)
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[a][b][r] = 0.f;

  // Stage st + 1 has landed for every wavefront, and every wavefront is done with the LDS reads
  // of stage st.
  auto join = [&](int st) {
    const TileWait wait = tile_wait<X4>(st, nst, whole);
    if (wait == TileWait::kAll)
      wait_and_join<0>();
    else if (wait == TileWait::kButX)
      wait_and_join<T::kXLeast>();
    else if (wave < T::kExtra)
      wait_and_join<T::kCopies + 1>();
    else
      wait_and_join<T::kCopies>();
  };

  const int row = lane & 31, half = lane >> 5;
  lds_u8* const my_w = lds_w + (wm * 32 * MT + row) * Geo::kWRow;
  lds_u8* const my_x = lds_x + (wn * 32 * NT + row) * Geo::kXRow;
  lds_u8* const my_fw = lds_f + (wm * 32 * MT + row) * kFetch;
  lds_u8* const my_fx = lds_f + (T::BM + wn * 32 * NT + row) * kFetch;
  auto rd16 = [](lds_u8* q) { return *(__attribute__((address_space(3))) i32x4*)q; };
  auto rd4 = [](lds_u8* q) { return *(__attribute__((address_space(3))) uint32_t*)q; };

  // A stage is worked through in steps; the operands of a step are read from LDS into the
  // second of two register sets while the matrix cores work on the first, and a stage's last
  // step runs beside the reads of the next stage's first one, behind the join.
#define QZ_FENCE __builtin_amdgcn_sched_barrier(0)
  // Products may be moved past branches (they have no side effects), down to the end of the
  // stage and with all its operands alive: this keeps those before it where they are.
  auto pin = [&] {
#pragma unroll
    for (int a = 0; a < MT; ++a)
#pragma unroll
      for (int b = 0; b < NT; ++b) asm volatile("" : "+v"(acc[a][b]));
  };
  fetch_factors(0);
#pragma unroll
  for (int i = 0; i < kRing; ++i)
    if (i < issues) issue(i);
  wait_and_join<0>();

  // The factors of stage st are in registers everywhere when a fetch replaces them: the last
  // stage of a fetch meets the others once more, and the fetch has the rest of it to land.
  auto refetch = [&](int st) {
    if ((st + 1) % kPer == 0 && st + 1 < nst) {
      asm volatile("" ::: "memory");
      __builtin_amdgcn_s_waitcnt(15 | (3 << 14) | (7 << 4));   // lgkmcnt = 0
      __builtin_amdgcn_s_barrier();
      asm volatile("" ::: "memory");
      fetch_factors((st + 1) * kBlocks);
    }
  };

  if constexpr (X4) {
    i32x4 w0[MT], x0[NT], w1[MT], x1[NT];
    uint32_t ew[MT], ex[NT], nw[MT], nx[NT];
    auto load = [&](int st, int s, i32x4 (&w)[MT], i32x4 (&x)[NT]) {
      const int c = 16 * ((4 * half + s) ^ swz<128>(row));
#pragma unroll
      for (int a = 0; a < MT; ++a) w[a] = rd16(my_w + (st % kRing) * T::kWBytes + a * 32 * 128 + c);
#pragma unroll
      for (int b = 0; b < NT; ++b) x[b] = rd16(my_x + (st % kRing) * T::kXBytes + b * 32 * 128 + c);
    };
    auto load_factors = [&](int st) {
      const int k = 4 * ((2 * (st % kPer) + half) ^ (row % 16));
#pragma unroll
      for (int a = 0; a < MT; ++a) nw[a] = rd4(my_fw + a * 32 * kFetch + k);
#pragma unroll
      for (int b = 0; b < NT; ++b) nx[b] = rd4(my_fx + b * 32 * kFetch + k);
    };
    auto multiply = [&](auto s, const i32x4 (&w)[MT], const i32x4 (&x)[NT]) {
#pragma unroll
      for (int a = 0; a < MT; ++a)
#pragma unroll
        for (int b = 0; b < NT; ++b) {
          const i32x8 wv = {w[a][0], w[a][1], w[a][2], w[a][3], 0, 0, 0, 0};
          const i32x8 xv = {x[b][0], x[b][1], x[b][2], x[b][3], 0, 0, 0, 0};
          acc[a][b] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(
              wv, xv, acc[a][b], 4, 4, decltype(s)::value, static_cast<int>(ew[a]),
              decltype(s)::value, static_cast<int>(ex[b]));
        }
    };
    using std::integral_constant;
    load(0, 0, w0, x0);
    load_factors(0);
    for (int st = 0; st < nst; ++st) {
#pragma unroll
      for (int a = 0; a < MT; ++a) ew[a] = nw[a];
#pragma unroll
      for (int b = 0; b < NT; ++b) ex[b] = nx[b];
      refetch(st);
      load(st, 1, w1, x1);
      QZ_FENCE;
      multiply(integral_constant<int, 0>{}, w0, x0);
      QZ_FENCE;
      load(st, 2, w0, x0);
      QZ_FENCE;
      multiply(integral_constant<int, 1>{}, w1, x1);
      QZ_FENCE;
      load(st, 3, w1, x1);
      QZ_FENCE;
      multiply(integral_constant<int, 2>{}, w0, x0);
      QZ_FENCE;
      pin();
      if (st + 1 < nst) {
        join(st);
        if (st + kRing < issues) issue(st + kRing);
        load(st + 1, 0, w0, x0);
        load_factors(st + 1);
      }
      QZ_FENCE;
      multiply(integral_constant<int, 3>{}, w1, x1);
      QZ_FENCE;
      pin();
    }
  } else {
    i32x4 c[MT], cn[MT], x0[NT], x1[NT];
    uint32_t f[MT], fn[MT];   // factors of the four blocks of a pair of stages
    auto load_w = [&](int st) {
      const int at = (st / 2 % 2) * T::kWBytes + 16 * ((2 * (st % 2) + half) ^ swz<64>(row));
      const int k = 4 * ((st % kPer / 2) ^ (row % 16));
#pragma unroll
      for (int a = 0; a < MT; ++a) {
        cn[a] = rd16(my_w + a * 32 * 64 + at);
        fn[a] = rd4(my_fw + a * 32 * kFetch + k);
      }
    };
    auto load_x = [&](int st, int j, i32x4 (&x)[NT]) {
      const int at = (st % kRing) * T::kXBytes + 16 * ((4 * half + j) ^ swz<128>(row));
#pragma unroll
      for (int b = 0; b < NT; ++b) x[b] = rd16(my_x + b * 32 * 128 + at);
    };
    auto multiply = [&](int j, const i32x4 (&x)[NT]) {
#pragma unroll
      for (int a = 0; a < MT; ++a) {
        const bf16x8 wv = mx_word_bf16(static_cast<uint32_t>(c[a][j]), __uint_as_float(f[a]));
#pragma unroll
        for (int b = 0; b < NT; ++b)
          acc[a][b] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(wv, __builtin_bit_cast(bf16x8, x[b]),
                                                              acc[a][b], 0, 0, 0);
      }
    };
    load_w(0);
    load_x(0, 0, x0);
    for (int st = 0; st < nst; ++st) {
#pragma unroll
      for (int a = 0; a < MT; ++a) {
        c[a] = cn[a];
        f[a] = (fn[a] >> (8 * (2 * (st % 2) + half)) & 255u) << 23;
      }
      refetch(st);
      load_x(st, 1, x1);
      QZ_FENCE;
      multiply(0, x0);
      QZ_FENCE;
      load_x(st, 2, x0);
      QZ_FENCE;
      multiply(1, x1);
      QZ_FENCE;
      load_x(st, 3, x1);
      QZ_FENCE;
      multiply(2, x0);
      QZ_FENCE;
      pin();
      if (st + 1 < nst) {
        join(st);
        if (st + kRing < issues) issue(st + kRing);
        load_w(st + 1);
        load_x(st + 1, 0, x0);
      }
      QZ_FENCE;
      multiply(3, x1);
      QZ_FENCE;
      pin();
    }
  }
#undef QZ_FENCE

  // Register r of lane l: row 8 (r / 4) + 4 (l / 32) + r % 4 of a tile, token l % 32.  32 tokens
  // at a time go through LDS of the wavefront's own, so that Y is written in whole lines.
  const int osize = p.partial || p.yt == QZ_F32 ? 4 : 2;
  uint8_t* const ybase = p.partial ? reinterpret_cast<uint8_t*>(p.partial + split * p.n * p.d_o)
                                   : static_cast<uint8_t*>(p.Y);
  const int64_t ld = p.partial ? p.d_o : p.ldy;
  const bool lines = ld * osize % 16 == 0 && reinterpret_cast<uintptr_t>(ybase) % 16 == 0;
  lds_u8* const out = (lds_u8*)smem + wave * 32 * T::kOutPitch;
  const int64_t wr0 = r0 + wm * 32 * MT;
  const bool biased = p.bias && !p.partial;
  lds_u8* const bias = (lds_u8*)smem + T::kOut;
  __syncthreads();
  if (biased) {   // once into LDS: a load for every four results cost a fifth of the kernel's time
    for (int i = tid; i < T::BM; i += T::kThreads)
      *(__attribute__((address_space(3))) float*)(bias + 4 * i) = r0 + i < p.d_o ? p.bias[r0 + i] : 0.f;
    __syncthreads();
  }
#pragma unroll
  for (int b = 0; b < NT; ++b) {
#pragma unroll
    for (int a = 0; a < MT; ++a)
#pragma unroll
      for (int r4 = 0; r4 < 4; ++r4) {
        const int rr = a * 32 + 8 * r4 + 4 * half;
        f32x4 v = {acc[a][b][4 * r4], acc[a][b][4 * r4 + 1], acc[a][b][4 * r4 + 2], acc[a][b][4 * r4 + 3]};
        if (biased) v += *(__attribute__((address_space(3))) f32x4*)(bias + 4 * (wm * 32 * MT + rr));
        if (osize == 4) {
          *(__attribute__((address_space(3))) f32x4*)(out + row * T::kOutPitch + 4 * rr) = v;
        } else {
          const uint32_t lo = f32_to_bf16(v[0]) | (static_cast<uint32_t>(f32_to_bf16(v[1])) << 16);
          const uint32_t hi = f32_to_bf16(v[2]) | (static_cast<uint32_t>(f32_to_bf16(v[3])) << 16);
          *(__attribute__((address_space(3))) uint64_t*)(out + row * T::kOutPitch + 2 * rr) = static_cast<uint64_t>(hi) << 32 | lo;
        }
      }
    const int64_t tb = t0 + (wn * NT + b) * 32;
    const int per_row = 32 * MT * osize / 16;           // pieces of 16 bytes
    for (int i = lane; i < 32 * per_row; i += 64) {
      const int t = i / per_row, k = i % per_row, e0 = k * 16 / osize;
      if (tb + t >= p.n || wr0 + e0 >= p.d_o) continue;
      const i32x4 v = rd16(out + t * T::kOutPitch + 16 * k);
      uint8_t* const dst = ybase + ((tb + t) * ld + wr0 + e0) * osize;
      if (lines && wr0 + e0 + 16 / osize <= p.d_o) {
        *reinterpret_cast<i32x4*>(dst) = v;
      } else if (osize == 4) {
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (wr0 + e0 + j < p.d_o) reinterpret_cast<int*>(dst)[j] = v[j];
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (wr0 + e0 + j < p.d_o)
            reinterpret_cast<uint16_t*>(dst)[j] = static_cast<uint16_t>(static_cast<uint32_t>(v[j / 2]) >> (16 * (j % 2)));
      }
    }
  }
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

// Y = the splits' sums in their order, with the bias.  Four results a thread.
__global__ __launch_bounds__(256) void mx4_join_kernel(const Mx4Product p, int splits) {
  const int64_t per_row = (p.d_o + 3) / 4, total = p.n * per_row;
  for (int64_t i = blockIdx.x * (int64_t)256 + threadIdx.x; i < total; i += (int64_t)gridDim.x * 256) {
    const int64_t t = i / per_row, r = i % per_row * 4;
    const float* src = p.partial + t * p.d_o + r;
    f32x4 v = {0.f, 0.f, 0.f, 0.f};
    if (p.d_o % 4 == 0) {
      for (int k = 0; k < splits; ++k) v += *reinterpret_cast<const f32x4*>(src + k * p.n * p.d_o);
    } else {
      for (int k = 0; k < splits; ++k)
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (r + j < p.d_o) v[j] += src[k * p.n * p.d_o + j];
    }
    store4(p, t, r, v);
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
                               hipFuncAttributeMaxDynamicSharedMemorySize, T::kShared));
    if (dev <= 63) allowed.fetch_or(uint64_t{1} << dev, std::memory_order_relaxed);
  }
  const int tw = static_cast<int>(ceil_div(p.d_o, T::BM)), tx = static_cast<int>(ceil_div(p.n, T::BN));
  const int all = static_cast<int>(ceil_div(p.G, TileGeom<X4>::kBlocks));
  const int per = static_cast<int>(round_up(ceil_div(all, splits), TileGeom<X4>::kWParts));
  const int parts = static_cast<int>(ceil_div(all, per));
  Mx4Product q = p;
  if (parts == 1) q.partial = nullptr;
  hipLaunchKernelGGL(kernel, dim3(static_cast<unsigned>(tw) * tx, parts), dim3(T::kThreads),
                     T::kShared, s, q, tw, tx, per);
  QZ_TRY(check_launch("mx4_tile"));
  if (parts == 1) return QZ_OK;
  const int64_t blocks = ceil_div(p.n * ceil_div(p.d_o, 4), 256);
  hipLaunchKernelGGL(mx4_join_kernel, dim3(static_cast<unsigned>(blocks < 4096 ? blocks : 4096)),
                     dim3(256), 0, s, q, parts);
  return check_launch("mx4_join");
}

}  // namespace

int launch_mx4_pad(const uint16_t* X, int64_t n, int64_t d_i, int64_t ldx, uint16_t* out,
                   int64_t ldo, hipStream_t s) {
  const int64_t b = ceil_div(n * ldo, 256);
  hipLaunchKernelGGL(mx4_pad_kernel, dim3(static_cast<unsigned>(b < 65536 ? b : 65536)), dim3(256),
                     0, s, X, n, d_i, ldx, out, ldo);
  return check_launch("mx4_pad");
}

namespace {

template <bool X4>
int launch_product(const Mx4Product& p, hipStream_t s) {
  using Choice = Mx4Choice;
  const Choice c = p.choice;
  switch (c.kind) {
    case Choice::kFew11x8: return launch_skinny<X4, 1, 1>(p, 8, s);
    case Choice::kFew11: return launch_skinny<X4, 1, 1>(p, 4, s);
    case Choice::kFew12:
      if constexpr (X4) return launch_skinny<X4, 1, 2>(p, 4, s);
      break;
    case Choice::kFew21:
      if constexpr (!X4) return launch_skinny<X4, 2, 1>(p, 4, s);
      break;
    case Choice::kFew22: return launch_skinny<X4, 2, 2>(p, 4, s);
    case Choice::kFew24:
      if constexpr (X4) return launch_skinny<X4, 2, 4>(p, 4, s);
      break;
    case Choice::kFew42:
      if constexpr (!X4) return launch_skinny<X4, 4, 2>(p, 4, s);
      break;
    case Choice::k256x256: return launch_tile<X4, 2, 4, 4, 2>(p, c.splits, s);
    case Choice::k256x128: return launch_tile<X4, 4, 2, 2, 2>(p, c.splits, s);
    case Choice::k128x128: return launch_tile<X4, 2, 2, 2, 2>(p, c.splits, s);
    case Choice::k128x64: return launch_tile<X4, 2, 2, 2, 1>(p, c.splits, s);
    case Choice::k64x64: return launch_tile<X4, 2, 2, 1, 1>(p, c.splits, s);
    case Choice::k128x32: return launch_tile<X4, 4, 1, 1, 1>(p, c.splits, s);
  }
  return fail(QZ_EHIP, "mx4_product: no kernel");
}

}  // namespace

Mx4Choice mx4_choose(bool x4, int64_t n, int64_t d_o, int64_t G) {
  return choose(x4, static_cast<int>(n), static_cast<int>(d_o), static_cast<int>(G));
}

int launch_mx4_product(const Mx4Product& p, hipStream_t s) {
  return p.X ? launch_product<false>(p, s) : launch_product<true>(p, s);
}

}  // namespace qz
