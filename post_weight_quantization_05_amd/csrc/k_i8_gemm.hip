// Products of 8-bit integer rows: Y = X W^T with a scale per row of X and of W, plain or grouped by
// expert.
#include <type_traits>

#include "i8_gemm.h"
#include "lds_copy.h"

namespace qz {

namespace {

using std::integral_constant;

// f(integral_constant<int, 0>) ... f(integral_constant<int, N - 1>)
template <class F, int... I>
__device__ __forceinline__ void each_of(F&& f, std::integer_sequence<int, I...>) {
  (f(integral_constant<int, I>{}), ...);
}
template <int N, class F>
__device__ __forceinline__ void each(F&& f) {
  each_of(f, std::make_integer_sequence<int, N>{});
}

// ---------------------------------------------------------------------------- large products
// Workgroup tile of BM rows of W by BN rows of X, BM = 32 MT WM, BN = 32 NT WN, in WM x WN wavefronts
// of 32 MT x 32 NT each.  The contraction goes in stages of 128 columns: whole lines of both.
template <int WM_, int WN_, int MT_, int NT_>
struct TileI8 {
  static constexpr int WM = WM_, WN = WN_, MT = MT_, NT = NT_;
  static constexpr int kWaves = WM * WN, kThreads = 64 * kWaves;
  static constexpr int BM = 32 * MT * WM, BN = 32 * NT * WN;
  static constexpr int kHalfW = BM / 2 * 128, kHalf = (BM + BN) / 2 * 128;   // bytes
  static constexpr int kLds = kWaves == 8 || MT * NT >= 8 ? 160 * 1024 : 80 * 1024;
  static constexpr int kRing = kLds / kHalf < 8 ? kLds / kHalf : 8;          // halves of a stage in LDS
  static constexpr int kCopiesW = BM / 16 / kWaves, kCopiesX = BN / 16 / kWaves;   // of a half, a wavefront
  static constexpr int kCopies = kCopiesW + kCopiesX;
  static constexpr int kProducts = MT * NT, kReads = MT + NT;
  static_assert(BM % (16 * kWaves) == 0 && BN % (16 * kWaves) == 0 && kRing >= 5);
  static constexpr int kOutPitch = 32 * MT * 4 + 16;
  static constexpr int kOut = kWaves * 32 * kOutPitch;
  static constexpr int kUsed = kRing * kHalf;
  static constexpr int kShared = kUsed > kOut + 12 * BM ? kUsed : kOut + 12 * BM;
  static_assert(kShared <= 160 * 1024);
};

template <Form FORM, class T>
__global__ __launch_bounds__(T::kThreads, T::kWaves / 4 * (T::kShared <= 80 * 1024 ? 2 : 1))
void i8_tile_kernel(const I8Product p, int tiles_w, int tiles_x, int stages_per_split) {
  constexpr int MT = T::MT, NT = T::NT, BM = T::BM, BN = T::BN, H = T::kRing;
  extern __shared__ __align__(1024) uint8_t smem[];
  lds_u8* const lds = (lds_u8*)smem;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave / T::WN, wn = wave % T::WN;

  // The hardware deals workgroups to the 8 XCDs in turn.  Each XCD gets a run of consecutive tiles,
  // and runs go through 8 rows of W tiles by all X tiles, so the tiles that are resident on an XCD
  // share panels in its L2.
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
  const int tw = __builtin_amdgcn_readfirstlane(g0 + pid % in_group % gh);
  const int tx = __builtin_amdgcn_readfirstlane(pid % in_group / gh);
  constexpr int kRows = FORM == kGateUp ? BM / 2 : BM;   // output rows of the tile
  const int64_t r0 = static_cast<int64_t>(tw) * kRows;
  int expert = 0, slot0 = 0, slot_end = 0;
  if constexpr (FORM != kPlain)
    if (!find_tile(p, tx, BN, &expert, &slot0, &slot_end)) return;
  const int64_t t0 = FORM == kPlain ? static_cast<int64_t>(tx) * BN : slot0;
  const int64_t t_end = FORM == kPlain ? p.n : slot_end;
  // last rows inside the matrices, counted in the tile: rows past them read these again
  const int last_r = static_cast<int>(p.d_o - 1 - r0 < kRows ? p.d_o - 1 - r0 : kRows);
  const int last_t = static_cast<int>(t_end - 1 - t0 < BN ? t_end - 1 - t0 : BN);
  const int64_t w_row0 = static_cast<int64_t>(expert) * (FORM == kGateUp ? 2 : 1) * p.d_o;   // the expert's

  const int all = static_cast<int>(p.P / 128);
  const int st0 = split * stages_per_split;
  const int nst = all - st0 < stages_per_split ? all - st0 : stages_per_split;   // >= 1
  const int halves = 2 * nst;

  // Sources of this wavefront's copies (of 8 rows, 1024 bytes of LDS each): offsets from the tile's
  // first row of W, and from the tile's first row of X or, gathered, from X.
  uint32_t from_w[2][T::kCopiesW], from_x[2][T::kCopiesX];
  const uint32_t pitch = static_cast<uint32_t>(p.P);
#pragma unroll
  for (int h = 0; h < 2; ++h) {
#pragma unroll
    for (int i = 0; i < T::kCopiesW; ++i) {
      const int r = (wave + T::kWaves * i) * 8 + lane / 8, chunk = (lane % 8) ^ swz<128>(r);
      uint32_t row;
      if constexpr (FORM == kGateUp) {   // 32 gate rows, the same up rows, and so on
        const int rr = h * BM / 2 + r, o = rr / 64 * 32 + rr % 32;
        row = (o < last_r ? o : last_r) + (rr / 32 % 2 ? static_cast<uint32_t>(p.d_o) : 0u);
      } else {
        const int rr = h * BM / 2 + r;
        row = rr < last_r ? rr : last_r;
      }
      from_w[h][i] = row * pitch + 16 * chunk;
    }
#pragma unroll
    for (int i = 0; i < T::kCopiesX; ++i) {
      const int r = (wave + T::kWaves * i) * 8 + lane / 8, chunk = (lane % 8) ^ swz<128>(r);
      const int rr = h * BN / 2 + r;
      uint32_t row = rr < last_t ? rr : last_t;
      if constexpr (FORM == kGateUp) row = static_cast<uint32_t>(p.order[t0 + row]) / static_cast<uint32_t>(p.k);
      from_x[h][i] = row * pitch + 16 * chunk;
    }
  }
  const uint8_t* const wbase = reinterpret_cast<const uint8_t*>(p.W) + (w_row0 + r0) * p.P + static_cast<int64_t>(st0) * 128;
  const uint8_t* const xbase = reinterpret_cast<const uint8_t*>(p.X) + (FORM == kGateUp ? 0 : t0 * p.P) + static_cast<int64_t>(st0) * 128;

  // Copy i of half h of stage st, to place `at` of the ring.
  auto copy = [&](auto h, auto i, int st, int at) {
    constexpr int hh = decltype(h)::value, ii = decltype(i)::value;
    lds_u8* const to = lds + at * T::kHalf;
    if constexpr (ii < T::kCopiesW)
      copy_lds<16>(to + (wave + T::kWaves * ii) * 1024, wbase + static_cast<int64_t>(st) * 128, from_w[hh][ii]);
    else
      copy_lds<16>(to + T::kHalfW + (wave + T::kWaves * (ii - T::kCopiesW)) * 1024,
                   xbase + static_cast<int64_t>(st) * 128, from_x[hh][ii - T::kCopiesW]);
  };
  auto copy_half = [&](auto h, int st, int at) { each<T::kCopies>([&](auto i) { copy(h, i, st, at); }); };

  i32x16 acc[MT][NT];
#pragma unroll
  for (int a = 0; a < MT; ++a)
#pragma unroll
    for (int b = 0; b < NT; ++b)
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[a][b][r] = 0;

  const int row = lane & 31, half = lane >> 5;
  const int wh = wm * 2 / T::WM, xh = wn * 2 / T::WN;   // the halves that this wavefront reads
  const int in_w = ((wm * 32 * MT) % (BM / 2) + row) * 128, in_x = T::kHalfW + ((wn * 32 * NT) % (BN / 2) + row) * 128;
  i32x4 w[2][MT], x[2][NT];
  auto rd16 = [](lds_u8* q) { return *(__attribute__((address_space(3))) i32x4*)q; };
  // Read i of step s into the operands `set`; aw, ax: LDS of this wavefront's rows of the stage.
  auto read = [&](auto set, auto i, lds_u8* aw, lds_u8* ax, int c) {
    constexpr int ii = decltype(i)::value;
    if constexpr (ii < MT)
      w[decltype(set)::value][ii] = rd16(aw + ii * 32 * 128 + c);
    else
      x[decltype(set)::value][ii - MT] = rd16(ax + (ii - MT) * 32 * 128 + c);
  };
  auto chunk_at = [&](int s) { return 16 * ((2 * s + half) ^ swz<128>(row)); };
  auto multiply = [&](auto set, auto i) {
    constexpr int ii = decltype(i)::value, a = ii / NT, b = ii % NT, s = decltype(set)::value;
    acc[a][b] = __builtin_amdgcn_mfma_i32_32x32x32_i8(w[s][a], x[s][b], acc[a][b], 0, 0, 0);
  };
#define QZ_FENCE __builtin_amdgcn_sched_barrier(0)
  // The products of operands `set`, with the reads of the next step's operands and `more` of them
  // (copies) dealt out between.
  constexpr int kP = T::kProducts, kR = T::kReads;
  auto step = [&](auto set, lds_u8* aw, lds_u8* ax, int c, auto reads, auto&& more) {
    constexpr int s = decltype(set)::value;
    each<kP>([&](auto i) {
      constexpr int ii = decltype(i)::value;
      if constexpr (decltype(reads)::value) {
        constexpr int before = ii * kR / kP, upto = (ii + 1) * kR / kP;
        each<upto - before>([&](auto j) {
          read(integral_constant<int, 1 - s>{}, integral_constant<int, before + decltype(j)::value>{}, aw, ax, c);
        });
      }
      more(i);
      QZ_FENCE;
      multiply(set, i);
      QZ_FENCE;
    });
  };
  auto nothing = [](auto) {};
  using Set0 = integral_constant<int, 0>;
  using Set1 = integral_constant<int, 1>;

  // Halves 0 .. H - 1 first; the first stage has landed when the others may be in flight.
  each<H>([&](auto i) {
    constexpr int ii = decltype(i)::value;
    if (ii < halves) copy_half(integral_constant<int, ii % 2>{}, ii / 2, ii);
  });
  if (H <= halves)
    wait_and_join<(H - 2) * T::kCopies>();
  else
    wait_and_join<0>();

  int at = 0;   // place of the stage's first half
  const auto wrap = [](int v) { return v >= H ? v - H : v; };
  each<kR>([&](auto i) {
    read(Set0{}, i, lds + wh * T::kHalf + in_w, lds + xh * T::kHalf + in_x, chunk_at(0));
  });

  // One stage.  Its last reads are made in the third step; behind them, all wavefronts meet: stage
  // st + 1 has landed for everyone, and the places of stage st are free for the halves 2 st + H and
  // 2 st + H + 1, whose copies go out beside the last step's products.
  auto first_steps = [&](lds_u8* aw, lds_u8* ax) {
    step(Set0{}, aw, ax, chunk_at(1), std::true_type{}, nothing);
    step(Set1{}, aw, ax, chunk_at(2), std::true_type{}, nothing);
    step(Set0{}, aw, ax, chunk_at(3), std::true_type{}, nothing);
  };
  int st = 0;
  for (; 2 * st + H + 1 < halves; ++st) {
    first_steps(lds + wrap(at + wh) * T::kHalf + in_w, lds + wrap(at + xh) * T::kHalf + in_x);
    wait_and_join<(H - 4) * T::kCopies>();
    const int next = wrap(at + 2), at1 = wrap(at + 1);
    const int far = st + H / 2;   // stage of half 2 st + H
    step(Set1{}, lds + wrap(next + wh) * T::kHalf + in_w, lds + wrap(next + xh) * T::kHalf + in_x, chunk_at(0),
         std::true_type{}, [&](auto i) {
           constexpr int ii = decltype(i)::value;
           constexpr int before = ii * 2 * T::kCopies / kP, upto = (ii + 1) * 2 * T::kCopies / kP;
           each<upto - before>([&](auto j) {
             constexpr int c = before + decltype(j)::value, second = c / T::kCopies;
             copy(integral_constant<int, (H + second) % 2>{}, integral_constant<int, c % T::kCopies>{},
                  far + (H % 2 + second) / 2, second ? at1 : at);
           });
         });
    at = next;
  }
  for (; st < nst; ++st) {
    first_steps(lds + wrap(at + wh) * T::kHalf + in_w, lds + wrap(at + xh) * T::kHalf + in_x);
    if (st + 1 < nst) {
      wait_and_join<0>();
      const int next = wrap(at + 2);
      if (2 * st + H < halves) copy_half(integral_constant<int, H % 2>{}, st + H / 2, at);
      each<kR>([&](auto i) {
        read(Set0{}, i, lds + wrap(next + wh) * T::kHalf + in_w, lds + wrap(next + xh) * T::kHalf + in_x, chunk_at(0));
      });
      at = next;
    }
    step(Set1{}, lds, lds, 0, std::false_type{}, nothing);
  }
#undef QZ_FENCE

  // Register r of lane l: row 8 (r / 4) + 4 (l / 32) + r % 4 of a tile, token l % 32.  32 tokens at a
  // time go through LDS of the wavefront's own, so that Y is written in whole lines.
  const bool sums = p.partial != nullptr;   // of a split product: the integers
  const int osize = sums || p.yt == QZ_F32 ? 4 : 2;
  const int64_t ld = sums ? p.d_o : p.ldy;
  uint8_t* const ybase = sums ? reinterpret_cast<uint8_t*>(p.partial + split * p.n * p.d_o) : static_cast<uint8_t*>(p.Y);
  const bool lines = ld * osize % 16 == 0 && reinterpret_cast<uintptr_t>(ybase) % 16 == 0;
  lds_u8* const out = lds + wave * 32 * T::kOutPitch;
  lds_u8* const par = lds + T::kOut;   // scales, zero points less 128, bias of the tile's rows
  __syncthreads();
  for (int i = tid; i < BM; i += T::kThreads) {
    const int o = FORM == kGateUp ? i / 64 * 32 + i % 32 : i;
    const int64_t r = w_row0 + r0 + (o < last_r ? o : last_r) + (FORM == kGateUp && i / 32 % 2 ? p.d_o : 0);
    *(__attribute__((address_space(3))) float*)(par + 4 * i) = p.sw[r];
    *(__attribute__((address_space(3))) int*)(par + 4 * (BM + i)) = p.zeros ? p.zeros[r] - 128 : 0;
    *(__attribute__((address_space(3))) float*)(par + 4 * (2 * BM + i)) = FORM == kPlain && p.bias ? p.bias[r] : 0.f;
  }
  __syncthreads();
  constexpr int kOutRows = FORM == kGateUp ? 16 * MT : 32 * MT;   // of a wavefront
  const int64_t wr0 = r0 + wm * kOutRows;
#pragma unroll
  for (int b = 0; b < NT; ++b) {
    const int64_t tb = t0 + (wn * NT + b) * 32;
    float sx = 0.f, pw = 1.f;
    int xsum = 0;
    if (tb + row < t_end && !sums) {
      const int64_t pair = FORM == kPlain ? 0 : p.order[tb + row];
      const int64_t xr = FORM == kGateUp ? pair / p.k : tb + row;
      sx = p.sx[xr];
      if (p.zeros) xsum = p.xsum[xr];
      if constexpr (FORM == kDown) pw = p.pair_weight[pair];
    }
    auto values = [&](int a, int r4) {
      const int rr = wm * 32 * MT + a * 32 + 8 * r4 + 4 * half;
      const f32x4 s = *(__attribute__((address_space(3))) f32x4*)(par + 4 * rr);
      const i32x4 z = *(__attribute__((address_space(3))) i32x4*)(par + 4 * (BM + rr));
      const f32x4 bias = *(__attribute__((address_space(3))) f32x4*)(par + 4 * (2 * BM + rr));
      f32x4 v;
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] = scaled(acc[a][b][4 * r4 + i], z[i], xsum, sx, s[i], bias[i]);
      return v;
    };
#pragma unroll
    for (int a = 0; a < MT; a += FORM == kGateUp ? 2 : 1)
#pragma unroll
      for (int r4 = 0; r4 < 4; ++r4) {
        const int rr = (FORM == kGateUp ? a / 2 : a) * 32 + 8 * r4 + 4 * half;
        if (sums) {
          *(__attribute__((address_space(3))) i32x4*)(out + row * T::kOutPitch + 4 * rr) =
              i32x4{acc[a][b][4 * r4], acc[a][b][4 * r4 + 1], acc[a][b][4 * r4 + 2], acc[a][b][4 * r4 + 3]};
          continue;
        }
        f32x4 v = values(a, r4);
        if constexpr (FORM == kGateUp) {
          const f32x4 u = values(a + 1, r4);
#pragma unroll
          for (int i = 0; i < 4; ++i) v[i] = silu(v[i]) * u[i];
        } else if constexpr (FORM == kDown) {
          v *= pw;
        }
        if (osize == 4)
          *(__attribute__((address_space(3))) f32x4*)(out + row * T::kOutPitch + 4 * rr) = v;
        else
          *(__attribute__((address_space(3))) uint64_t*)(out + row * T::kOutPitch + 2 * rr) =
              static_cast<uint64_t>(bf16_pair(v[2], v[3])) << 32 | bf16_pair(v[0], v[1]);
      }
    const int per_row = kOutRows * osize / 16;           // pieces of 16 bytes
    for (int i = lane; i < 32 * per_row; i += 64) {
      const int t = i / per_row, k = i % per_row, e0 = k * 16 / osize;
      if (tb + t >= t_end || wr0 + e0 >= p.d_o) continue;
      const i32x4 v = rd16(out + t * T::kOutPitch + 16 * k);
      const int64_t yr = FORM == kDown ? static_cast<int64_t>(p.order[tb + t]) : tb + t;
      uint8_t* const dst = ybase + (yr * ld + wr0 + e0) * osize;
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

// Y from the splits' sums.  Four results a thread.
__global__ __launch_bounds__(256) void i8_join_kernel(const I8Product p, int splits) {
  const int64_t per_row = (p.d_o + 3) / 4, total = p.n * per_row;
  const bool whole = p.d_o % 4 == 0;
  const int osize = p.yt == QZ_BF16 ? 2 : 4;
  const bool vec = whole && p.ldy % 4 == 0 && reinterpret_cast<uintptr_t>(p.Y) % (4 * osize) == 0;
  for (int64_t i = blockIdx.x * (int64_t)256 + threadIdx.x; i < total; i += (int64_t)gridDim.x * 256) {
    const int64_t t = i / per_row, r = i % per_row * 4;
    const int32_t* src = p.partial + t * p.d_o + r;
    i32x4 a = {0, 0, 0, 0};
    for (int k = 0; k < splits; ++k, src += p.n * p.d_o) {
      if (whole) {
        a += *reinterpret_cast<const i32x4*>(src);
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (r + j < p.d_o) a[j] += src[j];
      }
    }
    const float sx = p.sx[t];
    const int xsum = p.zeros ? p.xsum[t] : 0;
    f32x4 v;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int64_t c = r + j < p.d_o ? r + j : p.d_o - 1;
      v[j] = scaled(a[j], p.zeros ? p.zeros[c] - 128 : 0, xsum, sx, p.sw[c], p.bias ? p.bias[c] : 0.f);
    }
    if (osize == 2) {
      uint16_t* o = static_cast<uint16_t*>(p.Y) + t * p.ldy + r;
      const uint2 w = make_uint2(bf16_pair(v[0], v[1]), bf16_pair(v[2], v[3]));
      if (vec) {
        *reinterpret_cast<uint2*>(o) = w;
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (r + j < p.d_o) o[j] = static_cast<uint16_t>((j < 2 ? w.x : w.y) >> (16 * (j % 2)));
      }
    } else {
      float* o = static_cast<float*>(p.Y) + t * p.ldy + r;
      if (vec) {
        *reinterpret_cast<f32x4*>(o) = v;
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (r + j < p.d_o) o[j] = v[j];
      }
    }
  }
}

template <Form FORM, class T>
int launch_tile(const I8Product& p, int splits, hipStream_t s) {
  const auto kernel = i8_tile_kernel<FORM, T>;
  static LdsAllowance allowed;
  QZ_TRY(allowed.ask(reinterpret_cast<const void*>(kernel), T::kShared));
  const int64_t tw = ceil_div(p.d_o, FORM == kGateUp ? T::BM / 2 : T::BM);
  const int64_t tx = FORM == kPlain ? ceil_div(p.n, T::BN) : most_tiles(p, T::BN);
  if (tw * tx > 0x7fffffff) return fail(QZ_EINVAL, "i8_product: too many tiles");
  const int all = static_cast<int>(p.P / 128), per = static_cast<int>(ceil_div(all, splits));
  const int parts = static_cast<int>(ceil_div(all, per));
  I8Product q = p;
  if (parts == 1) q.partial = nullptr;
  hipLaunchKernelGGL(kernel, dim3(static_cast<unsigned>(tw * tx), parts), dim3(T::kThreads), T::kShared, s, q,
                     static_cast<int>(tw), static_cast<int>(tx), per);
  QZ_TRY(check_launch("i8_tile"));
  if (parts == 1) return QZ_OK;
  const int64_t blocks = ceil_div(p.n * ceil_div(p.d_o, 4), 256);
  hipLaunchKernelGGL(i8_join_kernel, dim3(static_cast<unsigned>(blocks < 4096 ? blocks : 4096)), dim3(256), 0, s, q, parts);
  return check_launch("i8_join");
}

template <Form FORM>
int launch(const I8Product& p, hipStream_t s) {
  if (p.n <= 64) return FORM == kPlain ? launch_i8_few(p, s) : FORM == kGateUp ? launch_i8_few_gate_up(p, s) : launch_i8_few_down(p, s);
  if (FORM != kPlain || p.n <= 2048) return launch_tile<FORM, TileI8<2, 2, 2, 2>>(p, 1, s);
  return launch_tile<FORM, TileI8<2, 4, 4, 2>>(p, 1, s);
}

}  // namespace

size_t i8_product_ws(int64_t, int64_t, int64_t) { return 0; }
int launch_i8_product(const I8Product& p, hipStream_t s) { return launch<kPlain>(p, s); }
int launch_i8_gate_up(const I8Product& p, hipStream_t s) { return launch<kGateUp>(p, s); }
int launch_i8_down(const I8Product& p, hipStream_t s) { return launch<kDown>(p, s); }

}  // namespace qz
