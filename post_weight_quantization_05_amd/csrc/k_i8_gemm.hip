// Products of 8-bit integer rows: Y = X W^T with a scale per row of X and of W, plain or grouped by
// expert.
//
// Y = fma((sum_c x_c w_c - (z - 128) sum_c x_c) sx, sw, b): the sums are whole and exact, so neither the
// tile, nor the order, nor the kernel changes a result.
//
// Stages of 128 columns come into LDS in two halves each (the upper and the lower rows of both
// operands), in a ring of places as deep as LDS allows: the finer the pieces, the more of LDS is on its way at
// any time.  Rows are whole lines, and 16-byte chunks lie permuted in a row so that the matrix
// instructions' reads meet no bank twice (conflicts 1% of the cycles).  A product's 32 x 32 x 32 step reads MT + NT
// pieces for MT NT instructions: 128 x 64 a wavefront in the large tile, which keeps LDS reads below the
// matrix time; in the smaller ones, whose steps are shorter than a read takes, the operands of a whole
// stage are read ahead.
//
// What bounds it, measured:
//  - 8192 x 5120 -> 25600, 256 x 256: 905 to 950 us, 2.26 to 2.37 POP/s, matrix cores busy for 64% of the
//    cycles at 1.74 GHz of 2.4: the power limit (on zeros, which draw less, 729 us at 2.4 GHz).  The
//    library's product of the same codes, without scales: 1025 to 1044 us.
//  - 2048 x 4096 -> 4096, 256 x 128: 36.5 us, busy for 40%: one tile a compute unit, so the first stages
//    and the results are not covered by another's products; the library's 40 us.
//  - 256 x 4096 -> 12288, 128 x 128: 22.9 us, 75 MB read (3.3 TB/s): 192 tiles on 256 compute units, each
//    bound by its own stream from memory into LDS; the library's 31 us.  64 x 64, four resident, would take 20.5 (the
//    choice's times err there, i8_plan.h).  Splitting the contraction, with the join in a second launch, lost at
//    every size.
//  - Expert layer, 4096 tokens 6 of 64, 2048 -> 2 x 1408: 206 us for 557 MB read and 138 written, busy for 33%:
//    384 tokens an expert use its weights for 1.5 tiles, so it reads nearly as long as it multiplies,
//    and a tile's ends (its slots, its results) are alone on their compute unit.  Down: 141 us for 286 MB read
//    and 201 written, busy for 23%.
#include <type_traits>

#include "i8_gemm.h"
#include "i8_plan.h"
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

template <Form FORM, class T>
__global__ __launch_bounds__(T::kThreads, T::kWaves / 4 * (T::kShared <= 80 * 1024 ? 2 : 1))
void i8_tile_kernel(const I8Product p, int tiles_w, int tiles_x) {
  constexpr int MT = T::MT, NT = T::NT, BM = T::BM, BN = T::BN, H = T::kRing;
  extern __shared__ __align__(1024) uint8_t smem[];
  lds_u8* const lds = (lds_u8*)smem;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  // Wavefronts of the same tokens on different SIMDs where a tile may have few (the hardware deals them in turn).
  const int wm = FORM == kPlain ? wave / T::WN : wave % T::WM, wn = FORM == kPlain ? wave % T::WN : wave / T::WM;

  // The hardware deals workgroups to the 8 XCDs in turn.  Each XCD gets a run of consecutive tiles,
  // and runs go through 8 rows of W tiles by all X tiles, so the tiles that are resident on an XCD
  // share panels in its L2.
  const auto mapped = [&](int nb) {
    const int per = nb / 8, extra = nb % 8, x = blockIdx.x % 8;
    return x * per + (x < extra ? x : extra) + static_cast<int>(blockIdx.x) / 8;
  };
  int pid, expert = 0, slot0 = 0, slot_end = 0, tw, tx;
  const auto place = [&] {
    constexpr int kGroup = 8;
    const int in_group = kGroup * tiles_x;
    const int g0 = pid / in_group * kGroup;
    const int gh = tiles_w - g0 < kGroup ? tiles_w - g0 : kGroup;
    tw = __builtin_amdgcn_readfirstlane(g0 + pid % in_group % gh);
    tx = __builtin_amdgcn_readfirstlane(pid % in_group / gh);
  };
  if constexpr (FORM == kPlain) {
    pid = mapped(gridDim.x);
    place();
  } else {
    // the launch has room for the most tiles there can be; those there are go evenly to the XCDs
    const Tiles tiles(p, BN);
    tiles_x = tiles.total;
    if (static_cast<int>(blockIdx.x) >= tiles_w * tiles_x) return;
    pid = mapped(tiles_w * tiles_x);
    place();
    tiles.find(tx, BN, &expert, &slot0, &slot_end);
  }
  constexpr int kRows = FORM == kGateUp ? BM / 2 : BM;   // output rows of the tile
  const int64_t r0 = static_cast<int64_t>(tw) * kRows;
  const int64_t t0 = FORM == kPlain ? static_cast<int64_t>(tx) * BN : slot0;
  const int64_t t_end = FORM == kPlain ? p.n : slot_end;
  // last rows inside the matrices, counted in the tile: rows past them read these again
  const int last_r = static_cast<int>(p.d_o - 1 - r0 < kRows ? p.d_o - 1 - r0 : kRows);
  const int last_t = static_cast<int>(t_end - 1 - t0 < BN ? t_end - 1 - t0 : BN);
  const int64_t w_row0 = static_cast<int64_t>(expert) * (FORM == kGateUp ? 2 : 1) * p.d_o;   // the expert's

  const int nst = static_cast<int>(p.P / 128);
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
  const uint8_t* const wbase = reinterpret_cast<const uint8_t*>(p.W) + (w_row0 + r0) * p.P;
  const uint8_t* const xbase = reinterpret_cast<const uint8_t*>(p.X) + (FORM == kGateUp ? 0 : t0 * p.P);

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

  // What the results are made with, fetched early: a row of W a thread, a token a lane for each 32.
  static_assert(BM <= T::kThreads);
  float my_sw = 0.f, my_bias = 0.f, sx[NT], pw[NT];
  int my_shift = 0, xsum[NT], pairs[NT];
  if (tid < BM) {
    const int o = FORM == kGateUp ? tid / 64 * 32 + tid % 32 : tid;
    const int64_t r = w_row0 + r0 + (o < last_r ? o : last_r) + (FORM == kGateUp && tid / 32 % 2 ? p.d_o : 0);
    my_sw = p.sw[r];
    if (p.zeros) my_shift = p.zeros[r] - 128;
    if (FORM == kPlain && p.bias) my_bias = p.bias[r];
  }
#pragma unroll
  for (int b = 0; b < NT; ++b) {
    const int64_t slot = t0 + (wn * NT + b) * 32 + (lane & 31);
    sx[b] = 0.f;
    pw[b] = 1.f;
    xsum[b] = 0;
    pairs[b] = 0;
    if (slot < t_end) {
      const int pair = FORM == kPlain ? 0 : p.order[slot];
      pairs[b] = pair;
      const int64_t xr = FORM == kGateUp ? pair / p.k : slot;
      sx[b] = p.sx[xr];
      if (p.zeros) xsum[b] = p.xsum[xr];
      if constexpr (FORM == kDown) pw[b] = p.pair_weight[pair];
    }
  }

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
  constexpr int S = T::kSteps;
  i32x4 w[2][S][MT], x[2][S][NT];
  auto rd16 = [](lds_u8* q) { return *(__attribute__((address_space(3))) i32x4*)q; };
  // Read i of a step at chunk offset c into place k of the operands `set`; aw, ax: LDS of this
  // wavefront's rows of the stage.
  auto read = [&](auto set, auto k, auto i, lds_u8* aw, lds_u8* ax, int c) {
    constexpr int ii = decltype(i)::value;
    if constexpr (ii < MT)
      w[decltype(set)::value][decltype(k)::value][ii] = rd16(aw + ii * 32 * 128 + c);
    else
      x[decltype(set)::value][decltype(k)::value][ii - MT] = rd16(ax + (ii - MT) * 32 * 128 + c);
  };
  auto chunk_at = [&](int s) { return 16 * ((2 * s + half) ^ swz<128>(row)); };
  auto multiply = [&](auto set, auto k, auto i) {
    constexpr int ii = decltype(i)::value, a = ii / NT, b = ii % NT, s = decltype(set)::value, kk = decltype(k)::value;
    acc[a][b] = __builtin_amdgcn_mfma_i32_32x32x32_i8(w[s][kk][a], x[s][kk][b], acc[a][b], 0, 0, 0);
  };
  using Zero = integral_constant<int, 0>;
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
          read(integral_constant<int, 1 - s>{}, Zero{}, integral_constant<int, before + decltype(j)::value>{}, aw, ax, c);
        });
      }
      more(i);
      QZ_FENCE;
      multiply(set, Zero{}, i);
      QZ_FENCE;
    });
  };
  auto nothing = [](auto) {};
  using Set0 = Zero;
  using Set1 = integral_constant<int, 1>;

  // Halves 0 .. H - 1 first; the first stage has landed when the others may be in flight.
  each<H>([&](auto i) {
    constexpr int ii = decltype(i)::value;
    if (ii < halves) copy_half(integral_constant<int, ii % 2>{}, ii / 2, ii);
  });
  if (tile_in_flight_first<T>(halves))
    wait_and_join<tile_in_flight_first<T>(H)>();
  else
    wait_and_join<0>();

  int at = 0;   // place of the stage's first half
  const auto wrap = [](int v) { return v >= H ? v - H : v; };
  // An expert's last tile may leave a wavefront without tokens: it copies and meets the others, no more.
  const bool idle = FORM != kPlain && t0 + wn * 32 * NT >= t_end;
  if (idle) {
    for (int st = 0; st + 1 < nst; ++st) {
      if (tile_in_flight<T>(st, halves))
        wait_and_join<tile_in_flight<T>(0, H + 2)>();
      else
        wait_and_join<0>();
      const int far = st + H / 2;
      if (2 * st + H < halves) copy_half(integral_constant<int, H % 2>{}, far, at);
      if (2 * st + H + 1 < halves) copy_half(integral_constant<int, (H + 1) % 2>{}, far + (H % 2 + 1) / 2, wrap(at + 1));
      at = wrap(at + 2);
    }
  } else {
  each<S>([&](auto k) {
    each<kR>([&](auto i) {
      read(Set0{}, k, i, lds + wh * T::kHalf + in_w, lds + xh * T::kHalf + in_x, chunk_at(k));
    });
  });

  int st = 0;
  if constexpr (S == 4) {
    // The operands of a whole stage are read while the one before is multiplied: a step's few products
    // are shorter than a read.  At the join of stage st its reads are done for everyone, so its places are
    // free for the halves 2 st + H and 2 st + H + 1, and stage st + 1 has landed.
    auto stage = [&](auto set, auto full) {   // full: with the copies of both halves
      constexpr bool kFull = decltype(full)::value;
      constexpr int s = decltype(set)::value;
      wait_and_join<kFull ? tile_in_flight<T>(0, H + 2) : 0>();   // what tile_in_flight says for st
      const int next = wrap(at + 2), at1 = wrap(at + 1), far = st + H / 2;
      lds_u8* const aw = lds + wrap(next + wh) * T::kHalf + in_w;
      lds_u8* const ax = lds + wrap(next + xh) * T::kHalf + in_x;
      if (!kFull && 2 * st + H < halves) copy_half(integral_constant<int, H % 2>{}, far, at);
      if (!kFull && 2 * st + H + 1 < halves) copy_half(integral_constant<int, (H + 1) % 2>{}, far + (H % 2 + 1) / 2, at1);
      constexpr int kSlots = 4 * kP, kAll = 4 * kR, kFew = kSlots * 3 / 4;   // reads in the first three quarters
      each<kSlots>([&](auto i) {
        constexpr int ii = decltype(i)::value;
        constexpr int first = ii < kFew ? ii * kAll / kFew : kAll, last = ii < kFew ? (ii + 1) * kAll / kFew : kAll;
        each<last - first>([&](auto j) {
          constexpr int r = first + decltype(j)::value;
          read(integral_constant<int, 1 - s>{}, integral_constant<int, r / kR>{}, integral_constant<int, r % kR>{}, aw, ax, chunk_at(r / kR));
        });
        if constexpr (kFull) {
          constexpr int before = ii * 2 * T::kCopies / kSlots, upto = (ii + 1) * 2 * T::kCopies / kSlots;
          each<upto - before>([&](auto j) {
            constexpr int c = before + decltype(j)::value, second = c / T::kCopies;
            copy(integral_constant<int, (H + second) % 2>{}, integral_constant<int, c % T::kCopies>{},
                 far + (H % 2 + second) / 2, second ? at1 : at);
          });
        }
        QZ_FENCE;
        multiply(set, integral_constant<int, ii / kP>{}, integral_constant<int, ii % kP>{});
        QZ_FENCE;
      });
      at = next;
      ++st;
    };
    while (tile_in_flight<T>(st + 1, halves)) {   // two whole stages
      stage(Set0{}, std::true_type{});
      stage(Set1{}, std::true_type{});
    }
    while (st + 1 < nst) {
      stage(Set0{}, std::false_type{});
#pragma unroll
      for (int k = 0; k < 4; ++k) {
#pragma unroll
        for (int a = 0; a < MT; ++a) w[0][k][a] = w[1][k][a];
#pragma unroll
        for (int b = 0; b < NT; ++b) x[0][k][b] = x[1][k][b];
      }
    }
    each<4 * kP>([&](auto i) { multiply(Set0{}, integral_constant<int, i / kP>{}, integral_constant<int, i % kP>{}); });
  } else {
  // One stage.  Its last reads are made in the third step; behind them, all wavefronts meet: stage
  // st + 1 has landed for everyone, and the places of stage st are free for the halves 2 st + H and
  // 2 st + H + 1, whose copies go out beside the last step's products.
  auto first_steps = [&](lds_u8* aw, lds_u8* ax) {
    step(Set0{}, aw, ax, chunk_at(1), std::true_type{}, nothing);
    step(Set1{}, aw, ax, chunk_at(2), std::true_type{}, nothing);
    step(Set0{}, aw, ax, chunk_at(3), std::true_type{}, nothing);
  };
  for (; tile_in_flight<T>(st, halves); ++st) {
    first_steps(lds + wrap(at + wh) * T::kHalf + in_w, lds + wrap(at + xh) * T::kHalf + in_x);
    wait_and_join<tile_in_flight<T>(0, H + 2)>();   // what it says for st
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
        read(Set0{}, Zero{}, i, lds + wrap(next + wh) * T::kHalf + in_w, lds + wrap(next + xh) * T::kHalf + in_x, chunk_at(0));
      });
      at = next;
    }
    step(Set1{}, lds, lds, 0, std::false_type{}, nothing);
  }
  }
  }
#undef QZ_FENCE

  // Register r of lane l: row 8 (r / 4) + 4 (l / 32) + r % 4 of a tile, token l % 32.  32 tokens at a
  // time go through LDS of the wavefront's own, so that Y is written in whole lines.
  uint8_t* const ybase = static_cast<uint8_t*>(p.Y);
  const bool lines = p.ldy * (p.yt == QZ_F32 ? 4 : 2) % 16 == 0 && reinterpret_cast<uintptr_t>(ybase) % 16 == 0;
  lds_u8* const out = lds + wave * 32 * T::kOutPitch;
  lds_u8* const par = lds + T::kOut;   // scales, zero points less 128, bias of the tile's rows
  __syncthreads();
  if (tid < BM) {
    *(__attribute__((address_space(3))) float*)(par + 4 * tid) = my_sw;
    *(__attribute__((address_space(3))) int*)(par + 4 * (BM + tid)) = my_shift;
    *(__attribute__((address_space(3))) float*)(par + 4 * (2 * BM + tid)) = my_bias;
  }
  __syncthreads();
  if (idle) return;
  constexpr int kOutRows = FORM == kGateUp ? 16 * MT : 32 * MT;   // of a wavefront
  const int64_t wr0 = r0 + wm * kOutRows;
  auto results = [&](int a, int b, int r4, auto shifted) {
    const int rr = wm * 32 * MT + a * 32 + 8 * r4 + 4 * half;
    const f32x4 s = *(__attribute__((address_space(3))) f32x4*)(par + 4 * rr);
    i32x4 z = {0, 0, 0, 0};
    f32x4 bias = {0.f, 0.f, 0.f, 0.f}, v;
    if constexpr (decltype(shifted)::value) {   // zero points or a bias
      z = rd16(par + 4 * (BM + rr));
      if constexpr (FORM == kPlain) bias = *(__attribute__((address_space(3))) f32x4*)(par + 4 * (2 * BM + rr));
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = scaled(acc[a][b][4 * r4 + i], z[i], xsum[b], sx[b], s[i], bias[i]);
    return v;
  };
  auto write = [&](auto size, auto shifted) {
    constexpr int osize = decltype(size)::value, per_row = kOutRows * osize / 16;   // pieces of 16 bytes
#pragma unroll
    for (int b = 0; b < NT; ++b) {
      const int64_t tb = t0 + (wn * NT + b) * 32;
#pragma unroll
      for (int a = 0; a < MT; a += FORM == kGateUp ? 2 : 1)
#pragma unroll
        for (int r4 = 0; r4 < 4; ++r4) {
          const int rr = (FORM == kGateUp ? a / 2 : a) * 32 + 8 * r4 + 4 * half;
          f32x4 v = results(a, b, r4, shifted);
          if constexpr (FORM == kGateUp) {
            v = silu(v) * results(a + 1, b, r4, shifted);
          } else if constexpr (FORM == kDown) {
#pragma unroll
            for (int i = 0; i < 4; ++i) v[i] *= pw[b];
          }
          if constexpr (osize == 4)
            *(__attribute__((address_space(3))) f32x4*)(out + row * T::kOutPitch + 4 * rr) = v;
          else
            *(__attribute__((address_space(3))) uint64_t*)(out + row * T::kOutPitch + 2 * rr) =
                static_cast<uint64_t>(bf16_pair(v[2], v[3])) << 32 | bf16_pair(v[0], v[1]);
        }
#pragma unroll
      for (int i = lane; i < 32 * per_row; i += 64) {
        const int t = i / per_row, k = i % per_row, e0 = k * 16 / osize;
        int64_t yr = tb + t;
        if constexpr (FORM == kDown) yr = __shfl(pairs[b], t);
        if (tb + t >= t_end || wr0 + e0 >= p.d_o) continue;
        const i32x4 v = rd16(out + t * T::kOutPitch + 16 * k);
        uint8_t* const dst = ybase + (yr * p.ldy + wr0 + e0) * osize;
        if (lines && wr0 + e0 + 16 / osize <= p.d_o) {
          if constexpr (FORM == kPlain)   // past the caches: the next launch reads hidden rows and pairs' results
            __builtin_nontemporal_store(v, reinterpret_cast<i32x4*>(dst));
          else
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
  };
  using std::false_type;
  using std::true_type;
  const bool shifted = p.zeros || (FORM == kPlain && p.bias);
  if (FORM != kPlain || p.yt == QZ_F32) {
    if (shifted)
      write(integral_constant<int, 4>{}, true_type{});
    else
      write(integral_constant<int, 4>{}, false_type{});
  } else if constexpr (FORM == kPlain) {
    if (shifted)
      write(integral_constant<int, 2>{}, true_type{});
    else
      write(integral_constant<int, 2>{}, false_type{});
  }
}

template <Form FORM, class T>
int launch_tile(const I8Product& p, hipStream_t s) {
  const auto kernel = i8_tile_kernel<FORM, T>;
  static LdsAllowance allowed;
  QZ_TRY(allowed.ask(reinterpret_cast<const void*>(kernel), T::kShared));
  const int64_t tw = ceil_div(p.d_o, FORM == kGateUp ? T::BM / 2 : T::BM);
  const int64_t tx = FORM == kPlain ? ceil_div(p.n, T::BN) : most_tiles(p, T::BN);
  if (tw * tx > 0xffffffffll / T::kThreads) return fail(QZ_EINVAL, "i8_product: too many tiles");   // a launch's limit
  hipLaunchKernelGGL(kernel, dim3(static_cast<unsigned>(tw * tx)), dim3(T::kThreads), T::kShared, s, p,
                     static_cast<int>(tw), static_cast<int>(tx));
  return check_launch("i8_tile");
}

template <Form FORM>
int launch(const I8Product& p, hipStream_t s) {
  const I8Kind kind = i8_choose(p.n, p.d_o * (FORM == kGateUp ? 2 : 1), p.P / 128, FORM == kPlain ? 0 : p.E, FORM == kGateUp);
  switch (kind) {
    case I8Kind::k256x256: return launch_tile<FORM, Tile256x256>(p, s);
    case I8Kind::k256x128: return launch_tile<FORM, Tile256x128>(p, s);
    case I8Kind::k128x128: return launch_tile<FORM, Tile128x128>(p, s);
    case I8Kind::k128x64: return launch_tile<FORM, Tile128x64>(p, s);
    case I8Kind::k64x64: if constexpr (FORM != kGateUp) return launch_tile<FORM, Tile64x64>(p, s); break;
    case I8Kind::k64x64by4: if constexpr (FORM != kGateUp) return launch_tile<FORM, Tile64x64By4>(p, s); break;
    default: return launch_i8_few(kind, FORM, p, s);
  }
  return fail(QZ_EHIP, "i8_product: no kernel");
}

}  // namespace

int launch_i8_product(const I8Product& p, hipStream_t s) { return launch<kPlain>(p, s); }
int launch_i8_gate_up(const I8Product& p, hipStream_t s) { return launch<kGateUp>(p, s); }
int launch_i8_down(const I8Product& p, hipStream_t s) { return launch<kDown>(p, s); }

}  // namespace qz
