// Plan of a product with MX4 weights: the shapes of the tile kernels, what their wavefronts wait
// for, and the choice of a kernel from the sizes.  Plain C++, so that host programs can include it.
#pragma once

#include <cstdint>
#include <initializer_list>

namespace qz {

// ------------------------------------------------------------------------------- tile kernels
// (k_mx4_gemm.hip; X4: X in MX4, else bf16)
template <bool X4>
struct TileGeom;
template <>
struct TileGeom<true> {
  static constexpr int kBlocks = 8, kRing = 2;      // of a stage; stages in LDS
  static constexpr int kWRow = 128, kXRow = 128;    // bytes of an LDS row
  static constexpr int kWParts = 1;                 // stages that share a W buffer
};
template <>
struct TileGeom<false> {
  static constexpr int kBlocks = 2, kRing = 3;
  static constexpr int kWRow = 64, kXRow = 128;
  static constexpr int kWParts = 2;
};
constexpr int kFetch = 64;   // factors of a row in LDS

template <bool X4, int WM, int WN, int MT, int NT>
struct TileShape {
  using G = TileGeom<X4>;
  static constexpr int kWaves = WM * WN, kThreads = 64 * kWaves;
  static constexpr int BM = 32 * MT * WM, BN = 32 * NT * WN;
  static constexpr int kWBytes = BM * G::kWRow, kXBytes = BN * G::kXRow;   // of a buffer
  static constexpr int kWBuffers = G::kWParts == 1 ? G::kRing : 2;
  static constexpr int kFRows = BM + (X4 ? BN : 0);                        // rows of factors
  static constexpr int kLds = kWBuffers * kWBytes + G::kRing * kXBytes + kFRows * kFetch;
  // copies (1024 bytes of LDS each) of a stage: a part of a W buffer and an X buffer
  static constexpr int kWPieces = kWBytes / 1024 / G::kWParts, kXPieces = kXBytes / 1024;
  static constexpr int kPieces = kWPieces + kXPieces;
  static constexpr int kCopies = kPieces / kWaves;   // of a wavefront; the first kExtra have one more
  static constexpr int kExtra = kPieces % kWaves;
  static constexpr int kXLeast = kCopies - (kWPieces + kWaves - 1) / kWaves;   // of X, at least
  static_assert(G::kRing == 2 || (G::kRing == 3 && kXLeast >= 0), "the waits of a stage");
  // the results of 32 tokens of a wavefront, on their way to whole lines of Y
  static constexpr int kOutPitch = 32 * MT * 4 + 16;
  static constexpr int kOut = kWaves * 32 * kOutPitch;
  static constexpr int kShared = kLds > kOut + 4 * BM ? kLds : kOut + 4 * BM;   // the bias behind them
  static_assert(kShared <= 160 * 1024, "LDS of a compute unit");
};

// What a wavefront may leave in flight at the join of stage st, where stage st + 1 has to have
// landed: with two buffers nothing.  With three, the batch issued last (stage st + 2) may be in
// flight where it is whole, so that the wavefront has issued its full number of copies; but where
// st + 1 begins a W buffer, that batch holds the second half of it, ahead of the copies of X.
// Copies land in the order of their issue: where st + 1 begins a fetch of factors, the fetch was
// issued behind that batch and nothing may be left.
enum class TileWait { kAll, kButX, kButStage };
template <bool X4>
constexpr TileWait tile_wait(int st, int nst, int whole) {
  using G = TileGeom<X4>;
  if (G::kRing == 2 || st + 2 >= nst || st + 2 + G::kWParts > whole) return TileWait::kAll;
  if ((st + 1) % (kFetch / G::kBlocks) == 0) return TileWait::kAll;
  return st % G::kWParts == G::kWParts - 1 ? TileWait::kButX : TileWait::kButStage;
}

// ------------------------------------------------------------------------- choice of a kernel
// Times of the alternatives, in microseconds, from their sizes.  A tile kernel's stage takes
// `alone` when its workgroup has a compute unit to itself (latency and the barriers), and `share`
// for each of the up to two resident ones when those are busy; then a launch, and for a split
// contraction the pass that joins the sums.  Fitted to 400 measurements (20 to 2048 tokens, seven
// layers of 512 to 12288 columns, 1 to 16 splits; 9% root mean square) and choosing within 8% of
// the best one measured there in all but six, where it is up to 20% off.  A few-token kernel's unit
// of 256 columns costs a wavefront `alone`, or `share` of the compute unit's time; fitted to 900
// measurements (1 to 1024 tokens, nine layers of 512 to 25600 columns; 4 to 9%).
// Both sides, measured, us (few-token shapes RT x NT of 16): 13 tokens 12288 -> 4096 bf16, 1 x 1 in
// eight wavefronts 8.9, in four 11.2; one token 5120 -> 25600 bf16, 1 x 1 18.8, 2 x 1 17.0; 64
// tokens 4096 -> 12288 bf16, 2 x 2 16.1 and the best tile, 128 x 32 in four splits, 21.8; 256 tokens
// 4096 -> 4096 bf16, 4 x 2 18.2, 2 x 2 20.0, tile 24.9; 512 tokens there, 31.9 and 31.8; 2048
// tokens, tiles of 256 x 256 81, of 256 x 128 72; MX4 X, 128 tokens 4096 -> 4096, 2 x 2 7.1, 2 x 4
// 7.7, tile 11.7; 256 tokens there, 11.1, 10.0, 11.9; 256 tokens 4096 -> 12288, 28.2, 27.7, 17.0.
// A product's kernel, from its sizes; splits: parts of the contraction whose sums go through
// Mx4Product::partial (1: none, partial unused).
struct Mx4Choice {
  enum Kind {
    kFew11x8, kFew11, kFew12, kFew21, kFew22, kFew24, kFew42,
    k256x256, k256x128, k128x128, k128x64, k64x64, k128x32
  } kind;
  int splits;
};

struct TileTime {
  int bm, bn, resident;
  double alone, share;
};
struct FewTime {
  int rt, nt, waves, resident;
  double fixed, alone, share;   // us; per unit of 256 columns of a wavefront
};
constexpr FewTime kFew[2][7] = {   // shapes without a time: slower everywhere for that type
    {{1, 1, 8, 3, 3.0, 1.00, 0.93}, {1, 1, 4, 4, 3.2, 0.62, 0.44}, {1, 2, 4, 0, 0, 0, 0},
     {2, 1, 4, 4, 3.2, 1.00, 0.67}, {2, 2, 4, 4, 3.0, 1.50, 1.07}, {2, 4, 4, 0, 0, 0, 0},
     {4, 2, 4, 2, 3.2, 2.40, 1.71}},
    {{1, 1, 8, 1, 3.2, 0.54, 0.54}, {1, 1, 4, 4, 3.2, 0.36, 0.21}, {1, 2, 4, 4, 3.2, 0.51, 0.34},
     {2, 1, 4, 0, 0, 0, 0}, {2, 2, 4, 3, 3.2, 0.71, 0.54}, {2, 4, 4, 2, 3.2, 1.22, 0.93},
     {4, 2, 4, 0, 0, 0, 0}}};

// `groups` workgroups of a compute unit, `resident` at once: one takes `alone`, r together at
// least r times `share`.
inline double rounds_time(int64_t groups, int resident, double alone, double share) {
  const int64_t full = groups / resident, rest = groups % resident;
  const auto together = [&](int64_t r) { return alone > r * share ? alone : r * share; };
  return full * together(resident) + (rest ? together(rest) : 0.);
}
constexpr TileTime kTiles[2][6] = {   // of a stage: 64 columns of bf16 X, 256 of MX4
    {{256, 256, 1, 1.746, 1.746}, {256, 128, 1, 1.021, 1.021}, {128, 128, 2, 1.027, 0.513},
     {128, 64, 2, 0.592, 0.369}, {64, 64, 2, 0.477, 0.239}, {128, 32, 2, 0.427, 0.256}},
    {{256, 256, 1, 2.072, 2.072}, {256, 128, 1, 1.419, 1.419}, {128, 128, 2, 1.272, 0.72},
     {128, 64, 2, 0.760, 0.495}, {64, 64, 2, 0.527, 0.264}, {128, 32, 2, 0.616, 0.308}}};

inline Mx4Choice choose(bool x4, int n, int d_o, int G) {
  using Choice = Mx4Choice;
  Choice best{Choice::kFew11, 1};
  double best_t = 1e30;
  const auto consider = [&](int kind, int splits, double t) {
    if (t < best_t) {
      best_t = t;
      best = {static_cast<Choice::Kind>(kind), splits};
    }
  };
  const auto parts = [](int a, int b) { return (a + b - 1) / b; };
  for (int i = 0; i < 7; ++i) {
    const FewTime& c = kFew[x4][i];
    if (!c.resident || parts(n, 16 * c.nt) > 65535) continue;   // a launch's limit
    const int64_t groups = static_cast<int64_t>(parts(d_o, 16 * c.rt)) * parts(n, 16 * c.nt);
    const int units = parts(parts(G, 8), c.waves);
    consider(Choice::kFew11x8 + i, 1,
             c.fixed + units * rounds_time((groups + 255) / 256, c.resident, c.alone, c.share));
  }
  if (n <= 16) return best;   // a large tile would be mostly empty
  const int blocks = x4 ? 8 : 2, even = x4 ? 1 : 2;
  const int all = parts(G, blocks);
  const double outputs = static_cast<double>(n) * d_o;
  for (int i = 0; i < 6; ++i) {
    const TileTime& c = kTiles[x4][i];
    const int64_t tiles = static_cast<int64_t>(parts(d_o, c.bm)) * parts(n, c.bn);
    for (const int want : {1, 2, 3, 4, 6, 8, 12, 16}) {
      const double join = want > 1 ? 4.0 + 1.3e-6 * want * outputs : 0.;   // written and read, fp32
      if (4.0 + join >= best_t || (want > 1 && want * outputs > 67108864.)) break;
      const int per = parts(parts(all, want), even) * even, splits = parts(all, per);
      if (splits != want || (want > 1 && per < 2)) continue;
      const int64_t groups = (tiles * splits + 255) / 256;
      consider(Choice::k256x256 + i, splits,
               4.0 + join + per * rounds_time(groups, c.resident, c.alone, c.share));
    }
  }
  return best;
}

}  // namespace qz
