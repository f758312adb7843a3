// Plan of a product of 8-bit integer rows: the kernels' shapes, what their wavefronts wait for, and the
// choice of a kernel from the sizes.  Plain C++, so that host programs can include it.
#pragma once

#include <cmath>
#include <cstdint>

namespace qz {

// ------------------------------------------------------------------------------- tile kernels
// Workgroup tile of BM rows of W by BN rows of X, BM = 32 MT WM, BN = 32 NT WN, in WM x WN wavefronts
// of 32 MT x 32 NT each.  The contraction goes in stages of 128 columns: whole lines of both.
template <int WM_, int WN_, int MT_, int NT_, int LDS_KB>
struct TileI8 {
  static constexpr int WM = WM_, WN = WN_, MT = MT_, NT = NT_;
  static constexpr int kWaves = WM * WN, kThreads = 64 * kWaves;
  static constexpr int BM = 32 * MT * WM, BN = 32 * NT * WN;
  static constexpr int kHalfW = BM / 2 * 128, kHalf = (BM + BN) / 2 * 128;   // bytes
  static constexpr int kFit = LDS_KB * 1024 / kHalf, kRing = kFit < 16 ? kFit : 16;   // halves of a stage in LDS
  static constexpr int kCopiesW = BM / 16 / kWaves, kCopiesX = BN / 16 / kWaves;   // of a half, a wavefront
  static constexpr int kCopies = kCopiesW + kCopiesX;
  static constexpr int kProducts = MT * NT, kReads = MT + NT;   // of a step of 32 columns
  static constexpr int kSteps = MT * NT <= 4 ? 4 : 1;           // whose operands are read ahead
  static_assert(BM % (16 * kWaves) == 0 && BN % (16 * kWaves) == 0 && kRing >= 5);
  static constexpr int kOutPitch = 32 * MT * 4 + 16;
  static constexpr int kOut = kWaves * 32 * kOutPitch;
  static constexpr int kUsed = kRing * kHalf;
  static constexpr int kShared = kUsed > kOut + 12 * BM ? kUsed : kOut + 12 * BM;
  static_assert(kShared <= 160 * 1024);
};
using Tile256x256 = TileI8<2, 4, 4, 2, 160>;
using Tile256x128 = TileI8<4, 2, 2, 2, 160>;
using Tile128x128 = TileI8<2, 2, 2, 2, 80>;
using Tile128x64 = TileI8<2, 2, 2, 1, 80>;
using Tile64x64 = TileI8<2, 2, 1, 1, 80>;
using Tile64x64By4 = TileI8<2, 2, 1, 1, 40>;

// Half p of the stages (2 st and 2 st + 1 of stage st) lies at place p % kRing of LDS.  Halves
// 0 .. kRing - 1 go out first; at the join of stage st its places are free, and halves 2 st + kRing and
// 2 st + kRing + 1 go out behind it.  Copies land in the order of their issue, and stage st + 1 has to have
// landed at the join: where both halves of every join so far were there to issue, the kRing - 4 halves
// behind it may be in flight; towards the end nothing may.
template <class T>
constexpr int tile_in_flight(int st, int halves) {
  return 2 * st + T::kRing + 1 < halves ? (T::kRing - 4) * T::kCopies : 0;
}
// Before the first stage: all halves but its own two.
template <class T>
constexpr int tile_in_flight_first(int halves) {
  return T::kRing <= halves ? (T::kRing - 2) * T::kCopies : 0;
}

// ---------------------------------------------------------------- very few tokens (k_i8_rows.hip)
// LDS of a workgroup for its tokens' codes, besides some for the sums.
constexpr int64_t kI8RowsLds = 56 * 1024;
inline bool i8_rows_fit(int64_t rows, int64_t pitch) { return rows * ((pitch + 1023) / 1024 * 1024) <= kI8RowsLds; }

// A product of one to four tokens: one launch, which quantizes them itself and needs no workspace.
inline bool i8_by_rows(int64_t n, int64_t pitch) { return n <= 4 && i8_rows_fit(n, pitch); }

// Few pairs of an expert layer, each with its expert's rows alone, in two launches: where the weights that
// several tokens ask for, read once for each, take less time (at 5.2 TB/s) than three more launches and what
// they do (16 us).
inline bool i8_moe_by_rows(int64_t n, int64_t d, int64_t f, int experts, int k) {
  const int64_t pairs = n * k;
  if (pairs > 256 || !i8_rows_fit(1, (d + 127) / 128 * 128) || !i8_rows_fit(k, (f + 127) / 128 * 128)) return false;
  const double part = k < experts ? 1. - static_cast<double>(k) / experts : 0.;
  const double reached = experts * (1. - std::pow(part, static_cast<double>(n)));   // on average
  return (pairs - reached) * 3. * d * f < 16. * 5.2e6;
}

// -------------------------------------------------------------------------- few-token kernels
// Each wavefront streams its part of the contraction through LDS of its own, 128 columns a stage,
// kDepth stages deep: whole lines of both operands, no registers in flight and no barrier before the
// sums are joined.  kGateUp: the first half of the rows are gate rows, the second their up rows.
template <int RT_, int NT_, int WAVES_, int LDS_KB>
struct FewI8 {
  static constexpr int RT = RT_, NT = NT_, kWaves = WAVES_;
  static constexpr int kCopies = 2 * (RT + NT);             // of a stage, 1024 bytes each
  static constexpr int kStage = kCopies * 1024;
  static constexpr int kFit = LDS_KB * 1024 / kWaves / kStage, kDepth = kFit < 8 ? kFit : 8;
  static constexpr int kLds = kWaves * kDepth * kStage;
  static_assert(kDepth >= 3 && kLds >= kWaves * RT * NT * 1024);
};
using Few11 = FewI8<1, 1, 4, 80>;
using Few21 = FewI8<2, 1, 4, 80>;
using Few22 = FewI8<2, 2, 4, 160>;
using Few24 = FewI8<2, 4, 4, 160>;

// ------------------------------------------------------------------------- choice of a kernel
// kFewRN: 16 R rows of W by 16 N of X, four wavefronts that share the contraction (k_i8_few.hip);
// kBMxBN: tiles (k_i8_gemm.hip); by4: with LDS for four workgroups a compute unit, not two.
enum class I8Kind { kFew11, kFew21, kFew22, kFew24, k256x256, k256x128, k128x128, k128x64, k64x64, k64x64by4 };

// Times in microseconds from the sizes: `fixed`, then for every round of resident workgroups of a
// compute unit `each` and a time for each stage of 128 columns of a wavefront: `alone`, or for r
// together at least r times `share`.  Fitted to 1100 measurements of seven layers.  On 274 sizes measured since (5 to 5000
// tokens, 128 to 12288 columns, half of the sizes drawn at random; the estimates 9 to 18% root mean square off) the
// kernel chosen is 1.6% slower than the best one on average, 21% at most.  Both sides, measured, us: 13 tokens
// 4096 -> 12288, few 2 x 1 9.6, 1 x 1 10.2; 64 tokens 4096 -> 4096, few 2 x 2 6.3, 2 x 1 7.0, 64 x 64 9.2; 1000 tokens
// 4096 -> 4096, 128 x 128 22.5, 128 x 64 24.1; 1600 tokens there, 256 x 128 31.2, 128 x 128 32.2; 4000 tokens
// 4096 -> 12288, 256 x 256 178, 256 x 128 199.  Sums split along the contraction and joined in a second launch lost
// against the best of these at every size measured.
//
// Where it errs: 128 x 128 is estimated 15 to 20% too fast where there is most of a tile a compute unit, but no more
// (256 tokens 4096 -> 12288, taken 22.0, 64 x 64 by four 20.5; 160 tokens there 20.9, 18.2), and tiles of 256 rows of W
// as much over several rounds (1600 tokens 2048 -> 10240, taken 256 x 128 55.5, 128 x 128 47.9).  Of the 272 products of
// 136 drawn and ordinary expert layers (2 to 4096 tokens, 2 to 128 experts, skewed) the one chosen is 3.6% slower than
// the best on average; the worst are narrow layers of many experts with 90 tokens each, whose tiles of 256 are two
// thirds empty (2910 tokens 2 of 64, 640 -> 2 x 416: 28.0, 128 x 64 16.8).
struct I8Time {
  I8Kind kind;
  int bm, bn, resident, waves;   // waves that share the contraction
  double fixed, each, alone, share;
};
constexpr I8Time kI8Times[] = {
    {I8Kind::kFew11, 16, 16, 2, 4, 2.089, 0.397, 0.192, 0.186},
    {I8Kind::kFew21, 32, 16, 2, 4, 1.787, 0.621, 0.181, 0.274},
    {I8Kind::kFew22, 32, 32, 1, 4, 0.305, 2.270, 0.358, 0.358},
    {I8Kind::kFew24, 32, 64, 1, 4, 0.000, 3.066, 0.481, 0.481},
    {I8Kind::k256x256, 256, 256, 1, 1, 0.000, 7.792, 1.125, 1.125},
    {I8Kind::k256x128, 256, 128, 1, 1, 0.000, 6.060, 0.586, 0.586},
    {I8Kind::k128x128, 128, 128, 2, 1, 2.051, 2.374, 0.286, 0.446},
    {I8Kind::k128x64, 128, 64, 2, 1, 1.877, 1.511, 0.291, 0.280},
    {I8Kind::k64x64, 64, 64, 2, 1, 2.351, 0.960, 0.029, 0.178},
    {I8Kind::k64x64by4, 64, 64, 4, 1, 1.726, 0.575, 0.349, 0.180}};

// n rows of X (of an expert layer: pairs) by d_o rows of W (of an expert), in `stages` of 128 columns;
// experts: 0 for a plain product; gate_up: gate and up rows side by side.
inline I8Kind i8_choose(int64_t n, int64_t d_o, int64_t stages, int experts, bool gate_up) {
  const auto parts = [](int64_t a, int64_t b) { return (a + b - 1) / b; };
  I8Kind best = I8Kind::kFew21;
  double best_t = 1e30;
  for (const I8Time& c : kI8Times) {
    const bool few = c.waves > 1;
    // not measured there, or gate and up rows do not fit side by side
    if (few ? n > 300 && !experts : n <= 16) continue;
    if (gate_up && (c.kind == I8Kind::kFew11 || c.bm == 64)) continue;
    // tiles of X: with experts, each has its share of the pairs and its last tile is half empty
    const int64_t used = n < experts ? n : experts;
    const int64_t tiles = !experts ? parts(n, c.bn) : n <= used * c.bn / 2 ? used : n / c.bn + used / 2;
    if (few && tiles > 65000) continue;   // a launch's limit
    const int64_t all = parts(d_o, c.bm) * tiles, groups = parts(all, 256);
    const double st = static_cast<double>(parts(stages, c.waves));
    const auto together = [&](int64_t r) {
      const double a = c.each + c.alone * st, s = r * (c.each + c.share * st);
      return c.resident == 1 || a > s ? a : s;
    };
    double t = c.fixed + (groups / c.resident) * together(c.resident) +
               (groups % c.resident ? together(groups % c.resident) : 0.);
    // Of several rounds of experts' tiles, full ones and short ones, half a round is left over on average: without this,
    // 4096 tokens 6 of 64 experts, 2048 -> 2 x 1408, take 256 x 128, 227 us, and not 256 x 256, 208.  Over those 272 products
    // it makes no difference (3.6 and 3.4%), and on the tiles of which several are resident it costs (4.0%).
    if (experts && c.resident == 1 && groups > 1) t = c.fixed + (all / 256. + 0.5) * together(1);
    if (t < best_t) {
      best_t = t;
      best = c.kind;
    }
  }
  return best;
}

}  // namespace qz
