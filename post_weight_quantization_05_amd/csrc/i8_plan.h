// Plan of a product of 8-bit integer rows: the choice of a kernel from the sizes.  Plain C++, so that
// host programs can include it.
#pragma once

#include <cstdint>

namespace qz {

// kFewRN: 16 R rows of W by 16 N of X, four wavefronts that share the contraction (k_i8_few.hip);
// kBMxBN: tiles (k_i8_gemm.hip); by4: with LDS for four workgroups a compute unit, not two.
enum class I8Kind { kFew11, kFew21, kFew22, kFew24, k256x256, k256x128, k128x128, k128x64, k64x64, k64x64by4 };

// Times in microseconds from the sizes: `fixed`, then for every round of resident workgroups of a
// compute unit `each` and a time for each stage of 128 columns of a wavefront: `alone`, or for r
// together at least r times `share`.  Fitted to 1100 measurements (5 to 4000 tokens, seven layers of
// 512 to 12288 columns; 7 to 15% root mean square); the kernel chosen is 1.5% slower than the best
// one measured there on average, 25% at most.  Both sides, measured, us: 13 tokens 4096 -> 12288, few
// 2 x 1 9.6, 1 x 1 10.2; 64 tokens 4096 -> 4096, few 2 x 2 6.3, 2 x 1 7.0, 64 x 64 9.2; 256 tokens
// 4096 -> 12288, 64 x 64 by four 20.7, 128 x 128 22.1; 1000 tokens 4096 -> 4096, 128 x 128 22.2,
// 128 x 64 23.9; 1600 tokens there, 256 x 128 31.2, 128 x 128 32.2; 4000 tokens 4096 -> 12288,
// 256 x 256 178, 256 x 128 199.  Sums split along the contraction and joined in a second launch lost
// against the best of these at every size measured.
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
    const int64_t groups = parts(parts(d_o, c.bm) * tiles, 256);
    const double st = static_cast<double>(parts(stages, c.waves));
    const auto together = [&](int64_t r) {
      const double a = c.each + c.alone * st, s = r * (c.each + c.share * st);
      return c.resident == 1 || a > s ? a : s;
    };
    const double t = c.fixed + (groups / c.resident) * together(c.resident) +
                     (groups % c.resident ? together(groups % c.resident) : 0.);
    if (t < best_t) {
      best_t = t;
      best = c.kind;
    }
  }
  return best;
}

}  // namespace qz
