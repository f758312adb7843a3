"""The plan of the products with MX4 weights (csrc/mx4_plan.h), on the host.

The tile kernels stream their operands into LDS by copies that a wavefront counts: at the join of
stage st it waits until at most N of its copies are in flight, and copies land in the order of their
issue.  The model below issues the copies of every wavefront in the kernel's order and asks at every
join whether what stage st + 1 reads has landed: its X, both halves of its W buffer and its factors."""
import os
import subprocess

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "post_weight_quantization_05_amd", "csrc")

MODEL = r"""
#include <cstdio>
#include <vector>
#include "mx4_plan.h"
using namespace qz;

// One wavefront over nst stages, `whole` of them (counted past the split's end too) full.  A copy of
// a ragged stage is issued where one of its lanes is inside the matrix: `ragged` says whether.
template <bool X4, class T>
int wavefront(int wave, int nst, int whole, bool words, bool ragged) {
  using G = TileGeom<X4>;
  constexpr int kPer = kFetch / G::kBlocks;
  int issued = 0, wrong = 0;
  std::vector<int> w(nst + 4, 0), x(nst + 4, 0), f(nst / kPer + 2, 0);   // copies up to the last one of each
  const auto fetch = [&](int gen) {
    if (!words) return;   // by registers, which the compiler waits for
    for (int p = wave; p < T::kFRows / 4; p += T::kWaves) ++issued;
    f[gen] = issued;
  };
  const auto issue = [&](int st) {
    const bool full = st / G::kWParts * G::kWParts + G::kWParts <= whole;
    for (int p = wave; p < T::kPieces; p += T::kWaves) {
      const bool is_w = p < T::kWPieces;
      if (!is_w && st >= nst) continue;
      if (full || ragged) ++issued;
      (is_w ? w : x)[st] = issued;
    }
  };
  const int issues = (nst + G::kWParts - 1) / G::kWParts * G::kWParts;
  fetch(0);
  for (int i = 0; i < G::kRing; ++i)
    if (i < issues) issue(i);
  int landed = issued;
  for (int st = 0; st + 1 < nst; ++st) {
    if ((st + 1) % kPer == 0) fetch((st + 1) / kPer);
    const TileWait wait = tile_wait<X4>(st, nst, whole);
    const int left = wait == TileWait::kAll ? 0 : wait == TileWait::kButX ? T::kXLeast : T::kCopies + (wave < T::kExtra);
    if (issued - left > landed) landed = issued - left;
    const int next = st + 1, pair = next / G::kWParts * G::kWParts;
    int need = x[next] > f[next / kPer] ? x[next] : f[next / kPer];
    for (int i = pair; i < pair + G::kWParts && i < issues; ++i) need = w[i] > need ? w[i] : need;
    if (need > landed) {
      if (!wrong) std::printf("tile %d x %d, wavefront %d of %d stages (%d whole, words %d): stage %d reads %d copies early\n",
                              T::BM, T::BN, wave, nst, whole, words, next, need - landed);
      ++wrong;
    }
    if (st + G::kRing < issues) issue(st + G::kRing);
  }
  return wrong;
}

template <bool X4, int WM, int WN, int MT, int NT>
int tile() {
  using T = TileShape<X4, WM, WN, MT, NT>;
  int wrong = 0;
  for (int nst = 1; nst <= 140; ++nst)
    for (int past : {-1, 0, 200}) {   // the last stage ragged, all whole, a split with others behind it
      if (past > 0 && nst % TileGeom<X4>::kWParts) continue;
      for (int wave = 0; wave < T::kWaves; ++wave)
        for (int bits = 0; bits < 4; ++bits)
          wrong += wavefront<X4, T>(wave, nst, nst + past, bits & 1, bits & 2);
    }
  return wrong;
}

int main() {
  int wrong = tile<false, 2, 4, 4, 2>() + tile<false, 4, 2, 2, 2>() + tile<false, 2, 2, 2, 2>() +
              tile<false, 2, 2, 2, 1>() + tile<false, 2, 2, 1, 1>() + tile<false, 4, 1, 1, 1>();
  wrong += tile<true, 2, 4, 4, 2>() + tile<true, 4, 2, 2, 2>() + tile<true, 2, 2, 2, 2>() +
           tile<true, 2, 2, 2, 1>() + tile<true, 2, 2, 1, 1>() + tile<true, 4, 1, 1, 1>();
  std::printf("%d wrong\n", wrong);
  return 0;
}
"""


def _run(tmp_path, source, stdin=""):
    src, exe = tmp_path / "a.cpp", tmp_path / "a.out"
    src.write_text(source)
    subprocess.run(["g++", "-O1", "-std=c++17", "-I", CSRC, str(src), "-o", str(exe)], check=True, timeout=100)
    return subprocess.run([str(exe)], input=stdin, capture_output=True, text=True, check=True, timeout=100).stdout


def test_a_stage_reads_only_copies_that_have_landed(tmp_path):
    out = _run(tmp_path, MODEL).splitlines()
    assert out[-1] == "0 wrong", "\n".join(out[:6] + out[-1:])


CHOICE = r"""
#include <cstdio>
#include "mx4_plan.h"
int main() {
  static const char* names[] = {"few 1x1 of 8", "few 1x1", "few 1x2", "few 2x1", "few 2x2", "few 2x4", "few 4x2",
                                "256x256", "256x128", "128x128", "128x64", "64x64", "128x32"};
  int x4;
  long n, d_i, d_o;
  while (std::scanf("%d %ld %ld %ld", &x4, &n, &d_i, &d_o) == 4) {
    const int G = static_cast<int>((d_i + 31) / 32);
    const qz::Mx4Choice c = qz::choose(x4, static_cast<int>(n), static_cast<int>(d_o), G);
    const int blocks = x4 ? qz::TileGeom<true>::kBlocks : qz::TileGeom<false>::kBlocks;
    const int parts = x4 ? qz::TileGeom<true>::kWParts : qz::TileGeom<false>::kWParts;
    const int all = (G + blocks - 1) / blocks, per = ((all + c.splits - 1) / c.splits + parts - 1) / parts * parts;
    std::printf("%s,%d,%d\n", names[c.kind], c.splits, per);
  }
}
"""


def _choices(tmp_path, sizes, x4):
    """(kernel, splits, stages of a split) of each (n, d_i, d_o)."""
    lines = _run(tmp_path, CHOICE, "\n".join(f"{int(x4)} {n} {d_i} {d_o}" for n, d_i, d_o in sizes)).split("\n")
    return [(k, int(s), int(p)) for k, s, p in (line.split(",") for line in lines if line)]


def test_the_long_products_reach_every_tile(tmp_path):
    from test_gpu_mx4_long import LONG_LINEAR
    got = _choices(tmp_path, LONG_LINEAR, False)
    assert [(k, s) for k, s, _ in got] == [
        ("256x256", 1), ("256x256", 2), ("256x128", 1), ("256x128", 3), ("128x128", 1), ("128x128", 3),
        ("128x64", 1), ("128x64", 3), ("64x64", 1), ("128x32", 3)]
    assert all(per >= 70 for _, _, per in got)
    assert all(d_i % 128 == 0 for _, d_i, _ in LONG_LINEAR)


def test_the_listed_products_reach_every_kernel(tmp_path):
    """Every few-token shape, and every tile with one split and with several."""
    from test_gpu_mx4 import EACH_LINEAR, EACH_MATMUL
    tiles = {(t, split) for t in ("256x256", "256x128", "128x128", "128x64", "64x64", "128x32")
             for split in (False, True)}
    for sizes, x4, few in ((EACH_LINEAR, False, {"few 1x1 of 8", "few 1x1", "few 2x1", "few 2x2", "few 4x2"}),
                           (EACH_MATMUL, True, {"few 1x1 of 8", "few 1x1", "few 1x2", "few 2x2", "few 2x4"})):
        got = {(k, s > 1) for k, s, _ in _choices(tmp_path, sizes, x4)}
        assert got == tiles | {(f, False) for f in few}, (x4, (tiles | {(f, False) for f in few}) ^ got)
