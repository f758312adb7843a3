"""The plan of the products of 8-bit integer rows (csrc/i8_plan.h), on the host.

The tile kernels stream halves of stages through a ring of places in LDS, by copies that a wavefront
counts.  The model below issues every wavefront's copies in the kernel's order and asks at every join
whether what stage st + 1 reads has landed, and at every issue whether the place it fills is free.  And the
sizes of the GPU tests have to reach every kernel there is."""
import os
import subprocess

import pytest

from test_gpu_i8 import REACH_LAYERS, REACH_PRODUCTS

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "post_weight_quantization_05_amd", "csrc")
KINDS = 10

MODEL = r"""
#include <cstdio>
#include <cstdlib>
#include <vector>
#include "i8_plan.h"
using namespace qz;

template <class T>
int tile(int nst) {
  constexpr int H = T::kRing;
  const int halves = 2 * nst;
  int wrong = 0, issued = 0, joined = -1, landed = 0;   // halves; joined: the last join's stage
  const auto issue = [&](int p) {   // in order; its place is free when the stage of half p - H is joined
    if (p != issued || (p >= H && (p - H) / 2 > joined)) ++wrong;
    ++issued;
  };
  const auto wait = [&](int left) {   // copies that may be in flight
    const int whole = issued - (left + T::kCopies - 1) / T::kCopies;
    if (whole > landed) landed = whole;
  };
  const auto reads = [&](int st) { if (landed < 2 * st + 2) ++wrong; };
  for (int i = 0; i < H && i < halves; ++i) issue(i);
  wait(tile_in_flight_first<T>(halves));
  reads(0);
  for (int st = 0; st + 1 < nst; ++st) {
    const int left = tile_in_flight<T>(st, halves);
    wait(left);
    joined = st;
    // two halves behind a whole join, or what there is
    for (int p = 2 * st + H; p <= 2 * st + H + 1; ++p)
      if (left || p < halves) issue(p);
    if (issued > halves) ++wrong;
    reads(st + 1);
  }
  if (issued != halves) ++wrong;
  if (wrong) std::printf("tile %d x %d, %d stages: %d wrong\n", T::BM, T::BN, nst, wrong);
  return wrong;
}

int main(int argc, char** argv) {
  if (argc == 1) {
    int wrong = 0;
    for (int nst = 1; nst <= 70; ++nst)
      wrong += tile<Tile256x256>(nst) + tile<Tile256x128>(nst) + tile<Tile128x128>(nst) + tile<Tile128x64>(nst) +
               tile<Tile64x64>(nst) + tile<Tile64x64By4>(nst);
    return wrong != 0;
  }
  const long n = atol(argv[1]), a = atol(argv[2]), b = atol(argv[3]);
  if (argc == 4) {   // a product: n, d_i, d_o
    std::printf("%d\n", static_cast<int>(i8_choose(n, b, (a + 127) / 128, 0, false)));
  } else {           // a layer: n, d, f, E, k
    const int E = atoi(argv[4]), k = atoi(argv[5]);
    if (i8_moe_by_rows(n, a, b, E, k)) std::printf("rows\n");
    else std::printf("%d %d\n", static_cast<int>(i8_choose(n * k, 2 * b, (a + 127) / 128, E, true)),
                     static_cast<int>(i8_choose(n * k, a, (b + 127) / 128, E, false)));
  }
}
"""


@pytest.fixture(scope="module")
def model(tmp_path_factory):
    d = tmp_path_factory.mktemp("i8_plan")
    (d / "model.cpp").write_text(MODEL)
    subprocess.run(["g++", "-std=c++17", "-O1", "-I", CSRC, str(d / "model.cpp"), "-o", str(d / "model")], check=True, timeout=100)
    return str(d / "model")


def test_every_read_waits_for_its_copies(model):
    r = subprocess.run([model], capture_output=True, text=True, timeout=60)
    assert r.returncode == 0, r.stdout


def test_the_gpu_tests_reach_every_product_kernel(model):
    out = lambda *a: subprocess.run([model, *map(str, a)], capture_output=True, text=True, check=True, timeout=10).stdout.split()  # noqa: E731
    assert {int(out(*p)[0]) for p in REACH_PRODUCTS} == set(range(KINDS))
    layers = [out(n, d, f, E, k) for n, E, k, d, f in REACH_LAYERS]
    assert ["rows"] in layers
    pairs = [tuple(map(int, r)) for r in layers if r != ["rows"]]
    assert {d for _, d in pairs} == set(range(KINDS))
    assert {g for g, _ in pairs} == set(range(KINDS)) - {0, 8, 9}    # gate and up rows do not fit side by side there
