"""Bounds of the grouped kernel's split last wave, on the host: the plan and the
addresses of the partial sums (csrc/tail_plan.h, which the kernel itself uses)
compiled with the host compiler and gone over for many calls.

Each form's last slot has to end inside the scratch, its counters inside theirs,
and no two (tile, piece, CTA, column) may share a value.
"""
import os
import shutil
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "blackwell_tile_gemm_gb300", "csrc")

PROGRAM = r"""
#include <cstdio>
#include <cstdlib>
#include <vector>
#include "tail_plan.h"
using namespace tg;

struct Form { int tile_n, cta_group; bool few, down; };

static long splits = 0, after_full = 0;

// One call: `tiles` tiles over `units`, `k_blocks` stages, rank values or not.
static void check(const Form& f, int64_t tiles, int units, int k_blocks, int rows, int rank) {
  const int width = tail_slot_width(f.down, rank);
  const int full = static_cast<int>(tiles / units) * units;
  const TailShape s{static_cast<int>(tiles) - full, units, k_blocks, f.cta_group, f.few, rows, rank,
                    tail_max_slots(f.tile_n, f.cta_group, width), tail_max_counters(f.cta_group)};
  uint32_t least = 0xFFFFFFFFu;
  int S = 1;
  for (int c = 0; c < 32; ++c)
    if (tail_cost(s, c) < least) least = tail_cost(s, c), S = c;
  if (least >= tail_limit(s)) return;
  ++splits;
  after_full += full > 0;
  const int64_t values = kTailPartialBytes / sizeof(float);
  // The last value of the last column of the last slot.
  const int64_t last = tail_column(s.rest - 1, S - 1, S, f.cta_group, f.cta_group - 1, f.tile_n,
                                   f.tile_n - 1, width) + width - 1;
  if (last >= values || s.rest * f.cta_group > kTailFlagWords || S > kTailMostPieces) {
    printf("out of range: tiles %lld units %d stages %d rank %d pieces %d: %lld of %lld values\n",
           (long long)tiles, units, k_blocks, rank, S, (long long)last, (long long)values);
    exit(1);
  }
}

int main() {
  const int units_of[] = {152, 148, 132, 76, 74, 8, 1};
  const int ks[] = {1, 8, 12, 16, 32, 47, 64, 96, 128, 175, 256};   // stages of 64
  // The rank values: 64 rows a tile, 128 of the rank.
  const Form down{64, 1, false, true};
  for (int units : units_of)
    for (int k : ks)
      for (int rank = 8; rank <= 256; rank += 8)
        for (int64_t M = 1; M <= 1000000; M += M < 24000 ? 61 : 3989)
          check(down, (M + 63) / 64 * ((rank + 127) / 128), units, k, 64, rank);
  // The products: single CTAs of 64 and 128 columns, CTA pairs of 256.
  const Form forms[] = {{64, 1, false, false}, {64, 1, true, false}, {128, 1, true, false},
                        {256, 2, false, false}};
  for (const Form& f : forms)
    for (int units : units_of)
      for (int k : ks)
        for (int64_t tiles = 1; tiles <= 3000; ++tiles)
          for (int rank = 8; rank <= (f.few ? 256 : 8); rank += 40)
            check(f, tiles, units, k, f.tile_n, rank);
  // Slots do not overlap.
  for (const Form& f : {down, forms[2], forms[3]})
    for (int width : {8, 72, 128}) {
      if (!f.down && width != 128) continue;
      const int rest = 5, S = 3;
      std::vector<char> used(static_cast<size_t>(rest) * S * f.cta_group * f.tile_n * width, 0);
      for (int t = 0; t < rest; ++t)
        for (int q = 0; q < S; ++q)
          for (int c = 0; c < f.cta_group; ++c)
            for (int col = 0; col < f.tile_n; ++col)
              for (int x = 0; x < width; ++x) {
                const size_t at = tail_column(t, q, S, f.cta_group, c, f.tile_n, col, width) + x;
                if (at >= used.size() || used[at]++) return printf("overlap\n"), 1;
              }
    }
  printf("%ld %ld\n", splits, after_full);
}
"""


def test_partial_sums_stay_inside_the_scratch(tmp_path):
    cxx = shutil.which("g++") or shutil.which("c++")
    if cxx is None:
        pytest.skip("no host compiler")
    src, exe = tmp_path / "plan.cc", tmp_path / "plan"
    src.write_text(PROGRAM)
    subprocess.run([cxx, "-std=c++17", "-O1", "-I", CSRC, str(src), "-o", str(exe)], check=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stdout
    splits, after_full = map(int, r.stdout.split())
    assert splits > 1000 and after_full > 1000      # the sweep reaches both kinds


def test_the_kernel_addresses_partial_sums_by_the_plan_alone():
    """Every use of the scratch in the kernel goes through tail_column."""
    text = open(os.path.join(CSRC, "grouped_kernel.cuh")).read()
    uses = [i for i in range(len(text)) if text.startswith("p.partials", i)]
    assert uses
    for i in uses:
        assert "tail_column(" in text[i:i + 120], text[i:i + 120]
