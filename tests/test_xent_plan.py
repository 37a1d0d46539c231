"""Plans of the vocabulary loss on the host (csrc/xent_plan.h, which the launches use),
compiled with the host compiler and gone over for many sizes: tiles cover the vocabulary,
the ring's slots and what the MMA reads beyond them stay inside shared memory, pieces
cover the vocabulary and fit their room, and what a reservation asks for serves every
smaller call."""
import os
import random
import shutil
import subprocess

import pytest

import blackwell_tile_gemm_gb300 as tg
from blackwell_tile_gemm_gb300 import build as tgbuild

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "blackwell_tile_gemm_gb300", "csrc")

PROGRAM = r"""
#include <cstdio>
#include <cstdlib>
#include <random>
#include "xent_plan.h"
using namespace tg;

static void fail(const char* what, long long M, long long N, long long K) {
  printf("%s: %lld %lld %lld\n", what, M, N, K);
  exit(1);
}

int main() {
  std::mt19937_64 gen(1);
  auto between = [&](double lo, double hi) {
    return static_cast<int64_t>(exp(std::uniform_real_distribution<>(log(lo), log(hi))(gen)));
  };
  for (int i = 0; i < 200000; ++i) {
    const int64_t M = between(1, 200000), N = between(1, 600000), K = between(1, 20000);
    const XentLossPlan q = xent_loss_plan(M, N);
    const bool few = M <= kXentFewRows;
    const int steps[2] = {few ? 16 : 32, 64};
    for (int step : steps) {
      const XentTiles t = xent_tiles(M, N, step);
      if (t.bn % step || t.bn < 32 || t.bn > 256 || (step == 64 && t.bn < 64)) fail("width", M, N, K);
      if (int64_t{t.bn} * t.n_tiles < N || int64_t{t.bn} * (t.n_tiles - 1) >= N) fail("cover", M, N, K);
      if (few ? t.m_tiles != 1 : int64_t{256} * t.m_tiles < M) fail("rows", M, N, K);
      if (few) {
        int b = 0, stages = 0;
        const int a_box = static_cast<int>((M + 7) / 8 * 8);
        const int a = xent_ring(a_box, t.bn, &b, &stages);
        if (stages < 4 || stages > 16 || stages * (a + b) > kXentRing) fail("ring", M, N, K);
        if (a % 1024 || b % 1024 || a < a_box * 128 || b < t.bn * 128) fail("slots", M, N, K);
        // The MMA reads 128 rows from the start of each slot of A.
        if ((stages - 1) * a + 128 * 128 > kXentRing) fail("reads past the ring", M, N, K);
      }
    }
    // [2 n_tiles][M] pairs before the targets' logits.
    if (int64_t{16} * q.tiles.n_tiles * M > static_cast<int64_t>(q.off_z)) fail("parts", M, N, K);
    for (int bf16 = 0; bf16 < 2; ++bf16) {
      const XentGradPlan g = xent_grad_plan(M, N, K, bf16);
      if (g.piece * g.pieces < N || g.piece * (g.pieces - 1) >= N) fail("pieces", M, N, K);
      if (g.pieces > 1 && g.piece % 256) fail("piece", M, N, K);
      if (g.rows % 64 || g.rows < M) fail("padding", M, N, K);
      const int64_t dz = int64_t{2} * g.terms * g.rows * ((g.piece + 63) / 64 * 64);
      if (static_cast<int64_t>(g.off_dz) < int64_t{2} * g.terms * g.rows * g.ld_a) fail("copy", M, N, K);
      if (static_cast<int64_t>(g.off_sum - g.off_dz) < dz) fail("dz", M, N, K);
      if (bf16 && g.pieces > 1 && static_cast<int64_t>(g.bytes - g.off_sum) < 4 * M * g.ld_sum)
        fail("sums", M, N, K);
    }
  }
  printf("ok\n");
}
"""


@pytest.mark.skipif(shutil.which("g++") is None, reason="needs g++")
def test_plans(tmp_path):
    src, exe = tmp_path / "plan.cpp", tmp_path / "plan"
    src.write_text("#include <cmath>\n" + PROGRAM)
    subprocess.run(["g++", "-std=c++17", "-O2", "-I", CSRC, str(src), "-o", str(exe)], check=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True)
    assert r.returncode == 0 and r.stdout.strip() == "ok", r.stdout


@pytest.mark.parametrize("call,kw", [
    (tg.TG_CALL_GEMM_BF16_XENT, {}),
    (tg.TG_CALL_GEMM_BF16_XENT_GRAD, dict(d_dtype=tg.TG_D_BF16)),
    (tg.TG_CALL_GEMM_BF16_XENT_GRAD, dict(d_dtype=tg.TG_D_F32)),
    (tg.TG_CALL_EMBED_ROWS_GRAD, {}), (tg.TG_CALL_BALANCE_LOSS, {})])
def test_a_reservation_serves_smaller_calls(call, kw):
    tgbuild.build()
    rng = random.Random(2)
    size = lambda hi: int(hi ** rng.random())  # noqa: E731
    for _ in range(3000):
        large = size(100000), size(200000 if call != tg.TG_CALL_BALANCE_LOSS else 4096), size(8192)
        small = tuple(rng.randint(1, x) for x in large)
        assert tg.workspace_bytes(call, *small, **kw) <= tg.workspace_bytes(call, *large, **kw), (
            small, large)


SLICES = r"""
#include <cmath>
#include <cstdio>
#include <cstdlib>
#include <random>
#include "xent_plan.h"
using namespace tg;

int main() {
  std::mt19937_64 gen(2);
  auto between = [&](double lo, double hi) {
    return static_cast<int64_t>(exp(std::uniform_real_distribution<>(log(lo), log(hi))(gen)));
  };
  int most = 0, both = 0;
  for (int i = 0; i < 200000; ++i) {
    const int64_t M = between(1, 200000), N = between(1, 600000), K = between(1, 20000);
    for (int bf16 = 0; bf16 < 2; ++bf16) {
      const XentGradPlan g = xent_grad_plan(M, N, K, bf16);
      const XentSlices a = g.rows_by, b = g.weights_by;
      // (One piece: the same room, one after the other.)
      const int64_t a_room = (g.pieces == 1 ? g.bytes : g.off_weights) - g.off_sum;
      const int64_t b_room = g.bytes - g.off_weights;
      const int64_t n = g.pieces > 1 ? g.piece : N;
      bool good = a.count >= 1 && a.count <= kXentMostSlices && b.count >= 1 &&
                  b.count <= kXentMostSlices;
      good &= a.columns % 32 == 0 && a.columns >= 160 && a.columns <= 256 && b.columns == 256;
      good &= (a.count == 1 && (!bf16 || g.pieces == 1)) || 4 * M * g.ld_sum * a.count <= a_room;
      good &= b.count == 1 || 4 * n * g.ld_sum * b.count <= b_room;
      // Rows of all slices and indices of all terms fit 32 bits.
      good &= a.count * M < int64_t{1} << 31 && b.count * (g.terms * g.rows + 64) < int64_t{1} << 31;
      good &= g.off_sum % 1024 == 0 && g.off_weights % 1024 == 0;
      if (!good) {
        printf("%lld %lld %lld %d\n", (long long)M, (long long)N, (long long)K, bf16);
        return 1;
      }
      most = a.count > most ? a.count : most;
      both += a.count > 1 && b.count > 1;
    }
  }
  puts(most > 16 && both > 100 ? "ok" : "never sliced");
}
"""


@pytest.mark.skipif(shutil.which("g++") is None, reason="needs g++")
def test_slices(tmp_path):
    src, exe = tmp_path / "slices.cpp", tmp_path / "slices"
    src.write_text(SLICES)
    subprocess.run(["g++", "-std=c++17", "-O2", "-I", CSRC, str(src), "-o", str(exe)], check=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True)
    assert r.returncode == 0 and r.stdout.strip() == "ok", r.stdout
