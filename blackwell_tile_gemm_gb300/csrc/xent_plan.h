// Plans of the vocabulary loss: tile widths, pieces of the vocabulary and the
// layout of the workspace.  Plain arithmetic, the same with and without a GPU.
#pragma once

#include <cstddef>
#include <cstdint>

namespace tg {

// SMs the widths are balanced for (another count changes the balance, not the
// results' validity).
constexpr int kXentSms = 152;
// Up to this many rows run as single CTAs.
constexpr int64_t kXentFewRows = 128;

// Fewest columns of a tile.
constexpr int64_t kXentFewLeast = 48;
constexpr int64_t kXentLeast = 128;

inline int64_t xent_up(int64_t a, int64_t b) { return (a + b - 1) / b * b; }

struct XentTiles {
  int bn;        // columns of a tile
  int m_tiles, n_tiles;
};

// Columns per tile: the width whose waves over the units take least.  A stage of
// a CTA pair costs the larger of its MMAs (2 cycles a column) and its loads (128
// rows of A and half the columns of B at 64 bytes a cycle).  One of few rows streams
// B from HBM, and A's rows with it, but no stage takes less than the 0.3 us of its four
// MMAs (0.1 whatever their width), its wait and commit, and its share of a chunk's
// hand-over (0.1); fewer loads or slots change nothing (one token x 64000 x 4096: tiles
// of 48 columns 186 us, 112 90, 224 78, i.e. 6.7 TB/s).  The last tile's epilogue is
// hidden by nothing.
inline XentTiles xent_tiles(int64_t M, int64_t N, int step) {
  const bool few = M <= kXentFewRows;
  const int64_t units = few ? kXentSms : kXentSms / 2;
  const int64_t mt = few ? 1 : (M + 255) / 256;
  const int64_t least = few ? (step > kXentFewLeast ? step : kXentFewLeast) : kXentLeast;
  int64_t best = 0, bn = 256;
  for (int64_t c = 256; c >= least; c -= step) {
    const int64_t waves = (mt * ((N + c - 1) / c) + units - 1) / units;
    const int64_t stage = c + M > 112 ? c + M : 112;
    const int64_t cost = few ? waves * (stage + 16) + c / 8
                             : waves * ((2 * c > 256 + c ? 2 * c : 256 + c) + 48);
    if (best == 0 || cost < best) {
      best = cost;
      bn = c;
    }
  }
  return XentTiles{static_cast<int>(bn), static_cast<int>(mt), static_cast<int>((N + bn - 1) / bn)};
}

// The ring of single CTAs: slots of a_box rows of A (from the start of the ring) and b_box
// of B (behind all of A's), 128 bytes a row, whole 1 KB swizzle atoms.  The MMA reads
// 128 rows from each slot of A: the last has to have as many bytes of the ring behind
// its start.
constexpr int kXentRing = 192 * 1024;
inline int xent_ring(int a_box, int b_box, int* b_bytes, int* stages) {
  const int a_bytes = static_cast<int>(xent_up(a_box, 8)) * 128;
  *b_bytes = static_cast<int>(xent_up(b_box, 8)) * 128;
  int s = kXentRing / (a_bytes + *b_bytes);
  if (s > 16) s = 16;
  *stages = s;
  return a_bytes;
}

// Workspace of the loss: [2 * n_tiles][M] pairs, then the targets' logits.  `bytes` is
// what the narrowest tiles would take, for this many rows or for few: it grows with M
// and N, so that a reservation for the largest call serves all smaller ones.
struct XentLossPlan {
  XentTiles tiles;
  size_t off_z, bytes;
};
inline XentLossPlan xent_loss_plan(int64_t M, int64_t N) {
  XentLossPlan q{};
  q.tiles = xent_tiles(M, N, M <= kXentFewRows ? 16 : 32);   // (MMAs of a pair: 16 a CTA)
  const int64_t few = (N + kXentFewLeast - 1) / kXentFewLeast * (M < kXentFewRows ? M : kXentFewRows);
  const int64_t many = M > kXentFewRows ? (N + kXentLeast - 1) / kXentLeast * M : 0;
  q.off_z = static_cast<size_t>(xent_up(16 * (few > many ? few : many), 256));
  q.bytes = q.off_z + static_cast<size_t>(4 * M);
  return q;
}

// Slices of a contraction: with few tiles the gradients' products are cut along it, the
// slices' f32 sums added afterwards.  A product of `tiles(columns)` tiles and `stages`
// stages; columns per tile and slices whose waves over the pairs of CTAs take least, in
// cycles: a stage the larger of its MMAs (2 a column) and its loads (128 rows and half
// the columns at 64 bytes a cycle); a tile its start and its stores; slices their
// `bytes` (of one) written and read at 3 KB a cycle, and a launch.
// Loss and gradients, without slices and with: 202 rows x 120448 x 384 in bf16 200 ->
// 145 us, 1 x 69040 x 149 90 -> 57, 20000 x 130 x 257 in f32 151 -> 79, 2259 x 1281 x
// 392 80 -> 50; 4096 x 128000 x 4096 has tiles enough and takes none.
constexpr int kXentMostSlices = 64;
constexpr int64_t kXentSliceBytes = int64_t{40} << 20;

struct XentSlices {
  int count;         // 1: none
  int columns;       // of a tile
};
inline XentSlices xent_slices(int64_t wide_tiles, int64_t rows, int64_t least_columns, int64_t stages,
                              int64_t bytes) {
  XentSlices q{1, 256};
  int64_t best = 0;
  for (int64_t c = 256; c >= least_columns; c -= 32) {
    const int64_t tiles = wide_tiles * ((rows + c - 1) / c);
    for (int64_t n = 1; n <= kXentMostSlices; ++n) {
      if (n > 1 && (n * bytes > kXentSliceBytes || stages < 4 * n)) break;
      const int64_t waves = (tiles * n + kXentSms / 2 - 1) / (kXentSms / 2);
      const int64_t stage = (2 * c > 256 + c ? 2 * c : 256 + c) + 70;
      const int64_t cost = waves * ((stages + n - 1) / n * stage + 4000) +
                           (n > 1 ? 6000 + n * bytes / 1500 : 0);
      if (best == 0 || cost < best) {
        best = cost;
        q = XentSlices{static_cast<int>(n), static_cast<int>(c)};
      }
      if (waves > 8) break;
    }
  }
  return q;
}

// Workspace of the gradient: the rows of A that have a target (the others as zeros),
// dz of one piece of the vocabulary, dA's f32 sums (of all pieces, each slice's) and
// dB's (of a piece).  With two terms of dz a row's second follows its first:
// [rows][2][ld_dz].  Read as rows twice as long, one contraction of dA takes both (B's
// rows a second time); read as twice the rows, so does one of dB, with each row of A
// twice.  Zeros fill the rows up to whole stages of that contraction: a ragged one takes
// a detour (1000 rows x 50304 x 1024 89 us, 1024 rows 74).
//
// Pieces are as wide as kXentDzBytes allow, but at least kXentLeastPiece columns:
// every piece adds its share of dA to all of it in memory, 8 bytes for 2 * width
// operations.
constexpr int64_t kXentDzBytes = int64_t{256} << 20;
constexpr int64_t kXentLeastPiece = 8192;

struct XentGradPlan {
  int terms;          // of dz: 2 where the gradients are f32
  int64_t rows;       // of dz: M in steps of 64
  int64_t piece;      // columns of a piece, a multiple of 256 (or all)
  int64_t pieces;
  XentSlices rows_by, weights_by;   // slices of dA's and of dB's contractions
  int64_t ld_a, ld_sum;
  size_t off_dz, off_sum, off_weights, bytes;
};
inline XentGradPlan xent_grad_plan(int64_t M, int64_t N, int64_t K, bool bf16) {
  XentGradPlan q{};
  q.terms = bf16 ? 1 : 2;
  q.rows = xent_up(M, 64);
  const int64_t column = 2 * q.terms * q.rows;               // bytes of dz
  int64_t most = kXentDzBytes / column / 256 * 256;
  if (most < kXentLeastPiece) most = kXentLeastPiece;
  q.pieces = (N + most - 1) / most;
  q.piece = q.pieces == 1 ? N : xent_up((N + q.pieces - 1) / q.pieces, 256);
  q.pieces = (N + q.piece - 1) / q.piece;
  q.ld_a = xent_up(K, 64);
  q.ld_sum = xent_up(K, 4);
  const int64_t wide = (K + 255) / 256;
  const int64_t a_bytes = 4 * M * q.ld_sum, b_bytes = 4 * q.piece * q.ld_sum;
  q.rows_by = xent_slices(wide, M, 160, q.terms * ((q.piece + 63) / 64), a_bytes);
  q.weights_by = xent_slices(wide, q.piece, 256, q.terms * q.rows / 64, b_bytes);
  // Room for the widest piece and the most slices there could be: it grows with M, N
  // and K, so that a reservation for the largest call serves all smaller ones.
  const int64_t widest = column * kXentLeastPiece > kXentDzBytes ? column * kXentLeastPiece
                                                                 : kXentDzBytes;
  const int64_t all = column * xent_up(N, 64);
  auto sliced = [](int64_t one) {
    return kXentMostSlices * one < kXentSliceBytes ? kXentMostSlices * one : kXentSliceBytes;
  };
  int64_t sums = sliced(a_bytes);
  if (bf16 && q.pieces > 1 && sums < a_bytes) sums = a_bytes;
  q.off_dz = static_cast<size_t>(xent_up(column * q.ld_a, 1024));
  q.off_sum = q.off_dz + static_cast<size_t>(xent_up(all < widest ? all : widest, 1024));
  const int64_t weights = sliced(4 * N * q.ld_sum);
  // One piece: dA's slices are added before dB's are made, in the same room.
  q.off_weights = q.off_sum + static_cast<size_t>(q.pieces == 1 ? 0 : xent_up(sums, 1024));
  q.bytes = q.off_weights + static_cast<size_t>(q.pieces == 1 && sums > weights ? sums : weights);
  return q;
}

}  // namespace tg
