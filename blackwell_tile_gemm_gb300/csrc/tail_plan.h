// Plan of the grouped kernel's last, partial wave: how many pieces its tiles'
// contractions are cut into, and where the pieces' partial sums lie in the
// stream's scratch.  Plain arithmetic without CUDA types, so that the kernel,
// its launch and host code that checks the bounds use the same.
#pragma once

#include <cstddef>
#include <cstdint>

#if defined(__CUDACC__)
#define TG_HD __host__ __device__ __forceinline__
#else
#define TG_HD inline
#endif

namespace tg {

// The scratch: f32 partial sums and the arrival counters.
constexpr size_t kTailPartialBytes = size_t{20} << 20;   // >= 152 slots of 128 KiB
constexpr int kTailFlagWords = 1024;

// Full waves of whole tiles, then the tiles of a last, partial wave in pieces
// of their contraction: the count (at most kTailMostPieces, each piece at least
// 4 stages) with the least waves * (stages per piece + join), against the whole
// tiles' stages + 2.  The join -- a piece's partial tile, its arrival, and the
// last piece's sum -- takes 14 stages (5 us) for single CTAs (with 0: 16 rows in
// 8 groups x 2048 x 2048 43 us instead of 14; without pieces: 4 rows x 4096 x
// 4096 24 us instead of 14); with the adapter term, where the tile's rows are
// known, 10 (3.7 us for 4 rows and 4 pieces) and the last piece's reads (7.8 us
// for 118 rows and 8); and 20 + 6 a piece for CTA pairs, whose partial tiles
// are 128 KB a CTA (wgrad of 22374 rows in 2 groups x 896 x 768 62 -> 40 us,
// 1444 rows x 1086 x 7085 40 -> 34 us).
struct GroupedPlan {
  int full;    // tiles run whole
  int S;       // pieces of the others
  int items;   // units of work
};
constexpr int kTailMostPieces = 8;

struct TailShape {
  int rest;         // tiles of the last wave
  int units;
  int k_blocks;     // stages of a contraction
  int cta_group;
  bool few_terms;   // few-row adapter product: its term is shared out too
  int rows, rank;   // of that form's tile
  int max_slots;    // partial tiles that fit (0: no scratch)
  int max_counters;
};

// A few-row tile's adapter term, which its pieces share out too, runs beside
// the contraction: about 6 stages' time for each 8 rows of a warp and 32 of
// the rank (39 rows x 1229 x 638, rank 128: 36 -> 28 us).
TG_HD int tail_work(const TailShape& s) {
  const int terms = s.few_terms ? (s.rows + 15) / 16 * ((s.rank + 31) / 32) * 6 : 0;
  return s.k_blocks > terms ? s.k_blocks : terms;
}
// The split has to stay below this (pieces have to gain a fifth).
TG_HD uint32_t tail_limit(const TailShape& s) {
  return static_cast<uint32_t>((tail_work(s) + 2) * 4 / 5);
}
// Cost of c pieces; 0xFFFFFFFF where they are not possible.
TG_HD uint32_t tail_cost(const TailShape& s, int c) {
  if (c < 2 || c > kTailMostPieces || s.rest <= 0 || s.k_blocks < (s.few_terms ? c : 4 * c) ||
      s.rest * c > s.max_slots || s.rest > s.max_counters)
    return 0xFFFFFFFFu;
  const int join = s.few_terms ? 10 + 3 * c * s.rows / 256 : s.cta_group == 1 ? 14 : 20 + 6 * c;
  return static_cast<uint32_t>((s.rest * c + s.units - 1) / s.units) *
         static_cast<uint32_t>((tail_work(s) + c - 1) / c + join);
}

// A slot: one CTA's partial tile, [column of the accumulator][width], the columns
// being rows of D and `width` the accumulator's 128 lanes.  Rank values (`down`)
// keep a tile of rank <= 128 in `rank` of them.
TG_HD int tail_slot_width(bool down, int wide) { return down && wide < 128 ? wide : 128; }
TG_HD int tail_max_slots(int tile_n, int cta_group, int width) {
  return static_cast<int>(kTailPartialBytes /
                          (static_cast<size_t>(tile_n) * cta_group * width * sizeof(float)));
}
TG_HD int tail_max_counters(int cta_group) { return kTailFlagWords / cta_group; }
// First value of column `col` of the slot of tile `tile` (counted from the first
// split one), piece `piece` of S and the CTA `cta` of its unit.
TG_HD int64_t tail_column(int tile, int piece, int S, int cta_group, int cta, int tile_n, int col,
                          int width) {
  return (((static_cast<int64_t>(tile) * S + piece) * cta_group + cta) * tile_n + col) * width;
}

}  // namespace tg
