// Products whose weights change with the row: one persistent, warp-specialised
// tcgen05 kernel for five of them, all bf16 with f32 accumulation.
//
//   kGroupedForward  D[i, :] = A[i, :] * B[g]^T      rows i of group g
//   kGroupedDgrad    dA[i, :] = G[i, :] * B[g]        (contraction over N)
//   kGroupedWgrad    dB[g] = G[rows of g]^T * A[rows of g]
//   kAdapter         D[i, :] = A[i, :] * B^T + H[i, :] * up[id_i]^T
//   kAdapterDown     H[i, :] = s * A[i, :] * down[id_i]^T
//
// Group g owns the rows offsets[g] <= i < offsets[g+1]; the offsets live on
// the device, so the host never learns the sizes and the tile list is made
// here (GroupWalk).
//
// Orientation.  The contiguous axis of D fills the MMA's M (the "wide" axis:
// N of the weights in the forward product, K in both gradients) and the other
// axis of D its N ("cols" below: the rows of a group, or N for the weight
// gradient).  The MMA's N is a runtime value in steps of 16 per CTA, so a
// group of 40 rows costs 48 or 64 columns, not a 128- or 256-row tile; and an
// accumulator row is a lane, so a warp that reads one accumulator column holds
// 32 consecutive elements of one row of D.  Single CTAs, and boxes that cross an
// edge, store them from registers (every ragged edge a predicate); CTA pairs
// stage whole boxes and write them with TMA.
//
// Operands in shared memory, 64 of the contraction index per stage, 128-byte
// rows, 128B swizzle:
//   K-major  [row][64 k]  (the contraction index is contiguous in memory),
//   MN-major [k][64 m]    (the other index is): boxes of 64 x 64, next 64
//            m at LBO = 8 KB, next 8 k at SBO = 1 KB, a K16 MMA step = 2 KB.
// The gradients need no transposed copy of anything: dgrad reads B[g]
// MN-major, wgrad both operands.
//
// Ragged contraction (wgrad): a group's last stage holds rows of the next
// group below its own.  0 * NaN is NaN, so both operands' rows past the
// group's end, up to the next multiple of 16 (fewer MMAs are issued instead
// of the rest), are overwritten with zeros by a fixing warp between the
// loads and the MMAs.
//
// Adapters: H[i] = scale * A[i] * down[id_i]^T was computed before and split
// into bf16 terms: two (17 bits) where D is rounded to bf16, three where D is
// f32 and the base product as exact as that (with two: 1.5e-6 of the term).
// After the tile's K stages each adapter that occurs among the tile's rows adds
// ceil(rank / 64) stages of up[id] and H for each term, into the same
// accumulator: D is written once.  Where all rows of the tile have one adapter,
// TMA's loads are all it takes (tiles start where a long run of rows with one
// adapter does: there the offsets are those of the runs), unless up[id] holds
// infinite or NaN weights: times a later term of H, which is zero or of either
// sign, they would turn an infinite sum into NaN, so the fixing warps take them
// out for the terms after the first.  (Whether it does they find out in memory
// while the tile's K stages run: 8000 rows, rank 64, x 8192 x 4096 423 us, with
// no look at the weights 420, with every such stage gone over in shared memory
// 455.)
// In other tiles the fixing warps put zeros over H's rows of other adapters.  A
// zero row times an infinite or NaN weight would still be NaN, so there they
// take such weights out for the first term too and mark the tile; the epilogue
// of a marked tile adds what they give in the rows they belong to.  A mixed
// stage takes about 0.65 us, a plain one 0.34 (551 rows of 50 requests, rank 128,
// x 6463 x 6084: 134 us).
//
// Few rows (kSplit, single CTAs): the product is bound by reading the
// weights, tiles are few, so S units share a tile's contraction; each writes
// an f32 partial and the one that arrives last adds them in piece order (the
// same bits every time; nobody waits).  There the adapter term stays out of
// the pipeline: the epilogue's warps compute it while the weights stream in.
//
// Roles: warp 0 TMA producer, warp 1 TMEM allocator and MMA issuer, warps 2
// and 3 fixing warps (gradients: 3 the second producer), warps 4..11 epilogue.
// Every wait is bounded.
//
// Bounds, measured on groups of equal size, weights of 2048 x 4096, bf16 D: 16
// groups of 2048 rows 310 us forward and dgrad, 319 wgrad (1770, 1770 and 1720
// TFLOP/s: the tensor pipe); 64 groups of 512 rows 342, 344 and 417 us: a tile
// takes in 64 KB and the weights' 1 GB of HBM traffic shares the time with the
// MMAs; f32 D 384 and 613 (wgrad) us: stores and loads take turns (32 groups of
// 1024 rows: tensor pipe 43%, DRAM 33%, L2 34%).  64 groups of 32 rows 174 us:
// 1.07 GB at 6.2 TB/s.  The walk over the offsets at the start: 512 rows in one of
// 64 groups of 128 x 128 6.6 us, of 1024 25, of 4096 87.
#pragma once

#include <cstdint>
#include <type_traits>
#include <cuda.h>

#include "epilogue.cuh"
#include "grouped_ptx.cuh"
#include "tail_plan.h"

namespace tg {

enum : int { kGroupedForward = 0, kGroupedDgrad = 1, kGroupedWgrad = 2, kAdapter = 3, kAdapterDown = 4 };

enum : uint32_t {
  kSiteGrEmpty = 31,
  kSiteGrFull = 32,
  kSiteGrFix = 33,
  kSiteGrAccEmpty = 34,
  kSiteGrAccFull = 35,
  kSiteGrFixIn = 36,
  kSiteGrOffsets = 40,   // not a wait: the offsets decrease or leave [0, M]
};

struct GroupedArgs {
  int M;               // rows of all groups together (extent of the offsets)
  int wide;            // extent of D's contiguous axis
  int cols;            // wgrad: rows of one group's D; else unused
  int num_wide_tiles;  // tiles of kCtaGroup * 128
  int num_col_tiles;   // wgrad: tiles of kTileN over cols
  int num_k_blocks;    // stages of 64 of the contraction index (wgrad: of an
                       // average group, for the choice of pieces only)
  int groups;
  const int* offsets;  // [groups + 1], or null: one group of all M rows
  void* D;
  int64_t ldd;
  int64_t group_stride_d;  // wgrad
  // kAdd
  int even;                // rows of a group: all but the last have as many
  int add;                 // dgrad: D += instead of D =
  int tile_cols;           // dgrad: most columns of a tile (a multiple of 32, at most kTileN)
  int slice;               // dgrad: contraction indices of a group (a multiple of 64) ...
  int second;              // ... after which follow as many of a second term: the column
                           // operand's, `second` columns behind the first, against the
                           // wide operand's rows again
  Epi epi;                 // bias: [groups][wide]
  // adapters
  const int* ids;          // [M]
  int adapters, rank;
  const int* row_idx;      // few rows forward, or null: row i is row row_idx[i] of the
  int num_rows;            // column operand's num_rows
  uint16_t* h;             // [M][h_terms][rank] bf16: each row of H as a sum of terms, which
  int h_terms;             // kAdapterDown writes: 2, or 3 where D is f32
  const float* scales;     // kAdapterDown: [adapters], or null for 1
  int wide_box;            // kAdapterDown: rows of `down` per load (the lanes
                           // above them hold leftovers and are not stored)
  const uint16_t* up;
  int64_t ld_up, group_stride_up;
  // split contraction
  int max_slots;           // partial tiles that fit (0: never split)
  int max_counters;
  float* partials;         // [tile][piece][CTA of pair][kTileN][128] f32 (tail_plan.h)
  uint32_t* counters;      // [tile][CTA of pair], 0 between launches
  uint32_t* status;
  uint64_t timeout_ns;
};

// Column-operand boxes of a quarter, half, three quarters and the whole of a
// CTA's rows of the operand: a stage's rows come in one load of the next size.
// A stage issues as few loads as it can: with 112 rows as boxes of 64 + 32 +
// 16 the producer, not the MMAs, set the pace (64 groups of 448 rows x 2048 x
// 4096: 493 us, against 357 us for 512 rows in single boxes).
// wgrad: box[0] is the 64 x 64 box of the MN-major operand, box[1] the pair
// of such boxes in one load.
constexpr int kColBoxes = 4;
struct ColumnMaps {
  CUtensorMap box[kColBoxes];
  CUtensorMap h[4];   // adapters: H's terms and, last, all of them; boxes of 128 rows
};

template <int kMode_, int kCtaGroup_, int kTileN_, int kStages_, bool kBf16Out_,
          bool kTail_ = kCtaGroup_ == 1, int kAdd_ = 0>
struct GroupedCfg {
  static constexpr int kMode = kMode_;
  static constexpr int kCtaGroup = kCtaGroup_;
  static constexpr int kTileN = kTileN_;          // most MMA columns of a tile
  static constexpr int kStages = kStages_;
  static constexpr bool kBf16Out = kBf16Out_;
  static constexpr bool kWideMn = kMode == kGroupedDgrad || kMode == kGroupedWgrad;
  static constexpr bool kColMn = kMode == kGroupedWgrad;
  static constexpr bool kSplit = kCtaGroup == 1;
  static constexpr bool kGather = kMode == kGroupedForward && kSplit;   // row_idx is read here
  // Whether a last wave may be cut into pieces (grouped_plan).  Pairs carry the
  // join only where it can pay: it costs the others registers and up to 8%
  // (wgrad of 16 groups x 2048 x 4096 with 128 rows each: 56 -> 60 us).
  static constexpr bool kTail = kTail_;
  // Adapter stages (MMA form) and ragged contractions are fixed up in shared
  // memory before the MMAs read them.
  static constexpr bool kExt = kMode == kAdapter && kCtaGroup == 2;
  // A contraction in slices (f32 D of CTA pairs), each the group of an equal share
  // (GroupedArgs::even, slice) with a D of its own.  Dgrad: of one operand's columns
  // and the other's rows; GroupedArgs::add adds the tile to D instead of writing it,
  // for contractions given one after the other.  1: sums that a rounding to bf16
  // follows, one accumulator each; 2: sums that stay f32, in chunks.  Wgrad (3): of
  // the rows.
  static constexpr int kAdd = kAdd_;
  static constexpr int kTerms = kBf16Out ? 2 : 3;   // bf16 terms of H
  static constexpr int kFixWarps = kExt ? 2 : kMode == kGroupedWgrad ? 1 : 0;
  static constexpr int kColStep = 16 * kCtaGroup;
  static constexpr int C_ROWS = kTileN / kCtaGroup;   // column-operand rows per CTA
  static constexpr int kBoxStep = C_ROWS / kColBoxes;
  static constexpr int W_BYTES = 128 * 128;
  static constexpr int C_BYTES = C_ROWS * 128;
  static constexpr int OFF_W = 0;
  static constexpr int OFF_C = OFF_W + kStages * W_BYTES;
  // CTA pairs store D by TMA from staged boxes of 32 rows x 128 bytes (bf16:
  // two warps fill one box); blocks that cross a group's end or D's right
  // edge are read back from the box and stored row by row.  wgrad of 64
  // groups x 2048 x 4096 with 64 rows each, i.e. the writing of 1.07 GB:
  // 515 us straight from registers (64 bytes a row and instruction), 312 us
  // with every box read back, 266 us with TMA boxes of 64 bytes.
  static constexpr bool kStaged = kCtaGroup == 2;
  static constexpr int OFF_STG = OFF_C + kStages * C_BYTES;
  static constexpr int OFF_BAR = OFF_STG + (kStaged ? 8 * 4096 : 0);
  static constexpr int kAccBufs = 2;
  // f32 D: the tensor cores truncate each time they add to an accumulator, so
  // its error grows with the number of K16 steps (measured 1e-6 of the result
  // after 1000 terms, 5e-6 after 5000).  Long contractions are therefore cut
  // into chunks of at most kChunk stages that are added in f32 with rounding
  // to nearest: each epilogue warp keeps its share of the tile (128 values a
  // lane) in registers.  (Adding the chunks to D in memory instead cost 80%:
  // 8192^3 wgrad 1579 us.)  bf16 D rounds at 2e-3 and needs none of it.  (kAdapterDown:
  // by the D that H is for, whose terms keep what the sums have.)
  static constexpr int kChunk = kAdd == 1 ? 1 << 30 : 12;
  static constexpr int NUM_BARS = 2 * kStages + 2 * kAccBufs + 1 + (kFixWarps ? 2 * kStages : 0) +
                                  (kExt ? 2 : 0);
  static constexpr int OFF_MISC = OFF_BAR + NUM_BARS * 8;
  static constexpr int SMEM_BYTES = OFF_MISC + 32 + (kExt ? 72 : 0) + 1024;
  static constexpr int TMEM_COLS = 2 * kTileN <= 32    ? 32
                                   : 2 * kTileN <= 64  ? 64
                                   : 2 * kTileN <= 128 ? 128
                                   : 2 * kTileN <= 256 ? 256
                                                       : 512;
  static constexpr int kEpiWarps = 8;
  static constexpr int kFixWarp0 = 2;
  static constexpr int kEpiWarp0 = 4;
  // The gradients' operands take two loads each (boxes of 64 x 64).
  static constexpr bool kTwoProducers = kWideMn && kCtaGroup == 2;
  static constexpr int kColWarp = 3;
  static_assert(!kTwoProducers || kFixWarps < 2, "warp 3 is free");
  static constexpr int kThreads = 32 * (kEpiWarp0 + kEpiWarps);
  static_assert(SMEM_BYTES <= 227 * 1024, "shared memory per CTA");
  static_assert(kTileN % 32 == 0 && kTileN <= 256, "MMA N");
  static_assert(C_BYTES % 1024 == 0, "swizzle atoms");
  static_assert(!kColMn || (kCtaGroup == 2 && kTileN == 256), "wgrad tiles");
  static_assert(!kWideMn || kCtaGroup == 2, "the gradients run as CTA pairs");
  static_assert(!kAdd || (kCtaGroup == 2 && !kBf16Out && kColMn == (kAdd == 3)), "slices are f32");
};

// One work item.
struct GroupedWork {
  int g;
  int wide0;    // first element of D's contiguous axis
  int row0;     // first row of D (wgrad: inside the group's D)
  int rows;     // rows of D this tile stores
  int ncols;    // MMA columns (rows rounded up)
  int nk;       // K stages of this unit
  int k0, ks;   // first stage, step
  int base;     // wgrad: first row of the contraction
  int len;      // wgrad: its length
  int tile;     // tile index (split scratch)
  int piece;
};

static __device__ __noinline__ int large_div(int a, int b) { return a / b; }
// a / b for a >= 0, b > 0: the float quotient of numbers below 2^22 is off by
// less than one.  (A call for the others: inlined, they made every use longer
// than the division it replaces.)
__device__ __forceinline__ int small_div(int a, int b) {
  if (a >= 1 << 22) return large_div(a, b);
  int q = __float2int_rd(__fdividef(static_cast<float>(a), static_cast<float>(b)));
  const int r = a - q * b;
  if (r < 0) --q;
  if (r >= b) ++q;
  return q;
}

__device__ __forceinline__ int grouped_clamp(int v, int hi) { return min(max(v, 0), hi); }

// Tile index -> group, by one warp.  The lanes hold the row ranges of 32
// consecutive groups and the running sum of their tiles; tile indices only
// grow, so the window only moves forwards.  Offsets outside [0, M] are
// clamped and decreasing ones raised to the running maximum: whatever the
// device holds, the ranges are disjoint and inside the arrays.
template <class C>
struct GroupWalk {
  int g0, t0, lo0;   // window: first group, tiles and first row before it
  int lo, hi, incl;  // this lane's group: rows [lo, hi), tiles up to and with it
  bool bad;
  // The group found last: its tiles [begin, end), rows [r0, r1), column tiles.
  int begin, end, r0, r1, group, nct, size;

  static __device__ __forceinline__ int tile_cols(const GroupedArgs& p) {
    return C::kAdd && !C::kColMn ? p.tile_cols : C::kTileN;
  }
  __device__ __forceinline__ void load(const GroupedArgs& p, int lane) {
    const int g = g0 + lane;
    int end = lo0;
    if constexpr (C::kAdd) {
      if (g < p.groups) {
        const int64_t all = static_cast<int64_t>(g + 1) * p.even;
        end = all < p.M ? static_cast<int>(all) : p.M;
      }
    } else if (p.offsets == nullptr) {
      end = g0 == 0 ? p.M : lo0;
    } else if (g < p.groups) {
      const int raw = p.offsets[g + 1];
      end = grouped_clamp(raw, p.M);
      bad |= raw != end;
    }
    const int own = end;
#pragma unroll
    for (int d = 1; d < 32; d *= 2) {
      const int o = __shfl_up_sync(0xFFFFFFFFu, end, d);
      if (lane >= d) end = max(end, o);
    }
    end = max(end, lo0);
    if (g < p.groups) bad |= end != own;
    hi = end;
    lo = __shfl_up_sync(0xFFFFFFFFu, end, 1);
    if (lane == 0) lo = lo0;
    int tiles = 0;
    if constexpr (C::kColMn) {
      if (g < p.groups) tiles = p.num_wide_tiles * p.num_col_tiles;
    } else {
      tiles = (hi - lo + tile_cols(p) - 1) / tile_cols(p) * p.num_wide_tiles;
    }
    incl = tiles;
#pragma unroll
    for (int d = 1; d < 32; d *= 2) {
      const int o = __shfl_up_sync(0xFFFFFFFFu, incl, d);
      if (lane >= d) incl += o;
    }
  }
  __device__ __forceinline__ void start(const GroupedArgs& p, int lane) {
    g0 = 0;
    t0 = 0;
    begin = end = 0;
    bad = false;
    lo0 = 0;
    if (p.offsets != nullptr) {
      const int raw = p.offsets[0];
      lo0 = grouped_clamp(raw, p.M);
      bad = raw != lo0;
    }
    load(p, lane);
  }
  __device__ __forceinline__ void advance(const GroupedArgs& p, int lane) {
    t0 += __shfl_sync(0xFFFFFFFFu, incl, 31);
    lo0 = __shfl_sync(0xFFFFFFFFu, hi, 31);
    g0 += 32;
    load(p, lane);
  }
  // Tiles of every group; first and end row of all groups.  Leaves the walk
  // at its start.
  __device__ __forceinline__ int total(const GroupedArgs& p, int lane, int* first, int* end) {
    start(p, lane);
    *first = lo0;
    while (g0 + 32 < p.groups) advance(p, lane);
    const int t = t0 + __shfl_sync(0xFFFFFFFFu, incl, 31);
    *end = __shfl_sync(0xFFFFFFFFu, hi, 31);
    if (g0 != 0) {
      const bool b = bad;
      start(p, lane);
      bad = b;
    }
    return t;
  }
  // The group that holds tile t (< total, not below the last one asked for).
  __device__ __forceinline__ void seek(const GroupedArgs& p, int lane, int t) {
    while (t >= t0 + __shfl_sync(0xFFFFFFFFu, incl, 31) && g0 + 32 < p.groups) advance(p, lane);
    const uint32_t above = __ballot_sync(0xFFFFFFFFu, t0 + incl > t);
    const int src = above ? __ffs(above) - 1 : 31;
    r0 = __shfl_sync(0xFFFFFFFFu, lo, src);
    r1 = __shfl_sync(0xFFFFFFFFu, hi, src);
    const int before = __shfl_sync(0xFFFFFFFFu, incl, src > 0 ? src - 1 : 0);
    begin = t0 + (src > 0 ? before : 0);
    end = t0 + __shfl_sync(0xFFFFFFFFu, incl, src);
    group = C::kMode == kAdapter ? 0 : g0 + src;   // (adapters: one shared operand)
    nct = C::kColMn ? p.num_col_tiles : (r1 - r0 + tile_cols(p) - 1) / tile_cols(p);
    // The group's rows in nct tiles of equal size (a multiple of kColStep).
    size = C::kMode == kAdapterDown || C::kColMn
               ? C::kTileN
               : (small_div(r1 - r0 + nct - 1, max(nct, 1)) + C::kColStep - 1) / C::kColStep *
                     C::kColStep;
  }
  __device__ __forceinline__ void find(const GroupedArgs& p, int lane, int t, int piece, int S,
                                       GroupedWork& w) {
    // Most tiles are in the last one's group: every role's warp asks for
    // every tile, and a short tile waits for the answer.
    if (t >= end || t < begin) seek(p, lane, t);
    const int l = t - begin;
    w.g = group;
    w.tile = t;
    w.piece = piece;
    // Tiles of a group: bands of 16 column tiles, within a band the column
    // tile fastest, so that the units running at the same time share a
    // weight panel and the band's rows stay in L2.
    int first = 0, gm = nct, r = l;
    if (nct > 16) {
      first = l / (16 * p.num_wide_tiles) * 16;
      gm = min(nct - first, 16);
      r = l - first * p.num_wide_tiles;
    }
    const int wt = small_div(r, gm);
    const int ct = first + r - wt * gm;
    w.wide0 = wt * (128 * C::kCtaGroup);
    if constexpr (C::kColMn) {
      w.row0 = ct * C::kTileN;
      w.rows = min(C::kTileN, p.cols - w.row0);
      w.ncols = w.rows <= 128 ? 128 : 256;
      w.base = r0;
      w.len = r1 - r0;
      // (0 for more pieces than stages)
      w.nk = small_div((w.len + 63) / 64 - piece + S - 1, S);
      w.k0 = piece;
      w.ks = S;
    } else {
      w.row0 = r0 + ct * size;
      w.rows = min(size, r1 - w.row0);
      w.ncols = (w.rows + C::kColStep - 1) / C::kColStep * C::kColStep;
      // Piece q of S takes stages q, q + S, ...: at any moment the pieces of
      // a tile read neighbouring 128-byte chunks of the same rows.
      w.k0 = piece;
      w.ks = S;
      w.nk = small_div(p.num_k_blocks - piece + S - 1, S);
      w.base = 0;
      w.len = 0;
    }
  }
};

// Chunks of a contraction of nk stages (0 for none), and where chunk c ends.
template <class C>
__device__ __forceinline__ int grouped_chunks(int nk) {
  if constexpr (C::kBf16Out) return nk > 0 ? 1 : 0;
  return (nk + C::kChunk - 1) / C::kChunk;
}
template <class C>
__device__ __forceinline__ int grouped_chunk_end(int nk, int chunks, int c) {
  if constexpr (C::kBf16Out) return nk;
  return static_cast<int>(static_cast<int64_t>(nk) * (c + 1) / chunks);
}

// Lane c weighs c pieces: one after the other, the divisions took 1.2 us before
// the first load (4 rows x 4096 x 4096, rank 16: the call 14.6 -> 14.0 us; 118
// rows x 667 x 735, rank 8, with fewer pieces too: 19.4 -> 18.0).
template <class C>
__device__ __forceinline__ GroupedPlan grouped_plan(const GroupedArgs& p, int tiles, int units,
                                                    int lane) {
  GroupedPlan g{tiles, 1, tiles};
  if constexpr (!C::kTail) return g;
  const int full = small_div(tiles, units) * units;
  const TailShape shape{tiles - full,
                        units,
                        p.num_k_blocks,
                        C::kCtaGroup,
                        C::kMode == kAdapter && C::kSplit,
                        min(p.M, C::kTileN),
                        p.rank,
                        p.max_slots,
                        p.max_counters};
  const uint32_t cost = tail_cost(shape, lane);
  const uint32_t least = __reduce_min_sync(0xFFFFFFFFu, cost);
  if (least < tail_limit(shape)) {
    const int S = __ffs(__ballot_sync(0xFFFFFFFFu, cost == least)) - 1;
    g = GroupedPlan{full, S, full + shape.rest * S};
  }
  return g;
}

// Warp-level MMA, 16 x 8 x 16, bf16 with f32 accumulation: a0, a1: rows
// lane / 4 and + 8 at k = 2 (lane % 4); a2, a3: the same at k + 8; b0, b1:
// column lane / 4; c: rows lane / 4 and + 8, columns 2 (lane % 4) and + 1.
__device__ __forceinline__ void mma_m16n8k16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                             uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// The smallest adapter above `last` among the ids of a tile's rows (each lane
// holds kTileN / 32 of them), or -1.  Rows without an adapter hold ids that
// compare as at least `adapters`.
template <int kPer>
__device__ __forceinline__ int next_adapter(const uint32_t (&ids)[kPer], int last,
                                            uint32_t adapters) {
  uint32_t m = adapters;
#pragma unroll
  for (int i = 0; i < kPer; ++i)
    if (static_cast<int>(min(ids[i], 0x7FFFFFFFu)) > last) m = min(m, ids[i]);
  m = __reduce_min_sync(0xFFFFFFFFu, m);
  return m < adapters ? static_cast<int>(m) : -1;
}

template <class C>
__device__ __forceinline__ void load_tile_ids(const GroupedArgs& p, const GroupedWork& w, int lane,
                                              uint32_t (&ids)[C::kTileN / 32]) {
#pragma unroll
  for (int i = 0; i < C::kTileN / 32; ++i) {
    const int r = lane + 32 * i;
    ids[i] = r < w.rows ? static_cast<uint32_t>(p.ids[w.row0 + r]) : 0xFFFFFFFFu;
  }
}

// Whether the tile's rows differ in their adapter (or some have none).
template <int kPer>
__device__ __forceinline__ bool mixed_adapters(const uint32_t (&ids)[kPer], int rows, int lane,
                                               uint32_t adapters) {
  uint32_t lo = 0xFFFFFFFFu, hi = 0u;
#pragma unroll
  for (int i = 0; i < kPer; ++i)
    if (lane + 32 * i < rows) {
      lo = min(lo, min(ids[i], adapters));
      hi = max(hi, min(ids[i], adapters));
    }
  return __reduce_min_sync(0xFFFFFFFFu, lo) != __reduce_max_sync(0xFFFFFFFFu, hi);
}

// kAdapterDown leaves tiles of more than kDownAdapters adapters to
// lora_down_kernel, which spreads them over more blocks: here they would run
// one after the other.
constexpr int kDownAdapters = 2;
template <int kPer>
__device__ __forceinline__ bool few_adapters(const uint32_t (&ids)[kPer], uint32_t adapters) {
  int id = -1;
  for (int n = 0; n <= kDownAdapters; ++n) {
    id = next_adapter(ids, id, adapters);
    if (id < 0) return true;
  }
  return false;
}

// Where the rank leaves room in the 128 lanes, one pass over a tile's rows does
// several of its adapters: slots of 32, 64 or 128 lanes, one adapter each.
__device__ __forceinline__ int down_slot(int rank) { return rank <= 32 ? 32 : rank <= 64 ? 64 : 128; }
// The pass's adapters: up to 128 / slot of them, -1 where there are no more;
// `last` moves on to the last one taken.
template <int kPer>
__device__ __forceinline__ int next_adapters(const uint32_t (&ids)[kPer], int& last, int most,
                                             uint32_t adapters, int (&out)[4]) {
  int n = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    out[i] = i < most && (i == 0 || out[i > 0 ? i - 1 : 0] >= 0) ? next_adapter(ids, last, adapters)
                                                                 : -1;
    if (out[i] >= 0) {
      last = out[i];
      ++n;
    }
  }
  return n;
}

// x as a sum of bf16 terms, `step` apart; what is infinite or NaN in the first
// is in the first alone.  (Finite values that would round to infinity take the
// largest finite term first.)
__device__ __forceinline__ void split_bf16(float x, uint16_t* h, int step, int terms) {
  uint32_t w = pack_bf16x2(x, x) & 0xFFFFu;
  if ((w & 0x7FFFu) == 0x7F80u && fabsf(x) < __uint_as_float(0x7F800000u)) --w;
  h[0] = static_cast<uint16_t>(w);
  for (int t = 1; t < terms; ++t) {
    const float rest = x - __uint_as_float(w << 16);
    x = fabsf(rest) < __uint_as_float(0x7F800000u) ? rest : 0.0f;
    w = pack_bf16x2(x, x) & 0xFFFFu;
    h[t * step] = static_cast<uint16_t>(w);
  }
}

// Adapter stages of 64 columns: columns 0.., 64.., ... of up[id] against H's
// first term, then the same against each other.  In a mixed tile, whose stages
// the fixing warps go over anyway, terms that fit into 64 columns together
// take one stage: next to each other, as they lie in memory, and up[id] as
// often.
template <int kTerms>
__device__ __forceinline__ bool adapter_packed(int rank, bool mixed) {
  return mixed && kTerms * rank <= 64;
}
template <int kTerms>
__device__ __forceinline__ int adapter_stages(int rank, bool mixed) {
  return adapter_packed<kTerms>(rank, mixed) ? 1 : kTerms * ((rank + 63) / 64);
}

// A word of two bf16 values without its infinite and NaN ones.
__device__ __forceinline__ uint32_t finite_bf16x2(uint32_t w) {
  if ((w & 0x7F800000u) == 0x7F800000u) w &= 0x0000FFFFu;
  if ((w & 0x00007F80u) == 0x00007F80u) w &= 0xFFFF0000u;
  return w;
}

// w * 0 + z on two bf16 values: z stays zero (of either sign) as long as every
// w is finite, and is NaN from the first that is not.
__device__ __forceinline__ uint32_t times_zero_bf16x2(uint32_t w, uint32_t z) {
  uint32_t d;
  asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(d) : "r"(w), "r"(0u), "r"(z));
  return d;
}

// Whether rows x0 .. x0 + 127 and columns r .. r + 63 of up[id] hold finite
// weights only.  By one warp: 4 rows of 8 16-byte pieces a step.
__device__ __forceinline__ bool finite_box(const GroupedArgs& p, int id, int x0, int r, int lane) {
  const int col = r + 8 * (lane & 7);
  uint32_t z[4] = {0u, 0u, 0u, 0u};
  if (col < p.rank) {
    const uint16_t* u = p.up + id * p.group_stride_up + col;
    const int rows = min(128, p.wide - x0);
#pragma unroll 1
    for (int i0 = lane >> 3; i0 < rows; i0 += 32) {
      uint4 v[8];
#pragma unroll
      for (int i = 0; i < 8; ++i)   // (past the last row: that again)
        v[i] = ld_global_nc_v4(u + static_cast<int64_t>(x0 + min(i0 + 4 * i, rows - 1)) * p.ld_up);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        z[0] = times_zero_bf16x2(v[i].x, z[0]);
        z[1] = times_zero_bf16x2(v[i].y, z[1]);
        z[2] = times_zero_bf16x2(v[i].z, z[2]);
        z[3] = times_zero_bf16x2(v[i].w, z[3]);
      }
    }
  }
  return !__any_sync(0xFFFFFFFFu, ((z[0] | z[1] | z[2] | z[3]) & 0x7FFF7FFFu) != 0u);
}

// epi(v) on the accumulators of one lane, whose column of D has bias b.
template <int kN>
__device__ __forceinline__ void grouped_epilogue(const Epi& e, float b, float (&v)[kN]) {
  if (e.op == kEpiNone) return;
  if (e.op == kEpiAddScalar || e.op == kEpiBiasCol) {
    const float a = e.op == kEpiAddScalar ? e.alpha : b;
#pragma unroll
    for (int i = 0; i < kN; ++i) v[i] += a;
  } else if (e.op == kEpiAffine) {
#pragma unroll
    for (int i = 0; i < kN; ++i) v[i] = v[i] * e.alpha + e.beta;
  } else if (e.op == kEpiSiluAffine) {
#pragma unroll
    for (int i = 0; i < kN; ++i) v[i] = silu_f32(v[i]) * e.alpha + e.beta;
  } else {
#pragma unroll
    for (int i = 0; i < kN; ++i) v[i] = silu_f32(v[i] + b);
  }
}

// Stores 32 accumulator columns (rows row .. row + 31 of D, those below
// `end`) of one warp; this lane holds element x of each.  f32: one 128-byte
// store a row.  bf16: lanes pair up and exchange one value for two rows, so
// that a store writes 64 contiguous bytes in each of two rows.
template <class C>
__device__ __forceinline__ void grouped_store(const GroupedArgs& p, int64_t d0, int row, int end,
                                              int x, const float (&v)[32]) {
  if constexpr (!C::kBf16Out) {
    if (x >= p.wide) return;
    float* d = reinterpret_cast<float*>(p.D) + d0 + row * p.ldd + x;
    if (row + 32 <= end) {
#pragma unroll
      for (int j = 0; j < 32; ++j) __stcs(d + j * p.ldd, v[j]);
    } else {
#pragma unroll
      for (int j = 0; j < 32; ++j)
        if (row + j < end) __stcs(d + j * p.ldd, v[j]);
    }
  } else {
    const int odd = x & 1;
    const int xe = x - odd;
    uint16_t* d = reinterpret_cast<uint16_t*>(p.D) + d0 + (row + odd) * p.ldd + xe;
    const bool both = xe + 1 < p.wide;
#pragma unroll
    for (int j = 0; j < 32; j += 2) {
      const float give = odd ? v[j] : v[j + 1];
      const float got = __shfl_xor_sync(0xFFFFFFFFu, give, 1);
      const uint32_t w = odd ? pack_bf16x2(got, v[j + 1]) : pack_bf16x2(v[j], got);
      if (xe < p.wide && row + j + odd < end) {
        uint16_t* q = d + j * p.ldd;
        if (both)
          __stcs(reinterpret_cast<uint32_t*>(q), w);
        else
          *q = static_cast<uint16_t>(w & 0xFFFFu);
      }
    }
  }
}

// 32 accumulator columns of this lane's row, into v or added to it.
template <bool kAdd>
__device__ __forceinline__ void grouped_read(uint32_t taddr, float (&v)[32]) {
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    uint32_t raw[16];
    tmem_ld_32x32b_x16(taddr + 16 * h, raw);
    tmem_ld_wait();
#pragma unroll
    for (int i = 0; i < 16; ++i)
      v[16 * h + i] = kAdd ? v[16 * h + i] + __uint_as_float(raw[i]) : __uint_as_float(raw[i]);
  }
}
__device__ __forceinline__ void grouped_zero(float (&v)[32]) {
#pragma unroll
  for (int i = 0; i < 32; ++i) v[i] = 0.0f;
}

// f32: the warp's 32 x 32 block into its staging box, one 128-byte line per
// row of D.
__device__ __forceinline__ void grouped_stage_f32(uint32_t stg, int lane, const float (&v)[32]) {
#pragma unroll
  for (int j = 0; j < 32; ++j) st_shared_b32(stg + 128 * j + 4 * lane, __float_as_uint(v[j]));
}

// bf16: the warp's 32 lanes x 32 accumulator columns at `taddr` (or zeros)
// into its half of a staging box of 32 rows x 128 bytes that it shares with
// the warp of the neighbouring 32 lanes.  The 16x256b read leaves two
// neighbouring columns of a lane in one thread, in the fragment layout of
// stmatrix, whose .trans form writes the transposed 8 x 8 blocks: rows of D.
// 128B swizzle (16-byte piece c of row r at c ^ (r & 7)) keeps that free of
// bank conflicts.  b[i]: bias of lane 8 i + (thread / 4).
__device__ __forceinline__ void grouped_stage_bf16(uint32_t stg, int lane, int slab, uint32_t taddr,
                                                   bool any, const Epi& e, const float (&b)[4]) {
  uint32_t v[2][16];
  if (any) {
    tmem_ld_16x256b_x4(taddr, v[0]);
    tmem_ld_16x256b_x4(taddr + (16u << 16), v[1]);
    tmem_ld_wait();
  } else {
#pragma unroll
    for (int i = 0; i < 16; ++i) v[0][i] = v[1][i] = 0u;
  }
  if (e.op != kEpiNone) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float t[8];
#pragma unroll
      for (int j = 0; j < 8; ++j)
        t[j] = __uint_as_float(v[i / 2][4 * (j / 2) + 2 * (i & 1) + (j & 1)]);
      grouped_epilogue(e, b[i], t);
#pragma unroll
      for (int j = 0; j < 8; ++j)
        v[i / 2][4 * (j / 2) + 2 * (i & 1) + (j & 1)] = __float_as_uint(t[j]);
    }
  }
  const uint32_t r = static_cast<uint32_t>(lane & 7);
  const uint32_t c = static_cast<uint32_t>(4 * (slab & 1) + (lane >> 3));
  const uint32_t a = stg + 128 * r + 16 * (c ^ r);
#pragma unroll
  for (int g = 0; g < 4; ++g) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      w[i] = pack_bf16x2(__uint_as_float(v[i / 2][4 * g + 2 * (i & 1)]),
                         __uint_as_float(v[i / 2][4 * g + 2 * (i & 1) + 1]));
    stmatrix_x4_trans(a + 1024 * g, w[0], w[1], w[2], w[3]);
  }
}

// Rows r0, r0 + step, ... of a staged box to D (element x0 of rows row ..,
// below `end`): eight lanes write one 128-byte line, four rows at a time.
template <class C>
__device__ __forceinline__ void grouped_unstage(const GroupedArgs& p, int64_t d0, uint32_t stg,
                                                int lane, int r0, int r1, int row, int end,
                                                int x0) {
  constexpr int kVec = C::kBf16Out ? 8 : 4;
  const int x = x0 + kVec * (lane & 7);
  using T = typename std::conditional<C::kBf16Out, uint16_t, float>::type;
#pragma unroll 4
  for (int r = r0 + (lane >> 3); r < r1; r += 4) {
    if (row + r >= end) break;
    const int c = C::kBf16Out ? (lane ^ r) & 7 : lane & 7;   // bf16 boxes are swizzled
    const uint4 q = ld_shared_v4(stg + 128 * r + 16 * c);
    T* d = reinterpret_cast<T*>(p.D) + d0 + (row + r) * p.ldd + x;
    if constexpr (C::kAdd) {
      if (p.add) {
        const float v[4] = {__uint_as_float(q.x), __uint_as_float(q.y), __uint_as_float(q.z),
                            __uint_as_float(q.w)};
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (x + e < p.wide) d[e] += v[e];
        continue;
      }
    }
    if (x + kVec <= p.wide) {
      __stcs(reinterpret_cast<uint4*>(d), q);
    } else {
      const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
      for (int e = 0; e < kVec; ++e)
        if (x + e < p.wide) {
          if constexpr (C::kBf16Out)
            d[e] = static_cast<uint16_t>(w[e / 2] >> (16 * (e & 1)));
          else
            d[e] = __uint_as_float(w[e]);
        }
    }
  }
}

// Rows of D in no group: [0, first) and [end, M) are set to zero, shared out
// over the epilogue warps of the grid.
template <class C>
__device__ __forceinline__ void grouped_zero_rows(const GroupedArgs& p, int first, int end,
                                                  int warp_id, int num_warps, int lane) {
  const int count = first + (p.M - end);
  constexpr int kEsize = C::kBf16Out ? 2 : 4;
  constexpr int kVec = 16 / kEsize;
  for (int i = warp_id; i < count; i += num_warps) {
    const int row = i < first ? i : end + (i - first);
    uint8_t* d = reinterpret_cast<uint8_t*>(p.D) + static_cast<int64_t>(row) * p.ldd * kEsize;
    const int nv = p.wide / kVec;
    for (int c = lane; c < nv; c += 32) st_global_v4(d + 16 * c, 0u, 0u, 0u, 0u);
    for (int c = nv * kVec + lane; c < p.wide; c += 32) {
      if constexpr (C::kBf16Out)
        reinterpret_cast<uint16_t*>(d)[c] = 0;
      else
        reinterpret_cast<float*>(d)[c] = 0.0f;
    }
  }
}

// up[id][x, r] * H[row, r], summed over the rank values r in [from, to): all, or
// those of infinite and NaN weights.
__device__ __forceinline__ float scalar_term(const GroupedArgs& p, uint32_t id, int row, int x,
                                             int from, int to, bool all) {
  float s = 0.0f;
  const uint16_t* u = p.up + id * p.group_stride_up + static_cast<int64_t>(x) * p.ld_up;
  const uint16_t* h = p.h + static_cast<int64_t>(row) * (p.h_terms * p.rank);
  for (int r = from; r < to; ++r)
    if (all || (u[r] & 0x7F80u) == 0x7F80u) {
      float sum = __uint_as_float(static_cast<uint32_t>(h[r]) << 16);
      for (int t = 1; t < p.h_terms; ++t)
        sum += __uint_as_float(static_cast<uint32_t>(h[t * p.rank + r]) << 16);
      s += __uint_as_float(static_cast<uint32_t>(u[r]) << 16) * sum;
    }
  return s;
}
// What the infinite and NaN weights of up[id] that were taken out of a marked
// tile give in the rows they belong to.
static __device__ __noinline__ float marked_term(const GroupedArgs& p, int row, int x) {
  const uint32_t id = static_cast<uint32_t>(p.ids[row]);
  return id < static_cast<uint32_t>(p.adapters) ? scalar_term(p, id, row, x, 0, p.rank, false) : 0.0f;
}
// The adapter term of row r0 + j of a few-row tile's batch, as far as it is this
// piece's: steps turn, turn + share, ... of the batch, of 32 rank values each.
// An infinite weight meets the whole rank value here; times a later term of H
// alone, which is zero or of either sign, it would give a NaN that the
// definition does not.
static __device__ __noinline__ float shared_term(const GroupedArgs& p, int r0, int j, int rows, int x,
                                                 int turn, int share) {
  if (j >= rows || x >= p.wide) return 0.0f;   // (neither is stored)
  const uint32_t id = static_cast<uint32_t>(p.ids[r0 + j]);
  if (id >= static_cast<uint32_t>(p.adapters)) return 0.0f;
  // The batch's adapters below this one, each counted at its first row.
  int step = 0;
  for (int i = 0; i < rows; ++i) {
    const uint32_t other = static_cast<uint32_t>(p.ids[r0 + i]);
    bool first = other < id;
    for (int k = 0; k < i; ++k) first = first && static_cast<uint32_t>(p.ids[r0 + k]) != other;
    if (first) step += (p.rank + 31) / 32;
  }
  float s = 0.0f;
  for (int r = 0; r < p.rank; r += 32, ++step)
    if (step % share == turn) s += scalar_term(p, id, r0 + j, x, r, min(r + 32, p.rank), true);
  return s;
}
__device__ __forceinline__ void add_marked_terms(const GroupedArgs& p, int row, int end, int x,
                                                 float (&v)[32]) {
  if (x >= p.wide) return;
#pragma unroll
  for (int j = 0; j < 32; ++j)
    if (row + j < end) v[j] += marked_term(p, row + j, x);
}

// Adapter term of a few-row tile: v[j] += up[id][x, :] . H[row + j, :] for 32
// rows.  It runs before the accumulator is waited for, beside the stream of
// the weights, on warp-level MMAs, in batches of 8 rows and steps of one
// adapter and 32 of the rank: 32 rows of up[id] by 8 rows of H, the result
// kept in the adapter's own rows' columns only (whatever the other columns
// hold).  Both operands come from memory in 16-byte pieces, 64 bytes of a row
// to each four lanes, so that a load instruction touches 8 lines; one lane per
// row of up[id] (32 lines each) took 71 us instead for 128 rows x 4096 with 48
// adapters of rank 64.
//
// A step takes about one trip to memory, so the tile's S pieces share the steps
// out: its batches first (batch0: this warp's before row), then, where there
// are more pieces than batches, each batch's steps.  (114 rows, 6 adapters of
// rank 32, x 1125 x 1721: 26 -> 22 us; 39 rows, 12 adapters of rank 128, x 1229 x
// 638, with H's ranks spread over blocks too: 28 -> 17.)
// Before `ready` only what the caller handed in is read: ids and up.
template <int kTerms>
__device__ __forceinline__ void add_adapter_terms(const GroupedArgs& p, const GroupedWork& w, int S,
                                                  int batch0, int row, int end, int x0, int lane,
                                                  bool& ready, float (&v)[32]) {
  const int g = lane >> 2, q = lane & 3;
  // The most batches one warp has: blocks of 32 rows go to two warps in turn.
  const int batches = min(4, (w.rows + 7) / 8) + (w.rows > 64 ? min(4, (w.rows - 57) / 8) : 0);
  const int share = S > batches ? small_div(S, batches) : 1;
  const int sets = S > batches ? small_div(S, share) : S;
  const int set = share > 1 ? small_div(w.piece, share) : w.piece;
  const int turn = w.piece - set * share;
  uint32_t again = 0;
#pragma unroll 1   // (one copy of a long body: instruction fetches are what a short call waits for)
  for (int b = 0; b < 4; ++b) {
    const int r0 = row + 8 * b;
    if (r0 >= end || (batch0 + b) % sets != set) continue;
    const int mine = r0 + (lane & 7);
    uint32_t ids[1] = {mine < end ? static_cast<uint32_t>(p.ids[mine]) : 0xFFFFFFFFu};
    const uint32_t id_b = __shfl_sync(0xFFFFFFFFu, ids[0], g);   // of the row this lane loads
    const uint32_t id_c0 = __shfl_sync(0xFFFFFFFFu, ids[0], 2 * q);
    const uint32_t id_c1 = __shfl_sync(0xFFFFFFFFu, ids[0], 2 * q + 1);
    const uint16_t* hrow = p.h + static_cast<int64_t>(r0 + g) * (kTerms * p.rank) + 8 * q;
    const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
    float sum[2][4] = {};
    int id = next_adapter(ids, -1, p.adapters), k = 0;
    // The step `n` steps on (id < 0: there is none).
    auto advance = [&](int n) {
      k += 32 * n;
      while (k >= p.rank && id >= 0) {
        k -= (p.rank + 31) / 32 * 32;
        id = next_adapter(ids, id, p.adapters);
      }
    };
    uint4 a[2][2], h[kTerms];
    auto load = [&]() {
      const bool in = 8 * q + k < p.rank;
      const uint16_t* u = p.up + id * p.group_stride_up + 8 * q + k;
#pragma unroll
      for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int x = x0 + 16 * t + 8 * i + g;
          a[t][i] = in && x < p.wide ? ld_global_nc_v4(u + static_cast<int64_t>(x) * p.ld_up) : zero;
        }
      if (!ready) {
        griddep_wait();
        ready = true;
      }
      const bool own = in && id_b == static_cast<uint32_t>(id);
#pragma unroll
      for (int t = 0; t < kTerms; ++t)
        h[t] = own ? *reinterpret_cast<const uint4*>(hrow + t * p.rank + k) : zero;
    };
    advance(turn);
    if (id < 0) continue;
    load();
    while (id >= 0) {
      const uint32_t cur = static_cast<uint32_t>(id);
      uint4 a0[2][2], h0[kTerms];
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        a0[t][0] = a[t][0];
        a0[t][1] = a[t][1];
      }
#pragma unroll
      for (int t = 0; t < kTerms; ++t) h0[t] = h[t];
      // The next step's loads are in flight during this one's products.
      advance(share);
      if (id >= 0) load();
      float c[2][4] = {};
#pragma unroll
      for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int i = 0; i < kTerms; ++i) {
          mma_m16n8k16(c[t], a0[t][0].x, a0[t][1].x, a0[t][0].y, a0[t][1].y, h0[i].x, h0[i].y);
          mma_m16n8k16(c[t], a0[t][0].z, a0[t][1].z, a0[t][0].w, a0[t][1].w, h0[i].z, h0[i].w);
        }
#pragma unroll
      for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if ((e & 1 ? id_c1 : id_c0) == cur) sum[t][e] += c[t][e];
    }
    // NaN: an infinite weight may have met a later term of H.  Nothing for now,
    // the batch's infinite and NaN sums after the others.
    bool nan = false;
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (sum[t][e] != sum[t][e]) {
          sum[t][e] = 0.0f;
          nan = true;
        }
    if (__any_sync(0xFFFFFFFFu, nan)) again |= 1u << b;
    // From (row of up g + 8 (e / 2) + 16 t, row of H 2 q + e % 2) to one lane
    // per row of up.
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int src = 4 * (lane & 7) + j / 2;
      float w[4];
#pragma unroll
      for (int i = 0; i < 4; ++i)
        w[i] = __shfl_sync(0xFFFFFFFFu, sum[i >> 1][2 * (i & 1) + (j & 1)], src);
      const float lo8 = lane & 16 ? w[2] : w[0], hi8 = lane & 16 ? w[3] : w[1];
      const float term = lane & 8 ? hi8 : lo8;
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (b == i) v[8 * i + j] += term;
    }
  }
  if (again == 0) return;
#pragma unroll 1
  for (int i = 0; i < 32; ++i) {
    if (!(again & (1u << (i / 8)))) continue;
    const int r0 = row + i / 8 * 8;
    const float term = shared_term(p, r0, i % 8, min(8, end - r0), x0 + lane, turn, share);
#pragma unroll
    for (int j = 0; j < 32; ++j)
      if (i == j && !(fabsf(term) < __uint_as_float(0x7F800000u))) v[j] += term;
  }
  __syncwarp();
}

template <class C>
__global__ void __launch_bounds__(C::kThreads, 1)
    gemm_grouped_kernel(const __grid_constant__ CUtensorMap tmW,
                        const __grid_constant__ CUtensorMap tmW2,
                        const __grid_constant__ ColumnMaps tmC,
                        const __grid_constant__ CUtensorMap tmUp,
                        const __grid_constant__ CUtensorMap tmD, const GroupedArgs p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::OFF_BAR);
  uint64_t* full_bar = bars;                       // [kStages] TMA -> MMA
  uint64_t* empty_bar = bars + C::kStages;         // [kStages] MMA -> TMA
  uint64_t* accf_bar = bars + 2 * C::kStages;      // [2] MMA -> epilogue
  uint64_t* acce_bar = accf_bar + C::kAccBufs;     // [2] epilogue -> MMA
  uint64_t* drain_bar = acce_bar + C::kAccBufs;
  uint64_t* fix_bar = drain_bar + 1;               // [kStages] fixing warps -> MMA
  uint64_t* tail_bar = fix_bar + C::kStages;       // [kStages] TMA -> this CTA's fixing warps
  uint64_t* checked_bar = tail_bar + C::kStages;   // fixing warps -> take_check
  uint64_t* checked_empty = checked_bar + 1;       // and back
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::OFF_MISC);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::OFF_MISC + 4);
  volatile int* join = reinterpret_cast<volatile int*>(smem + C::OFF_MISC + 8);
  volatile int* go = reinterpret_cast<volatile int*>(smem + C::OFF_MISC + 16);   // [4]
  // Marked tiles: entry n % 16 is n + 1 for the unit's n-th tile (the fixing
  // warps are never 16 tiles ahead: the ring is shorter).
  volatile int* marked = reinterpret_cast<volatile int*>(smem + C::OFF_MISC + 32);
  volatile int* checked = reinterpret_cast<volatile int*>(smem + C::OFF_MISC + 96);   // [2]

  const int warp = threadIdx.x >> 5;
  const int lane = static_cast<int>(threadIdx.x & 31);
  const uint32_t rank = C::kCtaGroup == 2 ? cluster_ctarank() : 0u;
  const bool leader = rank == 0;

  if (threadIdx.x == 0) {
    for (int s = 0; s < C::kStages; ++s) {
      mbar_init(&full_bar[s], 1);
      mbar_init(&empty_bar[s], 1);
      if constexpr (C::kFixWarps > 0) {
        mbar_init(&fix_bar[s], C::kCtaGroup);
        mbar_init(&tail_bar[s], 1);
      }
    }
    for (int b = 0; b < C::kAccBufs; ++b) {
      mbar_init(&accf_bar[b], 1);
      mbar_init(&acce_bar[b], C::kEpiWarps * C::kCtaGroup);
    }
    mbar_init(drain_bar, 1);
    *abort_flag = 0;
    if constexpr (C::kExt) {
      mbar_init(checked_bar, C::kFixWarps);
      mbar_init(checked_empty, C::kFixWarps + (leader ? 2 : 1));   // (one MMA issuer a pair)
    }
    if constexpr (C::kExt)
      for (int i = 0; i < 16; ++i) marked[i] = 0;
    fence_barrier_init();
  }
  if (warp == 0 && lane == 0) {
    prefetch_tensormap(&tmW);
    if constexpr (C::kWideMn) prefetch_tensormap(&tmW2);
    for (int b = 0; b < kColBoxes; ++b) prefetch_tensormap(&tmC.box[b]);
    if constexpr (C::kExt) prefetch_tensormap(&tmUp);
    if constexpr (C::kStaged) prefetch_tensormap(&tmD);
  }
  if (warp == 1) {
    tmem_alloc<C::kCtaGroup>(tmem_slot, C::TMEM_COLS);
    tmem_relinquish<C::kCtaGroup>();
  }
  tc_fence_before_sync();
  __syncthreads();
  if constexpr (C::kCtaGroup == 2) cluster_sync();
  tc_fence_after_sync();
  const uint32_t tmem_base = *tmem_slot;
  // The few-row adapter product streams its weights beside the kernel that
  // computes H, which started only when its own inputs (this one's A, B, up
  // and ids among them) were there, and so does kAdapterDown beside the kernels
  // before it: only the epilogue, which reads H and writes, waits for them
  // (the few-row product's only where it does either).
  constexpr bool kFewRows = C::kMode == kAdapter && C::kSplit;
  constexpr bool kEarly = kFewRows || C::kMode == kAdapterDown;
  bool inputs_ready = !kFewRows;
  if (!kEarly || (!kFewRows && warp >= C::kEpiWarp0)) griddep_wait();

  const WaitGuard guard{p.status, abort_flag, p.timeout_ns};
  // The fixing warps' word on the next tile of one adapter, whether the terms of
  // H after the first need care: by one thread each of the producer, the MMA
  // issuer and the fixing warps themselves.
  auto take_check = [&](uint32_t& parity, int& care) -> bool {
    if (!mbar_try_wait(smem_addr(checked_bar), parity) &&
        !mbar_wait(checked_bar, parity, guard, kSiteGrFixIn))
      return false;
    care = checked[0] | checked[1];
    mbar_arrive(checked_empty);
    parity ^= 1u;
    return true;
  };
  const int unit = blockIdx.x / C::kCtaGroup;
  const int num_units = gridDim.x / C::kCtaGroup;
  // Every role's warp walks the groups itself.
  GroupWalk<C> walk;
  int first_row, end_row;
  const int tiles = walk.total(p, lane, &first_row, &end_row);
  const GroupedPlan plan = grouped_plan<C>(p, tiles, num_units, lane);
  const int num_items = plan.items;
  GroupedWork w;
  // Work item u of the grid: S pieces from tile plan.full on.
  int S = 1;
  auto take = [&](int u) {
    if (C::kTail && u >= plan.full) {
      const int v = u - plan.full;
      S = plan.S;
      const int t = small_div(v, S);
      walk.find(p, lane, plan.full + t, v - t * S, S, w);
      w.tile -= plan.full;
    } else {
      S = 1;
      walk.find(p, lane, u, 0, 1, w);
    }
  };

  if (warp == 0 || (C::kTwoProducers && warp == C::kColWarp)) {
    // ------------------------------------------------------------ producers
    // Warp 0 posts the expected bytes and loads the wide operand; the column
    // operand is its own or, where a stage takes three or four loads, the
    // second producer's.
    const bool do_wide = warp == 0;
    const bool do_cols = !C::kTwoProducers || warp != 0;
    if (blockIdx.x == 0 && warp == 0) {
      const bool bad = __any_sync(0xFFFFFFFFu, walk.bad);
      if (bad && lane == 0 && atomicCAS(p.status, 0u, 1u) == 0u) {
        p.status[1] = kSiteGrOffsets;
        p.status[2] = 0;
        p.status[3] = 0;
      }
    }
    const uint64_t pol = policy_evict_last();
    const uint32_t sW = smem_addr(smem + C::OFF_W);
    const uint32_t sC = smem_addr(smem + C::OFF_C);
    const uint32_t empty0 = smem_addr(&empty_bar[0]);
    const uint32_t full0 = smem_addr(&full_bar[0]);
    const uint32_t full_dst0 = C::kCtaGroup == 2 ? map_to_cta(full0, 0u) : full0;
    int stage = 0;
    uint32_t phase = 0;
    uint32_t issued = 0, issued_parity = 0;    // full_bar
    uint32_t tailed = 0, tail_parity = 0;      // tail_bar: used, parity of the last use
    uint32_t check_parity = 0;
    int ok = 1;
    auto wait_slot = [&]() -> bool {
      return mbar_try_wait(empty0 + 8u * stage, phase ^ 1u) ||
             mbar_wait(&empty_bar[stage], phase ^ 1u, guard, kSiteGrEmpty);
    };
    auto note_tail = [&]() {
      tail_parity = (tailed >> stage) & 1u ? tail_parity ^ (1u << stage)
                                           : tail_parity & ~(1u << stage);
      tailed |= 1u << stage;
    };
    auto next_slot = [&]() {
      issued |= 1u << stage;
      issued_parity = (issued_parity & ~(1u << stage)) | (phase << stage);
      if (++stage == C::kStages) {
        stage = 0;
        phase ^= 1u;
      }
    };
    for (int u = unit; u < num_items && ok; u += num_units) {
      take(u);
      const int wx = w.wide0 + static_cast<int>(rank) * 128;
      const int crows = w.ncols / C::kCtaGroup;       // column-operand rows of this CTA
      const int cbox = (crows - 1) / C::kBoxStep;     // K-major: the box that holds them
      const int loaded = C::kColMn ? crows : (cbox + 1) * C::kBoxStep;
      // (Slices of dgrad read the same rows.)
      const int crow0 = w.row0 + static_cast<int>(rank) * crows -
                        (C::kAdd && !C::kColMn ? w.g * p.even : 0);
      // MN-major: both of a box pair's 64-element chunks lie inside the row.
      const bool w_chunks = C::kWideMn && wx + 128 <= p.wide;
      // Read here, used after the K stages.
      uint32_t tile_ids[C::kTileN / 32];
      if constexpr (C::kExt) load_tile_ids<C>(p, w, lane, tile_ids);
      const bool c_chunks = C::kColMn && crows == 128 && crow0 + 128 <= p.cols;
      if constexpr (C::kMode == kAdapterDown) {
        uint32_t ids[C::kTileN / 32];
        load_tile_ids<C>(p, w, lane, ids);
        if (!few_adapters(ids, p.adapters)) continue;
        const int slot = down_slot(p.rank);
        int last = -1, group[4];
        for (int n = next_adapters(ids, last, 128 / slot, p.adapters, group); n > 0 && ok;
             n = next_adapters(ids, last, 128 / slot, p.adapters, group)) {
          if (lane == 0) {
            for (int j = 0, kb = w.k0; j < w.nk; ++j, kb += w.ks) {
              if (!wait_slot()) {
                ok = 0;
                break;
              }
              const uint32_t fb = full0 + 8u * stage;
              mbar_arrive_expect_tx(&full_bar[stage],
                                    static_cast<uint32_t>(n * p.wide_box + loaded) * 128u);
#pragma unroll
              for (int i = 0; i < 4; ++i)
                if (group[i] >= 0)
                  tma_load_3d(sW + stage * C::W_BYTES + 128 * slot * i, &tmW, fb, kb * 64, wx,
                              group[i], pol);
              tma_load_2d(sC + stage * C::C_BYTES, &tmC.box[cbox], fb, kb * 64, crow0, pol);
              next_slot();
            }
          }
          ok = __shfl_sync(0xFFFFFFFFu, ok, 0);
        }
        continue;
      }
      if constexpr (C::kGather) {
        if (p.row_idx != nullptr) {
          // Rows picked by index: each lane four of them, in one gather (box
          // one row high); rows past the tile or outside the operand read zeros.
          int r[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const int i = 4 * lane + j;
            const int src = i < w.rows ? p.row_idx[w.row0 + i] : -1;
            r[j] = static_cast<uint32_t>(src) < static_cast<uint32_t>(p.num_rows) ? src : p.num_rows;
          }
          for (int j = 0, kb = w.k0; j < w.nk; ++j, kb += w.ks) {
            if (lane == 0) {
              ok = wait_slot();
              if (ok)
                mbar_arrive_expect_tx(&full_bar[stage],
                                      C::W_BYTES + static_cast<uint32_t>(w.ncols) * 128u);
            }
            ok = __shfl_sync(0xFFFFFFFFu, ok, 0);
            if (!ok) break;
            const uint32_t fb = full0 + 8u * stage;
            if (4 * lane < w.ncols)
              tma_gather4_2d(sC + stage * C::C_BYTES + 512u * static_cast<uint32_t>(lane),
                             &tmC.box[0], fb, kb * 64, r[0], r[1], r[2], r[3], pol);
            if (lane == 0)
              tma_load_3d(sW + stage * C::W_BYTES, &tmW, fb, kb * 64, wx, w.g, pol);
            next_slot();
          }
          continue;
        }
      }
      if (lane == 0) {
        const uint32_t cbytes = static_cast<uint32_t>(loaded) * 128u;
        for (int j = 0, kb = w.k0; j < w.nk; ++j, kb += w.ks) {
          if (!wait_slot()) {
            ok = 0;
            break;
          }
          const int kx = kb * 64;
          const uint32_t dW = sW + stage * C::W_BYTES;
          const uint32_t dC = sC + stage * C::C_BYTES;
          const bool tail = C::kColMn && w.len - kx < 64;
          if (tail) {
            // Both CTAs' loads of a ragged stage complete locally, for the
            // CTA's own fixing warp.
            const uint32_t tb = smem_addr(&tail_bar[stage]);
            if (do_wide) {
              if (leader) mbar_arrive(&full_bar[stage]);
              mbar_arrive_expect_tx(&tail_bar[stage], C::W_BYTES + cbytes);
              if (w_chunks)
                tma_load_4d(dW, &tmW2, tb, 0, w.base + kx, wx / 64, 0, pol);
              else
                for (int c = 0; c < 2; ++c)
                  tma_load_2d(dW + 8192 * c, &tmW, tb, wx + 64 * c, w.base + kx, pol);
            }
            if (do_cols) {
              if (c_chunks)
                tma_load_4d(dC, &tmC.box[1], tb, 0, w.base + kx, crow0 / 64, 0, pol);
              else
                for (int c = 0; c < crows / 64; ++c)
                  tma_load_2d(dC + 8192 * c, &tmC.box[0], tb, crow0 + 64 * c, w.base + kx, pol);
            }
            note_tail();
            next_slot();
            continue;
          }
          const uint32_t fb = full_dst0 + 8u * stage;
          if (leader && do_wide)
            mbar_arrive_expect_tx(&full_bar[stage], C::kCtaGroup * (C::W_BYTES + cbytes));
          if constexpr (C::kMode == kGroupedWgrad) {
            if (do_wide) {
              if (w_chunks)
                tma_load_4d_pair(dW, &tmW2, fb, 0, w.base + kx, wx / 64, 0, pol);
              else
                for (int c = 0; c < 2; ++c)
                  tma_load_2d_pair(dW + 8192 * c, &tmW, fb, wx + 64 * c, w.base + kx, pol);
            }
            if (do_cols) {
              if (c_chunks)
                tma_load_4d_pair(dC, &tmC.box[1], fb, 0, w.base + kx, crow0 / 64, 0, pol);
              else
                for (int c = 0; c < crows / 64; ++c)
                  tma_load_2d_pair(dC + 8192 * c, &tmC.box[0], fb, crow0 + 64 * c, w.base + kx,
                                   pol);
            }
          } else if constexpr (C::kCtaGroup == 2) {
            if (do_wide) {
              const int kw = C::kAdd ? w.g * p.slice + (kx < p.slice ? kx : kx - p.slice) : kx;
              const int wg = C::kAdd ? 0 : w.g;
              if (C::kWideMn && w_chunks) {
                tma_load_4d_pair(dW, &tmW2, fb, 0, kw, wx / 64, wg, pol);
              } else if constexpr (C::kWideMn) {
                for (int c = 0; c < 2; ++c)
                  tma_load_3d_pair(dW + 8192 * c, &tmW, fb, wx + 64 * c, kw, wg, pol);
              } else {
                tma_load_3d_pair(dW, &tmW, fb, kx, wx, w.g, pol);
              }
            }
            if (do_cols) {
              const int kc = C::kAdd ? w.g * p.slice +
                                           (kx < p.slice ? kx : p.second + kx - p.slice)
                                     : kx;
              tma_load_2d_pair(dC, &tmC.box[cbox], fb, kc, crow0, pol);
            }
          } else {
            tma_load_3d(dW, &tmW, fb, kx, wx, w.g, pol);
            tma_load_2d(dC, &tmC.box[cbox], fb, kx, crow0, pol);
          }
          next_slot();
        }
      }
      ok = __shfl_sync(0xFFFFFFFFu, ok, 0);
      if constexpr (C::kExt) {
        const bool mixed = mixed_adapters(tile_ids, w.rows, lane, p.adapters);
        // (A split tile's adapter stages belong to its first piece.)
        const int per = (p.rank + 63) / 64 * 64;
        const int end = w.piece == 0 ? 64 * adapter_stages<C::kTerms>(p.rank, mixed) : 0;
        int care = 0;
        for (int r = 0; r < end && ok; r += 64) {
          for (int id = next_adapter(tile_ids, -1, p.adapters); id >= 0 && ok;
               id = next_adapter(tile_ids, id, p.adapters)) {
            if (lane == 0) {
              // One adapter: the check's word before the second term's first stage.
              ok = (mixed || r != per || take_check(check_parity, care)) && wait_slot();
              if (ok) {
                const int term = small_div(r, per), rx = r - term * per;
                if (mixed || (care && term > 0)) {
                  // Like a ragged stage's, the load completes in each CTA for
                  // its own fixing warps.
                  if (leader) mbar_arrive(&full_bar[stage]);
                  mbar_arrive_expect_tx(&tail_bar[stage], C::W_BYTES + C::C_BYTES);
                  const uint32_t tb = smem_addr(&tail_bar[stage]);
                  tma_load_3d(sW + stage * C::W_BYTES, &tmUp, tb, rx, wx, id, pol);
                  tma_load_2d(sC + stage * C::C_BYTES,
                              &tmC.h[adapter_packed<C::kTerms>(p.rank, mixed) ? 3 : term], tb, rx,
                              crow0, pol);
                  note_tail();
                } else {
                  if (leader)
                    mbar_arrive_expect_tx(&full_bar[stage], 2 * (C::W_BYTES + C::C_BYTES));
                  const uint32_t fb = full_dst0 + 8u * stage;
                  tma_load_3d_pair(sW + stage * C::W_BYTES, &tmUp, fb, rx, wx, id, pol);
                  tma_load_2d_pair(sC + stage * C::C_BYTES, &tmC.h[term], fb, rx,
                                   crow0, pol);
                }
                next_slot();
              }
            }
            ok = __shfl_sync(0xFFFFFFFFu, ok, 0);
          }
        }
      }
    }
    if (lane == 0) {
      if (do_wide) griddep_launch_dependents();
      if (!ok) {
        for (int s = 0; s < C::kStages; ++s) {
          if (leader && (issued & (1u << s)))
            mbar_wait_drain(&full_bar[s], (issued_parity >> s) & 1u, p.timeout_ns);
          if (tailed & (1u << s))
            mbar_wait_drain(&tail_bar[s], (tail_parity >> s) & 1u, p.timeout_ns);
        }
      }
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer
    if (leader) {
      const uint32_t acce0 = smem_addr(&acce_bar[0]);
      const uint32_t full0 = smem_addr(&full_bar[0]);
      const uint64_t wdesc0 = make_smem_desc(smem_addr(smem + C::OFF_W), C::kWideMn ? 8192 : 16,
                                             1024, kDescSwizzle128B);
      const uint64_t cdesc0 = make_smem_desc(smem_addr(smem + C::OFF_C), C::kColMn ? 8192 : 16,
                                             1024, kDescSwizzle128B);
      // One K16 step: 32 bytes of a K-major row, 16 rows of an MN-major box.
      constexpr uint32_t kStepW = C::kWideMn ? 128 : 2;
      constexpr uint32_t kStepC = C::kColMn ? 128 : 2;
      int stage = 0;
      uint32_t phase = 0;
      int acc = 0;
      uint32_t acc_phase = 0;
      uint32_t fix_parity = 0;      // parity of each stage's next fix
      uint32_t check_parity = 0;
      int ok = 1;
      bool ready = false;
      auto wait_fix = [&]() -> bool {
        const uint32_t par = (fix_parity >> stage) & 1u;
        fix_parity ^= 1u << stage;
        return mbar_try_wait_cluster(smem_addr(&fix_bar[stage]), par) ||
               mbar_wait_cluster(&fix_bar[stage], par, guard, kSiteGrFix);
      };
      // The accumulator is complete: the next one follows.
      auto commit_acc = [&]() {
        if constexpr (C::kCtaGroup == 1)
          mma_commit(&accf_bar[acc]);
        else
          mma_commit_pair(&accf_bar[acc], static_cast<uint16_t>(3u));
        if (++acc == C::kAccBufs) {
          acc = 0;
          acc_phase ^= 1u;
        }
      };
      for (int u = unit; u < num_items && ok; u += num_units) {
        take(u);
        const uint32_t idesc =
            idesc_bf16_f32_major(128 * C::kCtaGroup, w.ncols, C::kWideMn, C::kColMn);
        uint32_t tile_ids[C::kTileN / 32];
        if constexpr (C::kExt) load_tile_ids<C>(p, w, lane, tile_ids);
        // kAdapterDown: one contraction for each of the tile's passes.
        int passes = 1;
        if constexpr (C::kMode == kAdapterDown) {
          uint32_t ids[C::kTileN / 32];
          load_tile_ids<C>(p, w, lane, ids);
          passes = 0;
          int last = -1, group[4];
          if (few_adapters(ids, p.adapters))
            while (next_adapters(ids, last, 128 / down_slot(p.rank), p.adapters, group) > 0) ++passes;
        }
        const int chunks = grouped_chunks<C>(w.nk);   // an empty contraction has none
        uint32_t d_tmem = 0;
        for (int pass = 0; pass < passes && ok; ++pass) {
        if (lane == 0) {
          for (int c = 0, j = 0, kb = w.k0; c < chunks && ok; ++c) {
            if (!mbar_try_wait(acce0 + 8u * acc, acc_phase ^ 1u) &&
                !mbar_wait(&acce_bar[acc], acc_phase ^ 1u, guard, kSiteGrAccEmpty)) {
              ok = 0;
              break;
            }
            tc_fence_after_sync();
            d_tmem = tmem_base + static_cast<uint32_t>(acc * C::kTileN);
            const int j0 = j;
            const int j1 = grouped_chunk_end<C>(w.nk, chunks, c);
            for (; j < j1; ++j, kb += w.ks) {
              if (!ready && !mbar_try_wait(full0 + 8u * stage, phase) &&
                  !mbar_wait(&full_bar[stage], phase, guard, kSiteGrFull)) {
                ok = 0;
                break;
              }
              int issues = 4;
              if constexpr (C::kColMn) {
                const int left = w.len - kb * 64;
                if (left < 64) {
                  issues = (left + 15) / 16;
                  if (!wait_fix()) {
                    ok = 0;
                    break;
                  }
                }
              }
              tc_fence_after_sync();
              const int ns = stage + 1 == C::kStages ? 0 : stage + 1;
              const uint32_t nph = stage + 1 == C::kStages ? phase ^ 1u : phase;
              const uint64_t wd = wdesc0 + static_cast<uint64_t>(stage * (C::W_BYTES >> 4));
              const uint64_t cd = cdesc0 + static_cast<uint64_t>(stage * (C::C_BYTES >> 4));
              if (!C::kColMn || issues == 4) {
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                  mma_bf16<C::kCtaGroup>(d_tmem, wd + kStepW * k, cd + kStepC * k, idesc,
                                         (j != j0 || k != 0));
                  if (k == 0) ready = mbar_try_wait(full0 + 8u * ns, nph);
                }
              } else {
                for (int k = 0; k < issues; ++k)
                  mma_bf16<C::kCtaGroup>(d_tmem, wd + kStepW * k, cd + kStepC * k, idesc,
                                         (j != j0 || k != 0));
                ready = mbar_try_wait(full0 + 8u * ns, nph);
              }
              if constexpr (C::kCtaGroup == 1)
                mma_commit(&empty_bar[stage]);
              else
                mma_commit_pair(&empty_bar[stage], static_cast<uint16_t>(3u));
              stage = ns;
              phase = nph;
            }
            if (ok && (c + 1 < chunks || C::kMode == kAdapterDown)) commit_acc();
          }
        }
        ok = __shfl_sync(0xFFFFFFFFu, ok, 0);
        }
        if constexpr (C::kExt) {
          const int per = (p.rank + 63) / 64 * 64;
          const bool mixed = mixed_adapters(tile_ids, w.rows, lane, p.adapters);
          const int end = w.piece == 0 ? 64 * adapter_stages<C::kTerms>(p.rank, mixed) : 0;
          int care = 0;
          for (int r = 0; r < end && ok; r += 64) {
            for (int id = next_adapter(tile_ids, -1, p.adapters); id >= 0 && ok;
                 id = next_adapter(tile_ids, id, p.adapters)) {
              if (lane == 0) {
                ok = (mixed || r != per || take_check(check_parity, care)) &&
                     (ready || mbar_try_wait(full0 + 8u * stage, phase) ||
                      mbar_wait(&full_bar[stage], phase, guard, kSiteGrFull)) &&
                     ((!mixed && (!care || r < per)) || wait_fix());
                if (ok) {
                  tc_fence_after_sync();
                  const uint64_t wd = wdesc0 + static_cast<uint64_t>(stage * (C::W_BYTES >> 4));
                  const uint64_t cd = cdesc0 + static_cast<uint64_t>(stage * (C::C_BYTES >> 4));
                  const int left = p.rank - (r - small_div(r, per) * per);
                  const int issues = adapter_packed<C::kTerms>(p.rank, mixed)
                                         ? (C::kTerms * p.rank + 15) / 16
                                     : left >= 64                  ? 4
                                                                   : (left + 15) / 16;
                  for (int k = 0; k < issues; ++k)
                    mma_bf16<C::kCtaGroup>(d_tmem, wd + 2 * k, cd + 2 * k, idesc, 1u);
                  mma_commit_pair(&empty_bar[stage], static_cast<uint16_t>(3u));
                  if (++stage == C::kStages) {
                    stage = 0;
                    phase ^= 1u;
                  }
                  ready = false;
                }
              }
              ok = __shfl_sync(0xFFFFFFFFu, ok, 0);
            }
          }
        }
        if (C::kMode != kAdapterDown && chunks > 0 && ok && lane == 0) commit_acc();
      }
      if (lane == 0 && (!ok || *abort_flag)) {
        if constexpr (C::kCtaGroup == 1)
          mma_commit(drain_bar);
        else
          mma_commit_pair(drain_bar, static_cast<uint16_t>(1u));
        mbar_wait_drain(drain_bar, 0, p.timeout_ns);
      }
    }
  } else if (warp < C::kEpiWarp0) {
    // ------------------------------------------------------------ fixing warps
    if (warp < C::kFixWarp0 + C::kFixWarps) {
      const int fw = warp - C::kFixWarp0;
      const uint32_t fix0 = map_to_cta(smem_addr(&fix_bar[0]), 0u);
      const uint32_t sW = smem_addr(smem + C::OFF_W);
      const uint32_t sC = smem_addr(smem + C::OFF_C);
      uint32_t pos = 0;            // ring slots used so far
      uint32_t tail_use = 0;       // parity of each stage's next tail
      uint32_t check_parity = 0;
      int ok = 1;
      int count = 0;               // tiles of this unit so far
      for (int u = unit; u < num_items && ok; u += num_units, ++count) {
        take(u);
        if constexpr (C::kMode == kGroupedWgrad) {
          const int rest = w.len & 63;
          // The ragged stage is the last one of the piece that has it.
          if (rest != 0 && w.len / 64 % w.ks == w.k0) {
            const int stage = static_cast<int>((pos + w.nk - 1) % C::kStages);
            const uint32_t par = (tail_use >> stage) & 1u;
            tail_use ^= 1u << stage;
            if (lane == 0)
              ok = mbar_try_wait(smem_addr(&tail_bar[stage]), par) ||
                   mbar_wait(&tail_bar[stage], par, guard, kSiteGrFixIn);
            ok = __shfl_sync(0xFFFFFFFFu, ok, 0);
            if (!ok) break;
            // Rows rest .. next multiple of 16 of each 64 x 64 box: one
            // contiguous piece (the swizzle permutes within a row).
            const int pieces = (((rest + 15) & ~15) - rest) * 8;
            const int cboxes = w.ncols / C::kCtaGroup / 64;
            for (int b = 0; b < 2 + cboxes; ++b) {
              const uint32_t a = (b < 2 ? sW + stage * C::W_BYTES + b * 8192
                                        : sC + stage * C::C_BYTES + (b - 2) * 8192) +
                                 static_cast<uint32_t>(rest) * 128u;
              for (int i = lane; i < pieces; i += 32) st_shared_v4(a + 16 * i, 0u, 0u, 0u, 0u);
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive_cluster(fix0 + 8u * stage);
          }
          pos += w.nk;
        } else {
          pos += w.nk;
          if (w.piece != 0) continue;
          uint32_t ids[C::kTileN / 32];
          load_tile_ids<C>(p, w, lane, ids);
          const int per = (p.rank + 63) / 64 * 64;
          const int crows = w.ncols / C::kCtaGroup;
          const int r0 = static_cast<int>(rank) * crows;   // this CTA's rows of the tile
          const bool mixed = mixed_adapters(ids, w.rows, lane, p.adapters);
          if (!mixed) {
            // One adapter: its stages are as TMA loads them, but for the terms
            // after the first where up[id] holds infinite or NaN weights.  Each
            // warp looks at one CTA's box in memory while the tile's K stages
            // run, and both CTAs at both.
            const int id = next_adapter(ids, -1, p.adapters);
            if (id < 0) continue;
            bool finite = true;
            for (int r = 0; r < p.rank && finite; r += 64)
              finite = finite_box(p, id, w.wide0 + 128 * fw, r, lane);
            int care = 0;
            if (lane == 0) {
              ok = mbar_try_wait(smem_addr(checked_empty), check_parity ^ 1u) ||
                   mbar_wait(checked_empty, check_parity ^ 1u, guard, kSiteGrFixIn);
              if (ok) {
                checked[fw] = finite ? 0 : 1;
                mbar_arrive(checked_bar);
                ok = take_check(check_parity, care);
              }
            }
            ok = __shfl_sync(0xFFFFFFFFu, ok, 0);
            if (!ok) break;
            if (!__shfl_sync(0xFFFFFFFFu, care, 0)) {
              pos += adapter_stages<C::kTerms>(p.rank, false);
              continue;
            }
            pos += per / 64;
          }
          // The adapters of this CTA's rows lane, lane + 32, ...
          uint32_t own[C::C_ROWS / 32];
#pragma unroll
          for (int i = 0; i < C::C_ROWS / 32; ++i) {
            const int r = lane + 32 * i;
            own[i] = r < crows && r0 + r < w.rows ? static_cast<uint32_t>(p.ids[w.row0 + r0 + r])
                                                  : 0xFFFFFFFFu;
          }
          // A warp goes over 4 rows x 8 16-byte pieces at a time; this lane's
          // piece, by the step's parity, with the rows' swizzle.  Packed:
          // up[id] again every `copy` pieces.
          const bool packed = adapter_packed<C::kTerms>(p.rank, mixed);
          const uint32_t lr = static_cast<uint32_t>(lane >> 3), q = static_cast<uint32_t>(lane & 7);
          const uint32_t copy = static_cast<uint32_t>(p.rank / 8);
          const uint32_t at[2] = {128u * lr + ((q ^ lr) << 4), 128u * lr + ((q ^ (lr + 4u)) << 4)};
          const int stages = 64 * adapter_stages<C::kTerms>(p.rank, mixed);
          for (int r = mixed ? 0 : per; r < stages && ok; r += 64) {
            const int cw = min(64, p.rank - (r - small_div(r, per) * per));   // columns (rest: zeros)
            for (int id = next_adapter(ids, -1, p.adapters); id >= 0 && ok;
                 id = next_adapter(ids, id, p.adapters), ++pos) {
              const int stage = static_cast<int>(pos % C::kStages);
              const uint32_t par = (tail_use >> stage) & 1u;
              tail_use ^= 1u << stage;
              // The warps take turns: one's waits are the other's work.
              if ((pos & 1u) != static_cast<uint32_t>(fw)) continue;
              if (lane == 0)
                ok = mbar_try_wait(smem_addr(&tail_bar[stage]), par) ||
                     mbar_wait(&tail_bar[stage], par, guard, kSiteGrFixIn);
              ok = __shfl_sync(0xFFFFFFFFu, ok, 0);
              if (!ok) break;
              // H: zeros in the rows of other adapters.
              const uint32_t hdst = sC + stage * C::C_BYTES;
#pragma unroll
              for (int i = 0; i < C::C_ROWS / 32; ++i) {
                const uint32_t others =
                    ~__ballot_sync(0xFFFFFFFFu, own[i] == static_cast<uint32_t>(id)) >> lr;
                if (mixed && 32 * i < crows) {
#pragma unroll
                  for (int t = 0; t < 8; ++t)
                    if (others & (1u << (4 * t)))
                      st_shared_v4(hdst + 4096u * i + 512u * t + at[t & 1], 0u, 0u, 0u, 0u);
                }
              }
              // up[id]: infinite and NaN weights go (those of one adapter's
              // tile have met the first term).  The pieces that hold weights,
              // eight loads on their way at a time.
              const uint32_t wsrc = sW + stage * C::W_BYTES;
              if (8 * static_cast<int>(q) < cw) {
#pragma unroll
                for (int i0 = 0; i0 < 32; i0 += 8) {
                  uint4 u[8];
#pragma unroll
                  for (int i = 0; i < 8; ++i) u[i] = ld_shared_v4(wsrc + 512u * (i0 + i) + at[i & 1]);
                  uint32_t z[4] = {0u, 0u, 0u, 0u};
#pragma unroll
                  for (int i = 0; i < 8; ++i) {
                    z[0] = times_zero_bf16x2(u[i].x, z[0]);
                    z[1] = times_zero_bf16x2(u[i].y, z[1]);
                    z[2] = times_zero_bf16x2(u[i].z, z[2]);
                    z[3] = times_zero_bf16x2(u[i].w, z[3]);
                  }
                  if (((z[0] | z[1] | z[2] | z[3]) & 0x7FFF7FFFu) != 0u) {
                    if (mixed) marked[count & 15] = count + 1;
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                      u[i] = make_uint4(finite_bf16x2(u[i].x), finite_bf16x2(u[i].y),
                                        finite_bf16x2(u[i].z), finite_bf16x2(u[i].w));
                      st_shared_v4(wsrc + 512u * (i0 + i) + at[i & 1], u[i].x, u[i].y, u[i].z,
                                   u[i].w);
                    }
                  }
                  if (packed) {
#pragma unroll
                    for (int t = 1; t < C::kTerms; ++t) {
                      const uint32_t c = q + t * copy;
#pragma unroll
                      for (int i = 0; i < 8; ++i)
                        st_shared_v4(wsrc + 512u * (i0 + i) + 128u * lr +
                                         ((c ^ (lr + 4u * (i & 1))) << 4),
                                     u[i].x, u[i].y, u[i].z, u[i].w);
                    }
                  }
                }
              }
              fence_proxy_async_smem();
              __syncwarp();
              if (lane == 0) mbar_arrive_cluster(fix0 + 8u * stage);
            }
          }
        }
      }
    }
  } else {
    // ------------------------------------------------------------ epilogue
    const int slab = warp & 3;                 // TMEM lanes 32 * slab ..
    const int half = (warp - C::kEpiWarp0) >> 2;   // column blocks half, half + 2, ...
    if constexpr (!C::kColMn && C::kMode != kAdapter)   // (adapters: every row has a tile)
      grouped_zero_rows<C>(p, first_row, end_row,
                           static_cast<int>(blockIdx.x) * C::kEpiWarps + warp - C::kEpiWarp0,
                           static_cast<int>(gridDim.x) * C::kEpiWarps, lane);
    int acc = 0;
    uint32_t acc_phase = 0;
    const int box = C::kBf16Out ? (warp - C::kEpiWarp0) >> 1 : warp - C::kEpiWarp0;
    // f32: one box a warp.  bf16: two boxes for each two warps (slabs 2i, 2i + 1).
    const uint32_t stg =
        smem_addr(smem + C::OFF_STG) + static_cast<uint32_t>(box) * (C::kBf16Out ? 8192u : 4096u);
    const bool box_lead = (warp & 1) == 0 && lane == 0;
    const uint64_t pol_d = policy_evict_first();   // D is written once
    uint32_t flip = 0;
    uint32_t acce_dst = smem_addr(&acce_bar[0]);
    if constexpr (C::kCtaGroup == 2) acce_dst = map_to_cta(acce_dst, 0u);
    // Waits for the next accumulator.
    auto acc_ready = [&]() -> bool {
      int got = 1;
      const bool all = C::kTail && plan.S > 1;
      if (all || (C::kStaged && C::kBf16Out)) {
        // Warps that meet at named barriers below (all of a split tile's, the
        // two that share a staging box) must agree whether the accumulator
        // arrived: one thread of them decides.  Where split tiles are to come,
        // it does for the whole tiles before them as well: a warp that gave up
        // there would be missing at the first split tile's barrier.
        const bool decides = all ? warp == C::kEpiWarp0 && lane == 0 : box_lead;
        const int id = all ? 1 : 2 + box, count = all ? 32 * C::kEpiWarps : 64;
        volatile int* flag = go + (all ? 0 : box);
        if (decides) *flag = mbar_wait(&accf_bar[acc], acc_phase, guard, kSiteGrAccFull) ? 1 : 0;
        named_bar_sync(id, count);
        got = *flag;
        named_bar_sync(id, count);
      } else {
        if (lane == 0) got = mbar_wait(&accf_bar[acc], acc_phase, guard, kSiteGrAccFull) ? 1 : 0;
        got = __shfl_sync(0xFFFFFFFFu, got, 0);
      }
      tc_fence_after_sync();
      return got != 0;
    };
    // Hands the accumulator back (this warp's reads of it are complete).
    auto hand_back = [&]() {
      tc_fence_before_sync();
      __syncwarp();
      if (lane == 0) {
        if constexpr (C::kCtaGroup == 1)
          mbar_arrive_relaxed(&acce_bar[acc]);
        else
          mbar_arrive_relaxed_cluster(acce_dst + 8u * static_cast<uint32_t>(acc));
      }
      if (++acc == C::kAccBufs) {
        acc = 0;
        acc_phase ^= 1u;
      }
    };
    // Split tiles: this lane's column of the piece's partial tile, [column of
    // the accumulator][128 lanes] for each CTA.
    constexpr int64_t kPart = C::kTileN * 128;
    auto part_of = [&](int piece) {
      return p.partials +
             tail_column(w.tile, piece, S, C::kCtaGroup, static_cast<int>(rank), C::kTileN, 0, 128) +
             slab * 32 + lane;
    };
    auto publish = [&](int col, int left, const float (&v)[32]) {
      float* dst = part_of(w.piece) + col * 128;
#pragma unroll
      for (int i = 0; i < 32; ++i)
        if (i < left) __stcg(dst + i * 128, v[i]);
    };
    // True in the CTA whose arrival is the tile's last: all partials are there.
    auto joined = [&]() -> bool {
      __threadfence();
      named_bar_sync(1, 32 * C::kEpiWarps);
      if (warp == C::kEpiWarp0 && lane == 0) {
        uint32_t* counter = p.counters + w.tile * C::kCtaGroup + static_cast<int>(rank);
        const int last = arrive_counter_gpu(counter) == static_cast<uint32_t>(S - 1);
        if (last) *counter = 0u;
        *join = last;
      }
      named_bar_sync(1, 32 * C::kEpiWarps);
      if (!*join) return false;
      __threadfence();
      return true;
    };
    // The pieces' sum, in piece order.  All 32 columns, also those past the
    // tile's rows (the slot has them; they are not stored): unconditional
    // loads fly together.
    auto collect = [&](int col, float (&v)[32]) {
      const float* src = part_of(0) + col * 128;
#pragma unroll
      for (int i = 0; i < 32; ++i) v[i] = __ldcg(src + i * 128);
      for (int r = 1; r < S; ++r) {
        src += C::kCtaGroup * kPart;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          float t[16];
#pragma unroll
          for (int i = 0; i < 16; ++i) t[i] = __ldcg(src + (16 * h + i) * 128);
#pragma unroll
          for (int i = 0; i < 16; ++i) v[16 * h + i] += t[i];
        }
      }
    };
    bool ok = true;
    int count = 0;                             // tiles of this unit so far
    for (int u = unit; u < num_items && ok; u += num_units, ++count) {
      take(u);
      const int chunks = grouped_chunks<C>(w.nk);
      const int x = w.wide0 + static_cast<int>(rank) * 128 + slab * 32 + lane;
      const float b = epi_uses_bias(p.epi.op) && x < p.wide
                          ? p.epi.bias[static_cast<int64_t>(w.g) * p.wide + x]
                          : 0.0f;
      const int64_t d0 = C::kColMn ? static_cast<int64_t>(w.g) * p.group_stride_d : 0;
      const int end = w.row0 + w.rows;
      const int blocks = (w.rows + 31) / 32;   // of 32 accumulator columns
      const uint32_t t_slab = tmem_base + (static_cast<uint32_t>(slab * 32) << 16);
      if constexpr (C::kMode == kAdapterDown) {
        // Column block `half` is this warp's 32 rows; its lanes are rank
        // indices xr of slot number `mine`.  Every row is written once, by its
        // own adapter's slot.
        uint32_t ids[C::kTileN / 32];
        load_tile_ids<C>(p, w, lane, ids);
        if (!few_adapters(ids, p.adapters)) continue;
        const int slot = down_slot(p.rank);
        const int mine = 32 * slab / slot;
        const int xr = w.wide0 + 32 * slab % slot + lane;
        const int row0 = w.row0 + 32 * half;
        // A split tile's partial sums: [row of the tile][rank value of it].
        const int width = tail_slot_width(true, p.rank);
        auto part_at = [&](int piece, int row, int r) {
          return p.partials +
                 tail_column(w.tile, piece, S, 1, 0, C::kTileN, row - w.row0, width) + (r - w.wide0);
        };
        auto keep = [&](int row, int r, float s) {
          split_bf16(s, p.h + static_cast<int64_t>(row) * (p.h_terms * p.rank) + r, p.rank,
                     p.h_terms);
        };
        int last_id = -1, group[4];
        while (next_adapters(ids, last_id, 128 / slot, p.adapters, group) > 0) {
          float v[32];
          if constexpr (!C::kBf16Out) grouped_zero(v);
          for (int c = 0; c < chunks && ok; ++c) {   // (bf16 D: one)
            ok = acc_ready();
            if (!ok) break;
            grouped_read<!C::kBf16Out>(
                t_slab + static_cast<uint32_t>(acc * C::kTileN + 32 * half), v);
            hand_back();
          }
          if (!ok) break;
          const int id = mine == 0 ? group[0] : mine == 1 ? group[1] : mine == 2 ? group[2] : group[3];
          if (id < 0 || xr >= p.wide) continue;
          const float scale = p.scales ? p.scales[id] : 1.0f;
#pragma unroll
          for (int j = 0; j < 32; ++j) {
            if (row0 + j >= end || p.ids[row0 + j] != id) continue;
            if (C::kTail && S > 1)
              __stcg(part_at(w.piece, row0 + j, xr), v[j] * scale);
            else
              keep(row0 + j, xr, v[j] * scale);
          }
        }
        if (!ok) break;
        if (C::kTail && S > 1) {
          __threadfence();
          named_bar_sync(1, 32 * C::kEpiWarps);
          if (warp == C::kEpiWarp0 && lane == 0) {
            const int last =
                arrive_counter_gpu(p.counters + w.tile) == static_cast<uint32_t>(S - 1);
            if (last) p.counters[w.tile] = 0u;
            *join = last;
          }
          named_bar_sync(1, 32 * C::kEpiWarps);
          if (!*join) continue;
          __threadfence();
          for (int j0 = 0; j0 < 32 && row0 + j0 < end && x < p.wide; j0 += 8) {
            // Rows past the end read the last one's again: the loads of eight
            // rows fly together.
            float s[8];
            const float* src[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              src[j] = part_at(0, min(row0 + j0 + j, end - 1), x);
              s[j] = __ldcg(src[j]);
            }
            for (int q = 1; q < S; ++q) {
              float t[8];
#pragma unroll
              for (int j = 0; j < 8; ++j) t[j] = __ldcg(src[j] + q * (C::kTileN * width));
#pragma unroll
              for (int j = 0; j < 8; ++j) s[j] += t[j];
            }
#pragma unroll
            for (int j = 0; j < 8; ++j)
              if (row0 + j0 + j < end && static_cast<uint32_t>(p.ids[row0 + j0 + j]) <
                                             static_cast<uint32_t>(p.adapters))
                keep(row0 + j0 + j, x, s[j]);
          }
        }
      } else if constexpr (C::kSplit) {
        // This warp's share (column blocks half, half + 2, ...) stays in
        // registers over the chunks.
        constexpr int kOwn = C::kTileN / 64;
        float m[kOwn][32];
#pragma unroll
        for (int q = 0; q < kOwn; ++q) grouped_zero(m[q]);
        // The adapter term comes before the last accumulators: while it waits
        // for H and for its own loads, the MMAs have those to fill.  (First of
        // all, the chunks of a long f32 contraction would wait for it: 256 rows
        // x 8192 x 8192, rank 16, 71 us instead of 64; 1444 x 1086 x 7085, rank
        // 128, 92 instead of 84.)
        const int before = max(0, chunks - C::kAccBufs);
        for (int c = 0; c <= chunks; ++c) {
          if constexpr (C::kMode == kAdapter) {
            if (c == before) {
#pragma unroll
              for (int q = 0; q < kOwn; ++q)
                add_adapter_terms<C::kTerms>(p, w, S, 4 * q, w.row0 + 32 * (half + 2 * q), end,
                                             x - lane, lane, inputs_ready, m[q]);
            }
          }
          if (c == chunks) break;
          if (!acc_ready()) {
            ok = false;
            break;
          }
#pragma unroll
          for (int q = 0; q < kOwn; ++q) {
            if (half + 2 * q < blocks)
              grouped_read<true>(
                  t_slab + static_cast<uint32_t>(acc * C::kTileN + 32 * (half + 2 * q)), m[q]);
          }
          hand_back();
        }
        if constexpr (C::kMode == kAdapter)
          if (!inputs_ready) {
            griddep_wait();
            inputs_ready = true;
          }
        if (!ok) break;
        if (C::kTail && S > 1) {
          // The last of the tile's pieces adds them all.
#pragma unroll
          for (int q = 0; q < kOwn; ++q)
            publish(32 * (half + 2 * q), w.rows - 32 * (half + 2 * q), m[q]);
          if (!joined()) continue;
#pragma unroll
          for (int q = 0; q < kOwn; ++q)
            if (half + 2 * q < blocks) collect(32 * (half + 2 * q), m[q]);
        }
#pragma unroll
        for (int q = 0; q < kOwn; ++q) {
          const int row = w.row0 + 32 * (half + 2 * q);
          if (row < end) {
            grouped_epilogue(p.epi, b, m[q]);
            grouped_store<C>(p, d0, row, end, x, m[q]);
          }
        }
      } else {
        constexpr int kOwn = C::kTileN / 64;
        if constexpr (C::kBf16Out) {
          // One accumulator: each block goes out as it is read, through two
          // boxes in turn.  box_lead (one thread of the box's two warps)
          // issues the stores and, before each meeting of the two warps, waits
          // until the store before the last has read its box.
          if (chunks > 0 && !acc_ready()) break;
          float bias[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int xb = x - lane + 8 * i + (lane >> 2);
            bias[i] = epi_uses_bias(p.epi.op) && xb < p.wide
                          ? p.epi.bias[static_cast<int64_t>(w.g) * p.wide + xb]
                          : 0.0f;
          }
          if (C::kTail && S > 1) {
            const bool mark = C::kExt && marked[count & 15] == count + 1;
            for (int q = half; q < blocks; q += 2) {
              float v[32];
              if (chunks > 0)
                grouped_read<false>(t_slab + static_cast<uint32_t>(acc * C::kTileN + 32 * q), v);
              else
                grouped_zero(v);
              if (mark) add_marked_terms(p, w.row0 + 32 * q, end, x, v);
              publish(32 * q, w.rows - 32 * q, v);
            }
            if (chunks > 0) hand_back();
            if (!joined()) continue;
            for (int q = half; q < blocks; q += 2) {
              float v[32];
              collect(32 * q, v);
              grouped_epilogue(p.epi, b, v);
              grouped_store<C>(p, d0, w.row0 + 32 * q, end, x, v);
            }
            continue;
          }
          if (C::kExt && marked[count & 15] == count + 1) {
            for (int q = half; q < blocks; q += 2) {
              const int row = w.row0 + 32 * q;
              float v[32];
              grouped_read<false>(t_slab + static_cast<uint32_t>(acc * C::kTileN + 32 * q), v);
              add_marked_terms(p, row, end, x, v);
              grouped_epilogue(p.epi, b, v);
              grouped_store<C>(p, d0, row, end, x, v);
            }
            hand_back();
            continue;
          }
          const int x0 = x - lane - 32 * (slab & 1);   // first element of the box
          for (int q = half; q < blocks; q += 2) {
            const int row = w.row0 + 32 * q;
            const uint32_t at = stg + 4096u * flip;
            flip ^= 1u;
            grouped_stage_bf16(at, lane, slab,
                               t_slab + static_cast<uint32_t>(acc * C::kTileN + 32 * q), chunks > 0,
                               p.epi, bias);
            fence_proxy_async_smem();
            if (box_lead) bulk_wait_group_read0();
            named_bar_sync(2 + box, 64);
            if ((C::kColMn || row + 32 <= end) && x0 + 64 <= p.wide) {
              if (box_lead) {
                tma_store_3d_hint(&tmD, at, x0, row, C::kColMn ? w.g : 0, pol_d);
                bulk_commit_group();
              }
            } else {
              const int r0 = 16 * (slab & 1);
              grouped_unstage<C>(p, d0, at, lane, r0, r0 + 16, row, end, x0);
            }
          }
          if (chunks > 0) hand_back();
        } else {
          // One block of 32 accumulator columns to D.
          auto finish = [&](int q, float (&v)[32]) {
            const int row = w.row0 + 32 * q;
            grouped_epilogue(p.epi, b, v);
            if (lane == 0) bulk_wait_group_read0();
            __syncwarp();
            grouped_stage_f32(stg, lane, v);
            if ((C::kColMn || row + 32 <= end) && x - lane + 32 <= p.wide) {
              fence_proxy_async_smem();
              __syncwarp();
              if (lane == 0) {
                if (C::kAdd && p.add)   // (one addend for each element: the same bits every time)
                  tma_reduce_add_3d(&tmD, stg, x, row, 0);
                else
                  tma_store_3d_hint(&tmD, stg, x, row, C::kColMn ? w.g : 0, pol_d);
                bulk_commit_group();
              }
            } else {
              __syncwarp();
              grouped_unstage<C>(p, d0, stg, lane, 0, 32, row, end, x - lane);
            }
          };
          // The warp's share of the tile stays in registers over the chunks.
          float m[kOwn][32];
#pragma unroll
          for (int q = 0; q < kOwn; ++q) grouped_zero(m[q]);
          for (int c = 0; c < chunks; ++c) {
            if (!acc_ready()) {
              ok = false;
              break;
            }
#pragma unroll
            for (int q = 0; q < kOwn; ++q)
              if (half + 2 * q < blocks)
                grouped_read<true>(
                    t_slab + static_cast<uint32_t>(acc * C::kTileN + 32 * (half + 2 * q)), m[q]);
            hand_back();
          }
          if (!ok) break;
          if (C::kExt && marked[count & 15] == count + 1) {
#pragma unroll
            for (int q = 0; q < kOwn; ++q)
              add_marked_terms(p, w.row0 + 32 * (half + 2 * q), end, x, m[q]);
          }
          if (C::kTail && S > 1) {
#pragma unroll
            for (int q = 0; q < kOwn; ++q)
              publish(32 * (half + 2 * q), w.rows - 32 * (half + 2 * q), m[q]);
            if (!joined()) continue;
#pragma unroll
            for (int q = 0; q < kOwn; ++q)
              if (half + 2 * q < blocks) collect(32 * (half + 2 * q), m[q]);
          }
#pragma unroll
          for (int q = 0; q < kOwn; ++q)
            if (half + 2 * q < blocks) finish(half + 2 * q, m[q]);
        }
      }
    }
    // Stores in flight finish before the block's shared memory goes away.
    if constexpr (C::kStaged)
      if (lane == 0) bulk_wait_group0();
  }

  tc_fence_before_sync();
  __syncthreads();
  if constexpr (C::kCtaGroup == 2) cluster_sync();
  if (warp == 1) {
    tc_fence_after_sync();
    tmem_dealloc<C::kCtaGroup>(tmem_base, C::TMEM_COLS);
  }
}

}  // namespace tg
