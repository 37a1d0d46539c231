// Products over a vocabulary whose logits are never stored: a persistent,
// warp-specialised tcgen05 kernel for z = scale * A * B^T with two epilogues.
//
//   kXentLoss   per row and tile of columns: the maximum m and the sum of
//               exp(z - m) of a softmax in one pass, and the target's logit
//   kXentGrad   dz = w * (exp(z - lse) - [column is the target]), w = grad *
//               scale, as bf16 (kXentGradTwo: as two bf16 terms), which the
//               products of both gradients read
//
// Rows of A (tokens) fill the MMA's M and so the lanes of the accumulator: a
// thread of the epilogue owns one row's columns, and neither the maximum nor
// the sum crosses lanes.  The columns of a tile are a runtime value (steps of
// 16, kXentGrad 64): the launch spreads the vocabulary evenly over the SMs.
//
// Up to 128 rows run as single CTAs that load only the rows there are and are
// bound by reading B; more rows as CTA pairs (256 x 256 tiles), bound by the
// tensor pipe: per tile and SM the epilogue takes 128 x 256 exponentials (about
// 2000 cycles beside the 34000 of 4096 terms) under the next tile's MMAs.
//
// Roles: warp 0 TMA producer, warp 1 TMEM allocator and MMA issuer, warps 2..9
// epilogue.  Every wait is bounded.
#pragma once

#include <cstdint>
#include <type_traits>
#include <cuda.h>

#include "tg_ptx.cuh"

namespace tg {

enum : int { kXentLoss = 0, kXentGrad = 1, kXentGradTwo = 2 };

enum : uint32_t {
  kSiteXentEmpty = 51,
  kSiteXentFull = 52,
  kSiteXentAccEmpty = 53,
  kSiteXentAccFull = 54,
};

struct XentArgs {
  int M, N;            // rows; columns of this launch
  int padded;          // kXentGrad: rows of dz and of the copy (zeros from M on)
  int col0, vocab;     // vocabulary index of its first column; size of the vocabulary
  int num_k_blocks;    // stages of 64 terms
  int num_m_tiles;     // of kCtaGroup * 128 rows
  int num_n_tiles;     // of bn columns
  int bn;
  int raster_group;    // m-tiles per band of the tile order
  int a_box;           // rows of A per load (128; few rows: theirs, rounded up to 8)
  int stages, a_bytes, b_bytes;   // the ring: slots, bytes of A and of B in each
  float scale;
  const int* targets;  // [M]
  // kXentLoss
  float scale2;        // scale * log2(e)
  float2* parts;       // [2 * num_n_tiles][M]: largest accumulator m, sum of exp(scale (a - m))
  float* target_z;     // [M] accumulator of the target, where that is among the columns
  // kXentGrad
  const float* lse;    // [M]
  const float* loss;   // [M], or null: the target's dz from z and lse
  const float* grad;   // [M], or null for 1
  // Where not null, the kernel also copies A's rows there (`terms` times in a row,
  // ld_copy apart), zeros for rows without a target: dz is 0 in those, but 0 times
  // what padding holds may be NaN, so the product for dB reads the copy.
  const uint16_t* A;
  int64_t lda, ld_copy;
  uint16_t* copy;
  int K;
  uint32_t* status;
  uint64_t timeout_ns;
};

template <int kCtaGroup_, int kMode_>
struct XentCfg {
  static constexpr int kCtaGroup = kCtaGroup_;
  static constexpr int kMode = kMode_;
  static constexpr bool kTwo = kMode == kXentGradTwo;
  static constexpr int BN = 256;                       // most columns of a tile
  // The ring, 192 KB.  CTA pairs: 6 slots of 128 rows of A and of B.  Few rows: as
  // many as fit of what they load, so that 6 MB and more are on their way to the SMs
  // (one token x 32000 x 4096 with 4 slots of 128 + 256 rows: 47.6 us).  The MMA
  // reads 128 rows of A all the same: what follows them is a later slot or B, and
  // lands in lanes that no row has.
  static constexpr int RING_BYTES = 192 * 1024;
  static constexpr int kStages = kCtaGroup == 2 ? 6 : 16;
  static constexpr int OFF_STG = RING_BYTES;
  static constexpr int kEpiWarps = 8;
  static constexpr int kAccBufs = 2;
  static constexpr int kStgBytes = kMode == kXentLoss ? 0 : 4096;   // a box of 32 rows x 64 bf16
  static constexpr int OFF_BAR = OFF_STG + kEpiWarps * kStgBytes;
  static constexpr int NUM_BARS = 2 * kStages + 2 * kAccBufs + 1;
  static constexpr int OFF_MISC = OFF_BAR + NUM_BARS * 8;
  static constexpr int SMEM_BYTES = OFF_MISC + 16 + 1024;
  static constexpr int kThreads = 64 + 32 * kEpiWarps;
  // The tensor cores truncate each time they add to an accumulator: z comes out
  // too small by 1e-6 of itself for each 1000 terms.  A loss between 0.1 and 1 of
  // a target far above the others takes ten times that on, f32 gradients take it on as
  // well, and bf16 ones where they are a rest: the target's dz, p - 1, takes on whatever
  // sets this z apart from the one that lse has seen.  So long contractions are cut into
  // chunks of kChunk stages, the same in every mode, that are added in registers with
  // rounding to nearest.  Few rows wait for
  // HBM, unless the vocabulary is small (83 x 2282 x 3734 with chunks of 256, 512 and
  // 1024 terms: 31.1, 28.9 and 26.9 us; error of 64 losses over 32000 x 2048 1.4e-7 and
  // 3.1e-7 with 256 and 512).  For pairs a chunk costs (1024 x 48640 x 4096, chunks of
  // 4096, 2048, 1024 and 512 terms: 217, 220, 226 and 234 us, error of the loss 2.8e-6,
  // 1.4e-6, 6e-7 and 3e-7).
  static constexpr int kChunk = kCtaGroup == 1 ? 4 : 16;
  static_assert(SMEM_BYTES <= 227 * 1024, "shared memory per CTA");
};

// Tile t: bands of `group` m-tiles, down the band before the next n-tile; every
// other band walks the n-tiles backwards, so that it starts on the panels of B
// the one before ended on.
__device__ __forceinline__ void xent_tile(const XentArgs& p, int t, int& tm, int& tn) {
  const int per_band = p.raster_group * p.num_n_tiles;
  const int band = t / per_band;
  const int first = band * p.raster_group;
  const int rows = min(p.num_m_tiles - first, p.raster_group);
  const int r = t - band * per_band;
  tm = first + r % rows;
  tn = r / rows;
  if (band & 1) tn = p.num_n_tiles - 1 - tn;
}

__device__ __forceinline__ float exp2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// What rounding x to r left (nothing where r is infinite or NaN: it is all there).
__device__ __forceinline__ float rest_of_bf16(float x, float r) {
  return fabsf(r) < __uint_as_float(0x7F800000u) ? x - r : 0.0f;
}

// kN accumulator columns of this lane's row, to z or added to it, 32 at a time.
template <bool kAdd, int kN>
__device__ __forceinline__ void xent_read(uint32_t taddr, float (&z)[kN]) {
#pragma unroll
  for (int e0 = 0; e0 < kN; e0 += 32) {
    uint32_t v[32];
    tmem_ld_32x32b_x16(taddr + e0, v);
    tmem_ld_32x32b_x16(taddr + e0 + 16, v + 16);
    tmem_ld_wait();
#pragma unroll
    for (int e = 0; e < 32; ++e) {
      const float x = __uint_as_float(v[e]);
      z[e0 + e] = kAdd ? z[e0 + e] + x : x;
    }
  }
}

// Rows warp, warp + warps, ... of A to the copy: whole 16-byte pieces, four a lane in
// flight, then the last K % 8 values.
template <int kTerms>
__device__ __forceinline__ void copy_learned_rows(const XentArgs& p, int warp, int warps,
                                                  int lane) {
  const int whole = p.K / 8;
#pragma unroll 1
  for (int i = warp; i < p.padded; i += warps) {
    const int t = i < p.M ? p.targets[i] : -1;
    const bool learned = t >= 0 && t < p.vocab;
    const uint16_t* s = p.A + i * p.lda;
    uint16_t* d = p.copy + static_cast<int64_t>(i) * kTerms * p.ld_copy;
#pragma unroll 1
    for (int k0 = lane; k0 < whole; k0 += 128) {
      uint4 v[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        v[u] = make_uint4(0u, 0u, 0u, 0u);
        if (learned && k0 + 32 * u < whole) v[u] = reinterpret_cast<const uint4*>(s)[k0 + 32 * u];
      }
#pragma unroll
      for (int u = 0; u < 4; ++u)
        if (k0 + 32 * u < whole)
          for (int h = 0; h < kTerms; ++h)
            reinterpret_cast<uint4*>(d + h * p.ld_copy)[k0 + 32 * u] = v[u];
    }
    const int k = whole * 8 + lane;
    if (lane < 8 && k < p.K)
      for (int h = 0; h < kTerms; ++h) d[h * p.ld_copy + k] = learned ? s[k] : 0;
  }
}

template <class C>
__global__ void __launch_bounds__(C::kThreads, 1)
    xent_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                const __grid_constant__ CUtensorMap tmD, const __grid_constant__ CUtensorMap tmD2,
                const XentArgs p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint64_t* full_bar = reinterpret_cast<uint64_t*>(smem + C::OFF_BAR);   // [kStages] TMA -> MMA
  uint64_t* empty_bar = full_bar + C::kStages;       // [kStages] MMA -> TMA
  uint64_t* accf_bar = empty_bar + C::kStages;       // [2] MMA -> epilogue
  uint64_t* acce_bar = accf_bar + C::kAccBufs;       // [2] epilogue -> MMA
  uint64_t* drain_bar = acce_bar + C::kAccBufs;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::OFF_MISC);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::OFF_MISC + 4);

  const int warp = threadIdx.x >> 5;
  const uint32_t lane = threadIdx.x & 31;
  const uint32_t rank = C::kCtaGroup == 2 ? cluster_ctarank() : 0u;
  const bool leader = rank == 0;

  const int stages = C::kCtaGroup == 2 ? C::kStages : p.stages;
  const uint32_t a_bytes = C::kCtaGroup == 2 ? 128u * 128u : static_cast<uint32_t>(p.a_bytes);
  const uint32_t b_bytes = C::kCtaGroup == 2 ? 128u * 128u : static_cast<uint32_t>(p.b_bytes);
  const uint32_t ring_a = smem_addr(smem);
  const uint32_t ring_b = ring_a + static_cast<uint32_t>(stages) * a_bytes;

  if (threadIdx.x == 0) {
    for (int s = 0; s < stages; ++s) {
      mbar_init(&full_bar[s], 1);
      mbar_init(&empty_bar[s], 1);
    }
    for (int b = 0; b < C::kAccBufs; ++b) {
      mbar_init(&accf_bar[b], 1);
      mbar_init(&acce_bar[b], C::kEpiWarps * C::kCtaGroup);
    }
    mbar_init(drain_bar, 1);
    *abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == 0 && lane == 0) {
    prefetch_tensormap(&tmA);
    prefetch_tensormap(&tmB);
    if constexpr (C::kMode != kXentLoss) prefetch_tensormap(&tmD);
    if constexpr (C::kTwo) prefetch_tensormap(&tmD2);
  }
  if (warp == 1) {
    tmem_alloc<C::kCtaGroup>(tmem_slot, 512);
    tmem_relinquish<C::kCtaGroup>();
  }
  tc_fence_before_sync();
  __syncthreads();
  if constexpr (C::kCtaGroup == 2) cluster_sync();
  tc_fence_after_sync();
  const uint32_t tmem_base = *tmem_slot;
  // What is above is on chip and may overlap the kernel before in the stream.
  griddep_wait();

  const WaitGuard guard{p.status, abort_flag, p.timeout_ns};
  const int unit = blockIdx.x / C::kCtaGroup;
  const int num_units = gridDim.x / C::kCtaGroup;
  const int num_tiles = p.num_m_tiles * p.num_n_tiles;
  const int nk = p.num_k_blocks;
  const int chunks = (nk + C::kChunk - 1) / C::kChunk;
  auto chunk_end = [&](int c) { return static_cast<int>(static_cast<int64_t>(nk) * (c + 1) / chunks); };

  if (warp == 0) {
    // ------------------------------------------------------------ producer
    if (lane == 0) {
      const uint64_t pol = policy_evict_last();
      // (The loss of few rows reads B once and for all.)
      const uint64_t pol_b =
          C::kCtaGroup == 1 && C::kMode == kXentLoss ? policy_evict_first() : pol;
      const uint32_t empty0 = smem_addr(&empty_bar[0]);
      const uint32_t full0 = smem_addr(&full_bar[0]);
      const uint32_t full_dst0 = C::kCtaGroup == 2 ? map_to_cta(full0, 0u) : full0;
      const int b_box = p.bn / C::kCtaGroup;
      const uint32_t bytes = static_cast<uint32_t>((p.a_box + b_box) * 128 * C::kCtaGroup);
      int stage = 0;
      uint32_t phase = 0;
      uint32_t issued = 0, issued_parity = 0;
      bool ok = true;
      for (int t = unit, wave = 0; ok && t < num_tiles; t += num_units, ++wave) {
        int tm, tn;
        xent_tile(p, t, tm, tn);
        const int a_row = (tm * C::kCtaGroup + static_cast<int>(rank)) * 128;
        const int b_row = tn * p.bn + static_cast<int>(rank) * b_box;
        const bool back = wave & 1;   // the slices read last are those L2 still holds
        for (int j = 0; j < nk; ++j) {
          if (!mbar_try_wait(empty0 + 8u * stage, phase ^ 1u) &&
              !mbar_wait(&empty_bar[stage], phase ^ 1u, guard, kSiteXentEmpty)) {
            ok = false;
            break;
          }
          const int kx = 64 * (back ? nk - 1 - j : j);
          const uint32_t fb = full_dst0 + 8u * stage;
          if (leader) mbar_arrive_expect_tx(&full_bar[stage], bytes);
          if constexpr (C::kCtaGroup == 1) {
            tma_load_2d(ring_a + stage * a_bytes, &tmA, fb, kx, a_row, pol);
            tma_load_2d(ring_b + stage * b_bytes, &tmB, fb, kx, b_row, pol_b);
          } else {
            tma_load_2d_pair(ring_a + stage * a_bytes, &tmA, fb, kx, a_row, pol);
            tma_load_2d_pair(ring_b + stage * b_bytes, &tmB, fb, kx, b_row, pol);
          }
          issued |= 1u << stage;
          issued_parity = (issued_parity & ~(1u << stage)) | (phase << stage);
          if (++stage == stages) {
            stage = 0;
            phase ^= 1u;
          }
        }
      }
      griddep_launch_dependents();
      if (!ok && leader) {
        // Gave up: the loads already issued land before the CTA exits.
        for (int s = 0; s < stages; ++s)
          if (issued & (1u << s))
            mbar_wait_drain(&full_bar[s], (issued_parity >> s) & 1u, p.timeout_ns);
      }
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer
    if (lane == 0 && leader) {
      const uint32_t acce0 = smem_addr(&acce_bar[0]);
      const uint32_t full0 = smem_addr(&full_bar[0]);
      const uint64_t adesc0 =
          make_smem_desc(ring_a, 16, 1024, kDescSwizzle128B);
      const uint64_t bdesc0 =
          make_smem_desc(ring_b, 16, 1024, kDescSwizzle128B);
      const uint32_t idesc = idesc_bf16_f32(128 * C::kCtaGroup, static_cast<uint32_t>(p.bn));
      int stage = 0;
      uint32_t phase = 0;
      int acc = 0;
      uint32_t acc_phase = 0;
      bool ok = true;
      bool ready = false;   // full barrier of `stage` already seen complete
      for (int t = unit; ok && t < num_tiles; t += num_units) {
        int j = 0;
        for (int c = 0; ok && c < chunks; ++c) {
          if (!mbar_try_wait(acce0 + 8u * acc, acc_phase ^ 1u) &&
              !mbar_wait(&acce_bar[acc], acc_phase ^ 1u, guard, kSiteXentAccEmpty)) {
            ok = false;
            break;
          }
          tc_fence_after_sync();
          const uint32_t d_tmem = tmem_base + static_cast<uint32_t>(acc * C::BN);
          const int end = chunk_end(c);
          bool add = false;
          for (; j < end; ++j) {
            if (!ready && !mbar_try_wait(full0 + 8u * stage, phase) &&
                !mbar_wait(&full_bar[stage], phase, guard, kSiteXentFull)) {
              ok = false;
              break;
            }
            tc_fence_after_sync();
            const int ns = stage + 1 == stages ? 0 : stage + 1;
            const uint32_t nph = stage + 1 == stages ? phase ^ 1u : phase;
            const uint64_t ad = adesc0 + static_cast<uint64_t>(stage * (a_bytes >> 4));
            const uint64_t bd = bdesc0 + static_cast<uint64_t>(stage * (b_bytes >> 4));
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              mma_bf16<C::kCtaGroup>(d_tmem, ad + 2 * k, bd + 2 * k, idesc, add || k != 0);
              if (k == 0) ready = mbar_try_wait(full0 + 8u * ns, nph);
            }
            add = true;
            if constexpr (C::kCtaGroup == 1)
              mma_commit(&empty_bar[stage]);
            else
              mma_commit_pair(&empty_bar[stage], 3);
            stage = ns;
            phase = nph;
          }
          if (!ok) break;
          if constexpr (C::kCtaGroup == 1)
            mma_commit(&accf_bar[acc]);
          else
            mma_commit_pair(&accf_bar[acc], 3);
          if (++acc == C::kAccBufs) {
            acc = 0;
            acc_phase ^= 1u;
          }
        }
      }
      if (!ok || *abort_flag) {
        // Gave up: every MMA issued finishes with shared and tensor memory.
        if constexpr (C::kCtaGroup == 1)
          mma_commit(drain_bar);
        else
          mma_commit_pair(drain_bar, 1);
        mbar_wait_drain(drain_bar, 0, p.timeout_ns);
      }
    }
  } else {
    // ------------------------------------------------------------ epilogue
    const int slab = warp & 3;              // TMEM lanes 32 * slab ..
    const int half = (warp - 2) >> 2;       // column blocks half, half + 2, ...
    const uint32_t t_slab = tmem_base + (static_cast<uint32_t>(slab * 32) << 16);
    const uint32_t stg =
        smem_addr(smem + C::OFF_STG) + static_cast<uint32_t>(warp - 2) * C::kStgBytes;
    const uint64_t pol_d = policy_evict_last();   // the gradients' products read dz next
    uint32_t acce_dst = smem_addr(&acce_bar[0]);
    if constexpr (C::kCtaGroup == 2) acce_dst = map_to_cta(acce_dst, 0u);
    int acc = 0;
    uint32_t acc_phase = 0;
    auto acc_ready = [&]() -> bool {
      int got = 1;
      if (lane == 0)
        got = mbar_wait(&accf_bar[acc], acc_phase, guard, kSiteXentAccFull) ? 1 : 0;
      got = __shfl_sync(0xFFFFFFFFu, got, 0);
      tc_fence_after_sync();
      return got != 0;
    };
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
    if constexpr (C::kMode != kXentLoss) {
      // The copy, while the first tile's product is under way.
      if (p.copy != nullptr)
        copy_learned_rows<C::kTwo ? 2 : 1>(p, static_cast<int>(blockIdx.x) * C::kEpiWarps + warp - 2,
                                           static_cast<int>(gridDim.x) * C::kEpiWarps,
                                           static_cast<int>(lane));
    }
    int last_tm = -1;
    int target = -1;                 // column of this launch, or negative
    bool learned = false;            // the row has a target in the vocabulary
    float lse = 0.0f, weight = 0.0f, own_dz = 0.0f;
    bool ok = true;
    for (int t = unit; ok && t < num_tiles; t += num_units) {
      int tm, tn;
      xent_tile(p, t, tm, tn);
      const int row0 = (tm * C::kCtaGroup + static_cast<int>(rank)) * 128 + slab * 32;
      const int row = row0 + static_cast<int>(lane);
      const int tile0 = tn * p.bn;
      const int cols = min(p.bn, p.N - tile0);   // of the tile's that there are
      if (tm != last_tm) {
        last_tm = tm;
        const int id = row < p.M ? p.targets[row] : -1;
        learned = id >= 0 && id < p.vocab;
        target = learned ? id - p.col0 : -1;
        if constexpr (C::kMode != kXentLoss) {
          lse = learned ? p.lse[row] : 0.0f;
          weight = learned ? (p.grad ? p.grad[row] : 1.0f) * p.scale : 0.0f;
          if (p.loss != nullptr) own_dz = learned ? expm1f(-p.loss[row]) : 0.0f;
        }
      }
      // The target's place in the tile, if this warp has it (else negative).
      const int here = target - tile0;
      if constexpr (C::kMode == kXentLoss) {
        // The warp's whole share stays in registers: the maximum and the sum are
        // two passes over them.  (Short contractions are bound by these instructions: the
        // first chunk not added to zeros, and four maxima, 20000 x 10000 x 64 113 -> 97 us.)
        float v[4][32];
        auto read = [&](auto add) {
          if (!acc_ready()) return false;
          const uint32_t t_row = t_slab + static_cast<uint32_t>(acc * C::BN);
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (32 * (half + 2 * i) < cols && row0 < p.M)
              xent_read<decltype(add)::value>(t_row + 32 * (half + 2 * i), v[i]);
          hand_back();
          return true;
        };
        ok = read(std::false_type{});
        for (int c = 1; ok && c < chunks; ++c) ok = read(std::true_type{});
        if (!ok) break;
        if (row0 >= p.M) continue;   // (lanes that no row has)
        const float none = __uint_as_float(0xFF800000u);   // -inf
        float most[4] = {none, none, none, none};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int left = cols - 32 * (half + 2 * i);
          if (left <= 0) continue;
          if (left < 32) {
#pragma unroll
            for (int e = 0; e < 32; ++e)
              if (e >= left) v[i][e] = none;
          }
#pragma unroll
          for (int e = 0; e < 32; ++e) most[e & 3] = fmaxf(most[e & 3], v[i][e]);
        }
        const float m = fmaxf(fmaxf(most[0], most[1]), fmaxf(most[2], most[3]));
        // (An infinite maximum is no reference.)  The difference first: it is exact
        // for the logits that count, whatever their size.
        const float r = fabsf(m) < __uint_as_float(0x7F800000u) ? m : 0.0f;
        // (In pairs: a sum that holds the maximum's 1 rounds the rest each time it is added
        // to.  One token's loss of 0.023 over 32000 x 4096 one after the other 1.2e-5 of
        // itself off, in pairs 6.4e-6; lse minus the target's logit in 32 bits 2.2e-5.)
        float s[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          if (32 * (half + 2 * i) >= cols) continue;
          float u[8];
#pragma unroll
          for (int e = 0; e < 32; e += 4) {
            float x[4];
#pragma unroll
            for (int d = 0; d < 4; ++d) x[d] = exp2_approx((v[i][e + d] - r) * p.scale2);
            u[e / 4] = (x[0] + x[1]) + (x[2] + x[3]);
          }
          s[i] = ((u[0] + u[1]) + (u[2] + u[3])) + ((u[4] + u[5]) + (u[6] + u[7]));
        }
        if (row < p.M) {
          p.parts[static_cast<int64_t>(2 * tn + half) * p.M + row] =
              make_float2(m, (s[0] + s[1]) + (s[2] + s[3]));
          if (here >= 0 && here < cols && ((here >> 5) & 1) == half) {
            float z = 0.0f;
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
              for (int e = 0; e < 32; ++e)
                if (here == 32 * (half + 2 * i) + e) z = v[i][e];
            p.target_z[row] = z;
          }
        }
      } else {
        // dz of a box of 64 columns, from its accumulators, in place.
        auto gradient = [&](float (&z)[64], int box0) {
#pragma unroll
          for (int e = 0; e < 64; ++e) z[e] = fmaf(z[e], p.scale, -lse);
          // The target's p - 1 without the subtraction: where p is near 1 the digits that
          // count are those of the exponent, and the loss has more of them than z - lse,
          // which two rounded numbers of its size leave.
          const int own = here - box0;
          if (own >= 0 && own < 64) {
            float x = 0.0f;
#pragma unroll
            for (int e = 0; e < 64; ++e)
              if (own == e) x = z[e];
            own_dz = p.loss != nullptr ? own_dz : expm1f(x);
          }
#pragma unroll
          for (int e = 0; e < 64; ++e) {
            const float pe = exp2_approx(z[e] * 1.4426950408889634f);
            z[e] = own == e ? own_dz : pe;
          }
#pragma unroll
          for (int e = 0; e < 64; ++e) z[e] = learned ? weight * z[e] : 0.0f;
          if (box0 + 64 > cols) {
#pragma unroll
            for (int e = 0; e < 64; ++e)
              if (box0 + e >= cols) z[e] = 0.0f;
          }
        };
        // Stores the box as bf16 (what rounding leaves stays in z).
        auto store = [&](float (&z)[64], int box0, const CUtensorMap* map) {
          if (lane == 0) bulk_wait_group_read0();
          __syncwarp();
          const uint32_t sw = lane & 7u;
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            uint32_t w[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              float& lo = z[8 * j + 2 * e];
              float& hi = z[8 * j + 2 * e + 1];
              w[e] = pack_bf16x2(lo, hi);
              if constexpr (C::kTwo) {
                lo = rest_of_bf16(lo, __uint_as_float(w[e] << 16));
                hi = rest_of_bf16(hi, __uint_as_float(w[e] & 0xFFFF0000u));
              }
            }
            st_shared_v4(stg + lane * 128u + ((static_cast<uint32_t>(j) ^ sw) << 4), w[0], w[1],
                         w[2], w[3]);
          }
          fence_proxy_async_smem();
          __syncwarp();
          // Rows past the last are clipped; dz has whole boxes of columns.
          if (lane == 0) {
            tma_store_2d_hint(map, stg, tile0 + box0, row0, pol_d);
            bulk_commit_group();
          }
        };
        // The warp's share of the tile stays in registers while the chunks are added (with
        // them, 4096 x 32000 x 4096 pieces in bf16 547 -> 579 us, 1% of a step; 64 x 32000 x 2048 1.5%).
        const int boxes = (cols + 63) / 64;
        float z[2][64];
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int e = 0; e < 64; ++e) z[i][e] = 0.0f;
        for (int c = 0; c < chunks; ++c) {
          if (!acc_ready()) {
            ok = false;
            break;
          }
          const uint32_t t_row = t_slab + static_cast<uint32_t>(acc * C::BN);
#pragma unroll
          for (int i = 0; i < 2; ++i)
            if (half + 2 * i < boxes) xent_read<true>(t_row + 64 * (half + 2 * i), z[i]);
          hand_back();
        }
        if (!ok) break;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int b = half + 2 * i;
          if (b >= boxes) continue;
          gradient(z[i], 64 * b);
          if (row0 >= p.padded) continue;
          store(z[i], 64 * b, &tmD);
          if constexpr (C::kTwo) store(z[i], 64 * b, &tmD2);
        }
      }
    }
    // Stores in flight finish before the block's shared memory goes away.
    if constexpr (C::kMode != kXentLoss)
      if (lane == 0) bulk_wait_group0();
  }

  tc_fence_before_sync();
  __syncthreads();
  if constexpr (C::kCtaGroup == 2) cluster_sync();
  if (warp == 1) {
    tc_fence_after_sync();
    tmem_dealloc<C::kCtaGroup>(tmem_base, 512);
  }
}

}  // namespace tg
