// Host launch of gemm_grouped_kernel<Cfg>: tensor maps, grid, cluster
// attribute and shared memory opt-in (once per device and configuration).
#pragma once

#include "gemm_launch.cuh"
#include "grouped_kernel.cuh"

namespace tg {

// The two streamed operands.  `wide` spans D's contiguous axis: the weights
// [slices][rows][...] (forward, dgrad, adapters) or A [rows of all groups]
// (wgrad).  `cols` spans its rows.  k: extent of the contraction index.
struct GroupedOperands {
  const void* wide;
  int64_t wide_ld, wide_rows, wide_slices, wide_slice_stride;
  const void* cols;
  int64_t cols_ld;
  int64_t k;
  const void* up;        // adapters: [adapters][wide][rank]
  int64_t up_ld, up_slice_stride, up_slices, up_rank;
};

// Most rows, columns and contraction terms.  The kernels count in 32 bits and go
// past an extent by less than this: whole tiles, boxes and a K step of a cluster
// (256 rows + 255, 128, 8 CTAs x 256).  2^31 - 1 rows in one group wrapped to no
// tile at all.
constexpr int64_t kGroupedMaxExtent = (int64_t{1} << 31) - 4096;

inline GroupedArgs grouped_args(DeviceCtx* ctx) {
  GroupedArgs a{};
  a.status = ctx->status;
  a.timeout_ns = wait_timeout_ns();
  a.groups = 1;
  a.epi = Epi{kEpiNone, 0.0f, 0.0f, nullptr};
  return a;
}

// The forward product with few rows per group on average: single CTAs with
// 64-column tiles, a deep ring of weight boxes and a split contraction; else CTA
// pairs with tiles of 256 x 256 (so the gradients always).  Groups of equal size,
// 64 x 2048 x 4096, 32 rows each: 174 us against 179 for pairs, 96 rows 277
// against 187; 5 rows in 10 groups x 896 x 2816 14 against 21; 32 rows in 8
// groups x 1024 x 1024 10.1 against 8.7.  (The sizes are the device's, so uneven
// groups go by their mean.)
inline bool grouped_few_rows(int64_t M, int64_t groups) { return M <= 48 * groups; }

// Of those, rows picked by index are gathered by the product's own loads (four
// rows an operation, which a short tile hides behind its weights), else copied
// together first.  64 groups x 2048 x 4096, 16 rows each: 173 us against 177,
// 32 rows 223 against 181; 5 rows in 10 groups x 896 x 2816 12.0 against 13.2.
inline bool grouped_gathers(int64_t M, int64_t groups) { return M <= 16 * groups; }

// CTA pairs with a split last wave: a contraction of at least 96 stages and
// tiles for less than two waves (`tiles`: at least so many, sizes of groups
// being the device's).  22374 rows in 2 groups x 896 x 768, wgrad (24 tiles of
// 175 stages) 62 -> 40 us; 14613 rows x 640 x 3456, forward (174 tiles of 54)
// 59 -> 62 us.
inline bool grouped_tail_pays(int64_t tiles, int64_t k_blocks, DeviceCtx* ctx) {
  return k_blocks >= 96 && tiles < ctx->num_sms;
}

template <class C>
int launch_grouped(const GroupedOperands& operands, const GroupedArgs& args, cudaStream_t stream,
                   DeviceCtx* ctx) {
  GroupedOperands o = operands;
  if (o.k == 0) {
    // Nothing is read (the caller may have passed null operands): any valid
    // map does.
    o.wide = o.cols = args.D;
    o.wide_ld = o.cols_ld = o.wide_slice_stride = 8;
    o.wide_rows = o.wide_slices = 1;
  }
  static std::atomic<int> prepared[64];
  auto kern = gemm_grouped_kernel<C>;
  std::atomic<int>& slot = prepared[ctx->device];
  int units = slot.load(std::memory_order_acquire);
  cudaLaunchConfig_t cfg{};
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = C::kCtaGroup;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.blockDim = dim3(C::kThreads, 1, 1);
  cfg.dynamicSmemBytes = C::SMEM_BYTES;
  cfg.attrs = attr;
  if (units == 0) {
    cudaError_t e =
        cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM_BYTES);
    if (e != cudaSuccess) return cuda_fail(e);
    units = ctx->num_sms / C::kCtaGroup;
    if constexpr (C::kCtaGroup == 2) {
      cfg.gridDim = dim3(static_cast<unsigned>(2 * units), 1, 1);
      cudaLaunchConfig_t q = cfg;
      q.attrs = attr + 1;
      q.numAttrs = 1;
      int clusters = 0;
      e = cudaOccupancyMaxActiveClusters(&clusters, kern, &q);
      if (e != cudaSuccess) return cuda_fail(e);
      if (clusters > 0 && clusters < units) units = clusters;
    }
    if (units < 1) units = 1;
    slot.store(units, std::memory_order_release);
  }
  GroupedArgs a = args;
  a.num_wide_tiles = ceil_div_i(a.wide, 128 * C::kCtaGroup);
  // The tail split's scratch: [tile][piece][CTA] partial tiles, a counter for
  // each tile and CTA.
  float* part = nullptr;
  uint32_t* counters = nullptr;
  if (tail_scratch(stream, &part, &counters)) {
    a.partials = part;
    a.counters = counters;
    a.max_slots = tail_max_slots(C::kTileN, C::kCtaGroup,
                                 tail_slot_width(C::kMode == kAdapterDown, a.wide));
    a.max_counters = tail_max_counters(C::kCtaGroup);
  }
  const CUtensorMapDataType bf = CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
  const CUtensorMapSwizzle sw = CU_TENSOR_MAP_SWIZZLE_128B;
  CUtensorMap tW, tW2, tUp, tD;
  ColumnMaps tC;
  int rc;
  if constexpr (C::kMode == kGroupedWgrad) {
    rc = make_tensor_map_2d(&tW, bf, o.wide, a.wide, o.wide_rows, o.wide_ld * 2, 64, 64, sw);
    if (rc != TG_OK) return rc;
    rc = make_tensor_map_2d(&tC.box[0], bf, o.cols, a.cols, o.wide_rows, o.cols_ld * 2, 64, 64, sw);
    if (rc != TG_OK) return rc;
    for (int b = 1; b < kColBoxes; ++b) tC.box[b] = tC.box[0];
    if (a.cols >= 128) {
      rc = make_tensor_map_chunks(&tC.box[1], o.cols, a.cols, o.wide_rows, 1, o.cols_ld * 2,
                                  o.cols_ld * 2);
      if (rc != TG_OK) return rc;
    }
  } else {
    // Weights: the contraction index contiguous (boxes of 128 rows), or for
    // dgrad the wide axis (boxes of 64 x 64).
    a.wide_box = a.wide < 128 ? (a.wide + 15) / 16 * 16 : 128;
    rc = make_tensor_map_3d(
        &tW, bf, o.wide, C::kWideMn ? a.wide : o.k, o.wide_rows, o.wide_slices, o.wide_ld * 2,
        o.wide_slice_stride * 2, 64,
        C::kWideMn ? 64 : C::kMode == kAdapterDown ? a.wide_box : 128, sw);
    if (rc != TG_OK) return rc;
    for (int b = 0; b < kColBoxes; ++b) {
      const bool gather = C::kGather && a.row_idx != nullptr;
      rc = make_tensor_map_2d(&tC.box[b], bf, o.cols, o.k, gather ? a.num_rows : a.M,
                              o.cols_ld * 2, 64, gather ? 1 : C::kBoxStep * (b + 1), sw);
      if (rc != TG_OK) return rc;
    }
  }
  tW2 = tC.h[0] = tC.h[1] = tC.h[2] = tC.h[3] = tW;
  if (C::kWideMn && a.wide >= 128) {
    const bool w = C::kMode == kGroupedWgrad;
    rc = make_tensor_map_chunks(&tW2, o.wide, a.wide, o.wide_rows, w ? 1 : o.wide_slices,
                                o.wide_ld * 2, (w ? o.wide_ld : o.wide_slice_stride) * 2);
    if (rc != TG_OK) return rc;
  }
  tUp = tW;
  if (C::kExt && o.up != nullptr) {
    rc = make_tensor_map_3d(&tUp, bf, o.up, o.up_rank, a.wide, o.up_slices, o.up_ld * 2,
                            o.up_slice_stride * 2, 64, 128, sw);
    if (rc != TG_OK) return rc;
    for (int t = 0; t <= C::kTerms; ++t) {
      const bool all = t == C::kTerms;
      rc = make_tensor_map_2d(&tC.h[all ? 3 : t], bf, all ? a.h : a.h + t * a.rank,
                              all ? C::kTerms * a.rank : a.rank, a.M, C::kTerms * a.rank * 2, 64,
                              128, sw);
      if (rc != TG_OK) return rc;
    }
  }
  tD = tW;
  if constexpr (C::kStaged) {
    // Boxes of 32 rows x 128 bytes; wgrad's rows end with the group's D.
    const int64_t esize = C::kBf16Out ? 2 : 4;
    const bool w = C::kMode == kGroupedWgrad;
    rc = make_tensor_map_3d(
        &tD, C::kBf16Out ? bf : CU_TENSOR_MAP_DATA_TYPE_FLOAT32, a.D, a.wide, w ? a.cols : a.M,
        w ? a.groups : 1, a.ldd * esize,
        (w && a.groups > 1 ? a.group_stride_d : a.ldd * (w ? a.cols : a.M)) * esize,
        C::kBf16Out ? 64 : 32, 32, C::kBf16Out ? sw : CU_TENSOR_MAP_SWIZZLE_NONE);
    if (rc != TG_OK) return rc;
  }
  cfg.gridDim = dim3(static_cast<unsigned>(units * C::kCtaGroup), 1, 1);
  cfg.stream = stream;
  cfg.numAttrs = C::kCtaGroup == 2 ? 2 : 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kern, tW, tW2, tC, tUp, tD, a);
  return e == cudaSuccess ? TG_OK : cuda_fail(e);
}

// CTA pairs in the form `tail` asks for.
template <int kMode, int kStages, bool kBf16Out>
int launch_grouped_pairs(bool tail, const GroupedOperands& o, const GroupedArgs& a,
                         cudaStream_t stream, DeviceCtx* ctx) {
  return tail ? launch_grouped<GroupedCfg<kMode, 2, 256, kStages, kBf16Out, true>>(o, a, stream, ctx)
              : launch_grouped<GroupedCfg<kMode, 2, 256, kStages, kBf16Out, false>>(o, a, stream,
                                                                                   ctx);
}

// One translation unit for each (they compile in parallel).
int launch_grouped_forward(bool bf16, const GroupedOperands& o, const GroupedArgs& a,
                           cudaStream_t stream, DeviceCtx* ctx);
int launch_grouped_dgrad(bool bf16, const GroupedOperands& o, const GroupedArgs& a,
                         cudaStream_t stream, DeviceCtx* ctx);
int launch_grouped_wgrad(bool bf16, const GroupedOperands& o, const GroupedArgs& a,
                         cudaStream_t stream, DeviceCtx* ctx);
int launch_grouped_adapter(bool bf16, const GroupedOperands& o, const GroupedArgs& a,
                           cudaStream_t stream, DeviceCtx* ctx);

}  // namespace tg
