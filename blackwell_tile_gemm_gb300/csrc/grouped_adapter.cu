// The adapter configurations of the grouped kernel: the shared product with the
// adapter term for few rows (tiles of 64 or 128 rows) and for many.
#include "grouped_launch.cuh"

namespace tg {

int launch_grouped_adapter(bool bf16, const GroupedOperands& o, const GroupedArgs& a,
                           cudaStream_t stream, DeviceCtx* ctx) {
  if (a.M <= 64)
    return bf16 ? launch_grouped<GroupedCfg<kAdapter, 1, 64, 8, true>>(o, a, stream, ctx)
                : launch_grouped<GroupedCfg<kAdapter, 1, 64, 8, false>>(o, a, stream, ctx);
  if (a.offsets == nullptr)
    return bf16 ? launch_grouped<GroupedCfg<kAdapter, 1, 128, 6, true>>(o, a, stream, ctx)
                : launch_grouped<GroupedCfg<kAdapter, 1, 128, 6, false>>(o, a, stream, ctx);
  const bool tail = grouped_tail_pays(
      static_cast<int64_t>(ceil_div_i(a.M, 256)) * ceil_div_i(a.wide, 256), a.num_k_blocks, ctx);
  return bf16 ? launch_grouped_pairs<kAdapter, 6, true>(tail, o, a, stream, ctx)
              : launch_grouped_pairs<kAdapter, 6, false>(tail, o, a, stream, ctx);
}

}  // namespace tg
