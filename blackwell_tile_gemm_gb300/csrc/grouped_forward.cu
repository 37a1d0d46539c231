// The forward configurations of the grouped kernel.
#include "grouped_launch.cuh"

namespace tg {

int launch_grouped_forward(bool bf16, const GroupedOperands& o, const GroupedArgs& a,
                           cudaStream_t stream, DeviceCtx* ctx) {
  // Few rows a group: single CTAs with 64-column tiles, a deep ring of weight
  // boxes and a split contraction.
  if (grouped_few_rows(a.M, a.groups))
    return bf16 ? launch_grouped<GroupedCfg<kGroupedForward, 1, 64, 9, true>>(o, a, stream, ctx)
                : launch_grouped<GroupedCfg<kGroupedForward, 1, 64, 9, false>>(o, a, stream, ctx);
  const bool tail = grouped_tail_pays(
      static_cast<int64_t>(ceil_div_i(a.M, 256)) * ceil_div_i(a.wide, 256), a.num_k_blocks, ctx);
  return bf16 ? launch_grouped_pairs<kGroupedForward, 6, true>(tail, o, a, stream, ctx)
              : launch_grouped_pairs<kGroupedForward, 6, false>(tail, o, a, stream, ctx);
}

}  // namespace tg
