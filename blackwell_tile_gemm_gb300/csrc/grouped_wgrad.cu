// The weight-gradient configurations of the grouped kernel.
#include "grouped_launch.cuh"

namespace tg {

int launch_grouped_wgrad(bool bf16, const GroupedOperands& o, const GroupedArgs& a,
                         cudaStream_t stream, DeviceCtx* ctx) {
  const bool tail = grouped_tail_pays(
      static_cast<int64_t>(a.groups) * a.num_col_tiles * ceil_div_i(a.wide, 256), a.num_k_blocks,
      ctx);
  return bf16 ? launch_grouped_pairs<kGroupedWgrad, 6, true>(tail, o, a, stream, ctx)
              : launch_grouped_pairs<kGroupedWgrad, 6, false>(tail, o, a, stream, ctx);
}

}  // namespace tg
