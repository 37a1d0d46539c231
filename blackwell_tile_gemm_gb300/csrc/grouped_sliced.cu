// The gradients' configurations for contractions in slices.
#include "grouped_launch.cuh"

namespace tg {

int launch_sliced_dgrad(bool chunked, const GroupedOperands& o, const GroupedArgs& a,
                        cudaStream_t stream, DeviceCtx* ctx) {
  return chunked
             ? launch_grouped<GroupedCfg<kGroupedDgrad, 2, 256, 6, false, false, 2>>(o, a, stream, ctx)
             : launch_grouped<GroupedCfg<kGroupedDgrad, 2, 256, 6, false, false, 1>>(o, a, stream, ctx);
}

int launch_sliced_wgrad(const GroupedOperands& o, const GroupedArgs& a, cudaStream_t stream,
                        DeviceCtx* ctx) {
  return launch_grouped<GroupedCfg<kGroupedWgrad, 2, 256, 6, false, false, 3>>(o, a, stream, ctx);
}

}  // namespace tg
