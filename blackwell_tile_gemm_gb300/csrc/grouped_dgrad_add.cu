// The input gradient given in parts of its contraction, added to D in f32.
#include "grouped_launch.cuh"

namespace tg {

namespace {
template <bool kTail, int kAdd>
using Cfg = GroupedCfg<kGroupedDgrad, 2, 256, 6, false, kTail, kAdd>;
}  // namespace

int launch_grouped_dgrad_add(bool chunked, const GroupedOperands& o, const GroupedArgs& a,
                             cudaStream_t stream, DeviceCtx* ctx) {
  const bool tail = grouped_tail_pays(
      static_cast<int64_t>(ceil_div_i(a.M, 256)) * ceil_div_i(a.wide, 256), a.num_k_blocks, ctx);
  if (chunked)
    return tail ? launch_grouped<Cfg<true, 2>>(o, a, stream, ctx)
                : launch_grouped<Cfg<false, 2>>(o, a, stream, ctx);
  return tail ? launch_grouped<Cfg<true, 1>>(o, a, stream, ctx)
              : launch_grouped<Cfg<false, 1>>(o, a, stream, ctx);
}

}  // namespace tg
