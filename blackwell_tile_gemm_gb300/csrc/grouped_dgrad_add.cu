// The input gradient given in parts of its contraction, added to D in f32.
#include "grouped_launch.cuh"

namespace tg {

namespace {
template <bool kTail, int kAdd>
using Cfg = GroupedCfg<kGroupedDgrad, 2, 256, 6, false, kTail, kAdd>;

// Columns per tile, of which the waves take least: a stage costs the larger of its
// MMAs (2 cycles a column) and its loads (4096 rows x 4096: 304 tiles of 224 columns
// in 4 waves, not 256 of 256).
int tile_columns(int64_t rows, int64_t wide, DeviceCtx* ctx) {
  const int64_t units = ctx->num_sms / 2, wide_tiles = (wide + 255) / 256;
  int64_t best = 0;
  int cols = 256;
  for (int c = 256; c >= 160; c -= 32) {
    const int64_t waves = (wide_tiles * ((rows + c - 1) / c) + units - 1) / units;
    const int64_t cost = waves * (2 * c > 256 + c ? 2 * c : 256 + c);
    if (best == 0 || cost < best) {
      best = cost;
      cols = c;
    }
  }
  return cols;
}

}  // namespace

int launch_grouped_dgrad_add(bool chunked, const GroupedOperands& o, const GroupedArgs& args,
                             cudaStream_t stream, DeviceCtx* ctx) {
  GroupedArgs a = args;
  const bool tail = grouped_tail_pays(
      static_cast<int64_t>(ceil_div_i(a.M, 256)) * ceil_div_i(a.wide, 256), a.num_k_blocks, ctx);
  a.tile_cols = tail ? 256 : tile_columns(a.M, a.wide, ctx);
  if (chunked)
    return tail ? launch_grouped<Cfg<true, 2>>(o, a, stream, ctx)
                : launch_grouped<Cfg<false, 2>>(o, a, stream, ctx);
  return tail ? launch_grouped<Cfg<true, 1>>(o, a, stream, ctx)
              : launch_grouped<Cfg<false, 1>>(o, a, stream, ctx);
}

}  // namespace tg
