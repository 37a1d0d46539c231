// Rows grouped by id: a stable counting sort of n small integers.
//
//   key_i = ids_i where 0 <= ids_i < G, else G (rows in no group go last)
//   offsets[g] = #{i : key_i < g}, order = positions by (key, position),
//   slot[order[j]] = j.
//
// It is the plan of every product whose weights change with the row, and its
// work is tiny (12 bytes a row), so latency decides.  The rows are cut into
// one contiguous chunk per warp.  A warp walks its chunk 32 rows at a time;
// votes give each lane the lanes with its key (same_key), so a row's rank
// among equal keys is a popcount and one lane per key updates the warp's own
// histogram in shared memory: no order is left to chance.  A first walk
// counts; the histograms are summed over the warps and CTAs and scanned over
// the keys; a second walk places.
//
// Up to kOneCta rows run in one CTA and one launch.  Above, a counting kernel
// writes every CTA's histogram to the workspace, and each CTA of the placing
// kernel sums the ones before its own: two launches, the second of which
// counts its own rows while the first ends.  256 rows in 64 groups take 3.0 us,
// 262144 rows in 256 groups 11.4 us in a replayed graph (one cluster of 8 CTAs,
// in one launch: 44 us); 3.1 MB are 0.5 us of HBM traffic, so what bounds it is
// the chain of a launch, two walks and the sums between them.
#include "tg_internal.h"
#include "tg_ptx.cuh"

namespace tg {
namespace {

constexpr int kMaxWarps = 32;
constexpr int kHistBytes = 192 * 1024;
constexpr int kOneCta = 2048;       // rows
constexpr int kRowsPerCta = 2048;   // above that, while SMs are free
constexpr int kRowsPerWarp = 64;    // at least

struct RowsArgs {
  const int* ids;
  int n, groups;
  int warps;     // per CTA
  int chunk;     // rows per warp, a multiple of 32
  int bits;      // of a key
  int* offsets;
  int* order;
  int* slot;     // may be null
  int* counts;   // [keys][CTA] of the counting kernel
};

__device__ __forceinline__ int key_of(const RowsArgs& p, int i) {
  const int id = p.ids[i];   // (a read-only load need not stay behind griddep_wait)
  return static_cast<unsigned>(id) < static_cast<unsigned>(p.groups) ? id : p.groups;
}

// The lanes whose key is this lane's: one vote per bit of the key (all lanes
// past the end hold -1).  __match_any_sync takes one step per distinct key
// instead: 262144 rows in 256 groups 70 us, in 8 groups 24 us.
__device__ __forceinline__ unsigned same_key(int key, int bits) {
  unsigned peers = 0xFFFFFFFFu;
  for (int b = 0; b < bits; ++b) {
    const unsigned v = __ballot_sync(0xFFFFFFFFu, (key >> b) & 1);
    peers &= (key >> b) & 1 ? v : ~v;
  }
  const unsigned valid = __ballot_sync(0xFFFFFFFFu, key >= 0);
  return peers & (key >= 0 ? valid : ~valid);
}

// Calls f(key, lanes with that key, row) for the rows [lo, hi), 32 at a time;
// key is -1 past the end.  The ids of kAhead steps are loaded together: one
// load a step left a warp waiting about 1 us for each.
template <class F>
__device__ __forceinline__ void walk(const RowsArgs& p, int lo, int hi, int lane, F f) {
  constexpr int kAhead = 8;
  for (int b = lo; b < hi; b += 32 * kAhead) {
    int key[kAhead];
#pragma unroll
    for (int j = 0; j < kAhead; ++j) key[j] = hi - b > 32 * j + lane ? key_of(p, b + 32 * j + lane) : -1;
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      if (hi - b <= 32 * j) break;
      f(key[j], same_key(key[j], p.bits), b + 32 * j + lane);
    }
  }
}

// Rows of each key among this CTA's rows.
__global__ void __launch_bounds__(1024, 1) count_rows_kernel(const RowsArgs p) {
  extern __shared__ int smem[];
  const int keys = p.groups + 1;
  for (int g = threadIdx.x; g < keys; g += blockDim.x) smem[g] = 0;
  griddep_wait();
  griddep_launch_dependents();
  __syncthreads();
  const int64_t per = static_cast<int64_t>(p.warps) * p.chunk;
  const int64_t lo = blockIdx.x * per;
  const int64_t hi = lo + per < p.n ? lo + per : p.n;
  for (int64_t i = lo + threadIdx.x; i < hi; i += blockDim.x)
    atomicAdd(smem + key_of(p, static_cast<int>(i)), 1);   // a count: any order gives it
  __syncthreads();
  for (int g = threadIdx.x; g < keys; g += blockDim.x)
    p.counts[static_cast<int64_t>(g) * gridDim.x + blockIdx.x] = smem[g];
}

template <bool kMany>
__global__ void __launch_bounds__(32 * kMaxWarps, 1) place_rows_kernel(const RowsArgs p) {
  extern __shared__ int smem[];
  const int keys = p.groups + 1;
  int* total = smem;                 // [keys] rows per key, of all CTAs
  int* start = smem + keys;          // [keys] this CTA's first slot of each key
  int* hist = smem + 2 * keys;       // [warps][keys]
  __shared__ int scan_part[kMaxWarps];
  const int warp = threadIdx.x >> 5;
  const int lane = static_cast<int>(threadIdx.x & 31);
  const int rank = static_cast<int>(blockIdx.x);
  const int threads = blockDim.x;

  for (int i = threadIdx.x; i < p.warps * keys; i += threads) hist[i] = 0;
  // The ids are there: the counting kernel lets this one start only after its
  // own wait for them.
  if constexpr (!kMany) griddep_wait();
  __syncthreads();

  const int64_t lo64 = (static_cast<int64_t>(rank) * p.warps + warp) * p.chunk;
  const int lo = warp < p.warps && lo64 < p.n ? static_cast<int>(lo64) : p.n;
  const int hi = p.n - lo > p.chunk ? lo + p.chunk : p.n;
  int* mine = hist + warp * keys;   // (only warps below p.warps have rows)
  walk(p, lo, hi, lane, [&](int key, unsigned peers, int) {
    if (key >= 0 && __ffs(peers) - 1 == lane) mine[key] += __popc(peers);
    __syncwarp();
  });
  __syncthreads();
  // Over the warps: each count becomes the rows of its key in earlier warps.
  // Over the CTAs: the same with the counting kernel's histograms.
  if constexpr (kMany) griddep_wait();
  for (int g = threadIdx.x; g < keys; g += threads) {
    int run = 0;
    for (int w = 0; w < p.warps; ++w) {
      const int c = hist[w * keys + g];
      hist[w * keys + g] = run;
      run += c;
    }
    total[g] = kMany ? 0 : run;
    start[g] = 0;
  }
  __syncthreads();
  if constexpr (kMany) {
    // Four keys at a time per warp, its lanes over the CTAs.
    const int ctas = static_cast<int>(gridDim.x);
    const int nw = threads / 32;
    for (int g0 = warp; g0 < keys; g0 += 4 * nw) {
      int all[4] = {0, 0, 0, 0}, before[4] = {0, 0, 0, 0};
      for (int c = lane; c < ctas; c += 32) {
        int v[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int g = g0 + k * nw;
          v[k] = g < keys ? __ldcg(p.counts + static_cast<int64_t>(g) * ctas + c) : 0;
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          all[k] += v[k];
          before[k] += c < rank ? v[k] : 0;
        }
      }
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        all[k] = __reduce_add_sync(0xFFFFFFFFu, all[k]);
        before[k] = __reduce_add_sync(0xFFFFFFFFu, before[k]);
        if (lane == 0 && g0 + k * nw < keys) {
          total[g0 + k * nw] = all[k];
          start[g0 + k * nw] = before[k];
        }
      }
    }
    __syncthreads();
  }
  // Over the keys: `base` = rows of smaller keys, in steps of one block.
  int carry = 0;
  for (int g0 = 0; g0 < keys; g0 += threads) {
    const int g = g0 + static_cast<int>(threadIdx.x);
    const int all = g < keys ? total[g] : 0;
    int incl = all;
#pragma unroll
    for (int d = 1; d < 32; d *= 2) {
      const int o = __shfl_up_sync(0xFFFFFFFFu, incl, d);
      if (lane >= d) incl += o;
    }
    if (lane == 31) scan_part[warp] = incl;
    __syncthreads();
    int prev = 0, sum = 0;
    for (int w = 0; w < threads / 32; ++w) {
      if (w < warp) prev += scan_part[w];
      sum += scan_part[w];
    }
    const int base = carry + prev + incl - all;
    carry += sum;
    if (g < keys) {
      if (rank == 0) p.offsets[g] = base;
      start[g] += base;
    }
    __syncthreads();
  }
  walk(p, lo, hi, lane, [&](int key, unsigned peers, int i) {
    int seen = 0;
    if (key >= 0) seen = mine[key];
    __syncwarp();
    if (key >= 0) {
      const int at = start[key] + seen + __popc(peers & ((1u << lane) - 1u));
      p.order[at] = i;
      if (p.slot != nullptr) p.slot[i] = at;
      if (__ffs(peers) - 1 == lane) mine[key] = seen + __popc(peers);
    }
    __syncwarp();
  });
}

template <class K>
int launch_one(K kern, int grid, int threads, size_t smem, const RowsArgs& a, cudaStream_t stream,
               DeviceCtx* ctx, std::atomic<int>* prepared) {
  if (prepared[ctx->device].load(std::memory_order_acquire) == 0) {
    const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               kHistBytes + 4 * (TG_MAX_GROUPS + 1));
    if (e != cudaSuccess) return cuda_fail(e);
    prepared[ctx->device].store(1, std::memory_order_release);
  }
  cudaLaunchConfig_t cfg{};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.gridDim = dim3(static_cast<unsigned>(grid), 1, 1);
  cfg.blockDim = dim3(static_cast<unsigned>(threads), 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kern, a);
  return e == cudaSuccess ? TG_OK : cuda_fail(e);
}

// CTAs of the placing kernel.
int rows_ctas(int64_t n, int num_sms) {
  if (n <= kOneCta) return 1;
  const int64_t c = (n + kRowsPerCta - 1) / kRowsPerCta;
  return static_cast<int>(c < num_sms ? c : num_sms);
}

int launch_rows(RowsArgs a, cudaStream_t stream, DeviceCtx* ctx) {
  static std::atomic<int> prepared[3][64];
  const int keys = a.groups + 1;
  const int ctas = rows_ctas(a.n, ctx->num_sms);
  const int64_t per_cta = (static_cast<int64_t>(a.n) + ctas - 1) / ctas;
  int warps = kHistBytes / (4 * keys) - 1;
  if (warps > kMaxWarps) warps = kMaxWarps;
  const int64_t need = (per_cta + kRowsPerWarp - 1) / kRowsPerWarp;
  if (need < warps) warps = need < 1 ? 1 : static_cast<int>(need);
  a.warps = warps;
  a.chunk = static_cast<int>(((per_cta + warps - 1) / warps + 31) / 32 * 32);
  while ((1 << a.bits) < keys) ++a.bits;
  const size_t smem = static_cast<size_t>(4) * keys * (warps + 2);
  if (ctas == 1)
    return launch_one(place_rows_kernel<false>, 1, 32 * warps, smem, a, stream, ctx, prepared[0]);
  int rc = TG_OK;
  a.counts = static_cast<int*>(device_workspace(group_rows_workspace_bytes(a.n, a.groups), stream, &rc));
  if (a.counts == nullptr) return rc;
  rc = launch_one(count_rows_kernel, ctas, 1024, static_cast<size_t>(4) * keys, a, stream, ctx,
                  prepared[1]);
  if (rc != TG_OK) return rc;
  return launch_one(place_rows_kernel<true>, ctas, 1024, smem, a, stream, ctx, prepared[2]);
}

}  // namespace

// Every CTA's histogram; no device has more SMs than this counts for.
size_t group_rows_workspace_bytes(int64_t n, int64_t groups) {
  const int c = rows_ctas(n, 256);
  return c == 1 ? 0 : static_cast<size_t>(c) * static_cast<size_t>(groups + 1) * 4u;
}

}  // namespace tg


using namespace tg;

extern "C" int tg_group_rows(const int32_t* ids, int64_t n, int64_t groups, int32_t* offsets,
                             int32_t* order, int32_t* slot, void* cuda_stream) {
  // Chunk ends stay below 2^31.
  if (n < 0 || n > (int64_t{1} << 30)) return TG_ERR_INVALID_ARG;
  if (groups < 1 || groups > TG_MAX_GROUPS || offsets == nullptr) return TG_ERR_INVALID_ARG;
  if (n > 0 && (ids == nullptr || order == nullptr)) return TG_ERR_INVALID_ARG;
  DeviceCtx* ctx = current_ctx();
  if (!ctx) return TG_ERR_CUDA;
  RowsArgs a{};
  a.ids = ids;
  a.n = static_cast<int>(n);
  a.groups = static_cast<int>(groups);
  a.offsets = offsets;
  a.order = order;
  a.slot = slot;
  cudaStream_t stream = static_cast<cudaStream_t>(cuda_stream);
  return launch_rows(a, stream, ctx);
}
