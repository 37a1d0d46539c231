// A shared projection with a low-rank adapter per row:
//
//   D[i, :] = epi( A[i, :] * B^T + s[id_i] * (A[i, :] * down[id_i]^T) * up[id_i]^T )
//
// H[i, :] = s[id_i] * A[i, :] * down[id_i]^T (rank values a row) comes first; the
// grouped kernel (kAdapter) then runs the shared product and adds H[i, :] *
// up[id_i]^T inside it, so that D is written once and the second term costs no
// pass of its own.  For many values of H it is computed by the same tcgen05
// kernel (kAdapterDown) in tiles of 64 rows; fewer, and tiles with more than
// kDownAdapters adapters, go through lora_down_kernel.
//
// lora_down_kernel.  2 M K rank flop against (M + adapters * rank) K values
// read: at most a few tens of flop per byte, so reading A and `down` bounds it
// and warp-level MMAs (m16n8k16, f32 accumulation) are ample.  The roles are
// swapped: 16 rows of `down` fill the MMA's M, 8 rows of A its N, so that
// one row of A alone wastes no more than 7 idle columns.  A fragment's k
// indices need not be neighbours in memory as long as both operands agree, so
// each thread loads 16 contiguous bytes of a row (8 values, two MMAs' worth)
// straight into its fragments: no shared memory, no transposition.
//
// A block takes 8 consecutive rows and a slice of K: its warps share the
// slice, the CTAs of the cluster share K, and the partial sums meet in
// (distributed) shared memory in a fixed order.  The rows' adapters are
// computed for the whole tile and kept for their own rows, each, and each
// 16 kRt of the rank, in a block of its own (blockIdx.y).  64 rows over 48
// adapters of rank 16, K = 8192: 11 us from a cold cache for 14 MB.
//
// The whole call in a replayed graph: 4 rows over 32 adapters of rank 16 x 4096
// x 4096 16 us (floor 5: two kernels, each a launch, a trip to memory and a
// join), 64 rows x 8192 x 8192 40 us (floor 24, the weights: 128 of 152 SMs read
// them), 8000 rows of 16 requests, rank 64, x 8192 x 4096 423 us (floor 295, the
// tensor pipe: 1300 TFLOP/s).
#include <algorithm>

#include "grouped_launch.cuh"

namespace tg {
namespace {

constexpr int kDownWarps = 8;

struct DownArgs {
  const uint16_t* A;
  int64_t lda;
  int M, K;
  const int* ids;
  const uint16_t* down;
  int64_t ld_down, stride_down;
  const float* scales;   // may be null: 1
  int adapters, rank;
  int k_per_cta;         // multiple of 32 * kDownWarps
  int parts;             // blocks that share an adapter's rank
  bool leave_few;        // kAdapterDown does the 64-row tiles of few adapters
  uint16_t* h;           // [M][h_terms][rank]: H as a sum of bf16 terms
  int h_terms;
};

// Values k .. k + 7 of a row; those from `end` on are zero and not read.
__device__ __forceinline__ uint4 load8(const uint16_t* row, int k, int end) {
  if (k + 8 <= end) return __ldg(reinterpret_cast<const uint4*>(row + k));
  uint32_t w[4] = {0u, 0u, 0u, 0u};
#pragma unroll
  for (int e = 0; e < 8; ++e)
    if (k + e < end) w[e / 2] |= static_cast<uint32_t>(row[k + e]) << (16 * (e & 1));
  return make_uint4(w[0], w[1], w[2], w[3]);
}

__device__ __forceinline__ float ld_dsmem(uint32_t addr) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
  return v;
}

// kRt 16-row tiles of `down` at a time.  kLong (f32 D): the tensor core truncates
// at every addition to an accumulator, so after kDownChunk steps (768 terms, as in
// grouped_kernel.cuh) a warp adds it to a total with rounding to nearest: adapter
// term against 64 bits, K 65536, 9.3e-6 -> 8.6e-7.  (kAdapterDown, K 16384: 9.2e-6
// -> 8.5e-7.)
//
// Blocks an SM holds hide the loads' latency: with kRt = 1 five instead of four
// take 110 rows of 110 requests, rank 128, x 613 x 6740 from 82 to 69 us, with kRt
// = 2 three instead of two 3077 rows of 46, rank 32, x 725 x 2004 from 34 to 30.
// (kLong and kRt = 1 spill at five: 4447 rows of 30, rank 16, x 634 x 4389 66 us,
// with four 60.)
constexpr int kDownChunk = 24;
template <int kRt, bool kLong>
__global__ void __launch_bounds__(32 * kDownWarps, kRt == 1 ? (kLong ? 4 : 5) : kRt == 2 ? 3 : 2)
    lora_down_kernel(const DownArgs p) {
  constexpr int kTok = 8;
  constexpr int kElems = 16 * kRt * kTok;
  extern __shared__ float part[];      // [warp][kElems], then the CTA's sum in [0]
  griddep_wait();
  // The kernel before may have written A, and a read-only load of an address
  // known before the wait need not stay behind it: A's address is made unknown
  // until here.  (`down` is read where the ids say, which are plain loads.)
  const uint16_t* A = p.A;
  asm volatile("" : "+l"(A));
  // What the next kernel reads early (A, B, ids) was there before this one.
  griddep_launch_dependents();
  const int warp = threadIdx.x >> 5;
  const int lane = static_cast<int>(threadIdx.x & 31);
  const int g = lane >> 2, q = lane & 3;
  const int csize = static_cast<int>(gridDim.z);
  const int crank = static_cast<int>(blockIdx.z);     // one cluster spans z
  const int row0 = static_cast<int>(blockIdx.x) * kTok;
  const int rows = min(kTok, p.M - row0);
  if (p.leave_few) {
    uint32_t all[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int r = row0 / 64 * 64 + lane + 32 * i;
      all[i] = r < p.M ? static_cast<uint32_t>(p.ids[r]) : 0xFFFFFFFFu;
    }
    if (few_adapters(all, p.adapters)) return;   // every CTA of the cluster
  }
  uint32_t ids[1] = {lane < rows ? static_cast<uint32_t>(p.ids[row0 + lane]) : 0xFFFFFFFFu};
  const int kbeg = crank * p.k_per_cta;
  const int kend = min(p.K, kbeg + p.k_per_cta);
  // Adapter number blockIdx.y / parts, + gridDim.y / parts, ... of the tile (the
  // same in every CTA of the cluster, so all of them meet at its barriers), and
  // of its rank the pieces blockIdx.y % parts, + parts, ...
  const int per = static_cast<int>(gridDim.y) / p.parts;
  const int first = static_cast<int>(blockIdx.y) / p.parts;
  const int part0 = static_cast<int>(blockIdx.y) - first * p.parts;
  int ordinal = 0;
  for (int id = next_adapter(ids, -1, p.adapters); id >= 0; id = next_adapter(ids, id, p.adapters)) {
    if (ordinal++ % per != first) continue;
    const uint16_t* down = p.down + id * p.stride_down;
    const float scale = p.scales ? p.scales[id] : 1.0f;
    for (int r0 = 16 * kRt * part0; r0 < p.rank; r0 += 16 * kRt * p.parts) {
      float acc[kRt][4] = {};
      float total[kLong ? kRt : 1][4] = {};
      int left = kDownChunk;
#pragma unroll 2
      for (int k = kbeg + 32 * warp; k < kend; k += 32 * kDownWarps) {
        const int kk = k + 8 * q;
        uint4 a[kRt][2];
#pragma unroll
        for (int t = 0; t < kRt; ++t)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const int r = r0 + 16 * t + 8 * h + g;
            a[t][h] = r < p.rank ? load8(down + r * p.ld_down, kk, kend) : make_uint4(0u, 0u, 0u, 0u);
          }
        const uint4 b = g < rows ? load8(A + static_cast<int64_t>(row0 + g) * p.lda, kk, kend)
                                 : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
        for (int t = 0; t < kRt; ++t) {
          mma_m16n8k16(acc[t], a[t][0].x, a[t][1].x, a[t][0].y, a[t][1].y, b.x, b.y);
          mma_m16n8k16(acc[t], a[t][0].z, a[t][1].z, a[t][0].w, a[t][1].w, b.z, b.w);
        }
        if constexpr (kLong) {
          if (--left == 0) {
            left = kDownChunk;
#pragma unroll
            for (int t = 0; t < kRt; ++t)
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                total[t][e] += acc[t][e];
                acc[t][e] = 0.0f;
              }
          }
        }
      }
      if constexpr (kLong) {
#pragma unroll
        for (int t = 0; t < kRt; ++t)
#pragma unroll
          for (int e = 0; e < 4; ++e) acc[t][e] += total[t][e];
      }
      // [down row][row of A]: c0, c1 at (g, 2q), (g, 2q + 1); c2, c3 8 rows on.
      float* mine = part + warp * kElems;
#pragma unroll
      for (int t = 0; t < kRt; ++t)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          mine[(16 * t + g + 8 * (e >> 1)) * kTok + 2 * q + (e & 1)] = acc[t][e];
      __syncthreads();
      for (int e = threadIdx.x; e < kElems; e += 32 * kDownWarps) {
        float s = part[e];
#pragma unroll
        for (int w = 1; w < kDownWarps; ++w) s += part[w * kElems + e];
        part[e] = s;     // read and written by this thread only
      }
      if (csize > 1)
        cluster_sync();
      else
        __syncthreads();
      // Each CTA finishes a share of the tile's values.
      for (int e = crank * 32 * kDownWarps + static_cast<int>(threadIdx.x); e < kElems;
           e += csize * 32 * kDownWarps) {
        const int i = e / (16 * kRt), r = r0 + e % (16 * kRt);
        const int at = (e % (16 * kRt)) * kTok + i;
        if (i < rows && r < p.rank && p.ids[row0 + i] == id) {
          float s = 0.0f;
          if (csize > 1) {
            const uint32_t a = smem_addr(part + at);
            for (int c = 0; c < csize; ++c) s += ld_dsmem(map_to_cta(a, c));
          } else {
            s = part[at];
          }
          s *= scale;
          split_bf16(s, p.h + static_cast<int64_t>(row0 + i) * (p.h_terms * p.rank) + r, p.rank,
                     p.h_terms);
        }
      }
      // The partial sums are free again once every CTA has read them.
      if (csize > 1)
        cluster_sync();
      else
        __syncthreads();
    }
  }
}

// Where the tiles of the shared product start: at the first row of each run of
// at least kLongRun rows with one adapter, and after it.  Shorter runs between
// them stay together.  One block: two ordered compactions (rows where the
// adapter changes; of those, the ones next to a long run).
constexpr int kLongRun = 192;
constexpr int kRunThreads = 1024;

// Position of the first of this thread's `items` among the block's, after
// *count of earlier steps (updated).
__device__ __forceinline__ int ordered_slot(int items, int* part, int* count) {
  const int warp = threadIdx.x >> 5, lane = static_cast<int>(threadIdx.x & 31);
  int incl = items;
#pragma unroll
  for (int d = 1; d < 32; d *= 2) {
    const int o = __shfl_up_sync(0xFFFFFFFFu, incl, d);
    if (lane >= d) incl += o;
  }
  if (lane == 31) part[warp] = incl;
  __syncthreads();
  int v = part[lane];
#pragma unroll
  for (int d = 1; d < 32; d *= 2) {
    const int o = __shfl_up_sync(0xFFFFFFFFu, v, d);
    if (lane >= d) v += o;
  }
  const int all = __shfl_sync(0xFFFFFFFFu, v, 31);
  const int before = warp ? __shfl_sync(0xFFFFFFFFu, v, warp - 1) : 0;
  __syncthreads();
  const int at = *count + before + incl - items;
  *count += all;
  return at;
}

__global__ void __launch_bounds__(kRunThreads) lora_runs_kernel(const int* ids, int M, int adapters,
                                                                int* runs, int* offsets, int most) {
  constexpr int kOwn = 8;   // consecutive rows of one thread
  __shared__ int part[kRunThreads / 32];
  static_assert(kRunThreads == 1024, "one partial sum a lane");
  // ids are older than the kernel before this one, and what this one writes
  // is read only after it (launch order in gemm_bf16_lora): it waits at its
  // end, so that whoever waits for it has waited for both.
  griddep_launch_dependents();
  int count = 0;
  for (int64_t b = 0; b < M; b += kOwn * kRunThreads) {
    const int64_t i0 = b + kOwn * static_cast<int64_t>(threadIdx.x);
    uint32_t key[kOwn + 1];
#pragma unroll
    for (int j = 0; j <= kOwn; ++j) {
      const int64_t i = i0 + j - 1;
      key[j] = i >= 0 && i < M ? min(static_cast<uint32_t>(ids[i]), static_cast<uint32_t>(adapters))
                               : 0xFFFFFFFFu;   // before the first row: unlike any key
    }
    uint32_t flags = 0;
#pragma unroll
    for (int j = 0; j < kOwn; ++j)
      if (i0 + j < M && key[j + 1] != key[j]) flags |= 1u << j;
    int at = ordered_slot(__popc(flags), part, &count);
#pragma unroll
    for (int j = 0; j < kOwn; ++j)
      if (flags & (1u << j)) runs[at++] = static_cast<int>(i0 + j);
  }
  __syncthreads();
  const int num = count;
  count = 0;
  for (int b = 0; b < num; b += kRunThreads) {
    const int j = b + static_cast<int>(threadIdx.x);
    bool flag = false;
    int start = 0;
    if (j < num) {
      start = runs[j];
      const int next = j + 1 < num ? runs[j + 1] : M;
      flag = j == 0 || next - start >= kLongRun || start - runs[j - 1] >= kLongRun;
    }
    const int at = ordered_slot(flag ? 1 : 0, part, &count);
    if (flag) offsets[at] = start;
  }
  for (int j = count + static_cast<int>(threadIdx.x); j <= most; j += kRunThreads) offsets[j] = M;
  griddep_wait();
}

// Most runs' starts there can be: two for each long run, and the first row.
int64_t lora_most_tiles(int64_t M) { return 2 * (M / kLongRun) + 1; }

int launch_runs(const int* ids, int M, int adapters, int* runs, int* offsets, cudaStream_t stream) {
  cudaLaunchConfig_t cfg{};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.gridDim = dim3(1, 1, 1);
  cfg.blockDim = dim3(kRunThreads, 1, 1);
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, lora_runs_kernel, ids, M, adapters, runs, offsets,
                                           static_cast<int>(lora_most_tiles(M)));
  return e == cudaSuccess ? TG_OK : cuda_fail(e);
}

template <int kRt, bool kLong>
int launch_down(DownArgs a, cudaStream_t stream, DeviceCtx* ctx) {
  static std::atomic<int> prepared[64];
  auto kern = lora_down_kernel<kRt, kLong>;
  constexpr int kTok = 8;
  constexpr int kSmem = kDownWarps * 16 * kRt * kTok * 4;
  if (prepared[ctx->device].load(std::memory_order_acquire) == 0) {
    const cudaError_t e =
        cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
    if (e != cudaSuccess) return cuda_fail(e);
    prepared[ctx->device].store(1, std::memory_order_release);
  }
  const int tiles = ceil_div_i(a.M, kTok);
  // A block per adapter of the tile and part of the rank; where many tiles are
  // left to the other kernel, fewer (8000 rows of 16 requests: 15 us of 8000
  // blocks that return at once; 1536 rows of 32, rank 128, x 1000 x 6000: the
  // call takes 122 us with one block a tile, 84 with 10).
  const int budget = a.leave_few ? std::max(1, 2048 / tiles) : 1 << 16;
  a.parts = std::min(budget, ceil_div_i(a.rank, 16 * kRt));
  const int y = std::min(budget / a.parts, std::min(std::min(a.M, kTok), a.adapters)) * a.parts;
  // K over a cluster of up to 8 CTAs, while that adds blocks the SMs have
  // room for and leaves a CTA at least one step per warp.
  int c = 1;
  while (c < 8 && tiles * y * c < 2 * ctx->num_sms && a.K > 32 * kDownWarps * c) c *= 2;
  a.k_per_cta = ceil_div_i(ceil_div_i(a.K, c), 32 * kDownWarps) * 32 * kDownWarps;
  cudaLaunchConfig_t cfg{};
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = 1;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = static_cast<unsigned>(c);
  cfg.gridDim = dim3(static_cast<unsigned>(tiles), static_cast<unsigned>(y), static_cast<unsigned>(c));
  cfg.blockDim = dim3(32 * kDownWarps, 1, 1);
  cfg.dynamicSmemBytes = kSmem;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = c > 1 ? 2 : 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kern, a);
  return e == cudaSuccess ? TG_OK : cuda_fail(e);
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// Whether the product runs on single CTAs, with a split contraction and the
// adapter term beside the weights' stream: always for one tile of rows, and as
// long as its tiles of 128 x 128 make one wave.  16 bf16 adapters, 1 / 32
// requests, against CTA pairs: 512 rows, rank 64, x 4096 x 4096 (128 tiles) 36 /
// 40 us against 36 / 58; 1024 rows, rank 128, x 1000 x 6000 (64) 51 / 65 against
// 70 / 108; 512 rows, rank 128, x 6000 x 1000 (188) 56 / 73 against 26 / 69.
bool lora_few_rows(int64_t M, int64_t N, const DeviceCtx* ctx) {
  return M <= 128 || ceil_div_i(M, 128) * ceil_div_i(N, 128) <= ctx->num_sms;
}
// H values (M * rank) up to which lora_down_kernel alone computes H; it reads
// `down` once per 8 rows.  1 / 32 requests, against kAdapterDown: rank 64, 2048
// rows x 4096 x 4096 73 / 122 us against 75 / 142, and 5000 rows 165 / 224
// against 148 / 208; rank 128, 1024 rows x 1000 x 6000 70 / 108 against 60 / 132.
constexpr int64_t kLoraDownValues = 1 << 17;

}  // namespace

// H: up to three bf16 terms; where CTA pairs may run also the runs and the tile starts.
size_t lora_workspace_bytes(int64_t M, int64_t rank) {
  const size_t h = (static_cast<size_t>(M) * static_cast<size_t>(rank) * 6u + 255u) / 256u * 256u;
  return M <= 128
             ? h
             : h + (static_cast<size_t>(M) + static_cast<size_t>(lora_most_tiles(M)) + 1u) * 4u;
}

}  // namespace tg

using namespace tg;

extern "C" int gemm_bf16_lora(const void* A, int64_t lda, const void* B, int64_t ldb,
                              const int32_t* ids, const void* down, int64_t ld_down,
                              int64_t stride_down, const void* up, int64_t ld_up,
                              int64_t stride_up, const float* scales, int64_t adapters,
                              int64_t rank, void* D, int64_t ldd, int64_t M, int64_t N, int64_t K,
                              int d_dtype, const tg_epilogue* epi, unsigned flags,
                              void* cuda_stream) {
  constexpr int64_t kMaxDim = (int64_t{1} << 31) - 1;
  Epi e;
  int rc = check_epilogue(epi, &e);
  if (rc != TG_OK) return rc;
  if (flags != 0) return TG_ERR_UNSUPPORTED;
  if (M < 0 || N < 0 || K < 0 || M > kMaxDim || N > kMaxDim || K > kMaxDim)
    return TG_ERR_INVALID_ARG;
  if (d_dtype != TG_D_F32 && d_dtype != TG_D_BF16) return TG_ERR_INVALID_ARG;
  if (adapters < 0 || adapters > kMaxDim || rank < 1) return TG_ERR_INVALID_ARG;
  if (rank % 8 != 0 || rank > TG_MAX_RANK) return TG_ERR_UNSUPPORTED;
  if (M > kGroupedMaxExtent || N > kGroupedMaxExtent || K > kGroupedMaxExtent)
    return TG_ERR_UNSUPPORTED;
  if ((M / 64 + 1) * (N / 128 + 1) > kMaxDim) return TG_ERR_UNSUPPORTED;
  if (M == 0 || N == 0) return TG_OK;
  const int d_esize = d_dtype == TG_D_F32 ? 4 : 2;
  if (D == nullptr || ldd < N) return TG_ERR_INVALID_ARG;
  if (!aligned16(D) || (ldd * d_esize) % 16 != 0) return TG_ERR_MISALIGNED;
  if (K > 0) {
    if (A == nullptr || B == nullptr || lda < K || ldb < K) return TG_ERR_INVALID_ARG;
    if (!aligned16(A) || !aligned16(B) || lda % 8 != 0 || ldb % 8 != 0) return TG_ERR_MISALIGNED;
    if (adapters > 0) {
      if (ids == nullptr || down == nullptr || up == nullptr || ld_down < K || ld_up < rank)
        return TG_ERR_INVALID_ARG;
      if (adapters > 1 &&
          (stride_down < (rank - 1) * ld_down + K || stride_up < (N - 1) * ld_up + rank))
        return TG_ERR_INVALID_ARG;
      if (!aligned16(down) || !aligned16(up) || ld_down % 8 != 0 || ld_up % 8 != 0)
        return TG_ERR_MISALIGNED;
      if (adapters > 1 && (stride_down % 8 != 0 || stride_up % 8 != 0)) return TG_ERR_MISALIGNED;
    }
  }
  DeviceCtx* ctx = current_ctx();
  if (!ctx) return TG_ERR_CUDA;
  cudaStream_t stream = static_cast<cudaStream_t>(cuda_stream);
  if (K == 0) return launch_fill_epilogue(D, ldd, M, N, d_dtype, e, stream);
  if (adapters == 0)
    return launch_gemm(kKindBf16, A, lda, B, ldb, nullptr, 0, nullptr, 0, D, ldd, M, N, K, d_dtype,
                       e, 0, stream, ctx);
  const bool few = lora_few_rows(M, N, ctx);
  void* ws = device_workspace(lora_workspace_bytes(M, rank), stream, &rc);
  if (ws == nullptr) return rc;
  DownArgs d{};
  d.A = static_cast<const uint16_t*>(A);
  d.lda = lda;
  d.M = static_cast<int>(M);
  d.K = static_cast<int>(K);
  d.ids = ids;
  d.down = static_cast<const uint16_t*>(down);
  d.ld_down = ld_down;
  d.stride_down = adapters > 1 ? stride_down : 0;
  d.scales = scales;
  d.adapters = static_cast<int>(adapters);
  d.rank = static_cast<int>(rank);
  d.h = static_cast<uint16_t*>(ws);
  GroupedArgs a = grouped_args(ctx);
  a.M = static_cast<int>(M);
  a.num_k_blocks = ceil_div_i(K, 64);
  a.ids = ids;
  a.adapters = static_cast<int>(adapters);
  a.rank = static_cast<int>(rank);
  d.h_terms = d_dtype == TG_D_BF16 ? 2 : 3;
  a.h = d.h;
  a.h_terms = d.h_terms;
  GroupedOperands o{};
  o.wide_slices = 1;
  o.cols = A;
  o.cols_ld = lda;
  o.k = K;
  d.leave_few = M * rank > kLoraDownValues;
  int* runs = reinterpret_cast<int*>(static_cast<uint8_t*>(ws) +
                                     (static_cast<size_t>(M) * rank * 6u + 255u) / 256u * 256u);
  int* starts = runs + M;
  // 64 of the rank a block, or less where that leaves SMs without one (1 row,
  // rank 128, 1260 x 7563: the call 22 us with 8 blocks of two passes, 14 with
  // 64 of 16).
  int rt = rank <= 16 ? 1 : rank <= 32 ? 2 : 4;
  while (!d.leave_few && rt > 1 && ceil_div_i(M, 8) * ceil_div_i(rank, 16 * rt) < ctx->num_sms)
    rt /= 2;
  if (d_dtype == TG_D_BF16)
    rc = rt == 1   ? launch_down<1, false>(d, stream, ctx)
         : rt == 2 ? launch_down<2, false>(d, stream, ctx)
                   : launch_down<4, false>(d, stream, ctx);
  else
    rc = rt == 1   ? launch_down<1, true>(d, stream, ctx)
         : rt == 2 ? launch_down<2, true>(d, stream, ctx)
                   : launch_down<4, true>(d, stream, ctx);
  if (rc != TG_OK) return rc;
  if (!few) {
    rc = launch_runs(ids, static_cast<int>(M), static_cast<int>(adapters), runs, starts, stream);
    if (rc != TG_OK) return rc;
  }
  if (d.leave_few) {
    GroupedArgs h = a;
    h.wide = static_cast<int>(rank);
    h.scales = scales;
    GroupedOperands od = o;
    od.wide = down;
    od.wide_ld = ld_down;
    od.wide_rows = rank;
    od.wide_slices = adapters;
    od.wide_slice_stride = adapters > 1 ? stride_down : ld_down * rank;
    rc = d_dtype == TG_D_BF16
             ? launch_grouped<GroupedCfg<kAdapterDown, 1, 64, 8, true>>(od, h, stream, ctx)
             : launch_grouped<GroupedCfg<kAdapterDown, 1, 64, 8, false>>(od, h, stream, ctx);
    if (rc != TG_OK) return rc;
  }
  a.wide = static_cast<int>(N);
  a.D = D;
  a.ldd = ldd;
  a.epi = e;
  a.up = static_cast<const uint16_t*>(up);
  a.ld_up = ld_up;
  a.group_stride_up = adapters > 1 ? stride_up : 0;
  o.wide = B;
  o.wide_ld = ldb;
  o.wide_rows = N;
  o.wide_slice_stride = ldb * N;
  o.up = up;
  o.up_ld = ld_up;
  o.up_slices = adapters;
  o.up_slice_stride = adapters > 1 ? stride_up : ld_up * N;
  o.up_rank = rank;
  if (!few) {
    a.offsets = starts;
    a.groups = static_cast<int>(lora_most_tiles(M));
  }
  return launch_grouped_adapter(d_dtype == TG_D_BF16, o, a, stream, ctx);
}
