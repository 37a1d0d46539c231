// Softmax cross entropy over a vocabulary and its gradient, logits never kept.
//
//   z = scale * A * B^T,  lse_i = log(sum_j exp z_ij),  loss_i = lse_i - z_i,t(i)
//   dz_ij = grad_i * scale * (exp(z_ij - lse_i) - [j = t(i)])
//   dA = dz * B,  dB = dz^T * A          (rows without a target: loss 0, dz 0)
//
// Forward: one pass of the product (xent_kernel.cuh) leaves a maximum and a sum
// per row and 128 columns, which xent_finish_kernel joins.  Backward: the
// vocabulary in pieces; for each, dz from the product made again, then the
// grouped gradients' kernels on it: dA's share (added up in f32 over the pieces)
// and the piece's rows of dB, which are complete.  Where their tiles are few, both are
// cut into slices of the contraction whose f32 sums are added in order.  dz passes between them as
// bf16, rounded once at 2^-9, as any gradient of a bf16 layer is; for f32
// gradients as two bf16 terms (2^-17), in one contraction over both.
#include <atomic>

#include "chained_launch.cuh"
#include "grouped_launch.cuh"
#include "xent_kernel.cuh"
#include "xent_plan.h"

using namespace tg;

namespace tg {
namespace {

// ---------------------------------------------------------------------------
// The product
// ---------------------------------------------------------------------------

template <class C>
int xent_units(DeviceCtx* ctx) {
  static std::atomic<int> prepared[64];
  std::atomic<int>& slot = prepared[ctx->device];
  int units = slot.load(std::memory_order_acquire);
  if (units > 0) return units;
  auto kern = xent_kernel<C>;
  cudaError_t e =
      cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM_BYTES);
  if (e != cudaSuccess) return -cuda_fail(e);
  units = ctx->num_sms / C::kCtaGroup;
  if constexpr (C::kCtaGroup == 2) {
    cudaLaunchConfig_t cfg{};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 2;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.gridDim = dim3(static_cast<unsigned>(2 * units), 1, 1);
    cfg.blockDim = dim3(C::kThreads, 1, 1);
    cfg.dynamicSmemBytes = C::SMEM_BYTES;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    int clusters = 0;
    e = cudaOccupancyMaxActiveClusters(&clusters, kern, &cfg);
    if (e != cudaSuccess) return -cuda_fail(e);
    if (clusters > 0 && clusters < units) units = clusters;
  }
  if (units < 1) units = 1;
  slot.store(units, std::memory_order_release);
  return units;
}

struct XentOperands {
  const void* A;
  int64_t lda;
  const void* B;
  int64_t ldb;
  int64_t K;
  void* dz;            // kXentGrad: [M][terms][ld_dz]
  int64_t ld_dz;
};

template <int kCtaGroup, int kMode>
int launch_xent_cfg(const XentOperands& o, const XentArgs& args, const XentTiles& tiles,
                    cudaStream_t stream, DeviceCtx* ctx) {
  using C = XentCfg<kCtaGroup, kMode>;
  const int units = xent_units<C>(ctx);
  if (units < 0) return TG_ERR_CUDA;
  XentArgs a = args;
  a.num_k_blocks = ceil_div_i(o.K, 64);
  a.num_m_tiles = tiles.m_tiles;
  a.num_n_tiles = tiles.n_tiles;
  a.bn = tiles.bn;
  // Bands of 4096 rows: the units that run at the same time share panels of B.
  a.raster_group = 4096 / (128 * kCtaGroup);
  a.a_box = kCtaGroup == 2 ? 128 : ceil_div_i(a.M, 8) * 8;
  a.a_bytes = xent_ring(a.a_box, a.bn / kCtaGroup, &a.b_bytes, &a.stages);
  a.status = ctx->status;
  a.timeout_ns = wait_timeout_ns();
  const CUtensorMapDataType bf = CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
  const CUtensorMapSwizzle sw = CU_TENSOR_MAP_SWIZZLE_128B;
  CUtensorMap tA, tB;
  int rc = make_tensor_map_2d(&tA, bf, o.A, o.K, a.M, o.lda * 2, 64, a.a_box, sw);
  if (rc != TG_OK) return rc;
  rc = make_tensor_map_2d(&tB, bf, o.B, o.K, a.N, o.ldb * 2, 64, a.bn / kCtaGroup, sw);
  if (rc != TG_OK) return rc;
  CUtensorMap tD = tA, tD2 = tA;
  if constexpr (kMode != kXentLoss) {
    const int64_t row_bytes = o.ld_dz * (C::kTwo ? 4 : 2);
    rc = make_tensor_map_2d(&tD, bf, o.dz, o.ld_dz, a.padded, row_bytes, 64, 32, sw);
    if (rc != TG_OK) return rc;
    if constexpr (C::kTwo) {
      rc = make_tensor_map_2d(&tD2, bf, static_cast<uint16_t*>(o.dz) + o.ld_dz, o.ld_dz, a.padded,
                              row_bytes, 64, 32, sw);
      if (rc != TG_OK) return rc;
    }
  }
  const int64_t num_tiles = static_cast<int64_t>(tiles.m_tiles) * tiles.n_tiles;
  cudaLaunchConfig_t cfg{};
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = kCtaGroup;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.gridDim = dim3(static_cast<unsigned>((num_tiles < units ? num_tiles : units) * kCtaGroup));
  cfg.blockDim = dim3(C::kThreads);
  cfg.dynamicSmemBytes = C::SMEM_BYTES;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = kCtaGroup == 2 ? 2 : 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, xent_kernel<C>, tA, tB, tD, tD2, a);
  return e == cudaSuccess ? TG_OK : cuda_fail(e);
}

template <int kMode>
int launch_xent(const XentOperands& o, const XentArgs& a, const XentTiles& tiles,
                cudaStream_t stream, DeviceCtx* ctx) {
  return a.M <= kXentFewRows ? launch_xent_cfg<1, kMode>(o, a, tiles, stream, ctx)
                             : launch_xent_cfg<2, kMode>(o, a, tiles, stream, ctx);
}

// ---------------------------------------------------------------------------
// Joining the tiles' maxima and sums
// ---------------------------------------------------------------------------

// Sums of exp(scale (a - m)): those of m2 join those of m.  The larger reference
// keeps its sum as it is, which also makes an infinite one meet itself without inf -
// inf.
__device__ __forceinline__ void join_sums(float& m, float& s, float m2, float s2, float scale2) {
  const float top = fmaxf(m, m2);
  s = s * (m == top ? 1.0f : exp2f((m - top) * scale2)) +
      s2 * (m2 == top ? 1.0f : exp2f((m2 - top) * scale2));
  m = top;
}

// Blocks of `rows` rows (a power of two: enough for two blocks an SM, then as many
// as make whole lines): neighbouring threads hold neighbouring rows, the block's
// others every kFinishThreads / rows-th part of them; joined in a fixed order.
// (8192 rows of 1000 parts, 65 MB: 28 us with 256 threads and 4 parts in flight.)
constexpr int kFinishThreads = 512;
constexpr int kFinishAhead = 8;

__global__ void __launch_bounds__(kFinishThreads) xent_finish_kernel(const float2* parts, int count,
                                                          const float* target_z, const int* targets,
                                                          float* loss, float* lse, int M, int vocab,
                                                          int rows, float scale, float scale2) {
  __shared__ float2 shared[kFinishThreads];
  griddep_wait();
  griddep_launch_dependents();
  const int r = static_cast<int>(threadIdx.x) % rows;
  const int group = static_cast<int>(threadIdx.x) / rows;
  const int groups = kFinishThreads / rows;
  const int row = static_cast<int>(blockIdx.x) * rows + r;
  float m = __uint_as_float(0xFF800000u), s = 0.0f;
  if (row < M) {
    const float2* at = parts + row;
    int q = group;
    for (; q + (kFinishAhead - 1) * groups < count; q += kFinishAhead * groups) {
      float2 v[kFinishAhead];
#pragma unroll
      for (int i = 0; i < kFinishAhead; ++i) v[i] = __ldcg(at + static_cast<int64_t>(q + i * groups) * M);
#pragma unroll
      for (int i = 0; i < kFinishAhead; ++i) join_sums(m, s, v[i].x, v[i].y, scale2);
    }
    for (; q < count; q += groups) {
      const float2 v = __ldcg(at + static_cast<int64_t>(q) * M);
      join_sums(m, s, v.x, v.y, scale2);
    }
  }
  shared[threadIdx.x] = make_float2(m, s);
  __syncthreads();
  for (int half = groups / 2; half > 0; half /= 2) {
    if (group < half) {
      const float2 v = shared[threadIdx.x + half * rows];
      join_sums(m, s, v.x, v.y, scale2);
      shared[threadIdx.x] = make_float2(m, s);
    }
    __syncthreads();
  }
  if (group == 0 && row < M) {
    // The loss from the reference, not from lse: where the target is the largest
    // logit, the difference is 0 and the small rest keeps its digits.
    const float l = logf(s);
    const int t = targets[row];
    lse[row] = fmaf(m, scale, l);
    loss[row] = t >= 0 && t < vocab ? fmaf(m - __ldcg(target_z + row), scale, l) : 0.0f;
  }
}

// K = 0: every logit is 0.  (No column: lse = log 0.)
__global__ void xent_zero_kernel(const int* targets, float* loss, float* lse, int M, int vocab) {
  const int64_t row = blockIdx.x * static_cast<int64_t>(blockDim.x) + threadIdx.x;
  if (row >= M) return;
  const float l = logf(static_cast<float>(vocab));
  const int t = targets[row];
  lse[row] = l;
  loss[row] = t >= 0 && t < vocab ? l : 0.0f;
}

// ---------------------------------------------------------------------------
// Sums of slices
// ---------------------------------------------------------------------------

// dst = the sum of `slices` arrays of f32 rows, in an order that the sizes alone give.
// kParts threads share the slices of four neighbouring elements: with few elements one
// thread's turns at memory would take longest (53 x 192, 63 slices: one thread 12 us, 16
// 3).
template <class TD, int kParts>
__global__ void __launch_bounds__(256) sum_slices_kernel(const float* src, int slices,
                                                         int64_t stride, int64_t ld, TD* dst,
                                                         int64_t ldd, int M, int K) {
  constexpr int kOwn = 256 / kParts;
  __shared__ float4 sums[kParts > 1 ? 256 : 1];
  griddep_wait();
  griddep_launch_dependents();
  const int per = (K + 3) / 4;       // the sums' rows end on 16 bytes
  const int64_t total = static_cast<int64_t>(M) * per;
  const int part = static_cast<int>(threadIdx.x) / kOwn;
  const int first = slices * part / kParts, end = slices * (part + 1) / kParts;
  for (int64_t i0 = static_cast<int64_t>(blockIdx.x) * kOwn; i0 < total;
       i0 += static_cast<int64_t>(gridDim.x) * kOwn) {
    const int64_t i = i0 + threadIdx.x % kOwn;
    const int64_t row = i / per;
    const int k = 4 * static_cast<int>(i - row * per);
    float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    if (i < total) {
      const float* at = src + row * ld + k;
      for (int s = first; s < end; s += 4) {
        float4 t[4];
#pragma unroll
        for (int u = 0; u < 4; ++u)
          if (s + u < end) t[u] = __ldcs(reinterpret_cast<const float4*>(at + (s + u) * stride));
#pragma unroll
        for (int u = 0; u < 4; ++u)
          if (s + u < end) {
            v.x += t[u].x;
            v.y += t[u].y;
            v.z += t[u].z;
            v.w += t[u].w;
          }
      }
    }
    if constexpr (kParts > 1) {
      sums[threadIdx.x] = v;
      __syncthreads();
      if (part == 0) {
#pragma unroll
        for (int q = 1; q < kParts; ++q) {
          const float4 t = sums[q * kOwn + threadIdx.x];
          v.x += t.x;
          v.y += t.y;
          v.z += t.z;
          v.w += t.w;
        }
      }
      __syncthreads();
    }
    if (part != 0 || i >= total) continue;
    TD* d = dst + row * ldd + k;
    const float f[4] = {v.x, v.y, v.z, v.w};
    if constexpr (sizeof(TD) == 2) {
      const uint32_t w[2] = {pack_bf16x2(v.x, v.y), pack_bf16x2(v.z, v.w)};
      if (k + 4 <= K) {
        *reinterpret_cast<uint2*>(d) = make_uint2(w[0], w[1]);
      } else {
#pragma unroll
        for (int e = 0; e < 3; ++e)
          if (k + e < K) d[e] = static_cast<TD>(w[e / 2] >> (16 * (e & 1)));
      }
    } else {
      if (k + 4 <= K) {
        *reinterpret_cast<float4*>(d) = v;
      } else {
#pragma unroll
        for (int e = 0; e < 3; ++e)
          if (k + e < K) d[e] = f[e];
      }
    }
  }
}

template <class TD>
int launch_sum_slices_to(const float* src, int slices, int64_t stride, int64_t ld, TD* dst,
                         int64_t ldd, int64_t M, int64_t K, cudaStream_t stream, DeviceCtx* ctx) {
  const int64_t total = M * ((K + 3) / 4);
  int parts = 1;
  while (parts < 16 && slices >= 4 * parts && total * parts < 256LL * 2 * ctx->num_sms) parts *= 4;
  const int own = 256 / parts;
  int64_t blocks = (total + own - 1) / own;
  if (blocks > 16 * ctx->num_sms) blocks = 16 * ctx->num_sms;
  auto* kern = parts == 1   ? &sum_slices_kernel<TD, 1>
               : parts == 4 ? &sum_slices_kernel<TD, 4>
                            : &sum_slices_kernel<TD, 16>;
  return launch_chained(kern, blocks, 256, 0, 1, stream, src, slices, stride, ld, dst, ldd,
                        static_cast<int>(M), static_cast<int>(K));
}

int launch_sum_slices(const float* src, int slices, int64_t stride, int64_t ld, void* dst,
                      int64_t ldd, int64_t M, int64_t K, bool bf16, cudaStream_t stream,
                      DeviceCtx* ctx) {
  return bf16 ? launch_sum_slices_to(src, slices, stride, ld, static_cast<uint16_t*>(dst), ldd, M,
                                     K, stream, ctx)
              : launch_sum_slices_to(src, slices, stride, ld, static_cast<float*>(dst), ldd, M, K,
                                     stream, ctx);
}

int clear_rows(void* D, int64_t ldd, int64_t rows, int64_t width, int esize, cudaStream_t stream) {
  if (rows == 0 || width == 0) return TG_OK;
  const cudaError_t e = cudaMemset2DAsync(D, static_cast<size_t>(ldd * esize), 0,
                                          static_cast<size_t>(width * esize),
                                          static_cast<size_t>(rows), stream);
  return e == cudaSuccess ? TG_OK : cuda_fail(e);
}

// ---------------------------------------------------------------------------
// Checks
// ---------------------------------------------------------------------------

constexpr int64_t kMaxDim = (int64_t{1} << 31) - 1;

int check_rows(const void* p, int64_t ld, int64_t width, int esize) {
  if (p == nullptr || ld < width) return TG_ERR_INVALID_ARG;
  if ((reinterpret_cast<uintptr_t>(p) & 15u) != 0 || (ld * esize) % 16 != 0)
    return TG_ERR_MISALIGNED;
  return TG_OK;
}

int check_sizes(int64_t M, int64_t N, int64_t K) {
  if (M < 0 || N < 0 || K < 0 || M > kMaxDim || N > kMaxDim || K > kMaxDim)
    return TG_ERR_INVALID_ARG;
  if (M > kGroupedMaxExtent || N > kGroupedMaxExtent || K > kGroupedMaxExtent)
    return TG_ERR_UNSUPPORTED;
  // Tile counts stay below 2^31, also those of the gradients' products.
  if ((M / 256 + 1) * (N / 64 + 1) > kMaxDim || (M / 256 + 1) * (K / 128 + 1) > kMaxDim ||
      (N / 256 + 1) * (K / 128 + 1) > kMaxDim)
    return TG_ERR_UNSUPPORTED;
  return TG_OK;
}

// (f32 gradients: two rows of dz for one of A.)
int check_grad_sizes(int64_t M, int64_t N, int64_t K, int d_dtype) {
  const int rc = check_sizes(M, N, K);
  if (rc != TG_OK) return rc;
  if (d_dtype != TG_D_F32 && d_dtype != TG_D_BF16) return TG_ERR_INVALID_ARG;
  return d_dtype == TG_D_F32 && 2 * M > kGroupedMaxExtent ? TG_ERR_UNSUPPORTED : TG_OK;
}

int check_form(float scale, unsigned flags) {
  // (A negative scale would make the smallest product the largest logit; log2(e)
  // times the largest is still finite.)
  if (!(scale > 0.0f) || scale > 1.0e38f) return TG_ERR_INVALID_ARG;
  return flags != 0 ? TG_ERR_UNSUPPORTED : TG_OK;
}

}  // namespace

int64_t xent_workspace_bytes(int64_t M, int64_t N, int64_t K) {
  const int rc = check_sizes(M, N, K);
  return rc != TG_OK ? -rc : static_cast<int64_t>(xent_loss_plan(M, N).bytes);
}
int64_t xent_grad_workspace_bytes(int64_t M, int64_t N, int64_t K, int d_dtype) {
  const int rc = check_grad_sizes(M, N, K, d_dtype);
  return rc != TG_OK ? -rc
                     : static_cast<int64_t>(xent_grad_plan(M, N, K, d_dtype == TG_D_BF16).bytes);
}

}  // namespace tg

extern "C" {

int gemm_bf16_xent(const void* A, int64_t lda, const void* B, int64_t ldb, const int32_t* targets,
                   float scale, float* loss, float* lse, int64_t M, int64_t N, int64_t K,
                   unsigned flags, void* cuda_stream) {
  int rc = check_sizes(M, N, K);
  if (rc == TG_OK) rc = check_form(scale, flags);
  if (rc != TG_OK || M == 0) return rc;
  if (targets == nullptr || loss == nullptr || lse == nullptr) return TG_ERR_INVALID_ARG;
  if (N > 0 && K > 0) {
    rc = check_rows(A, lda, K, 2);
    if (rc == TG_OK) rc = check_rows(B, ldb, K, 2);
    if (rc != TG_OK) return rc;
  }
  DeviceCtx* ctx = current_ctx();
  if (!ctx) return TG_ERR_CUDA;
  cudaStream_t stream = static_cast<cudaStream_t>(cuda_stream);
  const int m = static_cast<int>(M), n = static_cast<int>(N);
  if (N == 0 || K == 0) {
    xent_zero_kernel<<<static_cast<unsigned>((M + 255) / 256), 256, 0, stream>>>(targets, loss, lse,
                                                                                m, n);
    const cudaError_t e = cudaGetLastError();
    return e == cudaSuccess ? TG_OK : cuda_fail(e);
  }
  const XentLossPlan plan = xent_loss_plan(M, N);
  uint8_t* ws = static_cast<uint8_t*>(device_workspace(plan.bytes, stream, &rc));
  if (ws == nullptr) return rc;
  XentArgs a{};
  a.M = m;
  a.N = a.vocab = n;
  a.scale = scale;
  a.scale2 = scale * 1.4426950408889634f;
  a.targets = targets;
  a.parts = reinterpret_cast<float2*>(ws);
  a.target_z = reinterpret_cast<float*>(ws + plan.off_z);
  const XentOperands o{A, lda, B, ldb, K, nullptr, 0};
  rc = launch_xent<kXentLoss>(o, a, plan.tiles, stream, ctx);
  if (rc != TG_OK) return rc;
  int rows = 1;
  while (rows < 32 && rows * 2 * ctx->num_sms < m) rows *= 2;
  return launch_chained(xent_finish_kernel, (M + rows - 1) / rows, kFinishThreads, 0, 1, stream,
                        a.parts, 2 * plan.tiles.n_tiles, a.target_z, targets, loss, lse, m, n, rows,
                        a.scale, a.scale2);
}

int gemm_bf16_xent_grad_ex(const void* A, int64_t lda, const void* B, int64_t ldb,
                           const int32_t* targets, const float* lse, const float* loss,
                           const float* grad, float scale, void* dA, int64_t ldda, void* dB,
                           int64_t lddb, int64_t M, int64_t N, int64_t K, int d_dtype,
                           unsigned flags, void* cuda_stream) {
  int rc = check_grad_sizes(M, N, K, d_dtype);
  if (rc == TG_OK) rc = check_form(scale, flags);
  if (rc != TG_OK) return rc;
  const bool bf16 = d_dtype == TG_D_BF16;
  if (K == 0) return TG_OK;
  const int esize = bf16 ? 2 : 4;
  const bool rows = dA != nullptr && M > 0, weights = dB != nullptr && N > 0;
  if (rows) rc = check_rows(dA, ldda, K, esize);
  if (rc == TG_OK && weights) rc = check_rows(dB, lddb, K, esize);
  if (rc != TG_OK || (!rows && !weights)) return rc;
  if (M > 0 && N > 0) {
    if (targets == nullptr || lse == nullptr) return TG_ERR_INVALID_ARG;
    rc = check_rows(A, lda, K, 2);
    if (rc == TG_OK) rc = check_rows(B, ldb, K, 2);
    if (rc != TG_OK) return rc;
  }
  DeviceCtx* ctx = current_ctx();
  if (!ctx) return TG_ERR_CUDA;
  cudaStream_t stream = static_cast<cudaStream_t>(cuda_stream);
  if (M == 0) return clear_rows(dB, lddb, N, K, esize, stream);
  if (N == 0) return clear_rows(dA, ldda, M, K, esize, stream);

  const XentGradPlan plan = xent_grad_plan(M, N, K, bf16);
  uint8_t* ws = static_cast<uint8_t*>(device_workspace(plan.bytes, stream, &rc));
  if (ws == nullptr) return rc;
  uint16_t* a_rows = reinterpret_cast<uint16_t*>(ws);
  uint16_t* dz = reinterpret_cast<uint16_t*>(ws + plan.off_dz);
  float* sums = reinterpret_cast<float*>(ws + plan.off_sum);
  float* weight_sums = reinterpret_cast<float*>(ws + plan.off_weights);
  const int64_t one_sum = M * plan.ld_sum;
  // dA directly: bf16 from one contraction, f32 from contractions that are not sliced.
  const bool whole = plan.rows_by.count == 1 && plan.pieces == 1;
  const bool direct = plan.rows_by.count == 1 && (!bf16 || plan.pieces == 1);
  const int m = static_cast<int>(M);
  XentArgs a{};
  a.M = m;
  a.vocab = static_cast<int>(N);
  a.scale = scale;
  a.targets = targets;
  a.lse = lse;
  a.loss = loss;
  a.grad = grad;
  a.A = static_cast<const uint16_t*>(A);
  a.lda = lda;
  a.ld_copy = plan.ld_a;
  a.padded = static_cast<int>(plan.rows);
  a.K = static_cast<int>(K);
  for (int64_t col0 = 0; col0 < N; col0 += plan.piece) {
    const int64_t n = N - col0 < plan.piece ? N - col0 : plan.piece;
    const int64_t ld_dz = xent_up(n, 64);   // (the piece's own: nothing of another's is left in it)
    const uint16_t* b = static_cast<const uint16_t*>(B) + col0 * ldb;
    a.N = static_cast<int>(n);
    a.col0 = static_cast<int>(col0);
    a.copy = weights && col0 == 0 ? a_rows : nullptr;
    const XentOperands o{A, lda, b, ldb, K, dz, ld_dz};
    const XentTiles tiles = xent_tiles(M, n, 64);
    rc = bf16 ? launch_xent<kXentGrad>(o, a, tiles, stream, ctx)
              : launch_xent<kXentGradTwo>(o, a, tiles, stream, ctx);
    if (rc != TG_OK) return rc;
    if (rows) {
      GroupedArgs g = grouped_args(ctx);
      g.M = m;
      g.wide = static_cast<int>(K);
      GroupedOperands p{};
      p.wide = b;
      p.wide_ld = ldb;
      p.wide_rows = n;
      p.wide_slices = 1;
      p.wide_slice_stride = ldb * n;
      p.cols = dz;
      p.cols_ld = plan.terms * ld_dz;
      // (dz is zero from column n on, and past B's row n nothing is read.)
      p.k = plan.terms * ld_dz;
      if (bf16 && whole) {
        g.num_k_blocks = static_cast<int>(p.k / 64);
        g.D = dA;
        g.ldd = ldda;
        rc = launch_grouped_dgrad(true, p, g, stream, ctx);
      } else {
        const int slices = plan.rows_by.count;
        g.M = static_cast<int>(slices * M);
        g.groups = slices;
        g.even = m;
        g.tile_cols = plan.rows_by.columns;
        g.slice = static_cast<int>(xent_up((ld_dz + slices - 1) / slices, 64));
        g.second = static_cast<int>(ld_dz);
        g.num_k_blocks = plan.terms * g.slice / 64;
        g.add = col0 > 0;
        g.D = direct ? dA : sums;
        g.ldd = direct ? ldda : plan.ld_sum;
        rc = launch_sliced_dgrad(!bf16, p, g, stream, ctx);
        if (rc == TG_OK && !direct && col0 + plan.piece >= N)
          rc = launch_sum_slices(sums, slices, one_sum, plan.ld_sum, dA, ldda, M, K, bf16, stream,
                                 ctx);
      }
      if (rc != TG_OK) return rc;
    }
    if (weights) {
      // (Two terms: twice the rows of dz against as many of A.)
      const int64_t terms_rows = plan.terms * plan.rows;
      const int slices = plan.weights_by.count;
      void* D = static_cast<uint8_t*>(dB) + col0 * lddb * esize;
      GroupedArgs g = grouped_args(ctx);
      g.M = static_cast<int>(terms_rows);
      g.wide = static_cast<int>(K);
      g.cols = static_cast<int>(n);
      g.num_col_tiles = ceil_div_i(n, 256);
      g.D = D;
      g.ldd = lddb;
      GroupedOperands p{};
      p.wide = a_rows;
      p.wide_ld = plan.ld_a;
      p.wide_rows = terms_rows;
      p.wide_slices = 1;
      p.cols = dz;
      p.cols_ld = ld_dz;
      p.k = terms_rows;
      if (slices == 1) {
        g.num_k_blocks = ceil_div_i(terms_rows, 64);
        rc = launch_grouped_wgrad(bf16, p, g, stream, ctx);
      } else {
        g.groups = slices;
        g.even = static_cast<int>(xent_up((terms_rows + slices - 1) / slices, 64));
        g.num_k_blocks = g.even / 64;
        g.D = weight_sums;
        g.ldd = plan.ld_sum;
        g.group_stride_d = n * plan.ld_sum;
        rc = launch_sliced_wgrad(p, g, stream, ctx);
        if (rc != TG_OK) return rc;
        rc = launch_sum_slices(weight_sums, slices, g.group_stride_d, plan.ld_sum, D, lddb, n, K,
                               bf16, stream, ctx);
      }
      if (rc != TG_OK) return rc;
    }
  }
  return rc;
}

int gemm_bf16_xent_grad(const void* A, int64_t lda, const void* B, int64_t ldb,
                        const int32_t* targets, const float* lse, const float* grad, float scale,
                        void* dA, int64_t ldda, void* dB, int64_t lddb, int64_t M, int64_t N,
                        int64_t K, int d_dtype, unsigned flags, void* cuda_stream) {
  return gemm_bf16_xent_grad_ex(A, lda, B, ldb, targets, lse, nullptr, grad, scale, dA, ldda, dB,
                                lddb, M, N, K, d_dtype, flags, cuda_stream);
}

}  // extern "C"
