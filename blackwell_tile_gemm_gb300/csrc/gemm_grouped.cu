// Products grouped by expert with ragged sizes: forward, input gradient and
// weight gradient (grouped_kernel.cuh has the kernel and its reasons).
#include "grouped_launch.cuh"

using namespace tg;

namespace {

constexpr int64_t kMaxDim = (int64_t{1} << 31) - 1;

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

int check_sizes(int64_t M, int64_t N, int64_t K, int64_t groups, int d_dtype) {
  if (M < 0 || N < 0 || K < 0 || M > kMaxDim || N > kMaxDim || K > kMaxDim)
    return TG_ERR_INVALID_ARG;
  if (groups < 1 || groups > TG_MAX_GROUPS) return TG_ERR_INVALID_ARG;
  if (d_dtype != TG_D_F32 && d_dtype != TG_D_BF16) return TG_ERR_INVALID_ARG;
  if (M > kGroupedMaxExtent || N > kGroupedMaxExtent || K > kGroupedMaxExtent)
    return TG_ERR_UNSUPPORTED;
  // Tiles of every group together stay below 2^31.
  const int64_t tiles = (M / 64 + groups) * ((N > K ? N : K) / 128 + 1);
  if (tiles > kMaxDim) return TG_ERR_UNSUPPORTED;
  return TG_OK;
}

// A row-major operand or result: pointer, row stride (elements), width.
int check_rows(const void* p, int64_t ld, int64_t width, int esize) {
  if (p == nullptr || ld < width) return TG_ERR_INVALID_ARG;
  if (!aligned16(p) || (ld * esize) % 16 != 0) return TG_ERR_MISALIGNED;
  return TG_OK;
}

// Slices of rows, `stride` elements apart.
int check_slices(int64_t stride, int64_t rows, int64_t ld, int64_t width, int64_t slices,
                 int esize) {
  if (slices > 1 && stride < (rows - 1) * ld + width) return TG_ERR_INVALID_ARG;
  if (slices > 1 && (stride * esize) % 16 != 0) return TG_ERR_MISALIGNED;
  return TG_OK;
}

}  // namespace

extern "C" {

int gemm_bf16_grouped(const void* A, int64_t lda, int64_t a_rows, const int32_t* row_idx,
                      const int32_t* offsets, int64_t groups, int64_t M, const void* B,
                      int64_t ldb, int64_t group_stride_b, void* D, int64_t ldd, int64_t N,
                      int64_t K, int d_dtype, const tg_epilogue* epi, unsigned flags,
                      void* cuda_stream) {
  Epi e;
  int rc = check_epilogue(epi, &e);
  if (rc != TG_OK) return rc;
  if (flags != 0) return TG_ERR_UNSUPPORTED;
  rc = check_sizes(M, N, K, groups, d_dtype);
  if (rc != TG_OK) return rc;
  if (a_rows < 0 || a_rows > kMaxDim) return TG_ERR_INVALID_ARG;
  if (M == 0 || N == 0) return TG_OK;
  if (offsets == nullptr) return TG_ERR_INVALID_ARG;
  rc = check_rows(D, ldd, N, d_dtype == TG_D_F32 ? 4 : 2);
  if (rc != TG_OK) return rc;
  if (K > 0) {
    if (a_rows == 0 || (row_idx == nullptr && a_rows < M)) return TG_ERR_INVALID_ARG;
    rc = check_rows(A, lda, K, 2);
    if (rc == TG_OK) rc = check_rows(B, ldb, K, 2);
    if (rc == TG_OK) rc = check_slices(group_stride_b, N, ldb, K, groups, 2);
    if (rc != TG_OK) return rc;
  }
  DeviceCtx* ctx = current_ctx();
  if (!ctx) return TG_ERR_CUDA;
  cudaStream_t stream = static_cast<cudaStream_t>(cuda_stream);
  const bool in_place = grouped_gathers(M, groups);
  if (row_idx != nullptr && K > 0 && !in_place) {
    const void* rows = nullptr;
    rc = gather_to_workspace(A, lda, static_cast<int>(a_rows), row_idx, M, K, &rows, &lda, stream,
                             ctx);
    if (rc != TG_OK) return rc;
    A = rows;
  }
  GroupedArgs a = grouped_args(ctx);
  a.M = static_cast<int>(M);
  a.wide = static_cast<int>(N);
  a.groups = static_cast<int>(groups);
  a.offsets = offsets;
  a.num_k_blocks = ceil_div_i(K, 64);
  a.D = D;
  a.ldd = ldd;
  a.epi = e;
  if (K > 0 && in_place) {
    a.row_idx = row_idx;
    a.num_rows = static_cast<int>(a_rows);
  }
  GroupedOperands o{};
  o.wide = B;
  o.wide_ld = ldb;
  o.wide_rows = N;
  o.wide_slices = groups;
  o.wide_slice_stride = groups > 1 ? group_stride_b : ldb * N;
  o.cols = A;
  o.cols_ld = lda;
  o.k = K;
  return launch_grouped_forward(d_dtype == TG_D_BF16, o, a, stream, ctx);
}

int gemm_bf16_grouped_dgrad(const void* G, int64_t ldg, const int32_t* offsets, int64_t groups,
                            int64_t M, const void* B, int64_t ldb, int64_t group_stride_b,
                            void* D, int64_t ldd, int64_t N, int64_t K, int d_dtype,
                            unsigned flags, void* cuda_stream) {
  if (flags != 0) return TG_ERR_UNSUPPORTED;
  int rc = check_sizes(M, N, K, groups, d_dtype);
  if (rc != TG_OK || M == 0 || K == 0) return rc;
  if (offsets == nullptr) return TG_ERR_INVALID_ARG;
  rc = check_rows(D, ldd, K, d_dtype == TG_D_F32 ? 4 : 2);
  if (rc != TG_OK) return rc;
  if (N > 0) {
    rc = check_rows(G, ldg, N, 2);
    if (rc == TG_OK) rc = check_rows(B, ldb, K, 2);
    if (rc == TG_OK) rc = check_slices(group_stride_b, N, ldb, K, groups, 2);
    if (rc != TG_OK) return rc;
  }
  DeviceCtx* ctx = current_ctx();
  if (!ctx) return TG_ERR_CUDA;
  cudaStream_t stream = static_cast<cudaStream_t>(cuda_stream);
  GroupedArgs a = grouped_args(ctx);
  a.M = static_cast<int>(M);
  a.wide = static_cast<int>(K);
  a.groups = static_cast<int>(groups);
  a.offsets = offsets;
  a.num_k_blocks = ceil_div_i(N, 64);
  a.D = D;
  a.ldd = ldd;
  GroupedOperands o{};
  o.wide = B;
  o.wide_ld = ldb;
  o.wide_rows = N;
  o.wide_slices = groups;
  o.wide_slice_stride = groups > 1 ? group_stride_b : ldb * N;
  o.cols = G;
  o.cols_ld = ldg;
  o.k = N;
  return launch_grouped_dgrad(d_dtype == TG_D_BF16, o, a, stream, ctx);
}

int gemm_bf16_grouped_wgrad(const void* G, int64_t ldg, const void* A, int64_t lda,
                            int64_t a_rows, const int32_t* row_idx, const int32_t* offsets,
                            int64_t groups, int64_t M, void* D, int64_t ldd,
                            int64_t group_stride_d, int64_t N, int64_t K, int d_dtype,
                            unsigned flags, void* cuda_stream) {
  if (flags != 0) return TG_ERR_UNSUPPORTED;
  int rc = check_sizes(M, N, K, groups, d_dtype);
  if (rc != TG_OK || N == 0 || K == 0) return rc;
  if (a_rows < 0 || a_rows > kMaxDim) return TG_ERR_INVALID_ARG;
  if ((N / 256 + 1) * (K / 256 + 1) * groups > kMaxDim) return TG_ERR_UNSUPPORTED;
  if (offsets == nullptr) return TG_ERR_INVALID_ARG;
  const int esize = d_dtype == TG_D_F32 ? 4 : 2;
  rc = check_rows(D, ldd, K, esize);
  if (rc == TG_OK) rc = check_slices(group_stride_d, N, ldd, K, groups, esize);
  if (rc != TG_OK) return rc;
  if (M > 0) {
    if (a_rows == 0 || (row_idx == nullptr && a_rows < M)) return TG_ERR_INVALID_ARG;
    rc = check_rows(G, ldg, N, 2);
    if (rc == TG_OK) rc = check_rows(A, lda, K, 2);
    if (rc != TG_OK) return rc;
  } else {
    // Every group is empty: the operands are never read (any valid map does).
    G = A = D;
    ldg = (N + 7) / 8 * 8;
    lda = (K + 7) / 8 * 8;
    row_idx = nullptr;
  }
  DeviceCtx* ctx = current_ctx();
  if (!ctx) return TG_ERR_CUDA;
  cudaStream_t stream = static_cast<cudaStream_t>(cuda_stream);
  if (row_idx != nullptr) {
    const void* rows = nullptr;
    rc = gather_to_workspace(A, lda, static_cast<int>(a_rows), row_idx, M, K, &rows, &lda, stream,
                             ctx);
    if (rc != TG_OK) return rc;
    A = rows;
  }
  GroupedArgs a = grouped_args(ctx);
  a.M = static_cast<int>(M);
  a.wide = static_cast<int>(K);
  a.cols = static_cast<int>(N);
  a.num_col_tiles = ceil_div_i(N, 256);
  a.num_k_blocks = ceil_div_i(M, 64 * groups);
  a.groups = static_cast<int>(groups);
  a.offsets = offsets;
  a.D = D;
  a.ldd = ldd;
  a.group_stride_d = groups > 1 ? group_stride_d : 0;
  GroupedOperands o{};
  o.wide = A;
  o.wide_ld = lda;
  o.wide_rows = M;
  o.wide_slices = 1;
  o.cols = G;
  o.cols_ld = ldg;
  o.k = M;
  return launch_grouped_wgrad(d_dtype == TG_D_BF16, o, a, stream, ctx);
}

}  // extern "C"
