// Balance loss of a router, its counts and its gradient.
//
//   p_t = softmax(logits_t) over E experts; count_e = choices of expert e
//   share_e = E * count_e / (sum of counts * tokens)
//   loss = sum_e share_e * sum_t p_te
//   dlogits_t = g * p_t * (share - sum_e p_te share_e)     (counts are constants)
//
// A token is one with a choice inside [0, E); others (padding) have no part in
// anything.  An expert whose logit is -inf has p = 0, and so has every expert of
// a row that is -inf throughout.
//
// Both directions read the logits once and are bound by HBM, short ones by the
// chain of launches.  A row belongs to a group of lanes (a power of two, a whole
// block from 513 experts on), each of which keeps its experts' p in registers and,
// in the forward pass, their sums over the group's rows; those are added over a
// block's groups as a tree and over the blocks by the one block of a second
// kernel, always in the same order.
#include <type_traits>

#include "tg_internal.h"
#include "tg_ptx.cuh"

using namespace tg;

namespace tg {
namespace {

constexpr int64_t kMaxDim = (int64_t{1} << 31) - 1;
constexpr int kMostChoices = 1024;

struct BalanceArgs {
  const void* logits;
  int64_t ld;
  const int* ids;       // [M][choices]
  int choices, M, E;
  int lanes;            // of a row's group (warps: 1 .. 32)
  float* sums;          // [blocks][E]: sums of p
  int* counts_of;       // [blocks][E + 1]: choices of each expert; tokens
  // gradient
  const float* shares;  // [E]
  const float* grad;    // one value, or null for 1
  void* D;
  int64_t ldd;
};

template <class T>
__device__ __forceinline__ float value_of(const T* p) {
  if constexpr (sizeof(T) == 2)
    return __uint_as_float(static_cast<uint32_t>(*reinterpret_cast<const uint16_t*>(p)) << 16);
  else
    return *reinterpret_cast<const float*>(p);
}

__device__ __forceinline__ float no_logit() { return __uint_as_float(0xFF800000u); }

// Softmax of a row spread over a group's lanes (experts lane, lane + lanes, ...):
// z becomes p.  kBlock: the group is the block.
template <bool kMax>
__device__ __forceinline__ float over_block(float v, float* shared) {
  const int warp = threadIdx.x >> 5;
#pragma unroll
  for (int d = 16; d > 0; d /= 2) {
    const float o = __shfl_xor_sync(0xFFFFFFFFu, v, d);
    v = kMax ? fmaxf(v, o) : v + o;
  }
  __syncthreads();   // (the last call's values are read)
  if ((threadIdx.x & 31) == 0) shared[warp] = v;
  __syncthreads();
  v = shared[0];
  for (int w = 1; w < static_cast<int>(blockDim.x) / 32; ++w)
    v = kMax ? fmaxf(v, shared[w]) : v + shared[w];
  return v;
}

template <bool kMax, bool kBlock>
__device__ __forceinline__ float over_group(float v, int lanes, float* shared) {
  if constexpr (kBlock) {
    return over_block<kMax>(v, shared);
  } else {
    for (int d = lanes / 2; d > 0; d /= 2) {
      const float o = __shfl_xor_sync(0xFFFFFFFFu, v, d);
      v = kMax ? fmaxf(v, o) : v + o;
    }
    return v;
  }
}

template <int kV, bool kBlock>
__device__ __forceinline__ void softmax_row(float (&z)[kV], int lanes, float* shared) {
  float m = no_logit();
#pragma unroll
  for (int i = 0; i < kV; ++i) m = fmaxf(m, z[i]);
  m = over_group<true, kBlock>(m, lanes, shared);
  // Nothing but -inf: every exponential below is exp(-inf) = 0.
  const float ref = m == no_logit() ? 0.0f : m;
  float s = 0.0f;
#pragma unroll
  for (int i = 0; i < kV; ++i) {
    z[i] = expf(z[i] - ref);
    s += z[i];
  }
  s = over_group<false, kBlock>(s, lanes, shared);
  const float inv = m == no_logit() && s == 0.0f ? 0.0f : 1.0f / s;
#pragma unroll
  for (int i = 0; i < kV; ++i) z[i] *= inv;
}

// Rows that a group takes together, their loads in flight at the same time.
template <int kV>
constexpr int rows_together() { return kV >= 8 ? 1 : kV >= 4 ? 2 : 4; }

// The walk over rows that both kernels share.  f(row, p, some): the row's p and
// whether it is a token; count(id) for each choice inside.
template <class T, int kV, bool kBlock, class F, class N>
__device__ __forceinline__ void walk_rows(const BalanceArgs& p, float* shared, F f, N count) {
  constexpr int kR = kBlock ? 1 : rows_together<kV>();
  const int lanes = kBlock ? static_cast<int>(blockDim.x) : p.lanes;
  const int lane = static_cast<int>(threadIdx.x) % lanes;
  const int groups = static_cast<int>(blockDim.x) / lanes;
  const int64_t all = static_cast<int64_t>(gridDim.x) * groups;
  const int64_t mine = static_cast<int64_t>(blockIdx.x) * groups + threadIdx.x / lanes;
  const T* logits = static_cast<const T*>(p.logits);
  // Whole warps walk together (their shuffles and votes): as many steps for all.
  const int64_t steps = (p.M + all * kR - 1) / (all * kR);
  for (int64_t s = 0; s < steps; ++s) {
    const int64_t r0 = (s * kR) * all + mine;
    float z[kR][kV];
    int some[kR];
#pragma unroll
    for (int r = 0; r < kR; ++r) {
      const int64_t row = r0 + r * all;
#pragma unroll
      for (int i = 0; i < kV; ++i) {
        const int e = lane + i * lanes;
        z[r][i] = row < p.M && e < p.E ? value_of(logits + row * p.ld + e) : no_logit();
      }
      some[r] = 0;
      if (row < p.M)
        for (int c = lane; c < p.choices; c += lanes) {
          const int id = p.ids[row * p.choices + c];
          if (static_cast<unsigned>(id) < static_cast<unsigned>(p.E)) {
            some[r] = 1;
            count(id);
          }
        }
    }
#pragma unroll
    for (int r = 0; r < kR; ++r) {
      const int64_t row = r0 + r * all;
      int any;
      if constexpr (kBlock) {
        any = __syncthreads_or(some[r]);
      } else {
        const unsigned votes = __ballot_sync(0xFFFFFFFFu, some[r]);
        const unsigned group = lanes == 32 ? 0xFFFFFFFFu : ((1u << lanes) - 1u)
                                                               << ((threadIdx.x & 31) / lanes * lanes);
        any = (votes & group) != 0;
      }
      softmax_row<kV, kBlock>(z[r], lanes, shared);
      f(row, z[r], any != 0 && row < p.M, lane, lanes);
    }
  }
}

template <class T, int kV, bool kBlock>
__global__ void __launch_bounds__(kBlock ? 256 : 512) balance_sums_kernel(const BalanceArgs p) {
  extern __shared__ float smem[];   // [E] counts, [1] tokens, then the tree's sums
  __shared__ float warp_part[32];
  int* hist = reinterpret_cast<int*>(smem);
  float* tree = smem + p.E + 1;
  for (int e = threadIdx.x; e <= p.E; e += blockDim.x) hist[e] = 0;
  griddep_wait();
  griddep_launch_dependents();
  __syncthreads();
  float sum[kV] = {};
  walk_rows<T, kV, kBlock>(
      p, warp_part,
      [&](int64_t, const float (&q)[kV], bool some, int lane, int) {
        if (!some) return;
        if (lane == 0) atomicAdd(hist + p.E, 1);
#pragma unroll
        for (int i = 0; i < kV; ++i) sum[i] += q[i];
      },
      [&](int id) { atomicAdd(hist + id, 1); });   // (counts: any order gives them)
  // Over the groups: halves of them add to the others until one is left.
  const int lanes = kBlock ? static_cast<int>(blockDim.x) : p.lanes;
  const int lane = static_cast<int>(threadIdx.x) % lanes;
  const int group = static_cast<int>(threadIdx.x) / lanes;
  for (int half = static_cast<int>(blockDim.x) / lanes / 2; half > 0; half /= 2) {
    __syncthreads();
    if (group >= half && group < 2 * half) {
#pragma unroll
      for (int i = 0; i < kV; ++i)
        if (lane + i * lanes < p.E) tree[(group - half) * p.E + lane + i * lanes] = sum[i];
    }
    __syncthreads();
    if (group < half) {
#pragma unroll
      for (int i = 0; i < kV; ++i)
        if (lane + i * lanes < p.E) sum[i] += tree[group * p.E + lane + i * lanes];
    }
  }
  if (group == 0) {
#pragma unroll
    for (int i = 0; i < kV; ++i)
      if (lane + i * lanes < p.E)
        p.sums[static_cast<int64_t>(blockIdx.x) * p.E + lane + i * lanes] = sum[i];
  }
  __syncthreads();
  for (int e = threadIdx.x; e <= p.E; e += blockDim.x)
    p.counts_of[static_cast<int64_t>(blockIdx.x) * (p.E + 1) + e] = hist[e];
}

// One block: sums over the blocks, shares and the loss.
__global__ void __launch_bounds__(1024) balance_join_kernel(const float* sums, const int* counts_of,
                                                            int blocks, int E, float* loss,
                                                            int* counts, float* shares) {
  extern __shared__ float smem[];          // [parts][E] sums, [parts][E + 1] counts
  __shared__ float part[32];
  griddep_wait();
  griddep_launch_dependents();
  // A power of two of threads for each expert, as many as there are.
  int width = 1;
  while (width < E + 1 && width < 1024) width *= 2;
  const int parts = 1024 / width;
  float* sum_of = smem;
  int* count_of = reinterpret_cast<int*>(smem + parts * E);
  const int x = static_cast<int>(threadIdx.x) % width, q = static_cast<int>(threadIdx.x) / width;
  for (int e = x; e <= E; e += width) {
    float s = 0.0f;
    int n = 0;
#pragma unroll 8
    for (int b = q; b < blocks; b += parts) {
      if (e < E) s += __ldcg(sums + static_cast<int64_t>(b) * E + e);
      n += __ldcg(counts_of + static_cast<int64_t>(b) * (E + 1) + e);
    }
    if (e < E) sum_of[q * E + e] = s;
    count_of[q * (E + 1) + e] = n;
  }
  __syncthreads();
  // Each expert's sum to the first part; the sum of all counts.
  int mine = 0;
  for (int e = threadIdx.x; e <= E; e += 1024) {
    float s = e < E ? sum_of[e] : 0.0f;
    int n = count_of[e];
    for (int r = 1; r < parts; ++r) {
      if (e < E) s += sum_of[r * E + e];
      n += count_of[r * (E + 1) + e];
    }
    if (e < E) {
      sum_of[e] = s;
      counts[e] = n;
      mine += n;
    }
    count_of[e] = n;
  }
  mine = __reduce_add_sync(0xFFFFFFFFu, mine);
  __shared__ int whole[32];
  if ((threadIdx.x & 31) == 0) whole[threadIdx.x >> 5] = mine;
  __syncthreads();
  int64_t total = 0;
  for (int w = 0; w < 32; ++w) total += whole[w];
  const int tokens = count_of[E];
  float l = 0.0f;
  for (int e = threadIdx.x; e < E; e += 1024) {
    // (In 64 bits: a count, and the product below, may pass 2^24.)
    const float share = tokens > 0 ? static_cast<float>(static_cast<double>(E) * count_of[e] /
                                                        (static_cast<double>(total) * tokens))
                                   : 0.0f;
    shares[e] = share;
    l += share * sum_of[e];
  }
#pragma unroll
  for (int d = 16; d > 0; d /= 2) l += __shfl_xor_sync(0xFFFFFFFFu, l, d);
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = l;
  __syncthreads();
  if (threadIdx.x == 0) {
    l = 0.0f;
    for (int w = 0; w < 32; ++w) l += part[w];
    *loss = l;
  }
}

template <class T, class TD, int kV, bool kBlock>
__global__ void __launch_bounds__(kBlock ? 256 : 512) balance_grad_kernel(const BalanceArgs p) {
  __shared__ float warp_part[32];
  griddep_wait();
  griddep_launch_dependents();
  const int lanes = kBlock ? static_cast<int>(blockDim.x) : p.lanes;
  const int lane0 = static_cast<int>(threadIdx.x) % lanes;
  const float g = p.grad ? *p.grad : 1.0f;
  float share[kV];
#pragma unroll
  for (int i = 0; i < kV; ++i) share[i] = lane0 + i * lanes < p.E ? p.shares[lane0 + i * lanes] : 0.0f;
  walk_rows<T, kV, kBlock>(
      p, warp_part,
      [&](int64_t row, const float (&q)[kV], bool some, int lane, int n) {
        float dot = 0.0f;
#pragma unroll
        for (int i = 0; i < kV; ++i) dot += q[i] * share[i];
        dot = over_group<false, kBlock>(dot, n, warp_part);
        if (row >= p.M) return;
        TD* d = static_cast<TD*>(p.D) + row * p.ldd;
#pragma unroll
        for (int i = 0; i < kV; ++i) {
          const int e = lane + i * n;
          if (e >= p.E) continue;
          const float v = some ? g * q[i] * (share[i] - dot) : 0.0f;
          if constexpr (sizeof(TD) == 2)
            *reinterpret_cast<uint16_t*>(d + e) = static_cast<uint16_t>(pack_bf16x2(v, v) & 0xFFFFu);
          else
            *reinterpret_cast<float*>(d + e) = v;
        }
      },
      [](int) {});
}

template <class... P>
int launch_chained(void (*kern)(P...), int64_t blocks, int threads, size_t smem,
                   cudaStream_t stream, P... args) {
  cudaLaunchConfig_t cfg{};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.gridDim = dim3(static_cast<unsigned>(blocks), 1, 1);
  cfg.blockDim = dim3(static_cast<unsigned>(threads), 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kern, args...);
  return e == cudaSuccess ? TG_OK : cuda_fail(e);
}

// Lanes of a row's group and values each keeps: 16 at most, a whole block (256
// lanes) from 513 experts on.
struct BalanceShape {
  int lanes, values;
  bool block;
};
BalanceShape balance_shape(int E) {
  if (E > 512) return BalanceShape{256, 16, true};
  int lanes = 1;
  while (lanes < 32 && lanes < E) lanes *= 2;
  int values = 1;
  while (values * lanes < E) values *= 2;
  return BalanceShape{lanes, values, false};
}

// Blocks of a pass: a group takes at least one step of rows.
constexpr int kSumBlocks = 152;
int64_t balance_blocks(int64_t M, int E, int64_t most) {
  const BalanceShape s = balance_shape(E);
  const int64_t groups = s.block ? 1 : 512 / s.lanes;
  const int64_t b = (M + groups - 1) / groups;
  return b < most ? b : most;
}


template <class T, int kV, bool kBlock>
int launch_sums(const BalanceArgs& a, int64_t blocks, cudaStream_t stream) {
  auto kern = balance_sums_kernel<T, kV, kBlock>;
  const int threads = kBlock ? 256 : 512;
  const int groups = kBlock ? 1 : threads / a.lanes;
  // (18 KB at most: 512 experts in 16 groups)
  const size_t smem = 4 * (static_cast<size_t>(a.E) + 1 + static_cast<size_t>(groups / 2) * a.E);
  return launch_chained(kern, blocks, threads, smem, stream, a);
}

// f(V, block) with the template arguments of E.
template <class F>
int by_shape(int E, F f) {
  const BalanceShape s = balance_shape(E);
  if (s.block) return f(std::integral_constant<int, 16>{}, std::true_type{});
  switch (s.values) {
    case 1: return f(std::integral_constant<int, 1>{}, std::false_type{});
    case 2: return f(std::integral_constant<int, 2>{}, std::false_type{});
    case 4: return f(std::integral_constant<int, 4>{}, std::false_type{});
    case 8: return f(std::integral_constant<int, 8>{}, std::false_type{});
    default: return f(std::integral_constant<int, 16>{}, std::false_type{});
  }
}

int check_balance(const void* logits, int64_t ld, int dtype, const int32_t* ids, int64_t choices,
                  int64_t M, int64_t E) {
  if (M < 0 || M > kMaxDim || E < 1 || E > TG_MAX_GROUPS || choices < 1 || choices > kMostChoices)
    return TG_ERR_INVALID_ARG;
  if (dtype != TG_D_F32 && dtype != TG_D_BF16) return TG_ERR_INVALID_ARG;
  // Counts stay below 2^31.
  if (M * choices > kMaxDim) return TG_ERR_UNSUPPORTED;
  if (M == 0) return TG_OK;
  if (logits == nullptr || ids == nullptr || ld < E) return TG_ERR_INVALID_ARG;
  return TG_OK;
}

}  // namespace

size_t balance_workspace_bytes(int64_t, int64_t E) {
  return static_cast<size_t>(kSumBlocks) * static_cast<size_t>(2 * E + 1) * 4u;
}

}  // namespace tg

extern "C" {

int tg_balance_loss(const void* logits, int64_t ld, int dtype, const int32_t* ids, int64_t choices,
                    int64_t M, int64_t E, float* loss, int32_t* counts, float* shares,
                    void* cuda_stream) {
  int rc = check_balance(logits, ld, dtype, ids, choices, M, E);
  if (rc != TG_OK) return rc;
  if (loss == nullptr || counts == nullptr || shares == nullptr) return TG_ERR_INVALID_ARG;
  DeviceCtx* ctx = current_ctx();
  if (!ctx) return TG_ERR_CUDA;
  cudaStream_t stream = static_cast<cudaStream_t>(cuda_stream);
  const int64_t blocks = balance_blocks(M, static_cast<int>(E), kSumBlocks);
  float* sums = static_cast<float*>(device_workspace(balance_workspace_bytes(M, E), stream, &rc));
  if (sums == nullptr) return rc;
  BalanceArgs a{};
  a.logits = logits;
  a.ld = ld;
  a.ids = ids;
  a.choices = static_cast<int>(choices);
  a.M = static_cast<int>(M);
  a.E = static_cast<int>(E);
  a.lanes = balance_shape(a.E).lanes;
  a.sums = sums;
  a.counts_of = reinterpret_cast<int*>(sums + blocks * E);
  if (blocks > 0) {
    rc = by_shape(a.E, [&](auto v, auto block) {
      constexpr int kV = decltype(v)::value;
      constexpr bool kBlock = decltype(block)::value;
      return dtype == TG_D_BF16 ? launch_sums<uint16_t, kV, kBlock>(a, blocks, stream)
                                : launch_sums<float, kV, kBlock>(a, blocks, stream);
    });
    if (rc != TG_OK) return rc;
  }
  int width = 1;
  while (width < E + 1 && width < 1024) width *= 2;
  const size_t smem = static_cast<size_t>(1024 / width) * static_cast<size_t>(2 * E + 1) * 4u;
  return launch_chained(balance_join_kernel, 1, 1024, smem, stream,
                        static_cast<const float*>(a.sums), static_cast<const int*>(a.counts_of),
                        static_cast<int>(blocks), a.E, loss, counts, shares);
}

int tg_balance_loss_grad(const void* logits, int64_t ld, int dtype, const int32_t* ids,
                         int64_t choices, int64_t M, int64_t E, const float* shares,
                         const float* grad, void* D, int64_t ldd, int d_dtype, void* cuda_stream) {
  const int rc = check_balance(logits, ld, dtype, ids, choices, M, E);
  if (rc != TG_OK) return rc;
  if (d_dtype != TG_D_F32 && d_dtype != TG_D_BF16) return TG_ERR_INVALID_ARG;
  if (M == 0) return TG_OK;
  if (shares == nullptr || D == nullptr || ldd < E) return TG_ERR_INVALID_ARG;
  DeviceCtx* ctx = current_ctx();
  if (!ctx) return TG_ERR_CUDA;
  cudaStream_t stream = static_cast<cudaStream_t>(cuda_stream);
  BalanceArgs a{};
  a.logits = logits;
  a.ld = ld;
  a.ids = ids;
  a.choices = static_cast<int>(choices);
  a.M = static_cast<int>(M);
  a.E = static_cast<int>(E);
  a.lanes = balance_shape(a.E).lanes;
  a.shares = shares;
  a.grad = grad;
  a.D = D;
  a.ldd = ldd;
  const int64_t blocks = balance_blocks(M, a.E, 4 * static_cast<int64_t>(ctx->num_sms));
  return by_shape(a.E, [&](auto v, auto block) {
    constexpr int kV = decltype(v)::value;
    constexpr bool kBlock = decltype(block)::value;
    const int threads = kBlock ? 256 : 512;
    const bool in16 = dtype == TG_D_BF16, out16 = d_dtype == TG_D_BF16;
    if (in16 && out16)
      return launch_chained(balance_grad_kernel<uint16_t, uint16_t, kV, kBlock>, blocks, threads, 0,
                            stream, a);
    if (in16)
      return launch_chained(balance_grad_kernel<uint16_t, float, kV, kBlock>, blocks, threads, 0,
                            stream, a);
    if (out16)
      return launch_chained(balance_grad_kernel<float, uint16_t, kV, kBlock>, blocks, threads, 0,
                            stream, a);
    return launch_chained(balance_grad_kernel<float, float, kV, kBlock>, blocks, threads, 0, stream,
                          a);
  });
}

}  // extern "C"
