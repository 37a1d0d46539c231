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
// block from 513 experts on), each of which keeps 16 experts' p in registers and,
// in the forward pass, their sums over the group's rows; those are added over a
// block's groups as a tree and over the blocks by one cluster of a second kernel,
// always in the same order.  Few lanes with many experts each, not the reverse: a
// row's maximum and sum cross the lanes of its group one step after the other (32
// lanes with 8 experts each, read by 2 bytes: 65536 x 256 bf16 60 us forward, 47
// backward).
#include <type_traits>

#include "chained_launch.cuh"
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
  float* sums;          // [blocks][E]: sums of p
  int* counts_of;       // [blocks][E + 1]: choices of each expert; tokens
  float* loss;          // results (one block alone writes them)
  int* counts;
  float* out_shares;
  // gradient
  const float* shares;  // [E]
  const float* grad;    // one value, or null for 1
  void* D;
  int64_t ldd;
};

constexpr int kV = 16;               // experts of a lane
constexpr int kThreads = 640;        // 20 warps of 96 registers
constexpr int kBlockLanes = 256;     // of a row's group from 513 experts on: a block
constexpr int kGroupExperts = 512;
// Rows that a group takes together; the next ones' loads are in flight meanwhile.
template <class T>
constexpr int rows_together() { return sizeof(T) == 2 ? 2 : 1; }

// Threads of a block whose rows' groups have kLanes lanes.
template <int kLanes>
constexpr int block_threads() { return kLanes == kBlockLanes ? kBlockLanes : kThreads; }

// The expert of a lane's i-th value.  kVec: 16 bytes at a time, the lanes side by
// side; else one.
template <class T, bool kVec, int kLanes>
__device__ __forceinline__ int expert_of(int lane, int i) {
  constexpr int kW = kVec ? 16 / static_cast<int>(sizeof(T)) : 1;
  return (lane + i / kW * kLanes) * kW + i % kW;
}

__device__ __forceinline__ float no_logit() { return __uint_as_float(0xFF800000u); }

// This lane's logits of a row as they lie in memory (-inf past the last expert, and
// without a row).
template <class T>
struct Logits {
  uint32_t w[kV * sizeof(T) / 4];

  template <bool kVec, int kLanes>
  __device__ __forceinline__ void load(const T* row, bool in, int E, int lane) {
    constexpr int kPer = 4 / static_cast<int>(sizeof(T));       // values of a word
    constexpr uint32_t kNone = sizeof(T) == 4 ? 0xFF800000u : 0xFF80FF80u;
    if constexpr (kVec) {
      constexpr int kW = 4 * kPer;
#pragma unroll
      for (int i = 0; i < kV; i += kW) {
        const int e = expert_of<T, kVec, kLanes>(lane, i);
        uint4 q = make_uint4(kNone, kNone, kNone, kNone);
        if (in && e + kW <= E) {
          q = *reinterpret_cast<const uint4*>(row + e);
        } else if (in && e < E) {
          uint32_t t[4] = {kNone, kNone, kNone, kNone};
#pragma unroll
          for (int j = 0; j < kW; ++j)
            if (e + j < E) put(t[j / kPer], j % kPer, row + e + j);
          q = make_uint4(t[0], t[1], t[2], t[3]);
        }
        w[i / kPer] = q.x;
        w[i / kPer + 1] = q.y;
        w[i / kPer + 2] = q.z;
        w[i / kPer + 3] = q.w;
      }
    } else {
#pragma unroll
      for (int i = 0; i < kV; ++i) {
        if (i % kPer == 0) w[i / kPer] = kNone;
        const int e = expert_of<T, kVec, kLanes>(lane, i);
        if (in && e < E) put(w[i / kPer], i % kPer, row + e);
      }
    }
  }
  static __device__ __forceinline__ void put(uint32_t& word, int at, const T* p) {
    if constexpr (sizeof(T) == 4)
      word = *reinterpret_cast<const uint32_t*>(p);
    else
      word = (word & (at ? 0x0000FFFFu : 0xFFFF0000u)) |
             static_cast<uint32_t>(*reinterpret_cast<const uint16_t*>(p)) << (16 * at);
  }
  __device__ __forceinline__ float value(int i) const {
    if constexpr (sizeof(T) == 4)
      return __uint_as_float(w[i]);
    else
      return __uint_as_float(i & 1 ? w[i / 2] & 0xFFFF0000u : w[i / 2] << 16);
  }
};

// Maximum or sum over a group's lanes (kBlockLanes: over the block, through
// `shared`), in every lane.
template <bool kMax, int kLanes>
__device__ __forceinline__ float over_group(float v, float* shared) {
#pragma unroll
  for (int d = (kLanes > 32 ? 32 : kLanes) / 2; d > 0; d /= 2) {
    const float o = __shfl_xor_sync(0xFFFFFFFFu, v, d);
    v = kMax ? fmaxf(v, o) : v + o;
  }
  if constexpr (kLanes > 32) {
    __syncthreads();   // (the last call's values are read)
    if ((threadIdx.x & 31) == 0) shared[threadIdx.x >> 5] = v;
    __syncthreads();
    v = shared[0];
#pragma unroll
    for (int w = 1; w < kLanes / 32; ++w) v = kMax ? fmaxf(v, shared[w]) : v + shared[w];
  }
  return v;
}

// Softmax of a row spread over a group's lanes: z becomes exp(z - the largest), and
// 1 / their sum is returned.
template <int kLanes>
__device__ __forceinline__ float softmax_row(float (&z)[kV], float* shared) {
  constexpr float kLog2e = 1.4426950408889634f;
  float m = no_logit();
#pragma unroll
  for (int i = 0; i < kV; ++i) m = fmaxf(m, z[i]);
  m = over_group<true, kLanes>(m, shared);
  // Nothing but -inf: every exponential below is exp(-inf) = 0.
  const float ref = m == no_logit() ? 0.0f : m;
  float s = 0.0f;
#pragma unroll
  for (int i = 0; i < kV; ++i) {
    // (The difference first: m log2(e) of the lowest f32 is none.)
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(z[i]) : "f"((z[i] - ref) * kLog2e));
    s += z[i];
  }
  s = over_group<false, kLanes>(s, shared);
  return m == no_logit() && s == 0.0f ? 0.0f : __fdividef(1.0f, s);
}

// The walk over rows that both kernels share.  f(row, e, inv, some): p is e inv, and
// whether the row is a token; count(id) for each choice inside.
template <class T, bool kVec, int kLanes, class F, class N>
__device__ __forceinline__ void walk_rows(const BalanceArgs& p, float* shared, F f, N count) {
  constexpr int kR = rows_together<T>();
  constexpr int kIds = kLanes < 16 ? 2 : 1;
  constexpr int kGroups = block_threads<kLanes>() / kLanes;
  const int lane = static_cast<int>(threadIdx.x) % kLanes;
  const int all = static_cast<int>(gridDim.x) * kGroups;
  const int mine = static_cast<int>(blockIdx.x) * kGroups + static_cast<int>(threadIdx.x) / kLanes;
  const unsigned group =
      kLanes >= 32 ? 0xFFFFFFFFu
                   : ((1u << (kLanes & 31)) - 1u) << ((threadIdx.x & 31) / kLanes * kLanes);
  // Rows mine, mine + all, ...; whole warps walk together (their shuffles and votes):
  // as many steps for all.
  const T* at = static_cast<const T*>(p.logits) + mine * p.ld;
  const int64_t stride = all * p.ld;
  Logits<T> next[kR];
  int next_id[kR][kIds];      // choices lane and lane + kLanes
  auto load = [&](int64_t row0) {
#pragma unroll
    for (int r = 0; r < kR; ++r) {
      const int64_t row = row0 + static_cast<int64_t>(r) * all;
      next[r].template load<kVec, kLanes>(at, row < p.M, p.E, lane);
      at += stride;
#pragma unroll
      for (int i = 0; i < kIds; ++i) {
        const int c = lane + i * kLanes;
        next_id[r][i] = row < p.M && c < p.choices ? p.ids[row * p.choices + c] : -1;
      }
    }
  };
  load(mine);
  for (int64_t first = mine; first - mine < p.M; first += static_cast<int64_t>(all) * kR) {
    float z[kR][kV];
    int some[kR];
#pragma unroll
    for (int r = 0; r < kR; ++r) {
      const int64_t row = first + static_cast<int64_t>(r) * all;
      some[r] = 0;
      auto take = [&](int id) {
        if (static_cast<unsigned>(id) < static_cast<unsigned>(p.E)) {
          some[r] = 1;
          count(id);
        }
      };
#pragma unroll
      for (int i = 0; i < kIds; ++i) take(next_id[r][i]);
      if (row < p.M)
        for (int c = lane + kIds * kLanes; c < p.choices; c += kLanes)
          take(p.ids[row * p.choices + c]);
#pragma unroll
      for (int i = 0; i < kV; ++i) z[r][i] = next[r].value(i);
    }
    load(first + static_cast<int64_t>(all) * kR);
#pragma unroll
    for (int r = 0; r < kR; ++r) {
      const int64_t row = first + static_cast<int64_t>(r) * all;
      bool any;
      if constexpr (kLanes == kBlockLanes)
        any = __syncthreads_or(some[r]) != 0;
      else
        any = (__ballot_sync(0xFFFFFFFFu, some[r]) & group) != 0;
      const float inv = softmax_row<kLanes>(z[r], shared);
      f(row, z[r], inv, any && row < p.M);
    }
  }
}

// The results, from every expert's sum of p and count (and the tokens behind them)
// in shared memory.  By a whole block.
__device__ __forceinline__ void finish_loss(const float* sum_of, const int* count_of, int E,
                                            float* loss, int* counts, float* shares) {
  __shared__ int choice_part[32];
  __shared__ float loss_part[32];
  __shared__ float2 scale_of;
  const int tid = static_cast<int>(threadIdx.x), warp = tid >> 5, lane = tid & 31;
  const int warps = static_cast<int>(blockDim.x) / 32;
  int choices = 0;
  for (int e = tid; e < E; e += blockDim.x) {
    counts[e] = count_of[e];
    choices += count_of[e];
  }
  choices = __reduce_add_sync(0xFFFFFFFFu, choices);
  if (lane == 0) choice_part[warp] = choices;
  __syncthreads();
  if (tid == 0) {
    // share_e / count_e as a sum of two f32 (one thread's 64-bit division: every
    // thread's own took 3 us).
    int64_t total = 0;
    for (int w = 0; w < warps; ++w) total += choice_part[w];
    const int tokens = count_of[E];
    const double scale =
        tokens > 0 ? static_cast<double>(E) / (static_cast<double>(total) * tokens) : 0.0;
    scale_of = make_float2(static_cast<float>(scale),
                           static_cast<float>(scale - static_cast<float>(scale)));
  }
  __syncthreads();
  const float2 scale = scale_of;
  float l = 0.0f;
  for (int e = tid; e < E; e += blockDim.x) {
    const float count = static_cast<float>(count_of[e]);
    const float s = fmaf(count, scale.x, count * scale.y);
    shares[e] = s;
    l = fmaf(s, sum_of[e], l);
  }
#pragma unroll
  for (int d = 16; d > 0; d /= 2) l += __shfl_xor_sync(0xFFFFFFFFu, l, d);
  if (lane == 0) loss_part[warp] = l;
  __syncthreads();
  if (tid == 0) {
    l = 0.0f;
    for (int w = 0; w < warps; ++w) l += loss_part[w];
    *loss = l;
  }
}

template <class T, bool kVec, int kLanes>
__global__ void __launch_bounds__(block_threads<kLanes>(), 1)
    balance_sums_kernel(const BalanceArgs p) {
  extern __shared__ float smem[];   // [E] counts, [1] tokens, then the groups' sums
  __shared__ float warp_part[32];
  int* hist = reinterpret_cast<int*>(smem);
  float* sums_of = smem + p.E + 1;
  for (int e = threadIdx.x; e <= p.E; e += blockDim.x) hist[e] = 0;
  griddep_wait();
  griddep_launch_dependents();
  __syncthreads();
  const int lane = static_cast<int>(threadIdx.x) % kLanes;
  float sum[kV] = {};
  walk_rows<T, kVec, kLanes>(
      p, warp_part,
      [&](int64_t, const float (&e)[kV], float inv, bool some) {
        if (!some) return;
        if (lane == 0) atomicAdd(hist + p.E, 1);
#pragma unroll
        for (int i = 0; i < kV; ++i) sum[i] = fmaf(e[i], inv, sum[i]);
      },
      [&](int id) { atomicAdd(hist + id, 1); });   // (counts: any order gives them)
  // Over the groups of a warp, then all warps' sums, each expert's in order.
#pragma unroll
  for (int d = kLanes; d < 32; d *= 2) {
#pragma unroll
    for (int i = 0; i < kV; ++i) sum[i] += __shfl_xor_sync(0xFFFFFFFFu, sum[i], d);
  }
  constexpr int kParts = kLanes < 32 ? 32 : kLanes;       // lanes of a part
  constexpr int kGroups = block_threads<kLanes>() / kParts;
  const int group = static_cast<int>(threadIdx.x) / kParts;
  if (static_cast<int>(threadIdx.x) % kParts < kLanes) {
#pragma unroll
    for (int i = 0; i < kV; ++i) {
      const int e = expert_of<T, kVec, kLanes>(lane, i);
      if (e < p.E) sums_of[group * p.E + e] = sum[i];
    }
  }
  __syncthreads();
  const bool alone = gridDim.x == 1;
  for (int e = threadIdx.x; e < p.E; e += blockDim.x) {
    float s[4] = {};
    for (int g = 0; g < kGroups; g += 4) {
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (g + j < kGroups) s[j] += sums_of[(g + j) * p.E + e];
    }
    const float all = (s[0] + s[1]) + (s[2] + s[3]);
    if (alone)
      sums_of[e] = all;             // (this thread's own column)
    else
      p.sums[static_cast<int64_t>(blockIdx.x) * p.E + e] = all;
  }
  __syncthreads();
  if (alone) {
    finish_loss(sums_of, hist, p.E, p.loss, p.counts, p.out_shares);
    return;
  }
  for (int e = threadIdx.x; e <= p.E; e += blockDim.x)
    p.counts_of[static_cast<int64_t>(blockIdx.x) * (p.E + 1) + e] = hist[e];
}

// Sums over the blocks, and the results: by one cluster, an eighth of the experts to
// each CTA, whose sums and counts the first one collects.  (One block of 1024
// threads: 16 us for 152 blocks of 256 experts.)
constexpr int kJoinCtas = 8;
constexpr int kJoinThreads = 1024;

__device__ __forceinline__ void st_cluster(uint32_t addr, uint32_t v) {
  asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}

__global__ void __launch_bounds__(kJoinThreads)
    balance_join_kernel(const float* sums, const int* counts_of, int blocks, int E, float* loss,
                        int* counts, float* shares) {
  extern __shared__ float smem[];            // of the first CTA: [E] sums, [E + 1] counts
  __shared__ float sum_part[kJoinThreads];
  __shared__ int count_part[kJoinThreads];
  const int rank = static_cast<int>(cluster_ctarank());
  const int tid = static_cast<int>(threadIdx.x);
  const int share = (E + kJoinCtas) / kJoinCtas;          // of E + 1 counts, the tokens last
  const int first = rank * share;
  const int mine = min(E + 1 - first, share);             // (may be negative)
  // A power of two of neighbouring threads for the experts, the others its parts.
  int width = 1;
  while (width < share && width < kJoinThreads) width *= 2;
  const int parts = kJoinThreads / width;
  const int x = tid % width, part = tid / width;
  const uint32_t sum_dst = map_to_cta(smem_addr(smem), 0u);
  const uint32_t count_dst = map_to_cta(smem_addr(smem + E), 0u);
  cluster_sync();                            // (the first CTA is there)
  griddep_wait();
  griddep_launch_dependents();
  for (int e0 = 0; e0 < share; e0 += width) {
    const int e = first + e0 + x;
    float s = 0.0f;
    int n = 0;
    if (e0 + x < mine) {
#pragma unroll 10
      for (int b = part; b < blocks; b += parts) {
        if (e < E) s += __ldcg(sums + static_cast<int64_t>(b) * E + e);
        n += __ldcg(counts_of + static_cast<int64_t>(b) * (E + 1) + e);
      }
    }
    sum_part[tid] = s;
    count_part[tid] = n;
    __syncthreads();
    for (int half = parts / 2; half > 0; half /= 2) {
      if (part < half) {
        sum_part[tid] += sum_part[tid + half * width];
        count_part[tid] += count_part[tid + half * width];
      }
      __syncthreads();
    }
    if (part == 0 && e0 + x < mine) {
      if (e < E) st_cluster(sum_dst + 4u * static_cast<uint32_t>(e), __float_as_uint(sum_part[tid]));
      st_cluster(count_dst + 4u * static_cast<uint32_t>(e), static_cast<uint32_t>(count_part[tid]));
    }
    __syncthreads();
  }
  cluster_sync();
  if (rank == 0)
    finish_loss(smem, reinterpret_cast<const int*>(smem + E), E, loss, counts, shares);
}

// A lane's gradients of a row.
template <class T, class TD, bool kVec, int kLanes>
__device__ __forceinline__ void store_gradients(TD* row, int E, int lane, const float (&v)[kV]) {
  // (Where the types differ in size, a lane's 16 bytes of one are 8 or 32 of the other.)
  constexpr int kW = kVec ? 16 / static_cast<int>(sizeof(T)) : 1;
#pragma unroll
  for (int i = 0; i < kV; i += kW) {
    const int e = expert_of<T, kVec, kLanes>(lane, i);
    if (kVec && e + kW <= E) {
      if constexpr (sizeof(TD) == 4) {
#pragma unroll
        for (int j = 0; j < kW; j += 4)
          *reinterpret_cast<float4*>(row + e + j) =
              make_float4(v[(i + j) % kV], v[(i + j + 1) % kV], v[(i + j + 2) % kV], v[(i + j + 3) % kV]);
      } else {
        uint32_t w[kW > 1 ? kW / 2 : 1];
#pragma unroll
        for (int j = 0; j + 1 < kW; j += 2) w[j / 2] = pack_bf16x2(v[i + j], v[(i + j + 1) % kV]);
        if constexpr (kW == 8)
          *reinterpret_cast<uint4*>(row + e) = make_uint4(w[0], w[1], w[2], w[3]);
        else if constexpr (kW == 4)
          *reinterpret_cast<uint2*>(row + e) = make_uint2(w[0], w[1]);
      }
    } else {
#pragma unroll
      for (int j = 0; j < kW; ++j) {
        if (e + j >= E) continue;
        if constexpr (sizeof(TD) == 2)
          *reinterpret_cast<uint16_t*>(row + e + j) =
              static_cast<uint16_t>(pack_bf16x2(v[i + j], v[i + j]) & 0xFFFFu);
        else
          *reinterpret_cast<float*>(row + e + j) = v[i + j];
      }
    }
  }
}

template <class T, class TD, bool kVec, int kLanes>
__global__ void __launch_bounds__(block_threads<kLanes>(), 1)
    balance_grad_kernel(const BalanceArgs p) {
  __shared__ float warp_part[32];
  griddep_wait();
  griddep_launch_dependents();
  const int lane = static_cast<int>(threadIdx.x) % kLanes;
  const float g = p.grad ? *p.grad : 1.0f;
  float share[kV];
#pragma unroll
  for (int i = 0; i < kV; ++i) {
    const int e = expert_of<T, kVec, kLanes>(lane, i);
    share[i] = e < p.E ? p.shares[e] : 0.0f;
  }
  walk_rows<T, kVec, kLanes>(
      p, warp_part,
      [&](int64_t row, const float (&e)[kV], float inv, bool some) {
        float dot = 0.0f;
#pragma unroll
        for (int i = 0; i < kV; ++i) dot = fmaf(e[i], share[i], dot);
        dot = over_group<false, kLanes>(dot, warp_part) * inv;
        if (row >= p.M) return;
        const float w = g * inv;
        float v[kV];
#pragma unroll
        for (int i = 0; i < kV; ++i) v[i] = some ? w * e[i] * (share[i] - dot) : 0.0f;
        store_gradients<T, TD, kVec, kLanes>(static_cast<TD*>(p.D) + row * p.ldd, p.E, lane, v);
      },
      [](int) {});
}

// Lanes of a row's group: 1, 4, 16 (up to 16, 64, 256 experts), 32 or a block.
int balance_lanes(int E) {
  if (E > kGroupExperts) return kBlockLanes;
  int lanes = 1;
  while (lanes * kV < E) lanes *= 4;
  return lanes < 32 ? lanes : 32;
}

// Blocks of a pass: one on each of 152 SMs (more would be more sums to join), every
// group taking at least a row.
constexpr int64_t kMostBlocks = 152;
int64_t balance_blocks(int64_t M, int E) {
  const int lanes = balance_lanes(E);
  const int64_t rows = lanes == kBlockLanes ? 1 : kThreads / lanes;
  const int64_t b = (M + rows - 1) / rows;
  return b < 1 ? 1 : b < kMostBlocks ? b : kMostBlocks;
}
// Of sums: one alone while that takes its groups no more than four rows (500 rows of
// 64 experts: a launch less).
int64_t sum_blocks(int64_t M, int E) {
  const int64_t b = balance_blocks(M, E);
  return b <= 4 ? 1 : b;
}

// Whether rows may be read (or written) 16 bytes at a time.
bool whole_pieces(const void* p, int64_t ld, int dtype) {
  return (reinterpret_cast<uintptr_t>(p) & 15u) == 0 && ld * (dtype == TG_D_BF16 ? 2 : 4) % 16 == 0;
}

template <class T, bool kVec, int kLanes>
int launch_sums(const BalanceArgs& a, int64_t blocks, cudaStream_t stream) {
  constexpr int threads = block_threads<kLanes>();
  // (43 KB at most: 512 experts in 20 warps)
  const size_t smem = 4 * (static_cast<size_t>(a.E) + 1 +
                           static_cast<size_t>(threads / (kLanes < 32 ? 32 : kLanes)) * a.E);
  return launch_chained(balance_sums_kernel<T, kVec, kLanes>, blocks, threads, smem, 1, stream, a);
}

template <class T, class TD, bool kVec, int kLanes>
int launch_gradients(const BalanceArgs& a, int64_t blocks, cudaStream_t stream) {
  return launch_chained(balance_grad_kernel<T, TD, kVec, kLanes>, blocks, block_threads<kLanes>(),
                        0, 1, stream, a);
}

// f(16-byte pieces, lanes of a group) with both as template arguments.
template <class F>
int by_form(bool vec, int lanes, F f) {
  auto with = [&](auto v) {
    switch (lanes) {
      case 1: return f(v, std::integral_constant<int, 1>{});
      case 4: return f(v, std::integral_constant<int, 4>{});
      case 16: return f(v, std::integral_constant<int, 16>{});
      case 32: return f(v, std::integral_constant<int, 32>{});
      default: return f(v, std::integral_constant<int, kBlockLanes>{});
    }
  };
  return vec ? with(std::true_type{}) : with(std::false_type{});
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

int64_t balance_workspace_bytes(int64_t E) {
  return E < 1 || E > TG_MAX_GROUPS ? -TG_ERR_INVALID_ARG : kMostBlocks * (2 * E + 1) * 4;
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
  const int64_t blocks = sum_blocks(M, static_cast<int>(E));
  float* sums = nullptr;   // (one block keeps its own)
  if (blocks > 1) {
    sums = static_cast<float*>(device_workspace(static_cast<size_t>(balance_workspace_bytes(E)), stream, &rc));
    if (sums == nullptr) return rc;
  }
  BalanceArgs a{};
  a.logits = logits;
  a.ld = ld;
  a.ids = ids;
  a.choices = static_cast<int>(choices);
  a.M = static_cast<int>(M);
  a.E = static_cast<int>(E);
  a.sums = sums;
  a.counts_of = blocks > 1 ? reinterpret_cast<int*>(sums + blocks * E) : nullptr;
  a.loss = loss;
  a.counts = counts;
  a.out_shares = shares;
  rc = by_form(whole_pieces(logits, ld, dtype), balance_lanes(a.E), [&](auto vec, auto lanes) {
    constexpr bool kVec = decltype(vec)::value;
    constexpr int kLanes = decltype(lanes)::value;
    return dtype == TG_D_BF16 ? launch_sums<uint16_t, kVec, kLanes>(a, blocks, stream)
                              : launch_sums<float, kVec, kLanes>(a, blocks, stream);
  });
  if (rc != TG_OK || blocks == 1) return rc;
  return launch_chained(balance_join_kernel, kJoinCtas, kJoinThreads,
                        4 * static_cast<size_t>(2 * E + 1), kJoinCtas, stream,
                        a.sums, a.counts_of, static_cast<int>(blocks), a.E, loss, counts, shares);
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
  a.shares = shares;
  a.grad = grad;
  a.D = D;
  a.ldd = ldd;
  const int64_t blocks = balance_blocks(M, a.E);
  const bool whole = whole_pieces(logits, ld, dtype) && whole_pieces(D, ldd, d_dtype);
  return by_form(whole, balance_lanes(a.E), [&](auto vec, auto lanes) {
    constexpr bool kVec = decltype(vec)::value;
    constexpr int kLanes = decltype(lanes)::value;
    const bool in16 = dtype == TG_D_BF16, out16 = d_dtype == TG_D_BF16;
    if (in16 && out16) return launch_gradients<uint16_t, uint16_t, kVec, kLanes>(a, blocks, stream);
    if (in16) return launch_gradients<uint16_t, float, kVec, kLanes>(a, blocks, stream);
    if (out16) return launch_gradients<float, uint16_t, kVec, kLanes>(a, blocks, stream);
    return launch_gradients<float, float, kVec, kLanes>(a, blocks, stream);
  });
}

}  // extern "C"
