// Rows of a table by token id, and the table's gradient.
//
//   embed_rows       D[i] = scale * W[ids[i]]
//   embed_rows_grad  dW[v] (+)= scale * sum over {i : ids[i] = v} of G[i]
//
// Both are bound by HBM: every row is moved once.  The lookup gives each warp a
// part of a row.  The gradient must not depend on the order in which anything
// runs, so the rows are first sorted by id (stable; few by counting the smaller
// ones, more by merging sorted chunks, many digit by digit with the sort of
// group_rows.cu; very few not at all: a block looks its row's id up among all), and
// a run of equal ids is summed in the order of its rows, in f32.  Runs are as uneven
// as words are: the sorted rows are cut into chunks of equal length, a warp for each
// and 256 columns; a run that lies inside its chunk goes straight to dW, what
// crosses a chunk's end goes to the workspace as an f32 partial sum, and a second
// kernel adds a run's partial sums in their order.  The rows of dW that no token has
// (nearly all of a large table's) are written as zeros by further blocks of the
// first kernel, meanwhile.
#include <atomic>

#include "chained_launch.cuh"
#include "tg_ptx.cuh"

using namespace tg;

namespace tg {
namespace {

constexpr int64_t kMaxDim = (int64_t{1} << 31) - 1;
constexpr int64_t kMaxTokens = int64_t{1} << 30;   // as tg_group_rows
constexpr int64_t kMostColumns = int64_t{256} * 65535;

// Eight values of a row, from column k on, as they lie in memory; what lies past
// column K is neither read nor written.
template <class T>
struct Eight {
  uint4 q[sizeof(T) / 2];

  __device__ __forceinline__ void load(const T* row, int k, int K) {
    constexpr int kPer = 16 / static_cast<int>(sizeof(T));
    if (k + 8 <= K) {
#pragma unroll
      for (int h = 0; h < static_cast<int>(sizeof(T)) / 2; ++h)
        q[h] = __ldcs(reinterpret_cast<const uint4*>(row + k + kPer * h));
    } else {
      uint32_t w[4 * sizeof(T) / 2] = {};
#pragma unroll
      for (int e = 0; e < 7; ++e) {
        if (k + e >= K) continue;
        if constexpr (sizeof(T) == 2)
          w[e / 2] |= static_cast<uint32_t>(row[k + e]) << (16 * (e & 1));
        else
          w[e] = __float_as_uint(row[k + e]);
      }
#pragma unroll
      for (int h = 0; h < static_cast<int>(sizeof(T)) / 2; ++h)
        q[h] = make_uint4(w[4 * h], w[4 * h + 1], w[4 * h + 2], w[4 * h + 3]);
    }
  }
  __device__ __forceinline__ float value(int e) const {
    const uint4& p = q[e * static_cast<int>(sizeof(T)) / 16];
    const int i = sizeof(T) == 2 ? e / 2 : e % 4;
    const uint32_t w = i == 0 ? p.x : i == 1 ? p.y : i == 2 ? p.z : p.w;
    if constexpr (sizeof(T) == 2) return __uint_as_float(e & 1 ? w & 0xFFFF0000u : w << 16);
    return __uint_as_float(w);
  }
};

template <class T>
__device__ __forceinline__ void load8(const T* row, int k, int K, float (&v)[8]) {
  Eight<T> r;
  r.load(row, k, K);
#pragma unroll
  for (int e = 0; e < 8; ++e) v[e] = r.value(e);
}

template <class T>
__device__ __forceinline__ void store8(T* row, int k, int K, const float (&v)[8]) {
  if constexpr (sizeof(T) == 2) {
    uint32_t w[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) w[e] = pack_bf16x2(v[2 * e], v[2 * e + 1]);
    if (k + 8 <= K) {
      __stcs(reinterpret_cast<uint4*>(row + k), make_uint4(w[0], w[1], w[2], w[3]));
    } else {
#pragma unroll
      for (int e = 0; e < 7; ++e)
        if (k + e < K) row[k + e] = static_cast<T>(w[e / 2] >> (16 * (e & 1)));
    }
  } else {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      if (k + 4 * h + 4 <= K)
        __stcs(reinterpret_cast<float4*>(row + k + 4 * h),
               make_float4(v[4 * h], v[4 * h + 1], v[4 * h + 2], v[4 * h + 3]));
      else
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (k + 4 * h + e < K) row[k + 4 * h + e] = v[4 * h + e];
    }
  }
}

// ---------------------------------------------------------------------------
// Lookup
// ---------------------------------------------------------------------------

// A warp's item: up to kLookup * 256 columns of one row, all loads in flight.
constexpr int kLookup = 2;

template <class TD>
__global__ void __launch_bounds__(256, 8) embed_kernel(const uint16_t* W, int64_t ldw, int vocab,
                                                    const int* ids, int64_t n, int K, int parts,
                                                    float scale, TD* D, int64_t ldd) {
  griddep_wait();
  griddep_launch_dependents();
  const int lane = static_cast<int>(threadIdx.x & 31);
  const int64_t items = n * parts;
  for (int64_t i = blockIdx.x * 8LL + (threadIdx.x >> 5); i < items; i += gridDim.x * 8LL) {
    const int64_t row = i / parts;
    const int k0 = static_cast<int>(i - row * parts) * (256 * kLookup) + 8 * lane;
    const int id = ids[row];
    const bool in = static_cast<unsigned>(id) < static_cast<unsigned>(vocab);
    Eight<uint16_t> w[kLookup];
#pragma unroll
    for (int u = 0; u < kLookup; ++u) {
      w[u].q[0] = make_uint4(0u, 0u, 0u, 0u);
      if (in && k0 + 256 * u < K) w[u].load(W + id * ldw, k0 + 256 * u, K);
    }
#pragma unroll
    for (int u = 0; u < kLookup; ++u) {
      if (k0 + 256 * u >= K) continue;
      float v[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = in ? w[u].value(e) * scale : 0.0f;
      store8(D + row * ldd, k0 + 256 * u, K, v);
    }
  }
}

// ---------------------------------------------------------------------------
// Gradient
// ---------------------------------------------------------------------------

// Sorting up to kFewTokens ids in one launch: a row's place is the number of smaller
// (id, row) pairs, packed into 32 bits.  A block holds all pairs in shared memory and
// places 64 rows, 16 threads to each.
constexpr int kFewTokens = 8192;
constexpr int kFewBits = 13;
constexpr int64_t kFewRows = (int64_t{1} << (32 - kFewBits)) - 1;

__global__ void __launch_bounds__(1024) rank_ids_kernel(const int* ids, int n, int vocab,
                                                        int* order, int* sorted, int* note_count) {
  extern __shared__ uint4 keys4[];
  uint32_t* keys = reinterpret_cast<uint32_t*>(keys4);
  griddep_wait();
  griddep_launch_dependents();
  const int tid = static_cast<int>(threadIdx.x);
  const int n4 = (n + 3) / 4;
  for (int i = tid; i < 4 * n4; i += 1024) {
    uint32_t key = 0xFFFFFFFFu;
    if (i < n) {
      const int id = ids[i];
      const bool in = static_cast<unsigned>(id) < static_cast<unsigned>(vocab);
      key = static_cast<uint32_t>(in ? id : vocab) << kFewBits | static_cast<uint32_t>(i);
    }
    keys[i] = key;
  }
  if (blockIdx.x == 0 && tid == 0) *note_count = 0;
  __syncthreads();
  const int i = static_cast<int>(blockIdx.x) * 64 + tid / 16;
  const uint32_t mine = keys[i < n ? i : 0];
  int rank = 0;
#pragma unroll 4
  for (int j = tid % 16; j < n4; j += 16) {
    const uint4 k = keys4[j];
    rank += (k.x < mine) + (k.y < mine) + (k.z < mine) + (k.w < mine);
  }
#pragma unroll
  for (int d = 8; d > 0; d /= 2) rank += __shfl_xor_sync(0xFFFFFFFFu, rank, d);
  if (i < n && tid % 16 == 0) {
    const int id = static_cast<int>(mine >> kFewBits);
    order[rank] = i;
    sorted[rank] = id < vocab ? id : -1;
  }
}

// Up to kMergeTokens in two launches.  The first sorts chunks of 1024 in the same way
// (64 rows a block); the second holds the sorted chunks' ids in shared memory, and an
// id's place is the sum of its places in all of them, one lane's binary search in
// each: behind equal ids in the chunks before its own, before those in later ones.
// (32768 ids, two digits of the counting sort: 30 us for four launches.)
constexpr int kChunkBits = 10;
constexpr int kChunkIds = 1 << kChunkBits;
constexpr int kMergeTokens = 48 * kChunkIds;
constexpr int64_t kMergeRows = (int64_t{1} << (32 - kChunkBits)) - 1;

__global__ void __launch_bounds__(1024) sort_chunks_kernel(const int* ids, int n, int vocab,
                                                           int* chunk_ids, int* chunk_rows,
                                                           int* note_count) {
  __shared__ uint4 keys4[kChunkIds / 4];
  uint32_t* keys = reinterpret_cast<uint32_t*>(keys4);
  griddep_wait();
  griddep_launch_dependents();
  const int tid = static_cast<int>(threadIdx.x);
  const int base = static_cast<int>(blockIdx.x) / (kChunkIds / 64) * kChunkIds;
  uint32_t key = 0xFFFFFFFFu;
  if (base + tid < n) {
    const int id = ids[base + tid];
    const bool in = static_cast<unsigned>(id) < static_cast<unsigned>(vocab);
    key = static_cast<uint32_t>(in ? id : vocab) << kChunkBits | static_cast<uint32_t>(tid);
  }
  keys[tid] = key;
  if (blockIdx.x == 0 && tid == 0) *note_count = 0;
  __syncthreads();
  const int i = static_cast<int>(blockIdx.x) % (kChunkIds / 64) * 64 + tid / 16;
  const uint32_t mine = keys[i];
  int rank = 0;
#pragma unroll 4
  for (int j = tid % 16; j < kChunkIds / 4; j += 16) {
    const uint4 k = keys4[j];
    rank += (k.x < mine) + (k.y < mine) + (k.z < mine) + (k.w < mine);
  }
#pragma unroll
  for (int d = 8; d > 0; d /= 2) rank += __shfl_xor_sync(0xFFFFFFFFu, rank, d);
  if (base + i < n && tid % 16 == 0) {
    chunk_ids[base + rank] = static_cast<int>(mine >> kChunkBits);
    chunk_rows[base + rank] = base + i;
  }
}

__global__ void __launch_bounds__(1024) merge_chunks_kernel(const int* chunk_ids,
                                                            const int* chunk_rows, int n, int vocab,
                                                            int* order, int* sorted) {
  // (Chunks a word further apart than they are long: the lanes' searches, each in its
  // own, would else meet in one bank: 32768 ids 40 us.)
  extern __shared__ int ids[];
  constexpr int kStride = kChunkIds + 1;
  griddep_wait();
  griddep_launch_dependents();
  const int tid = static_cast<int>(threadIdx.x), lane = tid & 31;
  for (int i0 = tid; i0 < n; i0 += 8 * 1024) {
    int v[8];
#pragma unroll
    for (int u = 0; u < 8; ++u) v[u] = i0 + 1024 * u < n ? __ldcg(chunk_ids + i0 + 1024 * u) : 0;
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      const int i = i0 + 1024 * u;
      if (i < n) ids[(i >> kChunkBits) * kStride + (i & (kChunkIds - 1))] = v[u];
    }
  }
  __syncthreads();
  const int chunks = (n + kChunkIds - 1) >> kChunkBits;
  for (int e = static_cast<int>(blockIdx.x) * 32 + (tid >> 5); e < n;
       e += static_cast<int>(gridDim.x) * 32) {
    const int own = e >> kChunkBits, id = ids[own * kStride + (e & (kChunkIds - 1))];
    int rank = 0;
    for (int c = lane; c < chunks; c += 32) {
      if (c == own) {
        rank += e & (kChunkIds - 1);
        continue;
      }
      // The first place whose id is above (chunks before) or not below (behind).
      const int bound = c < own ? id : id - 1;
      const int* at = ids + c * kStride;
      int lo = 0, hi = min(kChunkIds, n - (c << kChunkBits));
      while (lo < hi) {
        const int mid = (lo + hi) / 2;
        if (at[mid] <= bound)
          lo = mid + 1;
        else
          hi = mid;
      }
      rank += lo;
    }
    rank = __reduce_add_sync(0xFFFFFFFFu, rank);
    if (lane == 0) {
      order[rank] = __ldcg(chunk_rows + e);
      sorted[rank] = id < vocab ? id : -1;
    }
  }
}

int launch_merge_sort(const int* ids, int n, int vocab, int* order, int* sorted, int* chunk_ids,
                      int* chunk_rows, int* note_count, cudaStream_t stream, DeviceCtx* ctx) {
  static std::atomic<int> prepared[64];
  if (prepared[ctx->device].load(std::memory_order_acquire) == 0) {
    const cudaError_t e = cudaFuncSetAttribute(
        merge_chunks_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
        4 * (kMergeTokens + kMergeTokens / kChunkIds));
    if (e != cudaSuccess) return cuda_fail(e);
    prepared[ctx->device].store(1, std::memory_order_release);
  }
  // (Whole chunks of 16 blocks; those past the last row have nothing to place.)
  int rc = launch_chained(sort_chunks_kernel, (n + 63) / 64, 1024, 0, 1, stream, ids, n, vocab,
                          chunk_ids, chunk_rows, note_count);
  if (rc != TG_OK) return rc;
  const int blocks = (n + 31) / 32 < ctx->num_sms ? (n + 31) / 32 : ctx->num_sms;
  return launch_chained(merge_chunks_kernel, blocks, 1024,
                        static_cast<size_t>(4 * (n + (n + kChunkIds - 1) / kChunkIds)), 1, stream,
                        chunk_ids, chunk_rows, n, vocab, order, sorted);
}

struct EmbedGradArgs {
  const void* G;
  int64_t ldg;
  int n, vocab, K;
  const int* ids;
  const int* order;       // rows by id
  const int* sorted;      // their ids, -1 for rows of none (last)
  const unsigned* marks;  // a bit for each id that occurs, or null: looked up in `sorted`
  float scale;
  void* D;
  int64_t ldd;
  int* note_count;        // runs to be joined, zero before; for each a note:
  int2* notes;            // its first chunk, its first slice (long runs: -1 - slice)
  float* parts;           // [chunk][2][ldp]: sums of a chunk's first and last run
  int64_t ldp;
  int chunk;              // sorted rows per warp, a multiple of kBatch
  int chunks, slices;     // warps of sums: chunks x slices of kSlice columns
};

constexpr int kSlice = 256;       // columns of a warp
constexpr int kWarps = 4;         // of a block, each with a slice of its own
constexpr int kBatch = 8;         // rows loaded together
constexpr int kLongRun = 32;      // chunks, from which on a whole block joins a slice

// The finished sum of an id's rows.
template <class TD, bool kAdd>
__device__ __forceinline__ void finish_run(const EmbedGradArgs& p, int id, int k, float (&v)[8]) {
  TD* d = static_cast<TD*>(p.D) + id * p.ldd;
#pragma unroll
  for (int e = 0; e < 8; ++e) v[e] *= p.scale;
  if constexpr (kAdd) {
    float old[8];
    load8(d, k, p.K, old);
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] += old[e];
  }
  store8(d, k, p.K, v);
}

// Untiled bulk copy shared -> global (16-byte aligned, size % 16 == 0).
__device__ __forceinline__ void bulk_store(void* dst, uint32_t src, uint32_t bytes) {
  asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(dst), "r"(src),
               "r"(bytes)
               : "memory");
}

// Whether v is among the sorted ids (behind which those of no row lie as -1).
__device__ __forceinline__ bool has_token(const int* sorted, int n, int64_t v) {
  int lo = 0, hi = n;
  while (lo < hi) {
    const int mid = (lo + hi) / 2;
    const int id = sorted[mid];
    if (id == v) return true;
    if (id >= 0 && id < v)
      lo = mid + 1;
    else
      hi = mid;
  }
  return false;
}

// Rows that no token has, a thread each, as bulk copies of zeros: 1 GB of them by
// 16-byte stores of whole warps, in blocks behind those of the sums, took 260 us
// with the sums of 32768 rows x 4096 in 128000.
constexpr int kZeros = 8192;      // bytes

// used(v): whether row v has a token.
template <class TD, class F>
__device__ __forceinline__ void clear_unused(const EmbedGradArgs& p, int64_t block, int64_t blocks,
                                             F used) {
  __shared__ __align__(128) uint4 zeros[kZeros / 16];
  for (int i = threadIdx.x; i < kZeros / 16; i += blockDim.x) zeros[i] = make_uint4(0u, 0u, 0u, 0u);
  fence_proxy_async_smem();
  __syncthreads();
  const uint32_t src = smem_addr(zeros);
  const int64_t bytes = static_cast<int64_t>(p.K) * sizeof(TD);
  const int64_t whole = bytes / 16 * 16;
  // (Rows far apart: a block's copies go out one after the other, and a small
  // table needs many blocks.)
  for (int64_t v = block + threadIdx.x * blocks; v < p.vocab; v += blocks * blockDim.x) {
    if (used(v)) continue;
    uint8_t* d = reinterpret_cast<uint8_t*>(static_cast<TD*>(p.D) + v * p.ldd);
    for (int64_t at = 0; at < whole; at += kZeros)
      bulk_store(d + at, src, static_cast<uint32_t>(whole - at < kZeros ? whole - at : kZeros));
    for (int64_t at = whole; at < bytes; at += sizeof(TD)) *reinterpret_cast<TD*>(d + at) = 0;
  }
  bulk_commit_group();
  bulk_wait_group0();
}

// Blocks of sums (a warp has a chunk of the rows and a slice of the columns) and
// blocks of zeros, evenly mixed: sums wait for memory's answers, zeros only for its
// room.
template <class TG, class TD, bool kAdd>
__global__ void __launch_bounds__(32 * kWarps) sum_runs_kernel(const EmbedGradArgs p) {
  griddep_wait();
  griddep_launch_dependents();
  const int64_t items = static_cast<int64_t>(p.chunks) * p.slices;
  const int64_t zeros = gridDim.x - (items + kWarps - 1) / kWarps;
  const int64_t before = blockIdx.x * zeros / gridDim.x;      // blocks of zeros
  if ((blockIdx.x + 1) * zeros / gridDim.x > before) {
    clear_unused<TD>(p, before, zeros, [&](int64_t v) -> bool {
      if (p.marks != nullptr) return (__ldcg(p.marks + (v >> 5)) >> (v & 31)) & 1u;
      return has_token(p.sorted, p.n, v);
    });
    return;
  }
  const int64_t item = (blockIdx.x - before) * kWarps + (threadIdx.x >> 5);
  if (item >= items) return;
  const int lane = static_cast<int>(threadIdx.x & 31);
  const int c = static_cast<int>(item / p.slices);
  const int k = static_cast<int>(item - static_cast<int64_t>(c) * p.slices) * kSlice + 8 * lane;
  const bool in = k < p.K;
  const int lo = c * p.chunk;
  const int hi = p.n - lo > p.chunk ? lo + p.chunk : p.n;
  const TG* G = static_cast<const TG*>(p.G);
  // The first run may have begun in an earlier chunk: then its sum is a part.
  int id = p.sorted[lo];
  bool whole = lo == 0 || p.sorted[lo - 1] != id;
  const int behind = hi < p.n ? p.sorted[hi] : -1;
  float sum[8] = {};
  for (int j0 = lo; j0 < hi && id >= 0; j0 += 32) {
    // 32 rows and their ids, a lane each, for the warp's shuffles.
    const int ids = j0 + lane < hi ? p.sorted[j0 + lane] : -1;
    const int rows = j0 + lane < hi ? p.order[j0 + lane] : 0;
    const int valid = __popc(__ballot_sync(0xFFFFFFFFu, ids >= 0));   // (sorted: the first ones)
#pragma unroll 1
    for (int u0 = 0; u0 < valid; u0 += kBatch) {
      Eight<TG> v[kBatch];
#pragma unroll
      for (int u = 0; u < kBatch; ++u) {
        const int row = __shfl_sync(0xFFFFFFFFu, rows, u0 + u);
        if (in && u0 + u < valid) v[u].load(G + row * p.ldg, k, p.K);
      }
#pragma unroll
      for (int u = 0; u < kBatch; ++u) {
        const int of = __shfl_sync(0xFFFFFFFFu, ids, u0 + u);
        if (u0 + u >= valid) break;
        if (of != id) {
          if (in) {
            if (whole)
              finish_run<TD, kAdd>(p, id, k, sum);
            else
              store8(p.parts + 2LL * c * p.ldp, k, p.K, sum);
          }
          id = of;
          whole = true;
#pragma unroll
          for (int e = 0; e < 8; ++e) sum[e] = 0.0f;
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) sum[e] += v[u].value(e);
      }
    }
  }
  if (id < 0) return;
  if (whole && behind == id && lane == 0) {
    // The run goes on: one note for eight slices, or for each of a long run.
    const int64_t far = lo + static_cast<int64_t>(kLongRun) * p.chunk;
    const bool is_long = far < p.n && p.sorted[far] == id;
    const int slice = static_cast<int>(item - static_cast<int64_t>(c) * p.slices);
    if (is_long || slice % 8 == 0) {
      p.notes[atomicAdd(p.note_count, 1)] = make_int2(c, is_long ? -1 - slice : slice);
    }
  }
  if (!in) return;
  if (whole && behind != id)
    finish_run<TD, kAdd>(p, id, k, sum);
  else
    store8(p.parts + (2LL * c + (whole ? 1 : 0)) * p.ldp, k, p.K, sum);
}

// Very few tokens, in one launch: a block for each token and slice of the columns, of
// which that of an id's first token sums all of them, in order; up to kRunOfWarp by
// one warp, more by the four in turn.
constexpr int kVeryFew = 1024;
constexpr int kVeryFewBlocks = 1536;
constexpr int kRunOfWarp = 32;

template <class TG, class TD, bool kAdd>
__global__ void __launch_bounds__(32 * kWarps) sum_few_kernel(const EmbedGradArgs p) {
  __shared__ int4 ids4[kVeryFew / 4];
  int* ids = reinterpret_cast<int*>(ids4);
  __shared__ int list[kVeryFew];
  __shared__ int counts[kWarps];
  __shared__ float part[kWarps][32][8];
  griddep_wait();
  griddep_launch_dependents();
  const int tid = static_cast<int>(threadIdx.x), warp = tid >> 5, lane = tid & 31;
  const int n4 = (p.n + 3) / 4;
  for (int i = tid; i < 4 * n4; i += 32 * kWarps) {
    const int id = i < p.n ? p.ids[i] : -1;
    ids[i] = static_cast<unsigned>(id) < static_cast<unsigned>(p.vocab) ? id : -1;
  }
  __syncthreads();
  const int64_t items = static_cast<int64_t>(p.n) * p.slices;
  const int64_t zeros = gridDim.x - items;
  const int64_t before = blockIdx.x * zeros / gridDim.x;      // blocks of zeros
  if ((blockIdx.x + 1) * zeros / gridDim.x > before) {
    clear_unused<TD>(p, before, zeros, [&](int64_t v) -> bool {
      bool found = false;
      for (int i = 0; i < n4; ++i) {
        const int4 q = ids4[i];
        found |= q.x == v || q.y == v || q.z == v || q.w == v;
      }
      return found;
    });
    return;
  }
  const int item = static_cast<int>(blockIdx.x - before);
  const int first = item / p.slices;
  const int k = (item - first * p.slices) * kSlice + 8 * lane;
  const int id = ids[first];
  if (id < 0) return;
  // The id's tokens in order: each warp has a quarter of them all.
  const int quarter = (p.n + 32 * kWarps - 1) / (32 * kWarps) * 32;
  const int lo = warp * quarter, hi = min(p.n, lo + quarter);
  int found = 0;
  bool earlier = false;
  for (int i0 = lo; i0 < hi; i0 += 32) {
    const bool same = i0 + lane < hi && ids[i0 + lane] == id;
    earlier |= same && i0 + lane < first;
    found += __popc(__ballot_sync(0xFFFFFFFFu, same));
  }
  if (lane == 0) counts[warp] = found;
  if (__syncthreads_or(earlier)) return;   // another block's
  int at = 0, count = 0;
  for (int w = 0; w < kWarps; ++w) {
    if (w < warp) at += counts[w];
    count += counts[w];
  }
  for (int i0 = lo; i0 < hi; i0 += 32) {
    const bool same = i0 + lane < hi && ids[i0 + lane] == id;
    const unsigned votes = __ballot_sync(0xFFFFFFFFu, same);
    if (same) list[at + __popc(votes & ((1u << lane) - 1u))] = i0 + lane;
    at += __popc(votes);
  }
  __syncthreads();
  const bool shared_out = count > kRunOfWarp;
  if (!shared_out && warp != 0) return;
  const TG* G = static_cast<const TG*>(p.G);
  const int by = shared_out ? kWarps : 1;
  float sum[8] = {};
  if (k < p.K) {
    for (int q0 = warp; q0 < count; q0 += kBatch * by) {
      Eight<TG> v[kBatch];
#pragma unroll
      for (int u = 0; u < kBatch; ++u)
        if (q0 + u * by < count) v[u].load(G + list[q0 + u * by] * p.ldg, k, p.K);
#pragma unroll
      for (int u = 0; u < kBatch; ++u)
        if (q0 + u * by < count) {
#pragma unroll
          for (int e = 0; e < 8; ++e) sum[e] += v[u].value(e);
        }
    }
  }
  if (shared_out) {
#pragma unroll
    for (int e = 0; e < 8; ++e) part[warp][lane][e] = sum[e];
    __syncthreads();
    if (warp != 0) return;
    for (int w = 1; w < kWarps; ++w)
#pragma unroll
      for (int e = 0; e < 8; ++e) sum[e] += part[w][lane][e];
  }
  if (k < p.K) finish_run<TD, kAdd>(p, id, k, sum);
}

// Runs that cross the end of the chunk they begin in, as noted by their first
// chunk: its last part and the first of each further one.  A short run's parts are
// added one after the other, a slice to each warp; a long one's slice by the block's
// eight warps in turn, whose sums are then added in order.  (The notes' order is
// chance, what each gives is not.)
template <class TD, bool kAdd>
__global__ void __launch_bounds__(256) join_runs_kernel(const EmbedGradArgs p) {
  __shared__ float shared[8][32][8];
  griddep_wait();
  griddep_launch_dependents();
  const int lane = static_cast<int>(threadIdx.x & 31), warp = static_cast<int>(threadIdx.x >> 5);
  const int notes = __ldcg(p.note_count);
  for (int i = blockIdx.x; i < notes; i += gridDim.x) {
    const int2 note = __ldcg(p.notes + i);
    const int c = note.x, code = note.y;
    auto id_behind = [&](int chunk) {
      const int64_t behind = static_cast<int64_t>(chunk + 1) * p.chunk;
      return behind < p.n ? p.sorted[behind] : -1;
    };
    const int id = id_behind(c);
    int last = c + 1;               // the chunk in which the run ends
    for (;;) {
      const unsigned over = __ballot_sync(0xFFFFFFFFu, id_behind(last + lane) != id);
      if (over) {
        last += __ffs(over) - 1;
        break;
      }
      last += 32;
    }
    const int count = last - c + 1;
    const int64_t step = 2 * p.ldp;
    const float* parts = p.parts + c * step;
    const bool is_long = code < 0;
    const int k = (is_long ? -1 - code : code + warp) * kSlice + 8 * lane;
    // Parts from, from + by, ..., eight in flight.
    const int from = is_long ? warp : 0, by = is_long ? 8 : 1;
    float sum[8] = {};
    if (k < p.K) {
      for (int q0 = from; q0 < count; q0 += 8 * by) {
        Eight<float> v[8];
#pragma unroll
        for (int u = 0; u < 8; ++u) {
          const int q = q0 + u * by;
          if (q < count) v[u].load(parts + q * step + (q == 0 ? p.ldp : 0), k, p.K);
        }
#pragma unroll
        for (int u = 0; u < 8; ++u)
          if (q0 + u * by < count) {
#pragma unroll
            for (int e = 0; e < 8; ++e) sum[e] += v[u].value(e);
          }
      }
    }
    if (is_long) {
#pragma unroll
      for (int e = 0; e < 8; ++e) shared[warp][lane][e] = sum[e];
      __syncthreads();
      if (warp == 0) {
        for (int w = 1; w < 8; ++w)
#pragma unroll
          for (int e = 0; e < 8; ++e) sum[e] += shared[w][lane][e];
      }
      __syncthreads();
    }
    if (k < p.K && (!is_long || warp == 0)) finish_run<TD, kAdd>(p, id, k, sum);
  }
}

// Sorted rows per warp: at most about a thousand chunks, so that a run as long as all
// of them still joins in little time, and no chunk of fewer than kBatch.
constexpr int64_t kMostChunks = 1024;
int grad_chunk(int64_t n) {
  int64_t c = kBatch;
  while (c * kMostChunks < n) c *= 2;
  return static_cast<int>(c);
}

constexpr size_t kNoteCount = 256;   // bytes

struct EmbedPlan {
  int chunk, chunks, slices;
  int64_t ldp;
  size_t other, rows, sorted, count, notes, marks, hist, parts, bytes;   // (marks: the count before)
};
EmbedPlan embed_plan(int64_t n, int64_t rows, int64_t K) {
  EmbedPlan q{};
  q.chunk = grad_chunk(n);
  q.chunks = static_cast<int>((n + q.chunk - 1) / q.chunk);
  q.slices = static_cast<int>((K + kSlice - 1) / kSlice);
  q.ldp = (K + 7) / 8 * 8;
  size_t at = 0;
  auto take = [&](size_t bytes) {
    const size_t was = at;
    at += (bytes + 255) / 256 * 256;
    return was;
  };
  const size_t list = static_cast<size_t>(4 * n);
  take(list);
  q.other = take(list);
  q.rows = take(n < kMergeTokens ? list : 4 * kMergeTokens);
  q.sorted = take(list);
  q.count = take(4 * ((size_t{1} << kSortDigit) + 1));
  // (As many chunks as fewer tokens may have: it grows with n.)
  const int64_t most = (n + kBatch - 1) / kBatch < kMostChunks ? (n + kBatch - 1) / kBatch : kMostChunks;
  q.notes = take(8 * static_cast<size_t>(most) * static_cast<size_t>(q.slices));
  q.marks = take(kNoteCount + static_cast<size_t>((rows + 31) / 32 * 4));
  q.hist = take(sort_ids_workspace_bytes(n));
  q.parts = take(8 * static_cast<size_t>(most) * static_cast<size_t>(q.ldp));
  q.bytes = at;
  return q;
}

template <class TG, class TD, bool kAdd>
int launch_grad(const EmbedGradArgs& a, DeviceCtx* ctx, cudaStream_t stream) {
  int64_t zero_blocks = 0;
  if (!kAdd) {
    zero_blocks = (static_cast<int64_t>(a.vocab) + 7) / 8;
    const int64_t most = 8 * static_cast<int64_t>(ctx->num_sms);
    if (zero_blocks > most) zero_blocks = most;
  }
  if (a.ids != nullptr) {
    // (The zeros look every row up: 1000 tokens are 1000 comparisons a thread.)
    return launch_chained(sum_few_kernel<TG, TD, kAdd>,
                          static_cast<int64_t>(a.n) * a.slices + zero_blocks, 32 * kWarps, 0, 1,
                          stream, a);
  }
  const int64_t blocks =
      (static_cast<int64_t>(a.chunks) * a.slices + kWarps - 1) / kWarps + zero_blocks;
  if (blocks == 0) return TG_OK;
  int rc = launch_chained(sum_runs_kernel<TG, TD, kAdd>, blocks, 32 * kWarps, 0, 1, stream, a);
  if (rc != TG_OK || a.chunks < 2) return rc;
  const int64_t notes = static_cast<int64_t>(a.chunks - 1) * a.slices;
  const int64_t most = 4 * static_cast<int64_t>(ctx->num_sms);
  return launch_chained(join_runs_kernel<TD, kAdd>, notes < most ? notes : most, 256, 0, 1,
                        stream, a);
}

template <class TG, class TD>
int launch_grad(const EmbedGradArgs& a, bool add, DeviceCtx* ctx, cudaStream_t stream) {
  return add ? launch_grad<TG, TD, true>(a, ctx, stream) : launch_grad<TG, TD, false>(a, ctx, stream);
}

int check_rows(const void* p, int64_t ld, int64_t width, int esize) {
  if (p == nullptr || ld < width) return TG_ERR_INVALID_ARG;
  if ((reinterpret_cast<uintptr_t>(p) & 15u) != 0 || (ld * esize) % 16 != 0)
    return TG_ERR_MISALIGNED;
  return TG_OK;
}

int check_embed(int64_t n, int64_t rows, int64_t K, int a_dtype, int d_dtype) {
  if (n < 0 || n > kMaxTokens || rows < 0 || rows > kMaxDim || K < 0 || K > kMaxDim)
    return TG_ERR_INVALID_ARG;
  if (a_dtype != TG_D_F32 && a_dtype != TG_D_BF16) return TG_ERR_INVALID_ARG;
  if (d_dtype != TG_D_F32 && d_dtype != TG_D_BF16) return TG_ERR_INVALID_ARG;
  if (K > kMostColumns) return TG_ERR_UNSUPPORTED;
  return TG_OK;
}

int esize(int dtype) { return dtype == TG_D_BF16 ? 2 : 4; }

}  // namespace

int64_t embed_grad_workspace_bytes(int64_t n, int64_t rows, int64_t K) {
  const int rc = check_embed(n, rows, K, TG_D_F32, TG_D_F32);
  return rc != TG_OK ? -rc : static_cast<int64_t>(embed_plan(n, rows, K).bytes);
}

}  // namespace tg

extern "C" {

int embed_rows(const void* W, int64_t ldw, int64_t rows, const int32_t* ids, int64_t n, int64_t K,
               float scale, void* D, int64_t ldd, int d_dtype, void* cuda_stream) {
  int rc = check_embed(n, rows, K, TG_D_BF16, d_dtype);
  if (rc != TG_OK || n == 0 || K == 0) return rc;
  if (ids == nullptr) return TG_ERR_INVALID_ARG;
  rc = check_rows(D, ldd, K, esize(d_dtype));
  if (rc == TG_OK && rows > 0) rc = check_rows(W, ldw, K, 2);
  if (rc != TG_OK) return rc;
  if (!current_ctx()) return TG_ERR_CUDA;
  cudaStream_t stream = static_cast<cudaStream_t>(cuda_stream);
  const int parts = static_cast<int>((K + 256 * kLookup - 1) / (256 * kLookup));
  // A warp for each part (32768 rows x 4096 of 128000, f32: 126 us; with four pieces a
  // lane 131; in a grid that stays, 150 to 200).
  int64_t blocks = (n * parts + 7) / 8;
  if (blocks > kMaxDim / 2) blocks = kMaxDim / 2;
  const uint16_t* w = static_cast<const uint16_t*>(W);
  const int v = static_cast<int>(rows), k = static_cast<int>(K);
  if (d_dtype == TG_D_BF16)
    return launch_chained(embed_kernel<uint16_t>, blocks, 256, 0, 1, stream, w, ldw, v, ids, n, k, parts,
                          scale, static_cast<uint16_t*>(D), ldd);
  return launch_chained(embed_kernel<float>, blocks, 256, 0, 1, stream, w, ldw, v, ids, n, k, parts,
                        scale, static_cast<float*>(D), ldd);
}

int embed_rows_grad(const void* G, int64_t ldg, int g_dtype, const int32_t* ids, int64_t n,
                    int64_t rows, int64_t K, float scale, void* D, int64_t ldd, int d_dtype,
                    int accumulate, void* cuda_stream) {
  int rc = check_embed(n, rows, K, g_dtype, d_dtype);
  if (rc != TG_OK) return rc;
  if (accumulate != 0 && accumulate != 1) return TG_ERR_INVALID_ARG;
  if (rows == 0 || K == 0 || (accumulate && n == 0)) return TG_OK;
  rc = check_rows(D, ldd, K, esize(d_dtype));
  if (rc != TG_OK) return rc;
  if (n > 0) {
    if (ids == nullptr) return TG_ERR_INVALID_ARG;
    rc = check_rows(G, ldg, K, esize(g_dtype));
    if (rc != TG_OK) return rc;
  }
  DeviceCtx* ctx = current_ctx();
  if (!ctx) return TG_ERR_CUDA;
  cudaStream_t stream = static_cast<cudaStream_t>(cuda_stream);
  EmbedGradArgs a{};
  a.G = G;
  a.ldg = ldg;
  a.n = static_cast<int>(n);
  a.vocab = static_cast<int>(rows);
  a.K = static_cast<int>(K);
  a.scale = scale;
  a.D = D;
  a.ldd = ldd;
  a.slices = static_cast<int>((K + kSlice - 1) / kSlice);
  if (n > 0 && n <= kVeryFew && n * a.slices <= kVeryFewBlocks) {
    a.ids = ids;
  } else if (n > 0) {
    const EmbedPlan plan = embed_plan(n, rows, K);
    if (static_cast<int64_t>(plan.chunks) * plan.slices > kMaxDim / 2) return TG_ERR_UNSUPPORTED;
    uint8_t* ws = static_cast<uint8_t*>(device_workspace(plan.bytes, stream, &rc));
    if (ws == nullptr) return rc;
    a.notes = reinterpret_cast<int2*>(ws + plan.notes);
    a.note_count = reinterpret_cast<int*>(ws + plan.marks);
    int* order = reinterpret_cast<int*>(ws);
    int* sorted = reinterpret_cast<int*>(ws + plan.sorted);
    if (n <= kFewTokens && rows <= kFewRows) {
      rc = launch_chained(rank_ids_kernel, (n + 63) / 64, 1024,
                          static_cast<size_t>((n + 3) / 4 * 16), 1, stream, ids, n, rows, order,
                          sorted, a.note_count);
    } else if (n <= kMergeTokens && rows <= kMergeRows) {
      rc = launch_merge_sort(ids, static_cast<int>(n), static_cast<int>(rows), order, sorted,
                             reinterpret_cast<int*>(ws + plan.other),
                             reinterpret_cast<int*>(ws + plan.rows), a.note_count, stream, ctx);
    } else {
      unsigned* marks =
          accumulate ? nullptr : reinterpret_cast<unsigned*>(ws + plan.marks + kNoteCount);
      const cudaError_t e = cudaMemsetAsync(
          a.note_count, 0,
          kNoteCount + (accumulate ? 0 : static_cast<size_t>((rows + 31) / 32 * 4)), stream);
      if (e != cudaSuccess) return cuda_fail(e);
      rc = sort_ids(ids, n, rows, order, reinterpret_cast<int*>(ws + plan.other), sorted,
                    reinterpret_cast<int*>(ws + plan.count), marks, ws + plan.hist, stream, ctx);
      a.marks = marks;
    }
    if (rc != TG_OK) return rc;
    a.order = order;
    a.sorted = sorted;
    a.parts = reinterpret_cast<float*>(ws + plan.parts);
    a.ldp = plan.ldp;
    a.chunk = plan.chunk;
    a.chunks = plan.chunks;
  }
  const bool add = accumulate != 0, g16 = g_dtype == TG_D_BF16, d16 = d_dtype == TG_D_BF16;
  if (g16 && d16) return launch_grad<uint16_t, uint16_t>(a, add, ctx, stream);
  if (g16) return launch_grad<uint16_t, float>(a, add, ctx, stream);
  if (d16) return launch_grad<float, uint16_t>(a, add, ctx, stream);
  return launch_grad<float, float>(a, add, ctx, stream);
}

}  // extern "C"
