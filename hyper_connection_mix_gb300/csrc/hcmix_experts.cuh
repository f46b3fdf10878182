// Tokens sorted by expert and back: a stable counting sort of the (token, choice)
// pairs, the rows copied to their experts' places and the weighted rows added up
// again, with the gradients.  No atomics: every row has one writer.
//
// The rows' copies are bound by HBM (copy rate 6787 GB/s).  Measured for 4096 tokens of 5120
// bf16 to 8 of 128 experts: sort 8.0 us, dispatch 56 us (378 MB, 6.7 TB/s), combine 53.5 us
// (378 MB, 7.1 TB/s), combine backward 107 us (713 MB, 6.7 TB/s).
#pragma once

#include <cooperative_groups.h>

#include "hcmix_vec.cuh"

namespace hcmix {
namespace sublayer {

struct SortArgs {
  const void* ids;
  int64_t n;  // pairs
  int E;
  int32_t *offsets, *slots, *source;
};

constexpr int kMostExperts = 4096;
constexpr int kSortCounters = 32 * 1024;  // warps * experts, 128 KB
// Pairs that one block sorts: 512 take it 3.3 us and 1024 4.7 us, a cluster 4.0 us.
constexpr int64_t kSortAlone = 512;
// Blocks of the cluster that sorts more.  The scattered stores of source, one sector
// a pair, are shared out over them: 32768 pairs of 128 experts take 16 blocks 8.0 us
// (8 blocks, before the loops were rolled, 10.3 us).  Each holds a row of totals for
// every block, 64 KB in all.
constexpr int kSortBlocks = 16, kSortBlocksWide = 4, kSortWide = 1024;  // past so many experts
inline int sort_blocks(int64_t n, int64_t E) { 
  return n <= kSortAlone ? 1 : E <= kSortWide ? kSortBlocks : kSortBlocksWide;
}
// The most shared memory that a sort takes: counters, totals, starts and the scan's sums.
constexpr int kSortRows = (kSortBlocks + 1) * kSortWide > (kSortBlocksWide + 1) * kMostExperts
                              ? (kSortBlocks + 1) * kSortWide
                              : (kSortBlocksWide + 1) * kMostExperts;
constexpr size_t kSortMost = ((size_t)kSortCounters + kSortRows + 32) * 4;

template <typename Id>
__device__ __forceinline__ int expert_of(const SortArgs& A, int64_t i) {
  const int64_t e = static_cast<const Id*>(A.ids)[i];
  return e >= 0 && e < A.E ? (int)e : A.E;  // A.E: of none
}

// The lanes whose key is this lane's, keys below 2^bits: a ballot for each bit.
// (__match_any_sync takes about 230 cycles of a sub-partition each, ballots of 8
// bits about 50.)
__device__ __forceinline__ unsigned same_key(int key, int bits) {
  unsigned same = 0xffffffffu;
  for (int b = 0; b < bits; ++b, key >>= 1) {
    const bool set = key & 1;
    const unsigned v = __ballot_sync(0xffffffffu, set);
    same &= set ? v : ~v;
  }
  return same;
}

// A barrier of the cluster's threads in two halves: arrive, and wait for all others'.
__device__ __forceinline__ void cluster_arrive() {
  asm volatile("barrier.cluster.arrive.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
  asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
}

// One cluster sorts all pairs.  Each of its warps takes a contiguous range of
// them and walks it in batches of 32, counting its experts in shared memory: a
// pair's rank in its warp is the count so far and the lower lanes with its expert.
// When the counts of the warps and blocks before are known, every pair has its
// place; until then the ranks wait in slots.
//
// Every phase runs once or a few times, so the time is that of latencies, fetching
// the code among them: the loops stay rolled.
template <typename Id>
__global__ void __launch_bounds__(1024) hcmix_expert_sort_kernel(const SortArgs A) {
  begin_kernel();
  namespace cg = cooperative_groups;
  extern __shared__ int sort_shared[];
  const cg::cluster_group cluster = cg::this_cluster();
  const int ctas = cluster.num_blocks(), cta = cluster.block_rank();
  if (ctas > 1) cluster_arrive();
  const int warps = blockDim.x / 32, warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int E = A.E, bits = 32 - __clz(E);  // of the keys 0 .. E
  int* count = sort_shared;         // [warps][E], then the counts of the warps before
  int* totals = count + warps * E;  // [ctas][E] the blocks' pairs of each expert
  int* start = totals + ctas * E;   // [E] the block's first row of each expert
  int* scan = start + E;            // [warps] sums of the scan over experts

  const int64_t ranges = (int64_t)ctas * warps;
  const int64_t span = ((A.n + ranges - 1) / ranges + 31) / 32 * 32;
  const int64_t first = ((int64_t)cta * warps + warp) * span;
  const int64_t last = first + span < A.n ? first + span : A.n;
  const auto key_at = [&](int64_t i) { return i < last ? expert_of<Id>(A, i) : E; };
  int key = key_at(first + lane);
  for (int i = threadIdx.x; i < warps * E; i += blockDim.x) count[i] = 0;
  __syncthreads();
  int* mine = count + warp * E;
  for (int64_t i = first + lane; i - lane < last; i += 32) {
    const int next = key_at(i + 32);
    const unsigned same = same_key(key, bits);
    const int lower = __popc(same & ((1u << lane) - 1));
    const int so_far = key < E ? mine[key] : 0;
    __syncwarp();
    if (lower == 0 && key < E) mine[key] = so_far + __popc(same);
    __syncwarp();
    if (i < last) A.slots[i] = so_far + lower;
    key = next;
  }
  __syncthreads();
  // A block's memory is there for others from its start to its end: they are touched
  // between the barrier on which every block arrives when it starts, and the next one.
  if (ctas > 1) cluster_wait();
  for (int e = threadIdx.x; e < E; e += blockDim.x) {
    int s = 0;
#pragma unroll 4
    for (int w = 0; w < warps; ++w) {
      const int c = count[w * E + e];
      count[w * E + e] = s;
      s += c;
    }
    for (int b = 0; b < ctas; ++b) cluster.map_shared_rank(totals, b)[cta * E + e] = s;
  }
  if (ctas > 1)
    cluster.sync();
  else
    __syncthreads();
  // start[e] = the pairs of all experts before e, and those of e in earlier blocks:
  // a thread takes `per` neighbouring experts
  const int per = (E + blockDim.x - 1) / blockDim.x;
  const int e0 = threadIdx.x * per, e1 = e0 + per < E ? e0 + per : E;
  int sum = 0;
  for (int e = e0; e < e1; ++e) {
    int here = 0;
#pragma unroll 4
    for (int b = 0; b < ctas; ++b) {
      if (b == cta) start[e] = here;
      here += totals[b * E + e];
    }
    totals[e] = here;  // the expert's pairs in all blocks
    sum += here;
  }
  int before = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int t = __shfl_up_sync(0xffffffffu, before, o);
    if (lane >= o) before += t;
  }
  if (lane == 31) scan[warp] = before;
  __syncthreads();
  int all = 0;
  before -= sum;
  const int with_experts = (E + 32 * per - 1) / (32 * per);  // warps
  for (int w = 0; w < with_experts; ++w) {
    const int t = scan[w];
    if (w < warp) before += t;
    all += t;
  }
  for (int e = e0; e < e1; ++e) {
    start[e] += before;
    if (cta == 0) A.offsets[e] = before;
    before += totals[e];
  }
  if (cta == 0 && threadIdx.x == 0) A.offsets[E] = all;
  __syncthreads();
#pragma unroll 2
  for (int64_t i = first + lane; i < last; i += 32) {
    const int e = key_at(i);
    const int place = e < E ? start[e] + mine[e] + A.slots[i] : -1;
    A.slots[i] = place;
    if (place >= 0) A.source[place] = (int)i;
  }
  for (int64_t r = all + (int64_t)cta * blockDim.x + threadIdx.x; r < A.n;
       r += (int64_t)ctas * blockDim.x)
    A.source[r] = -1;
}

template <typename Id>
hcmix_status launch_sort(const SortArgs& A, cudaStream_t stream) {
  const int ctas = sort_blocks(A.n, A.E);
  // a warp for each 32 pairs, as far as there are, so that few pairs need few counters
  int64_t warps = (A.n + 32 * ctas - 1) / (32 * ctas);
  const int most = kSortCounters / A.E < 32 ? kSortCounters / A.E : 32;
  warps = warps < 4 ? 4 : warps > most ? most : warps;
  const size_t smem = (((size_t)warps + ctas + 1) * A.E + 32) * 4;
  if (ctas > 8) {
    const hcmix_status st = checked(cudaFuncSetAttribute(
        hcmix_expert_sort_kernel<Id>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1));
    if (st != HCMIX_OK) return st;
  }
  return launch(hcmix_expert_sort_kernel<Id>, dim3(ctas), dim3((unsigned)warps * 32), smem,
                kSortMost, stream, A, ctas);
}

inline hcmix_status run_sort(const SortArgs& A, bool wide_ids, cudaStream_t stream) {
  return wide_ids ? launch_sort<int64_t>(A, stream) : launch_sort<int32_t>(A, stream);
}

// ---------------------------------------------------------------- rows

struct RowsArgs {
  const void *x, *ys;  // tokens' rows; experts' rows
  int64_t x_stride, ys_stride;
  int64_t T, k, D, rows;
  const int32_t *slots, *offsets;
  int64_t E;
  const float* weights;
  void* out;
  float* dweights;
  int chunks;
};

// Rows from offsets[E] on carry no pair: worker `b` of `workers` zeroes its share of
// them, in its columns c, c + step, ... below `end`.
template <typename T, int kVec>
__device__ __forceinline__ void zero_tail(const RowsArgs& A, int64_t b, int64_t workers, int64_t c,
                                          int step, int64_t end) {
  if (A.offsets == nullptr) return;
  int64_t used = A.offsets[A.E];
  if (used < 0) used = 0;
  const float zero[kVec] = {};
  for (int64_t r = used + b; r < A.rows; r += workers)
    for (int64_t q = c; q < end; q += step)
      store_f32<T, kVec>(static_cast<T*>(A.out) + r * A.D + q, zero);
}

// A token's row is read once and written to each of its slots.
template <typename T, int kVec, int kU>
__global__ void __launch_bounds__(256) hcmix_expert_dispatch_kernel(const RowsArgs A) {
  begin_kernel();
  const int64_t t = blockIdx.x / A.chunks;
  const int step = blockDim.x * kVec;
  const int64_t c = ((int64_t)(blockIdx.x % A.chunks) * kU * blockDim.x + threadIdx.x) * kVec;
  if (c >= A.D) return;
  Cols<T, kVec, kU> v;
  v.load(static_cast<const T*>(A.x) + t * A.x_stride, c, step, A.D);
  for (int64_t j = 0; j < A.k; ++j) {
    const int64_t s = A.slots[t * A.k + j];
    if (s >= 0 && s < A.rows) v.store(static_cast<T*>(A.out) + s * A.D, c, step, A.D);
  }
  const int64_t end = c + kU * step < A.D ? c + kU * step : A.D;
  zero_tail<T, kVec>(A, t, A.T, c, step, end);
}

// kBatch of a token's rows are under way at a time.
template <typename T, int kVec, int kU, int kBatch>
__global__ void __launch_bounds__(256) hcmix_expert_combine_kernel(const RowsArgs A) {
  begin_kernel();
  const int64_t t = blockIdx.x / A.chunks;
  const int step = blockDim.x * kVec;
  const int64_t c = ((int64_t)(blockIdx.x % A.chunks) * kU * blockDim.x + threadIdx.x) * kVec;
  if (c >= A.D) return;
  using Count = uint32_t;  // k can be 2^31 - 1
  constexpr int64_t kPast = (int64_t)INT32_MAX + kBatch;  // and j passes k by a batch
  static_assert((int64_t)(Count)kPast == kPast, "");
  const Count k = (Count)A.k;
  const uint32_t rows = (uint32_t)A.rows;
  const int32_t* slots = A.slots + t * A.k;
  const float* weights = A.weights != nullptr ? A.weights + t * A.k : nullptr;
  float sum[kU * kVec] = {};
  for (Count j = 0; j < k; j += kBatch) {
    Cols<T, kVec, kU> q[kBatch];
    uint32_t s[kBatch];
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      s[i] = kBatch == 1 || j + i < k ? (uint32_t)slots[j + i] : ~0u;  // a negative slot is large
      if (s[i] < rows) q[i].load(static_cast<const T*>(A.ys) + s[i] * A.ys_stride, c, step, A.D);
    }
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      if (s[i] < rows) {
        float v[kU * kVec];
        q[i].unpack(v);
        vfma(sum, weights != nullptr ? weights[j + i] : 1.f, v, sum);
      }
    }
  }
  store_cols<T, kVec, kU>(static_cast<T*>(A.out) + t * A.D, c, step, A.D, sum);
}

// A warp takes a pair: its one dot product needs no other warp.  The block's warps
// take the pairs of neighbouring tokens, so dy[t] comes from L1 for all but the
// first of a token's pairs.
constexpr int kPairWarps = 4;

template <typename T, int kVec, int kU>
__global__ void __launch_bounds__(32 * kPairWarps) hcmix_expert_combine_backward_kernel(
    const RowsArgs A) {
  begin_kernel();
  const int lane = threadIdx.x % 32, step = 32 * kVec;
  const int64_t pairs = A.T * A.k;
  const int64_t pair = (int64_t)blockIdx.x * kPairWarps + threadIdx.x / 32;
  const int64_t s = pair < pairs ? A.slots[pair] : -1;
  Acc dot;
  if (s >= 0 && s < A.rows) {
    const int64_t t = pair / A.k;
    const float w = A.weights[pair];
    const T* dy = static_cast<const T*>(A.x) + t * A.x_stride;
    const T* ys = static_cast<const T*>(A.ys) + s * A.ys_stride;
    T* dys = static_cast<T*>(A.out) + s * A.D;
    // four steps through the row are under way at a time (of narrow vectors two): 107 us for 4096 tokens of 8 rows of
    // 5120 bf16, two 108 us, one 121 us
    constexpr int kSteps = kU > 1 ? 2 : 4;
    for (int64_t c = lane * kVec; c < A.D; c += kSteps * kU * step) {
      Cols<T, kVec, kU> pg[kSteps], pv[kSteps];
#pragma unroll
      for (int i = 0; i < kSteps; ++i) {
        const int64_t at = c + i * kU * step;
        if (i == 0 || at < A.D) {
          pg[i].load_cached(dy, at, step, A.D);
          pv[i].load(ys, at, step, A.D);
        }
      }
#pragma unroll
      for (int i = 0; i < kSteps; ++i) {
        const int64_t at = c + i * kU * step;
        if (i == 0 || at < A.D) {
          float g[kU * kVec], v[kU * kVec];
          pg[i].unpack(g);
          pv[i].unpack(v);
          dot.add(g, v);
          vmul(g, w, g);
          store_cols<T, kVec, kU>(dys, at, step, A.D, g);
        }
      }
    }
  }
  const float total = warp_sum(dot.sum());
  if (lane == 0 && pair < pairs) A.dweights[pair] = total;
  zero_tail<T, kVec>(A, pair, (int64_t)gridDim.x * kPairWarps, lane * kVec, step, A.D);
}

enum class RowsOp { kDispatch, kCombine, kCombineBackward };

template <typename T, int kVec, int kU>
hcmix_status launch_rows(RowsOp op, RowsArgs A, cudaStream_t stream) {
  if (op == RowsOp::kCombineBackward) {
    int64_t blocks = (A.T * A.k + kPairWarps - 1) / kPairWarps;
    blocks = blocks > 0 ? blocks : 1;
    return launch(hcmix_expert_combine_backward_kernel<T, kVec, kU>, dim3((unsigned)blocks),
                  dim3(32 * kPairWarps), 0, 0, stream, A);
  }
  // Combine has four of a token's rows under way, in blocks of 128 threads: 4096 tokens of 8
  // rows of 5120 bf16 take 53.4 us, in blocks of 256 threads 54.9 us, two rows at a time 59.8 us,
  // eight 56.3 us.  Narrow vectors have four loads a row already: 3000 tokens of 7 rows of
  // 3001 bf16 take 59 us two at a time, 68 us four.  One row a token is a kernel of its own
  // with more of the row a thread: 13074 tokens of 6976 bf16 take 65 us, one vector a thread
  // 73 us, a batch of four 115 us.
  constexpr int kBatch = kU > 1 ? 2 : 4, kOneU = kU > 1 ? kU : 2;
  const bool combine = op == RowsOp::kCombine, one = combine && A.k == 1;
  const int64_t share = kVec * (one ? kOneU : kU), shares = (A.D + share - 1) / share;
  const int most = combine && !one ? 128 : 256;
  A.chunks = (int)((shares + most - 1) / most);
  const unsigned threads = (unsigned)((shares + A.chunks - 1) / A.chunks + 31) / 32 * 32;
  const int64_t blocks = A.T * A.chunks;
  if (blocks >= ((int64_t)1 << 31)) return HCMIX_ERR_UNSUPPORTED;
  const auto kernel = one       ? hcmix_expert_combine_kernel<T, kVec, kOneU, 1>
                      : combine ? hcmix_expert_combine_kernel<T, kVec, kU, kBatch>
                                : hcmix_expert_dispatch_kernel<T, kVec, kU>;
  return launch(kernel, dim3((unsigned)blocks), dim3(threads), 0, 0, stream, A);
}

inline hcmix_status run_rows(RowsOp op, const RowsArgs& A, hcmix_type type, cudaStream_t stream) {
  const int bytes =
      vector_bytes(size_of(type), {{A.x, A.x_stride}, {A.ys, A.ys_stride}, {A.out, A.D}});
  return with_vector(type, bytes, [&](auto t, auto vec, auto u) {
    return launch_rows<decltype(t), decltype(vec)::value, decltype(u)::value>(op, A, stream);
  });
}

}  // namespace sublayer
}  // namespace hcmix
