// Tokens sorted by expert and back: a stable counting sort of the (token, choice)
// pairs, the rows copied to their experts' places and the weighted rows added up
// again, with the gradients.  No atomics: every row has one writer.
#pragma once

#include <cooperative_groups.h>

#include "hcmix_vec.cuh"

namespace hcmix {
namespace sublayer {

struct SortArgs {
  const void* ids;
  int wide_ids;  // int64
  int64_t n;     // pairs
  int E;
  int32_t *offsets, *slots, *source;
};

constexpr int kMostExperts = 4096;
constexpr int kSortCounters = 32 * 1024;  // warps * experts, 128 KB
constexpr int kSortCluster = 8;

__device__ __forceinline__ int expert_of(const SortArgs& A, int64_t i) {
  const int64_t e = A.wide_ids ? static_cast<const int64_t*>(A.ids)[i]
                               : static_cast<const int32_t*>(A.ids)[i];
  return e >= 0 && e < A.E ? (int)e : -1;
}

inline int sort_warps(int E) {
  const int w = kSortCounters / E;
  return w > 32 ? 32 : w;
}

inline size_t sort_smem(int E) { return ((size_t)sort_warps(E) * E + 2 * (size_t)E + 64) * 4; }

// One cluster sorts all pairs: each of its warps takes a contiguous range of
// them, counts its experts, and after the counts of the warps before it are
// known walks its range again and places each pair.  Within 32 pairs a pair's
// rank is the number of lower lanes with its expert.
__global__ void __launch_bounds__(1024) hcmix_expert_sort_kernel(const SortArgs A) {
  namespace cg = cooperative_groups;
  extern __shared__ int sort_shared[];
  const cg::cluster_group cluster = cg::this_cluster();
  const int ctas = cluster.num_blocks(), cta = cluster.block_rank();
  const int warps = blockDim.x / 32, warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int E = A.E;
  int* count = sort_shared;         // [warps][E]
  int* total = count + warps * E;   // [E] this block's pairs of each expert
  int* start = total + E;           // [E] the block's first row of each expert
  int* scan = start + E;            // [warps] sums of the scan over experts

  for (int i = threadIdx.x; i < warps * E; i += blockDim.x) count[i] = 0;
  __syncthreads();
  const int64_t ranges = (int64_t)ctas * warps;
  const int64_t span = ((A.n + ranges - 1) / ranges + 31) / 32 * 32;
  const int64_t first = ((int64_t)cta * warps + warp) * span;
  const int64_t last = first + span < A.n ? first + span : A.n;
  int* mine = count + warp * E;
  for (int64_t i = first + lane; i - lane < last; i += 32) {
    const int e = i < last ? expert_of(A, i) : -1;
    const unsigned same = __match_any_sync(0xffffffffu, e);
    if (e >= 0 && __ffs(same) - 1 == lane) mine[e] += __popc(same);
    __syncwarp();
  }
  __syncthreads();
  for (int e = threadIdx.x; e < E; e += blockDim.x) {
    int s = 0;
    for (int w = 0; w < warps; ++w) {
      const int c = count[w * E + e];
      count[w * E + e] = s;
      s += c;
    }
    total[e] = s;
  }
  cluster.sync();
  // start[e] = the pairs of all experts before e, and those of e in earlier blocks
  const int per = (E + blockDim.x - 1) / blockDim.x;
  int sum = 0;
  for (int q = 0; q < per; ++q) {
    const int e = threadIdx.x * per + q;
    if (e < E)
      for (int b = 0; b < ctas; ++b) sum += cluster.map_shared_rank(total, b)[e];
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
  for (int w = 0; w < warps; ++w) {
    if (w < warp) before += scan[w];
    all += scan[w];
  }
  for (int q = 0; q < per; ++q) {
    const int e = threadIdx.x * per + q;
    if (e >= E) break;
    if (cta == 0) A.offsets[e] = before;
    int here = before;
    for (int b = 0; b < ctas; ++b) {
      const int t = cluster.map_shared_rank(total, b)[e];
      if (b < cta) here += t;
      before += t;
    }
    start[e] = here;
  }
  if (cta == 0 && threadIdx.x == 0) A.offsets[E] = all;
  __syncthreads();
  for (int64_t i = first + lane; i - lane < last; i += 32) {
    const int e = i < last ? expert_of(A, i) : -1;
    const unsigned same = __match_any_sync(0xffffffffu, e);
    if (e >= 0) {
      const int place = start[e] + mine[e] + __popc(same & ((1u << lane) - 1));
      A.slots[i] = place;
      A.source[place] = (int)i;
    } else if (i < last) {
      A.slots[i] = -1;
    }
    __syncwarp();
    if (e >= 0 && __ffs(same) - 1 == lane) mine[e] += __popc(same);
    __syncwarp();
  }
  for (int64_t r = all + (int64_t)cta * blockDim.x + threadIdx.x; r < A.n;
       r += (int64_t)ctas * blockDim.x)
    A.source[r] = -1;
  cluster.sync();  // the other blocks may still read this one's totals
}

inline hcmix_status run_sort(const SortArgs& A, cudaStream_t stream) {
  const size_t smem = sort_smem(A.E);
  if (cudaFuncSetAttribute(hcmix_expert_sort_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           (int)smem) != cudaSuccess)
    return HCMIX_ERR_CUDA;
  const int ctas = A.n <= 4096 ? 1 : kSortCluster;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(ctas);
  cfg.blockDim = dim3(sort_warps(A.E) * 32);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = ctas;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, hcmix_expert_sort_kernel, A) != cudaSuccess) return HCMIX_ERR_CUDA;
  return launched();
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

// Rows from offsets[E] on carry no pair: block `b` of `blocks` zeroes its share
// of them, in its columns.
template <typename T, int kVec>
__device__ __forceinline__ void zero_tail(const RowsArgs& A, int64_t b, int64_t blocks, int64_t c,
                                          int64_t step) {
  if (A.offsets == nullptr) return;
  int64_t used = A.offsets[A.E];
  if (used < 0) used = 0;
  const float zero[kVec] = {};
  for (int64_t r = used + b; r < A.rows; r += blocks)
    for (int64_t q = c; q < A.D; q += step) store_f32<T, kVec>(static_cast<T*>(A.out) + r * A.D + q, zero);
}

// A token's row is read once and written to each of its slots.
template <typename T, int kVec>
__global__ void __launch_bounds__(256) hcmix_expert_dispatch_kernel(const RowsArgs A) {
  const int64_t t = blockIdx.x / A.chunks;
  const int64_t c = ((int64_t)(blockIdx.x % A.chunks) * blockDim.x + threadIdx.x) * kVec;
  if (c >= A.D) return;
  const Packed<T, kVec> v = load_vec<T, kVec>(static_cast<const T*>(A.x) + t * A.x_stride + c);
  for (int64_t j = 0; j < A.k; ++j) {
    const int64_t s = A.slots[t * A.k + j];
    if (s >= 0 && s < A.rows) store_vec<T, kVec>(static_cast<T*>(A.out) + s * A.D + c, v);
  }
  zero_tail<T, kVec>(A, t, A.T, c, A.D);
}

template <typename T, int kVec>
__global__ void __launch_bounds__(256) hcmix_expert_combine_kernel(const RowsArgs A) {
  const int64_t t = blockIdx.x / A.chunks;
  const int64_t c = ((int64_t)(blockIdx.x % A.chunks) * blockDim.x + threadIdx.x) * kVec;
  if (c >= A.D) return;
  float sum[kVec] = {};
  for (int64_t j = 0; j < A.k; ++j) {
    const int64_t s = A.slots[t * A.k + j];
    if (s < 0 || s >= A.rows) continue;
    const float w = A.weights != nullptr ? A.weights[t * A.k + j] : 1.f;
    float v[kVec];
    load_f32<T, kVec>(static_cast<const T*>(A.ys) + s * A.ys_stride + c, v);
#pragma unroll
    for (int e = 0; e < kVec; ++e) sum[e] = fmaf(w, v[e], sum[e]);
  }
  store_f32<T, kVec>(static_cast<T*>(A.out) + t * A.D + c, sum);
}

// One block a pair.  dy[t] comes from L2 for all but the first of a token's pairs.
template <typename T, int kVec>
__global__ void __launch_bounds__(256) hcmix_expert_combine_backward_kernel(const RowsArgs A) {
  __shared__ float part[32];
  const int64_t pair = blockIdx.x, pairs = A.T * A.k;
  const int64_t c0 = (int64_t)threadIdx.x * kVec, step = (int64_t)blockDim.x * kVec;
  const int64_t s = pair < pairs ? A.slots[pair] : -1;
  float dot[1] = {0.f};
  if (s >= 0 && s < A.rows) {
    const int64_t t = pair / A.k;
    const float w = A.weights[pair];
    const T* dy = static_cast<const T*>(A.x) + t * A.x_stride;
    const T* ys = static_cast<const T*>(A.ys) + s * A.ys_stride;
    T* dys = static_cast<T*>(A.out) + s * A.D;
    for (int64_t c = c0; c < A.D; c += step) {
      float g[kVec], v[kVec];
      load_f32<T, kVec>(dy + c, g);
      load_f32<T, kVec>(ys + c, v);
#pragma unroll
      for (int e = 0; e < kVec; ++e) {
        dot[0] = fmaf(g[e], v[e], dot[0]);
        g[e] *= w;
      }
      store_f32<T, kVec>(dys + c, g);
    }
  }
  block_sums_all<1>(dot, part);
  if (threadIdx.x == 0 && pair < pairs) A.dweights[pair] = dot[0];
  zero_tail<T, kVec>(A, pair, gridDim.x, c0, step);
}

enum class RowsOp { kDispatch, kCombine, kCombineBackward };

template <typename T, int kVec>
hcmix_status launch_rows(RowsOp op, RowsArgs A, cudaStream_t stream) {
  const int64_t vecs = (A.D + kVec - 1) / kVec;
  if (op == RowsOp::kCombineBackward) {
    const unsigned threads = vecs >= 256 ? 256 : (unsigned)(vecs + 31) / 32 * 32;
    hcmix_expert_combine_backward_kernel<T, kVec>
        <<<(unsigned)(A.T * A.k > 0 ? A.T * A.k : 1), threads, 0, stream>>>(A);
    return launched();
  }
  A.chunks = (int)((vecs + 255) / 256);
  const int threads = (int)((vecs + A.chunks - 1) / A.chunks + 31) / 32 * 32;
  const int64_t blocks = A.T * A.chunks;
  if (blocks >= ((int64_t)1 << 31)) return HCMIX_ERR_UNSUPPORTED;
  if (op == RowsOp::kDispatch)
    hcmix_expert_dispatch_kernel<T, kVec><<<(unsigned)blocks, threads, 0, stream>>>(A);
  else
    hcmix_expert_combine_kernel<T, kVec><<<(unsigned)blocks, threads, 0, stream>>>(A);
  return launched();
}

inline hcmix_status run_rows(RowsOp op, const RowsArgs& A, hcmix_type type, cudaStream_t stream) {
  const int n = size_of(type);
  const bool wide = aligned_rows(A.x, A.x_stride, n) && aligned_rows(A.ys, A.ys_stride, n) &&
                    aligned_rows(A.out, A.D, n);
  return with_type(type, [&](auto t) {
    using T = decltype(t);
    return wide ? launch_rows<T, kWide<T>>(op, A, stream) : launch_rows<T, 1>(op, A, stream);
  });
}

}  // namespace sublayer
}  // namespace hcmix
