// Hyper-connection coefficients applied to the four residual streams of a row:
// collapse (h = sum_i pre_i x_i), expand (x'_i = post_i y + sum_j comb_ij x_j)
// and their gradients.  Every output element needs the same column of every
// stream, so a thread takes one column vector of all of them and each operand
// is read and written once.  A thread reads only elements that it will write, after
// all its reads of them, so results may replace their operands.
//
// All are bound by HBM (copy rate 6787 GB/s).  Measured with four streams of 5120 bf16:
// collapse of 16384 rows 118 us (839 MB, 7.1 TB/s), expand of 16384 rows 213 us (1.51 GB, 7.1 TB/s), expand backward of 4096 rows 90 us
// (588 MB, 6.5 TB/s), collapse backward of 4096 rows 81 us (545 MB, 6.7 TB/s).
#pragma once

#include "hcmix_vec.cuh"

namespace hcmix {
namespace sublayer {

struct StreamsArgs {
  const void *x, *y, *g, *add;  // streams; sublayer output; gradient; gradient to add
  int64_t x_stride, y_stride, g_stride, add_stride;
  const float *pre, *post, *comb;
  void *out, *dy;
  float *dpre, *dpost, *dcomb;
  int64_t M, D;
  int chunks;  // thread blocks across a row (forward kernels)
};

constexpr int kStreamsThreads = 128;

// A thread's first column in the chunk-th block across a row.
template <int kVec, int kU>
__device__ __forceinline__ int64_t first_column(int chunk) {
  return ((int64_t)chunk * kU * blockDim.x + threadIdx.x) * kVec;
}

template <typename T, int kVec, int kU>
__global__ void __launch_bounds__(kStreamsThreads) hcmix_collapse_kernel(const StreamsArgs A) {
  begin_kernel();
  const int64_t row = blockIdx.x / A.chunks;
  const int64_t c = first_column<kVec, kU>(blockIdx.x % A.chunks);
  const int step = blockDim.x * kVec;
  if (c >= A.D) return;
  const T* x = static_cast<const T*>(A.x) + row * A.x_stride;
  Cols<T, kVec, kU> px[kStreams];
#pragma unroll
  for (int i = 0; i < kStreams; ++i) px[i].load(x + i * A.D, c, step, A.D);
  float h[kU * kVec] = {};
#pragma unroll
  for (int i = 0; i < kStreams; ++i) {
    float v[kU * kVec];
    px[i].unpack(v);
    vfma(h, A.pre[row * kStreams + i], v, h);
  }
  store_cols<T, kVec, kU>(static_cast<T*>(A.out) + row * A.D, c, step, A.D, h);
}

template <typename T, int kVec, int kU>
__global__ void __launch_bounds__(kStreamsThreads) hcmix_expand_kernel(const StreamsArgs A) {
  begin_kernel();
  const int64_t row = blockIdx.x / A.chunks;
  const int64_t c = first_column<kVec, kU>(blockIdx.x % A.chunks);
  const int step = blockDim.x * kVec;
  if (c >= A.D) return;
  const T* x = static_cast<const T*>(A.x) + row * A.x_stride;
  const float* comb = A.comb + row * kStreams * kStreams;
  Cols<T, kVec, kU> px[kStreams], py;
#pragma unroll
  for (int j = 0; j < kStreams; ++j) px[j].load(x + j * A.D, c, step, A.D);
  py.load(static_cast<const T*>(A.y) + row * A.y_stride, c, step, A.D);
  float v[kStreams][kU * kVec], y[kU * kVec];
#pragma unroll
  for (int j = 0; j < kStreams; ++j) px[j].unpack(v[j]);
  py.unpack(y);
  T* out = static_cast<T*>(A.out) + row * kStreams * A.D;
#pragma unroll
  for (int i = 0; i < kStreams; ++i) {
    float o[kU * kVec];
    vmul(o, A.post[row * kStreams + i], y);
#pragma unroll
    for (int j = 0; j < kStreams; ++j) vfma(o, comb[i * kStreams + j], v[j], o);
    store_cols<T, kVec, kU>(out + i * A.D, c, step, A.D, o);
  }
}

// One block a row: the row's four dot products need all of its columns.
template <typename T, int kVec, int kU>
__global__ void __launch_bounds__(kStreamsThreads) hcmix_collapse_backward_kernel(const StreamsArgs A) {
  begin_kernel();
  __shared__ float part[kStreams * 32];
  const int64_t row = blockIdx.x;
  const int step = blockDim.x * kVec;
  const T* x = static_cast<const T*>(A.x) + row * A.x_stride;
  const T* g = static_cast<const T*>(A.g) + row * A.g_stride;
  const T* add = static_cast<const T*>(A.add) + row * A.add_stride;
  T* dx = static_cast<T*>(A.out) + row * kStreams * A.D;
  float pre[kStreams];
  Acc dot[kStreams];
#pragma unroll
  for (int i = 0; i < kStreams; ++i) pre[i] = A.pre[row * kStreams + i];
  for (int64_t c = first_column<kVec, kU>(0); c < A.D; c += kU * step) {
    Cols<T, kVec, kU> px[kStreams], pa[kStreams], pg;
    pg.load(g, c, step, A.D);
#pragma unroll
    for (int i = 0; i < kStreams; ++i) px[i].load(x + i * A.D, c, step, A.D);
    if (A.add != nullptr) {
#pragma unroll
      for (int i = 0; i < kStreams; ++i) pa[i].load(add + i * A.D, c, step, A.D);
    }
    float dh[kU * kVec];
    pg.unpack(dh);
#pragma unroll
    for (int i = 0; i < kStreams; ++i) {
      float v[kU * kVec], d[kU * kVec];
      px[i].unpack(v);
      dot[i].add(dh, v);
      if (A.add != nullptr) {
        pa[i].unpack(d);
        vfma(d, pre[i], dh, d);
      } else {
        vmul(d, pre[i], dh);
      }
      store_cols<T, kVec, kU>(dx + i * A.D, c, step, A.D, d);
    }
  }
  float sums[kStreams];
#pragma unroll
  for (int i = 0; i < kStreams; ++i) sums[i] = dot[i].sum();
  const float total = block_sums<kStreams>(sums, part);
  if (threadIdx.x < kStreams) A.dpre[row * kStreams + threadIdx.x] = total;
}

// One block a row, as above; 4 + 16 dot products, 40 FMA a column.  The 20 accumulators,
// the coefficients and nine vectors under way fill 128 registers: four blocks of 128
// threads a multiprocessor.
template <typename T, int kVec, int kU>
__global__ void __launch_bounds__(kStreamsThreads, 4) hcmix_expand_backward_kernel(const StreamsArgs A) {
  begin_kernel();
  constexpr int kDots = kStreams + kStreams * kStreams;
  __shared__ float part[kDots * 32];
  const int64_t row = blockIdx.x;
  const int step = blockDim.x * kVec;
  const T* x = static_cast<const T*>(A.x) + row * A.x_stride;
  const T* y = static_cast<const T*>(A.y) + row * A.y_stride;
  const T* g = static_cast<const T*>(A.g) + row * A.g_stride;
  T* dx = static_cast<T*>(A.out) + row * kStreams * A.D;
  T* dy = static_cast<T*>(A.dy) + row * A.D;
  float post[kStreams], comb[kStreams][kStreams];
  Acc dot[kDots];
#pragma unroll
  for (int i = 0; i < kStreams; ++i) {
    post[i] = A.post[row * kStreams + i];
#pragma unroll
    for (int j = 0; j < kStreams; ++j)
      comb[i][j] = A.comb[(row * kStreams + i) * kStreams + j];
  }
  for (int64_t c = first_column<kVec, kU>(0); c < A.D; c += kU * step) {
    Cols<T, kVec, kU> pg[kStreams], px[kStreams], py;
#pragma unroll
    for (int i = 0; i < kStreams; ++i) pg[i].load(g + i * A.D, c, step, A.D);
    py.load(y, c, step, A.D);
#pragma unroll
    for (int i = 0; i < kStreams; ++i) px[i].load(x + i * A.D, c, step, A.D);
    float d[kStreams][kU * kVec], v[kU * kVec], o[kU * kVec] = {};
    py.unpack(v);
#pragma unroll
    for (int i = 0; i < kStreams; ++i) {
      pg[i].unpack(d[i]);
      vfma(o, post[i], d[i], o);
      dot[i].add(d[i], v);
    }
    store_cols<T, kVec, kU>(dy, c, step, A.D, o);
#pragma unroll
    for (int j = 0; j < kStreams; ++j) {
      px[j].unpack(v);
      vmul(o, comb[0][j], d[0]);
#pragma unroll
      for (int i = 1; i < kStreams; ++i) vfma(o, comb[i][j], d[i], o);
#pragma unroll
      for (int i = 0; i < kStreams; ++i) dot[kStreams + i * kStreams + j].add(d[i], v);
      store_cols<T, kVec, kU>(dx + j * A.D, c, step, A.D, o);
    }
  }
  float sums[kDots];
#pragma unroll
  for (int i = 0; i < kDots; ++i) sums[i] = dot[i].sum();
  const float total = block_sums<kDots>(sums, part);
  const int t = threadIdx.x;
  if (t < kStreams) A.dpost[row * kStreams + t] = total;
  else if (t < kDots) A.dcomb[row * kStreams * kStreams + t - kStreams] = total;
}

enum class StreamsOp { kCollapse, kExpand, kCollapseBackward, kExpandBackward };

template <typename T, int kVec, int kU>
hcmix_status launch_streams(StreamsOp op, StreamsArgs A, cudaStream_t stream) {
  // a row in as many equal parts as blocks of 128 threads need: blocks, or the steps
  // of one block.  (Of 256 threads: expand backward 98.6 us for 90.1 us at 4096 rows of
  // 4 x 5120 bf16, expand 216 us for 213 us at 16384.)
  const int64_t shares = (A.D + kVec * kU - 1) / (kVec * kU);
  const int64_t parts = (shares + kStreamsThreads - 1) / kStreamsThreads;
  const unsigned threads = (unsigned)((shares + parts - 1) / parts + 31) / 32 * 32;
  if (op == StreamsOp::kCollapse || op == StreamsOp::kExpand) {
    A.chunks = (int)parts;
    const int64_t blocks = A.M * A.chunks;
    if (blocks >= ((int64_t)1 << 31)) return HCMIX_ERR_UNSUPPORTED;
    return launch(op == StreamsOp::kCollapse ? hcmix_collapse_kernel<T, kVec, kU>
                                             : hcmix_expand_kernel<T, kVec, kU>,
                  dim3((unsigned)blocks), dim3(threads), 0, 0, stream, A);
  }
  return launch(op == StreamsOp::kCollapseBackward ? hcmix_collapse_backward_kernel<T, kVec, kU>
                                                   : hcmix_expand_backward_kernel<T, kVec, kU>,
                dim3((unsigned)A.M), dim3(threads), 0, 0, stream, A);
}

inline hcmix_status run_streams(StreamsOp op, const StreamsArgs& A, hcmix_type type,
                                cudaStream_t stream) {
  // a row's streams start D apart, whatever its stride
  const int bytes = vector_bytes(size_of(type), {{A.x, A.x_stride}, {A.y, A.y_stride},
                                                 {A.g, A.g_stride}, {A.add, A.add_stride},
                                                 {A.out, A.D}, {A.dy, A.D}});
  return with_vector(type, bytes, [&](auto t, auto vec, auto u) {
    return launch_streams<decltype(t), decltype(vec)::value, decltype(u)::value>(op, A, stream);
  });
}

}  // namespace sublayer
}  // namespace hcmix
