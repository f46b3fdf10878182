// Hyper-connection coefficients applied to the four residual streams of a row:
// collapse (h = sum_i pre_i x_i), expand (x'_i = post_i y + sum_j comb_ij x_j)
// and their gradients.  Every output element needs the same column of every
// stream, so a thread takes one column vector of all of them and each operand
// is read and written once.
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

template <typename T, int kVec>
__global__ void __launch_bounds__(256) hcmix_collapse_kernel(const StreamsArgs A) {
  begin_kernel();
  const int64_t row = blockIdx.x / A.chunks;
  const int64_t c = ((int64_t)(blockIdx.x % A.chunks) * blockDim.x + threadIdx.x) * kVec;
  if (c >= A.D) return;
  const T* x = static_cast<const T*>(A.x) + row * A.x_stride + c;
  float h[kVec] = {};
#pragma unroll
  for (int i = 0; i < kStreams; ++i) {
    float v[kVec];
    load_f32<T, kVec>(x + i * A.D, v);
    const float w = A.pre[row * kStreams + i];
    vfma(h, w, v, h);
  }
  store_f32<T, kVec>(static_cast<T*>(A.out) + row * A.D + c, h);
}

template <typename T, int kVec>
__global__ void __launch_bounds__(256) hcmix_expand_kernel(const StreamsArgs A) {
  begin_kernel();
  const int64_t row = blockIdx.x / A.chunks;
  const int64_t c = ((int64_t)(blockIdx.x % A.chunks) * blockDim.x + threadIdx.x) * kVec;
  if (c >= A.D) return;
  const T* x = static_cast<const T*>(A.x) + row * A.x_stride + c;
  const float* comb = A.comb + row * kStreams * kStreams;
  float v[kStreams][kVec], y[kVec];
#pragma unroll
  for (int j = 0; j < kStreams; ++j) load_f32<T, kVec>(x + j * A.D, v[j]);
  load_f32<T, kVec>(static_cast<const T*>(A.y) + row * A.y_stride + c, y);
#pragma unroll
  for (int i = 0; i < kStreams; ++i) {
    const float p = A.post[row * kStreams + i];
    float o[kVec];
    vmul(o, p, y);
#pragma unroll
    for (int j = 0; j < kStreams; ++j) vfma(o, comb[i * kStreams + j], v[j], o);
    store_f32<T, kVec>(static_cast<T*>(A.out) + row * kStreams * A.D + i * A.D + c, o);
  }
}

// One block a row: the row's four dot products need all of its columns.
template <typename T, int kVec>
__global__ void __launch_bounds__(256) hcmix_collapse_backward_kernel(const StreamsArgs A) {
  begin_kernel();
  __shared__ float part[kStreams * 32];
  const int64_t row = blockIdx.x;
  const T* x = static_cast<const T*>(A.x) + row * A.x_stride;
  const T* g = static_cast<const T*>(A.g) + row * A.g_stride;
  const T* add = static_cast<const T*>(A.add) + row * A.add_stride;
  T* dx = static_cast<T*>(A.out) + row * kStreams * A.D;
  float pre[kStreams];
  Acc dot[kStreams];
#pragma unroll
  for (int i = 0; i < kStreams; ++i) pre[i] = A.pre[row * kStreams + i];
  for (int64_t c = (int64_t)threadIdx.x * kVec; c < A.D; c += blockDim.x * kVec) {
    Packed<T, kVec> px[kStreams], pa[kStreams];
    const Packed<T, kVec> pg = load_vec<T, kVec>(g + c);
#pragma unroll
    for (int i = 0; i < kStreams; ++i) px[i] = load_vec<T, kVec>(x + i * A.D + c);
    if (A.add != nullptr) {
#pragma unroll
      for (int i = 0; i < kStreams; ++i) pa[i] = load_vec<T, kVec>(add + i * A.D + c);
    }
    float dh[kVec];
    pg.unpack(dh);
#pragma unroll
    for (int i = 0; i < kStreams; ++i) {
      float v[kVec], d[kVec];
      px[i].unpack(v);
      dot[i].add(dh, v);
      if (A.add != nullptr) {
        pa[i].unpack(d);
        vfma(d, pre[i], dh, d);
      } else {
        vmul(d, pre[i], dh);
      }
      store_f32<T, kVec>(dx + i * A.D + c, d);
    }
  }
  float sums[kStreams];
#pragma unroll
  for (int i = 0; i < kStreams; ++i) sums[i] = dot[i].sum();
  const float total = block_sums<kStreams>(sums, part);
  if (threadIdx.x < kStreams) A.dpre[row * kStreams + threadIdx.x] = total;
}

// One block a row, as above; 4 + 16 dot products.
template <typename T, int kVec>
__global__ void __launch_bounds__(256, 2) hcmix_expand_backward_kernel(const StreamsArgs A) {
  begin_kernel();
  constexpr int kDots = kStreams + kStreams * kStreams;
  __shared__ float part[kDots * 32];
  const int64_t row = blockIdx.x;
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
  for (int64_t c = (int64_t)threadIdx.x * kVec; c < A.D; c += blockDim.x * kVec) {
    Packed<T, kVec> pg[kStreams], px[kStreams];
#pragma unroll
    for (int i = 0; i < kStreams; ++i) pg[i] = load_vec<T, kVec>(g + i * A.D + c);
    const Packed<T, kVec> py = load_vec<T, kVec>(y + c);
#pragma unroll
    for (int i = 0; i < kStreams; ++i) px[i] = load_vec<T, kVec>(x + i * A.D + c);
    float d[kStreams][kVec], v[kVec], o[kVec] = {};
    py.unpack(v);
#pragma unroll
    for (int i = 0; i < kStreams; ++i) {
      pg[i].unpack(d[i]);
      vfma(o, post[i], d[i], o);
      dot[i].add(d[i], v);
    }
    store_f32<T, kVec>(dy + c, o);
#pragma unroll
    for (int j = 0; j < kStreams; ++j) {
      px[j].unpack(v);
      vmul(o, comb[0][j], d[0]);
#pragma unroll
      for (int i = 1; i < kStreams; ++i) vfma(o, comb[i][j], d[i], o);
#pragma unroll
      for (int i = 0; i < kStreams; ++i) dot[kStreams + i * kStreams + j].add(d[i], v);
      store_f32<T, kVec>(dx + j * A.D + c, o);
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

template <typename T, int kVec>
hcmix_status launch_streams(StreamsOp op, StreamsArgs A, cudaStream_t stream) {
  const int64_t vecs = (A.D + kVec - 1) / kVec;
  if (op == StreamsOp::kCollapse || op == StreamsOp::kExpand) {
    A.chunks = (int)((vecs + 255) / 256);
    const int threads = (int)((vecs + A.chunks - 1) / A.chunks + 31) / 32 * 32;
    const int64_t blocks = A.M * A.chunks;
    if (blocks >= ((int64_t)1 << 31)) return HCMIX_ERR_UNSUPPORTED;
    return launch(op == StreamsOp::kCollapse ? hcmix_collapse_kernel<T, kVec>
                                             : hcmix_expand_kernel<T, kVec>,
                  dim3((unsigned)blocks), threads, 0, stream, A);
  }
  // as many equal steps through the row as blocks of 256 threads need
  const int64_t steps = (vecs + 255) / 256;
  const int threads = (int)((vecs + steps - 1) / steps + 31) / 32 * 32;
  return launch(op == StreamsOp::kCollapseBackward ? hcmix_collapse_backward_kernel<T, kVec>
                                                   : hcmix_expand_backward_kernel<T, kVec>,
                dim3((unsigned)A.M), threads, 0, stream, A);
}

inline hcmix_status run_streams(StreamsOp op, const StreamsArgs& A, hcmix_type type,
                                cudaStream_t stream) {
  const int n = size_of(type);
  const bool wide = aligned_rows(A.x, A.x_stride, n) && aligned_rows(A.y, A.y_stride, n) &&
                    aligned_rows(A.g, A.g_stride, n) && aligned_rows(A.add, A.add_stride, n) &&
                    aligned_rows(A.out, A.D, n) && aligned_rows(A.dy, A.D, n);
  return with_type(type, [&](auto t) {
    using T = decltype(t);
    return wide ? launch_streams<T, kWide<T>>(op, A, stream) : launch_streams<T, 1>(op, A, stream);
  });
}

}  // namespace sublayer
}  // namespace hcmix
