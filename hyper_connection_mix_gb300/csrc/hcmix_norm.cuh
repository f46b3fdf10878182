// Layer norm forward (of a plain row, or of the collapsed streams) and backward.
#pragma once

#include "hcmix_vec.cuh"

namespace hcmix {
namespace sublayer {

struct NormArgs {
  const void* x;
  int64_t x_stride;
  const float* pre;  // collapse: the streams' coefficients
  const void *weight, *bias;
  bool p32;  // weight and bias are fp32
  float eps;
  void *y, *h;
  float *mean, *rstd;
  int64_t M, N;
  // backward
  const void* dy;
  int64_t dy_stride;
  void* dx;
  float *dweight, *dbias, *part;
  int blocks;  // partial rows of the weight's gradient
};

// kVec values of column c of a row: x itself, or sum_i pre[i] x_i.
template <typename T, int kVec, bool kCollapse>
__device__ __forceinline__ void norm_source(const NormArgs& A, const T* x, const float* pre,
                                            int64_t c, float (&v)[kVec]) {
  if constexpr (!kCollapse) {
    load_f32<T, kVec>(x + c, v);
  } else {
    float s[kStreams][kVec];
#pragma unroll
    for (int i = 0; i < kStreams; ++i) load_f32<T, kVec>(x + i * A.N + c, s[i]);
#pragma unroll
    for (int e = 0; e < kVec; ++e) {
      v[e] = pre[0] * s[0][e];
#pragma unroll
      for (int i = 1; i < kStreams; ++i) v[e] = fmaf(pre[i], s[i][e], v[e]);
    }
  }
}

template <typename T, int kVec>
__device__ __forceinline__ void norm_apply(const NormArgs& A, int64_t row, int64_t c, float mean,
                                           float rstd, float (&v)[kVec]) {
  float w[kVec], b[kVec];
#pragma unroll
  for (int e = 0; e < kVec; ++e) w[e] = 1.f, b[e] = 0.f;
  if (A.weight != nullptr) load_param<T, kVec>(A.weight, A.p32, c, w);
  if (A.bias != nullptr) load_param<T, kVec>(A.bias, A.p32, c, b);
#pragma unroll
  for (int e = 0; e < kVec; ++e) v[e] = fmaf((v[e] - mean) * rstd, w[e], b[e]);
  store_f32<T, kVec>(static_cast<T*>(A.y) + row * A.N + c, v);
}

// One block a row, the row in registers: kPer vectors a thread.  The mean is
// taken first and the variance from the differences, so that a large mean
// costs no digits.
template <typename T, int kVec, int kPer, bool kCollapse>
__global__ void __launch_bounds__(1024) hcmix_norm_kernel(const NormArgs A) {
  __shared__ float part[2][32];
  const int64_t row = blockIdx.x;
  const T* x = static_cast<const T*>(A.x) + row * A.x_stride;
  float pre[kStreams] = {};
  if constexpr (kCollapse) {
#pragma unroll
    for (int i = 0; i < kStreams; ++i) pre[i] = A.pre[row * kStreams + i];
  }
  float v[kPer][kVec];
  float sum[1] = {0.f};
#pragma unroll
  for (int k = 0; k < kPer; ++k) {
    const int64_t c = ((int64_t)k * blockDim.x + threadIdx.x) * kVec;
    if (c < A.N) {
      norm_source<T, kVec, kCollapse>(A, x, pre, c, v[k]);
    } else {
#pragma unroll
      for (int e = 0; e < kVec; ++e) v[k][e] = 0.f;
    }
#pragma unroll
    for (int e = 0; e < kVec; ++e) sum[0] += v[k][e];
  }
  const float inv = 1.f / (float)A.N;
  block_sum<1>(sum, part[0]);
  const float mean = sum[0] * inv;
  float sq[1] = {0.f};
#pragma unroll
  for (int k = 0; k < kPer; ++k) {
    const int64_t c = ((int64_t)k * blockDim.x + threadIdx.x) * kVec;
    if (c < A.N) {
#pragma unroll
      for (int e = 0; e < kVec; ++e) sq[0] = fmaf(v[k][e] - mean, v[k][e] - mean, sq[0]);
    }
  }
  block_sum<1>(sq, part[1]);
  const float rstd = 1.f / sqrtf(sq[0] * inv + A.eps);
#pragma unroll
  for (int k = 0; k < kPer; ++k) {
    const int64_t c = ((int64_t)k * blockDim.x + threadIdx.x) * kVec;
    if (c < A.N) {
      if (kCollapse && A.h != nullptr)
        store_f32<T, kVec>(static_cast<T*>(A.h) + row * A.N + c, v[k]);
      norm_apply<T, kVec>(A, row, c, mean, rstd, v[k]);
    }
  }
  if (threadIdx.x == 0) {
    if (A.mean != nullptr) A.mean[row] = mean;
    if (A.rstd != nullptr) A.rstd[row] = rstd;
  }
}

// Rows too wide for registers: three passes over the row, the later two mostly
// from L2.
template <typename T, int kVec, bool kCollapse>
__global__ void __launch_bounds__(512) hcmix_norm_wide_kernel(const NormArgs A) {
  __shared__ float part[2][32];
  const int64_t row = blockIdx.x;
  const T* x = static_cast<const T*>(A.x) + row * A.x_stride;
  const int64_t step = (int64_t)blockDim.x * kVec, c0 = (int64_t)threadIdx.x * kVec;
  float pre[kStreams] = {};
  if constexpr (kCollapse) {
#pragma unroll
    for (int i = 0; i < kStreams; ++i) pre[i] = A.pre[row * kStreams + i];
  }
  float v[kVec], sum[1] = {0.f}, sq[1] = {0.f};
  for (int64_t c = c0; c < A.N; c += step) {
    norm_source<T, kVec, kCollapse>(A, x, pre, c, v);
#pragma unroll
    for (int e = 0; e < kVec; ++e) sum[0] += v[e];
  }
  const float inv = 1.f / (float)A.N;
  block_sum<1>(sum, part[0]);
  const float mean = sum[0] * inv;
  for (int64_t c = c0; c < A.N; c += step) {
    norm_source<T, kVec, kCollapse>(A, x, pre, c, v);
#pragma unroll
    for (int e = 0; e < kVec; ++e) sq[0] = fmaf(v[e] - mean, v[e] - mean, sq[0]);
  }
  block_sum<1>(sq, part[1]);
  const float rstd = 1.f / sqrtf(sq[0] * inv + A.eps);
  for (int64_t c = c0; c < A.N; c += step) {
    norm_source<T, kVec, kCollapse>(A, x, pre, c, v);
    if (kCollapse && A.h != nullptr) store_f32<T, kVec>(static_cast<T*>(A.h) + row * A.N + c, v);
    norm_apply<T, kVec>(A, row, c, mean, rstd, v);
  }
  if (threadIdx.x == 0) {
    if (A.mean != nullptr) A.mean[row] = mean;
    if (A.rstd != nullptr) A.rstd[row] = rstd;
  }
}

template <typename T, int kVec, bool kCollapse>
hcmix_status launch_norm(const NormArgs& A, cudaStream_t stream) {
  constexpr int kMost = kVec == 1 ? 16 : 4;  // vectors a thread: at most 32 values
  const int64_t vecs = (A.N + kVec - 1) / kVec;
  const unsigned grid = (unsigned)A.M;
  const auto threads = [&](int per) { return (unsigned)((vecs + per - 1) / per + 31) / 32 * 32; };
  if (vecs <= 256)
    hcmix_norm_kernel<T, kVec, 1, kCollapse><<<grid, threads(1), 0, stream>>>(A);
  else if (vecs <= 1024 * kMost)
    hcmix_norm_kernel<T, kVec, kMost, kCollapse><<<grid, threads(kMost), 0, stream>>>(A);
  else
    hcmix_norm_wide_kernel<T, kVec, kCollapse><<<grid, 512, 0, stream>>>(A);
  return launched();
}

inline hcmix_status run_norm(const NormArgs& A, hcmix_type type, bool collapse,
                             cudaStream_t stream) {
  const int n = size_of(type);
  const bool wide = aligned_rows(A.x, A.x_stride, n) && aligned_rows(A.y, A.N, n) &&
                    aligned_rows(A.h, A.N, n) && A.N * n % 16 == 0;
  return with_type(type, [&](auto t) {
    using T = decltype(t);
    if (collapse)
      return wide ? launch_norm<T, kWide<T>, true>(A, stream) : launch_norm<T, 1, true>(A, stream);
    return wide ? launch_norm<T, kWide<T>, false>(A, stream) : launch_norm<T, 1, false>(A, stream);
  });
}

// ---------------------------------------------------------------- backward

// dx, one block a row.
template <typename T, int kVec>
__global__ void __launch_bounds__(512) hcmix_norm_dx_kernel(const NormArgs A) {
  __shared__ float part[2 * 32];
  const int64_t row = blockIdx.x;
  const T* x = static_cast<const T*>(A.x) + row * A.x_stride;
  const T* dy = static_cast<const T*>(A.dy) + row * A.dy_stride;
  const float mean = A.mean[row], rstd = A.rstd[row];
  const int64_t step = (int64_t)blockDim.x * kVec, c0 = (int64_t)threadIdx.x * kVec;
  float sum[2] = {0.f, 0.f}, v[kVec], g[kVec], w[kVec];
#pragma unroll
  for (int e = 0; e < kVec; ++e) w[e] = 1.f;
  for (int64_t c = c0; c < A.N; c += step) {
    load_f32<T, kVec>(x + c, v);
    load_f32<T, kVec>(dy + c, g);
    if (A.weight != nullptr) load_param<T, kVec>(A.weight, A.p32, c, w);
#pragma unroll
    for (int e = 0; e < kVec; ++e) {
      const float t = g[e] * w[e];
      sum[0] += t;
      sum[1] = fmaf(t, (v[e] - mean) * rstd, sum[1]);
    }
  }
  block_sum<2>(sum, part);
  const float inv = 1.f / (float)A.N;
  const float c1 = sum[0] * inv, c2 = sum[1] * inv;
  for (int64_t c = c0; c < A.N; c += step) {
    load_f32<T, kVec>(x + c, v);
    load_f32<T, kVec>(dy + c, g);
    if (A.weight != nullptr) load_param<T, kVec>(A.weight, A.p32, c, w);
#pragma unroll
    for (int e = 0; e < kVec; ++e)
      v[e] = rstd * (fmaf(g[e], w[e], -c1) - (v[e] - mean) * rstd * c2);
    store_f32<T, kVec>(static_cast<T*>(A.dx) + row * A.N + c, v);
  }
}

constexpr int kColumnThreads = 128;

// Partial sums of the weight's and bias's gradient: block (b, s) takes columns
// from b * kColumnThreads * kVec and rows s, s + slabs, ...
template <typename T, int kVec>
__global__ void __launch_bounds__(kColumnThreads) hcmix_norm_columns_kernel(const NormArgs A) {
  const int64_t c = ((int64_t)blockIdx.x * kColumnThreads + threadIdx.x) * kVec;
  if (c >= A.N) return;
  float dw[kVec] = {}, db[kVec] = {};
  for (int64_t row = blockIdx.y; row < A.M; row += gridDim.y) {
    float v[kVec], g[kVec];
    load_f32<T, kVec>(static_cast<const T*>(A.x) + row * A.x_stride + c, v);
    load_f32<T, kVec>(static_cast<const T*>(A.dy) + row * A.dy_stride + c, g);
    const float mean = A.mean[row], rstd = A.rstd[row];
#pragma unroll
    for (int e = 0; e < kVec; ++e) {
      dw[e] = fmaf(g[e], (v[e] - mean) * rstd, dw[e]);
      db[e] += g[e];
    }
  }
  float* part = A.part + (int64_t)blockIdx.y * 2 * A.N + c;
#pragma unroll
  for (int e = 0; e < kVec; ++e) {
    part[e] = dw[e];
    part[A.N + e] = db[e];
  }
}

// The partial rows added in order.
__global__ void __launch_bounds__(256) hcmix_norm_join_kernel(const NormArgs A) {
  const int64_t c = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (c >= 2 * A.N) return;
  float s = 0.f;
  for (int b = 0; b < A.blocks; ++b) s += A.part[(int64_t)b * 2 * A.N + c];
  (c < A.N ? A.dweight[c] : A.dbias[c - A.N]) = s;
}

constexpr int kMostPartials = 64;

inline int norm_partials(int64_t M) { return (int)(M < kMostPartials ? M : kMostPartials); }

inline size_t norm_workspace(int64_t M, int64_t N) {
  return ((size_t)norm_partials(M) * 2 * (size_t)N * 4 + 255) / 256 * 256;
}

template <typename T, int kVec>
hcmix_status launch_norm_backward(NormArgs A, cudaStream_t stream) {
  if (A.M > 0) {
    const int64_t vecs = (A.N + kVec - 1) / kVec;
    const unsigned threads = vecs >= 256 ? 256 : (unsigned)(vecs + 31) / 32 * 32;
    hcmix_norm_dx_kernel<T, kVec><<<(unsigned)A.M, threads, 0, stream>>>(A);
  }
  if (A.dweight == nullptr) return launched();
  A.blocks = norm_partials(A.M);
  const int64_t per = (int64_t)kColumnThreads * kVec;
  if (A.blocks > 0)
    hcmix_norm_columns_kernel<T, kVec>
        <<<dim3((unsigned)((A.N + per - 1) / per), A.blocks), kColumnThreads, 0, stream>>>(A);
  hcmix_norm_join_kernel<<<(unsigned)((2 * A.N + 255) / 256), 256, 0, stream>>>(A);
  return launched();
}

inline hcmix_status run_norm_backward(const NormArgs& A, hcmix_type type, cudaStream_t stream) {
  const int n = size_of(type);
  const bool wide = aligned_rows(A.x, A.x_stride, n) && aligned_rows(A.dy, A.dy_stride, n) &&
                    aligned_rows(A.dx, A.N, n) && A.N * n % 16 == 0;
  return with_type(type, [&](auto t) {
    using T = decltype(t);
    return wide ? launch_norm_backward<T, kWide<T>>(A, stream)
                : launch_norm_backward<T, 1>(A, stream);
  });
}

}  // namespace sublayer
}  // namespace hcmix
