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

// kVec values of column c of a row, x itself or sum_i pre[i] x_i: first loaded,
// then worked out.
template <typename T, int kVec, bool kCollapse>
struct NormSource {
  Packed<T, kVec> s[kCollapse ? kStreams : 1];
  __device__ __forceinline__ void load(const NormArgs& A, const T* x, int64_t c) {
#pragma unroll
    for (int i = 0; i < (kCollapse ? kStreams : 1); ++i)
      s[i] = load_vec<T, kVec>(x + i * A.N + c);
  }
  __device__ __forceinline__ void values(const float* pre, float (&v)[kVec]) const {
    s[0].unpack(v);
    if constexpr (kCollapse) {
      vmul(v, pre[0], v);
#pragma unroll
      for (int i = 1; i < kStreams; ++i) {
        float t[kVec];
        s[i].unpack(t);
        vfma(v, pre[i], t, v);
      }
    }
  }
};

template <typename T, int kVec, bool kCollapse>
__device__ __forceinline__ void norm_source(const NormArgs& A, const T* x, const float* pre,
                                            int64_t c, float (&v)[kVec]) {
  NormSource<T, kVec, kCollapse> s;
  s.load(A, x, c);
  s.values(pre, v);
}

// Weight and bias of column c, ones and zeros where there are none.
template <typename T, int kVec>
__device__ __forceinline__ void norm_params(const NormArgs& A, int64_t c, float (&w)[kVec],
                                            float (&b)[kVec]) {
#pragma unroll
  for (int e = 0; e < kVec; ++e) w[e] = 1.f, b[e] = 0.f;
  if (A.weight != nullptr) load_param<T, kVec>(A.weight, A.p32, c, w);
  if (A.bias != nullptr) load_param<T, kVec>(A.bias, A.p32, c, b);
}

template <typename T, int kVec>
__device__ __forceinline__ void norm_apply(const NormArgs& A, int64_t row, int64_t c, float mean,
                                           float rstd, float (&v)[kVec]) {
  float w[kVec], b[kVec];
  norm_params<T, kVec>(A, c, w, b);
  vadd(v, -mean, v);
  vmul(v, rstd, v);
  vfma(v, v, w, b);
  store_f32<T, kVec>(static_cast<T*>(A.y) + row * A.N + c, v);
}

// One block a row, the row in registers: kPer vectors a thread.  The mean is
// taken first and the variance from the differences, so that a large mean
// costs no digits.
template <typename T, int kVec, int kPer, int kThreads, bool kCollapse>
__global__ void __launch_bounds__(kThreads) hcmix_norm_kernel(const NormArgs A) {
  begin_kernel();
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
  NormSource<T, kVec, kCollapse> raw[kPer];
#pragma unroll
  for (int k = 0; k < kPer; ++k) {
    const int64_t c = ((int64_t)k * blockDim.x + threadIdx.x) * kVec;
    if (c < A.N) raw[k].load(A, x, c);
  }
#pragma unroll
  for (int k = 0; k < kPer; ++k) {
    const int64_t c = ((int64_t)k * blockDim.x + threadIdx.x) * kVec;
    if (c < A.N) {
      raw[k].values(pre, v[k]);
    } else {
#pragma unroll
      for (int e = 0; e < kVec; ++e) v[k][e] = 0.f;
    }
#pragma unroll
    for (int e = 0; e < kVec; ++e) sum[0] += v[k][e];
  }
  const float inv = 1.f / (float)A.N;
  block_sums_all<1>(sum, part[0]);
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
  block_sums_all<1>(sq, part[1]);
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
  begin_kernel();
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
  block_sums_all<1>(sum, part[0]);
  const float mean = sum[0] * inv;
  for (int64_t c = c0; c < A.N; c += step) {
    norm_source<T, kVec, kCollapse>(A, x, pre, c, v);
#pragma unroll
    for (int e = 0; e < kVec; ++e) sq[0] = fmaf(v[e] - mean, v[e] - mean, sq[0]);
  }
  block_sums_all<1>(sq, part[1]);
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

// Resident blocks take groups of rows b, b + blocks, ... through a ring of
// kStages groups in shared memory.  Each thread copies the vectors that it will
// read itself (cp.async), so no barrier stands between the copies and their use,
// and what belongs to its columns (weight, bias, sums over rows) stays in
// registers.  A group is kRows source rows (streams; x and dy of several rows).
template <typename T, int kVec, int kPer, int kRows, int kStages>
struct Ring {
  using V = Packed<T, kVec>;
  unsigned char* mine;
  int pitch;  // bytes from one of the thread's vectors to its next
  int at;     // byte offset of the stage that is read
  int columns, first, step;  // the thread's columns: first + k * step, below columns
  __device__ __forceinline__ Ring(unsigned char* smem, int64_t width)
      : mine(smem + threadIdx.x * sizeof(V)),
        pitch(blockDim.x * sizeof(V)),
        at(0),
        columns((int)width),
        first(threadIdx.x * kVec),
        step(blockDim.x * kVec) {}
  __device__ __forceinline__ bool has(int k) const { return first + k * step < columns; }
  __device__ __forceinline__ int column(int k) const { return first + k * step; }
  __device__ __forceinline__ int group() const { return kRows * kPer * pitch; }
  // Starts the copy of source row i, given its first element, into the stage at
  // byte offset `to`.
  __device__ __forceinline__ void copy(int to, int i, const T* row) const {
#pragma unroll
    for (int k = 0; k < kPer; ++k)
      if (has(k))
        async_copy(reinterpret_cast<V*>(mine + to + (i * kPer + k) * pitch), row + column(k));
  }
  // The stage to refill while this group is worked on: the one read a group ago.
  __device__ __forceinline__ int refill() const {
    return at == 0 ? (kStages - 1) * group() : at - group();
  }
  __device__ __forceinline__ const V& read(int i, int k) const {
    return *reinterpret_cast<const V*>(mine + at + (i * kPer + k) * pitch);
  }
  __device__ __forceinline__ void advance() {
    at += group();
    if (at == kStages * group()) at = 0;
  }
};

constexpr int kSms = 152;

// Stages that fit a multiprocessor with kBlocks blocks of kThreads threads: 200 KB,
// from two to eight.
template <int kRows, int kPer, int kThreads, int kBlocks>
constexpr int kRingFit = 200 * 1024 / (kBlocks * kRows * kPer * kThreads * 16);
template <int kRows, int kPer, int kThreads, int kBlocks>
constexpr int kRingStages = kRingFit<kRows, kPer, kThreads, kBlocks> > 8   ? 8
                            : kRingFit<kRows, kPer, kThreads, kBlocks> < 2 ? 2
                                : kRingFit<kRows, kPer, kThreads, kBlocks>;

struct RingPlan {
  int threads, each;  // each: blocks a multiprocessor
  size_t stage;       // bytes
};

// `each` blocks of `most` threads fit a multiprocessor; smaller ones in proportion.
inline RingPlan ring_plan(int64_t vecs, int per, int most, int each, int rows, int vec_bytes) {
  RingPlan p;
  p.threads = (int)((vecs + per - 1) / per + 31) / 32 * 32;
  p.each = each * most / p.threads;
  p.each = p.each > 16 ? 16 : p.each;
  p.stage = (size_t)rows * per * p.threads * vec_bytes;
  return p;
}

// The norm of 16-byte vectors through the ring.
template <typename T, int kVec, int kPer, int kThreads, int kBlocks, bool kCollapse>
__global__ void __launch_bounds__(kThreads, kBlocks) hcmix_norm_ring_kernel(const NormArgs A) {
  begin_kernel();
  extern __shared__ __align__(16) unsigned char smem[];
  __shared__ float part[2][32];
  constexpr int kRows = kCollapse ? kStreams : 1;
  constexpr int kStages = kRingStages<kRows, kPer, kThreads, kBlocks>;
  Ring<T, kVec, kPer, kRows, kStages> ring(smem, A.N);
  const T* from = static_cast<const T*>(A.x) + blockIdx.x * A.x_stride;
  const int64_t jump = gridDim.x * A.x_stride;
  int64_t next = blockIdx.x;
  const auto fetch = [&](int to) {
    if (next < A.M) {
#pragma unroll
      for (int i = 0; i < kRows; ++i) ring.copy(to, i, from + i * A.N);
    }
    async_commit();  // an empty group past the last row keeps the count
    next += gridDim.x;
    from += jump;
  };
#pragma unroll
  for (int s = 0; s < kStages - 1; ++s) fetch(s * ring.group());
  float w[kPer][kVec], b[kPer][kVec];
#pragma unroll
  for (int k = 0; k < kPer; ++k)
    if (ring.has(k)) norm_params<T, kVec>(A, ring.column(k), w[k], b[k]);
  const float inv = 1.f / (float)A.N;
  for (int64_t row = blockIdx.x; row < A.M; row += gridDim.x) {
    float pre[kStreams] = {};
    if constexpr (kCollapse) {
#pragma unroll
      for (int i = 0; i < kStreams; ++i) pre[i] = A.pre[row * kStreams + i];
    }
    fetch(ring.refill());
    async_wait<kStages - 1>();
    float v[kPer][kVec];
    Acc acc;
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
      if (ring.has(k)) {
        NormSource<T, kVec, kCollapse> raw;
#pragma unroll
        for (int i = 0; i < kRows; ++i) raw.s[i] = ring.read(i, k);
        raw.values(pre, v[k]);
        acc.add(v[k]);
      }
    }
    float sum[1] = {acc.sum()};
    block_sums_all<1>(sum, part[0]);
    const float mean = sum[0] * inv;
    Acc square;
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
      if (ring.has(k)) {
        if (kCollapse && A.h != nullptr)
          store_f32<T, kVec>(static_cast<T*>(A.h) + row * A.N + ring.column(k), v[k]);
        vadd(v[k], -mean, v[k]);
        square.add(v[k], v[k]);
      }
    }
    float sq[1] = {square.sum()};
    block_sums_all<1>(sq, part[1]);
    const float rstd = 1.f / sqrtf(sq[0] * inv + A.eps);
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
      if (ring.has(k)) {
        vmul(v[k], rstd, v[k]);
        vfma(v[k], v[k], w[k], b[k]);
        store_f32<T, kVec>(static_cast<T*>(A.y) + row * A.N + ring.column(k), v[k]);
      }
    }
    if (threadIdx.x == 0) {
      if (A.mean != nullptr) A.mean[row] = mean;
      if (A.rstd != nullptr) A.rstd[row] = rstd;
    }
    ring.advance();
  }
}

template <typename T, int kVec, int kPer, int kThreads, int kBlocks, bool kCollapse>
hcmix_status launch_norm_ring(const NormArgs& A, int64_t vecs, cudaStream_t stream) {
  constexpr int kRows = kCollapse ? kStreams : 1;
  const RingPlan p = ring_plan(vecs, kPer, kThreads, kBlocks, kRows, kVec * (int)sizeof(T));
  const size_t smem = kRingStages<kRows, kPer, kThreads, kBlocks> * p.stage;
  const int64_t blocks = A.M < kSms * p.each ? A.M : kSms * p.each;
  return launch(hcmix_norm_ring_kernel<T, kVec, kPer, kThreads, kBlocks, kCollapse>,
                dim3((unsigned)blocks), p.threads, smem, stream, A);
}

// The variant goes by type, alignment and width, never by the number of rows: a
// row's result is the same bits in a call of one row and of many.
template <typename T, int kVec, bool kCollapse>
hcmix_status launch_norm(const NormArgs& A, cudaStream_t stream) {
  // vectors a thread and threads of the usual block: what a thread loads before it
  // adds anything up (four streams' worth when collapsing) has to fit its registers
  constexpr int kMost = (kVec == 1 ? 16 : 4) / (kCollapse ? 2 : 1);
  constexpr int kThreads = kCollapse ? 512 : 256;
  const int64_t vecs = (A.N + kVec - 1) / kVec;
  const dim3 grid((unsigned)A.M);
  const auto threads = [&](int per) { return (unsigned)((vecs + per - 1) / per + 31) / 32 * 32; };
  if constexpr (kVec > 1) {
    if (vecs <= 256) return launch_norm_ring<T, kVec, 1, 256, 4, kCollapse>(A, vecs, stream);
    if (vecs <= 640) return launch_norm_ring<T, kVec, 2, 320, 2, kCollapse>(A, vecs, stream);
    if (vecs <= 1024) return launch_norm_ring<T, kVec, 2, 512, 1, kCollapse>(A, vecs, stream);
  } else {
    if (vecs <= kThreads * kMost)
      return launch(hcmix_norm_kernel<T, kVec, kMost, kThreads, kCollapse>, grid, threads(kMost), 0,
                    stream, A);
  }
  if (vecs <= 1024 * kMost)
    return launch(hcmix_norm_kernel<T, kVec, kMost, 1024, kCollapse>, grid, threads(kMost), 0,
                  stream, A);
  return launch(hcmix_norm_wide_kernel<T, kVec, kCollapse>, grid, 512, 0, stream, A);
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
  begin_kernel();
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
  block_sums_all<2>(sum, part);
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
  begin_kernel();
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

// dx and the partial sums of the weight's and bias's gradient in one pass over x
// and dy, through the ring; a block works on kGroup rows at a time, with one
// barrier for all their sums.  A thread keeps dweight and dbias of its columns in
// registers.  With one vector a thread (kPer 1) weight, (x - mean) rstd and
// dy weight stay there too; with more they are read and worked out again, from
// L1 and the stage.
template <typename T, int kVec, int kPer, int kGroup, int kThreads, int kBlocks>
__global__ void __launch_bounds__(kThreads, kBlocks) hcmix_norm_backward_kernel(const NormArgs A) {
  begin_kernel();
  extern __shared__ __align__(16) unsigned char smem[];
  __shared__ float part[2][2 * kGroup * 32];
  constexpr bool kKeep = kPer == 1;
  constexpr int kKept = kKeep ? kGroup : 1;
  constexpr int kStages = kRingStages<2 * kGroup, kPer, kThreads, kBlocks>;
  Ring<T, kVec, kPer, 2 * kGroup, kStages> ring(smem, A.N);
  const T* x = static_cast<const T*>(A.x) + blockIdx.x * kGroup * A.x_stride;
  const T* dy = static_cast<const T*>(A.dy) + blockIdx.x * kGroup * A.dy_stride;
  const int64_t x_jump = gridDim.x * kGroup * A.x_stride;
  const int64_t dy_jump = gridDim.x * kGroup * A.dy_stride;
  const int M = (int)A.M, jump = gridDim.x * kGroup;
  int64_t next = blockIdx.x * kGroup;
  const auto fetch = [&](int to) {
#pragma unroll
    for (int r = 0; r < kGroup; ++r) {
      if (next + r < M) {
        ring.copy(to, 2 * r, x + r * A.x_stride);
        ring.copy(to, 2 * r + 1, dy + r * A.dy_stride);
      }
    }
    async_commit();  // an empty group past the last row keeps the count
    next += jump;
    x += x_jump;
    dy += dy_jump;
  };
#pragma unroll
  for (int s = 0; s < kStages - 1; ++s) fetch(s * ring.group());
  float dw[kPer][kVec] = {}, db[kPer][kVec] = {}, w[kVec];
  const auto load_weight = [&](int k) {
#pragma unroll
    for (int e = 0; e < kVec; ++e) w[e] = 1.f;
    if (A.weight != nullptr && ring.has(k))
      load_param<T, kVec>(A.weight, A.p32, ring.column(k), w);
  };
  if (kKeep) load_weight(0);
  const float inv = 1.f / (float)A.N;
  int odd = 0;
  float next_mean[kGroup], next_rstd[kGroup];
  const auto fetch_stats = [&](int64_t row) {
#pragma unroll
    for (int r = 0; r < kGroup; ++r) {
      if (row + r < M) {
        next_mean[r] = A.mean[row + r];
        next_rstd[r] = A.rstd[row + r];
      }
    }
  };
  fetch_stats(next - (int64_t)(kStages - 1) * jump);
  for (int64_t row = blockIdx.x * kGroup; row < M; row += jump, odd ^= 1) {
    float mean[kGroup], rstd[kGroup];
#pragma unroll
    for (int r = 0; r < kGroup; ++r) mean[r] = next_mean[r], rstd[r] = next_rstd[r];
    fetch_stats(row + jump);
    fetch(ring.refill());
    async_wait<kStages - 1>();
    float xh[kKept][kVec], t[kKept][kVec], g[kVec];
    const auto load_row = [&](int r, int k) {
      const int q = kKeep ? r : 0;
      ring.read(2 * r, k).unpack(xh[q]);
      ring.read(2 * r + 1, k).unpack(g);
      if (!kKeep) load_weight(k);
      vadd(xh[q], -mean[r], xh[q]);
      vmul(xh[q], rstd[r], xh[q]);
      vmul(t[q], g, w);
    };
    float sums[2 * kGroup];
#pragma unroll
    for (int r = 0; r < kGroup; ++r) {
      Acc acc[2];
#pragma unroll
      for (int k = 0; k < kPer; ++k) {
        if (ring.has(k) && row + r < M) {
          const int q = kKeep ? r : 0;
          load_row(r, k);
          vfma(dw[k], g, xh[q], dw[k]);
          vadd(db[k], g, db[k]);
          acc[0].add(t[q]);
          acc[1].add(t[q], xh[q]);
        }
      }
      sums[2 * r] = acc[0].sum();
      sums[2 * r + 1] = acc[1].sum();
    }
    // two groups apart, a barrier lies between the uses of `part`
    block_sums_all<2 * kGroup>(sums, part[odd]);
#pragma unroll
    for (int r = 0; r < kGroup; ++r) {
      const float c1 = sums[2 * r] * inv, c2 = sums[2 * r + 1] * inv;
#pragma unroll
      for (int k = 0; k < kPer; ++k) {
        if (ring.has(k) && row + r < M) {
          const int q = kKeep ? r : 0;
          if (!kKeep) load_row(r, k);
          vadd(t[q], -c1, t[q]);
          vfma(t[q], -c2, xh[q], t[q]);
          vmul(t[q], rstd[r], t[q]);
          store_f32<T, kVec>(static_cast<T*>(A.dx) + (row + r) * A.N + ring.column(k), t[q]);
        }
      }
    }
    ring.advance();
  }
  float* out = A.part + (int64_t)blockIdx.x * 2 * A.N;
#pragma unroll
  for (int k = 0; k < kPer; ++k) {
    if (ring.has(k)) {
      // the workspace is aligned, and so are whole vectors' columns
      constexpr int kQuad = kVec % 4 == 0 ? 4 : 1;
#pragma unroll
      for (int e = 0; e < kVec; e += kQuad) {
        float q[kQuad], p[kQuad];
#pragma unroll
        for (int i = 0; i < kQuad; ++i) q[i] = dw[k][e + i], p[i] = db[k][e + i];
        store_f32<float, kQuad>(out + ring.column(k) + e, q);
        store_f32<float, kQuad>(out + A.N + ring.column(k) + e, p);
      }
    }
  }
}

// The partial rows added up: 32 columns a block, 16 groups of rows, each group's
// rows and then the groups in order.
constexpr int kJoinGroups = 16;

__global__ void __launch_bounds__(32 * kJoinGroups) hcmix_norm_join_kernel(const NormArgs A) {
  begin_kernel();
  __shared__ float part[kJoinGroups][32];
  const int lane = threadIdx.x % 32, group = threadIdx.x / 32;
  const int64_t c = (int64_t)blockIdx.x * 32 + lane;
  float s = 0.f;
  if (c < 2 * A.N) {
#pragma unroll 8
    for (int b = group; b < A.blocks; b += kJoinGroups) s += A.part[(int64_t)b * 2 * A.N + c];
  }
  part[group][lane] = s;
  __syncthreads();
  if (group != 0 || c >= 2 * A.N) return;
  for (int i = 1; i < kJoinGroups; ++i) s += part[i][lane];
  (c < A.N ? A.dweight[c] : A.dbias[c - A.N]) = s;
}

// How a backward call runs.
struct NormPlan {
  int variant;  // of launch_norm_backward; 0: dx and the column sums by separate kernels
  int blocks;   // partial rows of the column sums
  RingPlan ring;
};

// The same for every call of a size and type, so that the workspace can be sized
// before the operands are known; rows of 16-byte vectors (`wide`) go through the
// ring, and so do unaligned fp32 ones, element by element.
inline NormPlan norm_plan(int size, bool wide, int64_t M, int64_t N) {
  NormPlan p = {};
  const int vec = wide ? 16 / size : 1;
  const int64_t vecs = (N + vec - 1) / vec;
  const int per[5] = {0, 1, 1, 2, 4}, most[5] = {0, 256, 640, 640, 640}, each[5] = {0, 3, 1, 1, 1};
  const int group[5] = {0, 2, 2, 1, 1};  // rows at a time
  if (vec * size >= 4 && M > 0)
    for (int v = 1; v < 5 && p.variant == 0; ++v)
      if (vecs <= per[v] * most[v]) p.variant = v;
  if (p.variant == 0) {
    p.blocks = (int)(M < 64 ? M : 64);
    return p;
  }
  const int v = p.variant;
  p.ring = ring_plan(vecs, per[v], most[v], each[v], 2 * group[v], vec * size);
  const int64_t groups = (M + group[v] - 1) / group[v];
  p.blocks = (int)(groups < kSms * p.ring.each ? groups : kSms * p.ring.each);
  return p;
}

// The larger of the two alignments' needs.
inline size_t norm_workspace(int size, int64_t M, int64_t N) {
  const int a = norm_plan(size, true, M, N).blocks, b = norm_plan(size, false, M, N).blocks;
  return ((size_t)(a > b ? a : b) * 2 * (size_t)N * 4 + 255) / 256 * 256;
}

template <typename T, int kVec, int kPer, int kGroup, int kThreads, int kBlocks>
hcmix_status launch_norm_backward_ring(const NormArgs& A, const RingPlan& p, cudaStream_t stream) {
  const size_t smem = kRingStages<2 * kGroup, kPer, kThreads, kBlocks> * p.stage;
  return launch(hcmix_norm_backward_kernel<T, kVec, kPer, kGroup, kThreads, kBlocks>,
                dim3(A.blocks), p.threads, smem, stream, A);
}

template <typename T, int kVec>
hcmix_status launch_norm_backward(NormArgs A, cudaStream_t stream) {
  const NormPlan p = norm_plan(sizeof(T), kVec > 1, A.M, A.N);
  A.blocks = p.blocks;
  hcmix_status st = HCMIX_OK;
  if (A.dweight == nullptr || p.variant == 0) {
    const int64_t vecs = (A.N + kVec - 1) / kVec;
    const unsigned threads = vecs >= 256 ? 256 : (unsigned)(vecs + 31) / 32 * 32;
    if (A.M > 0)
      st = launch(hcmix_norm_dx_kernel<T, kVec>, dim3((unsigned)A.M), threads, 0, stream, A);
    if (st != HCMIX_OK || A.dweight == nullptr) return st;
    const int64_t per = (int64_t)kColumnThreads * kVec;
    if (p.blocks > 0)
      st = launch(hcmix_norm_columns_kernel<T, kVec>,
                  dim3((unsigned)((A.N + per - 1) / per), p.blocks), kColumnThreads, 0, stream, A);
  } else if constexpr (kVec * sizeof(T) >= 4) {
    switch (p.variant) {
      case 1: st = launch_norm_backward_ring<T, kVec, 1, 2, 256, 3>(A, p.ring, stream); break;
      case 2: st = launch_norm_backward_ring<T, kVec, 1, 2, 640, 1>(A, p.ring, stream); break;
      case 3: st = launch_norm_backward_ring<T, kVec, 2, 1, 640, 1>(A, p.ring, stream); break;
      default: st = launch_norm_backward_ring<T, kVec, 4, 1, 640, 1>(A, p.ring, stream); break;
    }
  }
  if (st != HCMIX_OK) return st;
  return launch(hcmix_norm_join_kernel, dim3((unsigned)((2 * A.N + 31) / 32)), 32 * kJoinGroups, 0,
                stream, A);
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
