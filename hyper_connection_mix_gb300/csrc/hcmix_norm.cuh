// Layer norm forward (of a plain row, or of the collapsed streams) and backward.
//
// Resident blocks take rows in turn through a ring of rows in shared memory, copied
// ahead of their use; what belongs to a thread's columns (weight, bias, sums over
// rows) stays in its registers.  Rows too wide for that are passed over several
// times.
//
// Bound by HBM (copy rate 6787 GB/s) less what a row's reduction stalls: measured, collapse
// + norm of 16384 x 4 x 5120 bf16 137 us (839 MB, 6.1 TB/s), norm of 16384 x 5120 bf16 64 us
// (5.2 TB/s), backward of 4096 x 5120 bf16 29.5 us (126 MB, 4.3 TB/s; 4 us of it the join).
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

// v = x itself, or sum_i pre[i] x_i, of the loaded vectors.
template <typename T, int kVec, bool kCollapse>
__device__ __forceinline__ void norm_values(const Packed<T, kVec> (&s)[kCollapse ? kStreams : 1],
                                            const float* pre, float (&v)[kVec]) {
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

// Rows too wide for the ring: three passes over the row, the later two mostly from
// L2.
template <typename T, int kVec, bool kCollapse>
__global__ void __launch_bounds__(512) hcmix_norm_wide_kernel(const NormArgs A) {
  begin_kernel();
  __shared__ float part[2][32];
  constexpr int kRows = kCollapse ? kStreams : 1;
  const int64_t row = blockIdx.x;
  const T* x = static_cast<const T*>(A.x) + row * A.x_stride;
  const int64_t step = (int64_t)blockDim.x * kVec, c0 = (int64_t)threadIdx.x * kVec;
  float pre[kStreams] = {};
  if constexpr (kCollapse) {
#pragma unroll
    for (int i = 0; i < kStreams; ++i) pre[i] = A.pre[row * kStreams + i];
  }
  float v[kVec];
  const auto load = [&](int64_t c) {
    Packed<T, kVec> s[kRows];
#pragma unroll
    for (int i = 0; i < kRows; ++i) s[i] = load_vec<T, kVec>(x + i * A.N + c);
    norm_values<T, kVec, kCollapse>(s, pre, v);
  };
  Acc sum, square;
#pragma unroll 4
  for (int64_t c = c0; c < A.N; c += step) {
    load(c);
    sum.add(v);
  }
  const float inv = 1.f / (float)A.N;
  float total[1] = {sum.sum()};
  team_sums<1>(total, part[0]);
  const float mean = total[0] * inv;
#pragma unroll 4
  for (int64_t c = c0; c < A.N; c += step) {
    load(c);
    vadd(v, -mean, v);
    square.add(v, v);
  }
  float sq[1] = {square.sum()};
  team_sums<1>(sq, part[1]);
  const float rstd = 1.f / sqrtf(sq[0] * inv + A.eps);
#pragma unroll 2
  for (int64_t c = c0; c < A.N; c += step) {
    load(c);
    if (kCollapse && A.h != nullptr) store_f32<T, kVec>(static_cast<T*>(A.h) + row * A.N + c, v);
    float w[kVec], b[kVec];
    load_param<T, kVec>(A.weight, A.p32, c, 1.f, w);
    load_param<T, kVec>(A.bias, A.p32, c, 0.f, b);
    vadd(v, -mean, v);
    vmul(v, rstd, v);
    vfma(v, v, w, b);
    store_f32<T, kVec>(static_cast<T*>(A.y) + row * A.N + c, v);
  }
  if (threadIdx.x == 0) {
    if (A.mean != nullptr) A.mean[row] = mean;
    if (A.rstd != nullptr) A.rstd[row] = rstd;
  }
}

// ---------------------------------------------------------------- the ring

// A matrix in memory, whose rows a ring copies.
struct Matrix {
  const unsigned char *begin, *end;
  uint32_t row_bytes;  // from a row to the next, as far as its low bits go
  template <typename T>
  static __device__ __forceinline__ Matrix of(const void* p, int64_t rows, int64_t stride,
                                              int64_t width) {
    const unsigned char* b = static_cast<const unsigned char*>(p);
    return {b, b + ((rows - 1) * stride + width) * (int64_t)sizeof(T),
            (uint32_t)stride * (uint32_t)sizeof(T)};
  }
  // How far past 16 bytes row r starts.
  __device__ __forceinline__ int misalignment(uint32_t r) const {
    return ((uint32_t)reinterpret_cast<uintptr_t>(begin) + r * row_bytes) & 15;
  }
};

// A ring of kStages groups of rows in shared memory, for one team of blockDim.x
// threads.  A group is kRows source rows (streams; x and dy of several rows); a thread
// works on kPer vectors of each, its columns the same in every group.  Rows come by
// asynchronous 16-byte copies.
//
// Rows of 16-byte vectors (kOwn): each thread copies the vectors that it will read
// itself, so that no barrier stands between the copies and their use.  Other rows are
// copied as the aligned 16-byte blocks that hold them, and read by 4-byte vectors or
// by elements as they lie there, after a barrier.  The bytes of a block beside its row
// belong to the rows next to it, except at the matrix's two ends, where the elements
// are copied one by one.
//
// The first kFull vectors of every thread lie within the row.
template <typename T, int kVec, int kPer, int kRows, int kStages, int kFull>
struct Ring {
  using V = Packed<T, kVec>;
  static constexpr bool kOwn = sizeof(V) == 16;
  unsigned char* base;  // of the team
  int pitch;   // bytes from one of the thread's vectors to its next
  int at;      // byte offset of the stage that is read
  int columns, first, step;  // the thread's columns: first + k * step, below columns
  __device__ __forceinline__ Ring(unsigned char* smem, int64_t width)
      : pitch(blockDim.x * sizeof(V)),
        at(0),
        columns((int)width),
        first(threadIdx.x * kVec),
        step(blockDim.x * kVec) {
    base = smem + threadIdx.y * (kStages * group());
  }
  // Bytes of a block's rings: `teams` of `threads` threads.
  static constexpr size_t bytes(int threads, int teams) {
    return (size_t)kStages * kRows * teams * (kPer * threads * sizeof(V) + (kOwn ? 0 : 16));
  }
  __device__ __forceinline__ int row() const { return kPer * pitch + (kOwn ? 0 : 16); }
  __device__ __forceinline__ int group() const { return kRows * row(); }
  __device__ __forceinline__ int column(int k) const { return first + k * step; }
  __device__ __forceinline__ bool has(int k) const { return k < kFull || column(k) < columns; }
  // Starts the copy of source row i, given its first element, into the stage at
  // byte offset `to`.
  __device__ __forceinline__ void copy(int to, int i, const T* from, const Matrix& all) const {
    unsigned char* dst = base + to + i * row();
    if constexpr (kOwn) {
#pragma unroll
      for (int k = 0; k < kPer; ++k)
        if (has(k)) async_copy16(dst + threadIdx.x * 16 + k * pitch, from + column(k));
    } else {
      const int m = (int)(reinterpret_cast<uintptr_t>(from) & 15);
      const int blocks = (m + columns * (int)sizeof(T) + 15) / 16;
      const unsigned char* src = reinterpret_cast<const unsigned char*>(from) - m;
      for (int b = threadIdx.x; b < blocks; b += blockDim.x) {
        const unsigned char* p = src + b * 16;
        if (p >= all.begin && p + 16 <= all.end) {
          async_copy16(dst + b * 16, p);
        } else {
#pragma unroll
          for (int e = 0; e < 16; e += (int)sizeof(T))
            if (p + e >= all.begin && p + e < all.end)
              *reinterpret_cast<T*>(dst + b * 16 + e) = *reinterpret_cast<const T*>(p + e);
        }
      }
    }
  }
  // The stage to refill while this group is worked on: the one read a group ago.
  __device__ __forceinline__ int refill() const {
    return at == 0 ? (kStages - 1) * group() : at - group();
  }
  // Starts the next group's copies by fetch(stage) and waits for this group's.
  template <typename Fetch>
  __device__ __forceinline__ void turn(Fetch&& fetch) const {
    if constexpr (kOwn) {
      fetch(refill());
      async_wait<kStages - 1>();
    } else {
      async_wait<kStages - 2>();
      team_sync(blockDim.x / 32);  // and the stage to refill has been read by all
      fetch(refill());
    }
  }
  // The thread's k-th vector of source row i, which starts m bytes past 16.
  __device__ __forceinline__ V read(int i, int k, int m) const {
    const unsigned char* p = base + at + i * row() + threadIdx.x * (int)sizeof(V) + k * pitch;
    return *reinterpret_cast<const V*>(kOwn ? p : p + m);
  }
  __device__ __forceinline__ void advance() {
    at += group();
    if (at == kStages * group()) at = 0;
  }
};

constexpr int kSms = 152;

// A shape of ring kernel: blocks of kThreads threads that hold kUnits times 16
// bytes of each of a group's kRows rows, kBlocks of them a multiprocessor; as many stages as fit
// 200 KB, up to eight.  Narrow rows take a team of fewer threads each, several teams
// a block.
//
// A shape is taken for rows of more than kOver bytes, so its teams have at least
// kLeast threads.  They have less than 32 threads' worth of vectors to spare: of kPer
// vectors a thread only the last ceil(32 kPer / kLeast) can lie past the row's end.
template <int kUnits_, int kThreads_, int kBlocks_, int kOver_>
struct Shape {
  static constexpr int kUnits = kUnits_, kThreads = kThreads_, kBlocks = kBlocks_;
  static constexpr int kRowBytes = kUnits * kThreads * 16;
  static constexpr int kLeast = (kOver_ / 16 / kUnits + 1 + 31) / 32 * 32;
  static constexpr int kTeams = kThreads / kLeast;  // at most
  template <int kPer>
  static constexpr int kFull = kPer - (32 * kPer + kLeast - 1) / kLeast;
};
template <typename S, int kRows>
constexpr int kFit = 200 * 1024 / (S::kBlocks * kRows * S::kRowBytes);
template <typename S, int kRows>
constexpr int kStagesOf = kFit<S, kRows> > 8 ? 8 : kFit<S, kRows> < 2 ? 2 : kFit<S, kRows>;

// The most shared memory that a kernel of ring R and shape S takes.
template <typename R, typename S>
constexpr size_t ring_most = R::bytes(S::kThreads / S::kTeams, S::kTeams);

struct RingPlan {
  int threads, teams, blocks;  // of a team; of a block
};
// `groups` groups of rows of `row_bytes`; as many teams a block as it takes threads,
// but blocks on every multiprocessor first.
template <typename S>
inline RingPlan ring_plan(int64_t row_bytes, int64_t groups) {
  const int64_t units = (row_bytes + 15) / 16;
  RingPlan p;
  p.threads = (int)((units + S::kUnits - 1) / S::kUnits + 31) / 32 * 32;
  const int64_t wanted = (groups + kSms * S::kBlocks - 1) / (kSms * S::kBlocks);
  p.teams = S::kThreads / p.threads;
  p.teams = p.teams < wanted ? p.teams : (int)wanted;
  const int64_t blocks = (groups + p.teams - 1) / p.teams;
  p.blocks = (int)(blocks < kSms * S::kBlocks ? blocks : kSms * S::kBlocks);
  return p;
}

// The norm, one row at a time.  A warp takes the mean of its columns and the squared
// differences from that, and one barrier later the warps' are joined:
//   mean = sum_w s_w / N,  N var = sum_w (q_w + n_w (s_w / n_w - mean)^2),
// so that a large mean costs no digits.  Weight and bias are kept in registers where they
// fit beside the row (16 values a thread or fewer); else they come for every row, 16
// values of each a thread at a time so that their loads overlap (3588 x 12562 fp32: 137 us,
// a vector at a time 222 us).
template <typename T, int kVec, typename S, bool kCollapse>
__global__ void __launch_bounds__(S::kThreads, S::kBlocks) hcmix_norm_kernel(const NormArgs A) {
  begin_kernel();
  extern __shared__ __align__(16) unsigned char smem[];
  __shared__ float2 parts[8][2][32];  // of each team: s_w and q_w
  __shared__ float counts[8][32];     // n_w
  float2(&part)[2][32] = parts[threadIdx.y];
  constexpr int kRows = kCollapse ? kStreams : 1;
  constexpr int kPer = S::kUnits * 16 / (kVec * (int)sizeof(T));
  constexpr int kStages = kStagesOf<S, kRows>;
  using R = Ring<T, kVec, kPer, kRows, kStages, S::template kFull<kPer>>;
  constexpr bool kKeep = kPer * kVec <= 16;
  constexpr int kKept = kKeep ? kPer : 16 / kVec;  // else as many at a time
  R ring(smem, A.N);
  const Matrix all = Matrix::of<T>(A.x, A.M, A.x_stride, kRows * A.N);
  const uint32_t M = (uint32_t)A.M, jump = gridDim.x * blockDim.y;
  const uint32_t first = blockIdx.x * blockDim.y + threadIdx.y;
  const T* from = static_cast<const T*>(A.x) + first * A.x_stride;
  const int64_t x_jump = jump * A.x_stride;
  uint32_t next = first;
  const auto fetch = [&](int to) {
    if (next < M) {
#pragma unroll
      for (int i = 0; i < kRows; ++i) ring.copy(to, i, from + i * A.N, all);
    }
    async_commit();  // an empty group past the last row keeps the count
    next += jump;
    from += x_jump;
  };
#pragma unroll
  for (int s = 0; s < kStages - 1; ++s) fetch(s * ring.group());
  float w[kKept][kVec], b[kKept][kVec];
  const auto load_params = [&](int from) {  // of vectors from .. from + kKept - 1
#pragma unroll
    for (int i = 0; i < kKept; ++i) {
      if (ring.has(from + i)) {
        load_param<T, kVec>(A.weight, A.p32, ring.column(from + i), 1.f, w[i]);
        load_param<T, kVec>(A.bias, A.p32, ring.column(from + i), 0.f, b[i]);
      }
    }
  };
  if constexpr (kKeep) load_params(0);
  const int warps = blockDim.x / 32, warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  int count = 0;
#pragma unroll
  for (int k = 0; k < kPer; ++k) count += ring.has(k) ? kVec : 0;
  const float n = (float)__reduce_add_sync(0xffffffffu, count), inv_n = n > 0.f ? 1.f / n : 0.f;
  if (lane == 0) counts[threadIdx.y][warp] = n;
  int odd = 0;
  const float inv = 1.f / (float)A.N;
  for (uint32_t row = first; row < M; row += jump, odd ^= 1) {
    float pre[kStreams] = {};
    if constexpr (kCollapse) {
#pragma unroll
      for (int i = 0; i < kStreams; ++i) pre[i] = A.pre[(int64_t)row * kStreams + i];
    }
    ring.turn(fetch);
    int m[kRows] = {};
    if constexpr (!R::kOwn) {
#pragma unroll
      for (int i = 0; i < kRows; ++i)
        m[i] = (all.misalignment(row) + i * (int)A.N * (int)sizeof(T)) & 15;
    }
    float v[kPer][kVec];
    Acc acc;
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
      if (ring.has(k)) {
        Packed<T, kVec> s[kRows];
#pragma unroll
        for (int i = 0; i < kRows; ++i) s[i] = ring.read(i, k, m[i]);
        norm_values<T, kVec, kCollapse>(s, pre, v[k]);
        acc.add(v[k]);
      }
    }
    const float sum = warp_sum(acc.sum()), own_mean = sum * inv_n;
    Acc square;
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
      if (ring.has(k)) {
        float d[kVec];
        vadd(d, -own_mean, v[k]);
        square.add(d, d);
      }
    }
    const float own_square = warp_sum(square.sum());
    float mean = own_mean, all_square = own_square;
    if (warps > 1) {
      // two rows apart, a barrier lies between the uses of `part`
      if (lane == 0) part[odd][warp] = make_float2(sum, own_square);
      team_sync(warps);
      const float2 p = lane < warps ? part[odd][lane] : make_float2(0.f, 0.f);
      const float c = lane < warps ? counts[threadIdx.y][lane] : 0.f;
      mean = warp_sum(p.x) * inv;
      const float d = c > 0.f ? p.x / c - mean : 0.f;
      all_square = warp_sum(fmaf(c * d, d, p.y));
    }
    const float rstd = 1.f / sqrtf(all_square * inv + A.eps);
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
      if (!kKeep && k % kKept == 0) load_params(k);
      if (ring.has(k)) {
        if (kCollapse && A.h != nullptr)
          store_f32<T, kVec>(static_cast<T*>(A.h) + row * A.N + ring.column(k), v[k]);
        vadd(v[k], -mean, v[k]);
        vmul(v[k], rstd, v[k]);
        vfma(v[k], v[k], w[k % kKept], b[k % kKept]);
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

template <typename T, int kVec, typename S, bool kCollapse>
hcmix_status launch_norm_ring(const NormArgs& A, cudaStream_t stream) {
  constexpr int kRows = kCollapse ? kStreams : 1;
  const RingPlan p = ring_plan<S>(A.N * (int64_t)sizeof(T), A.M);
  using R = Ring<T, kVec, S::kUnits * 16 / (kVec * (int)sizeof(T)), kRows, kStagesOf<S, kRows>, 0>;
  return launch(hcmix_norm_kernel<T, kVec, S, kCollapse>, dim3(p.blocks),
                dim3(p.threads, p.teams), R::bytes(p.threads, p.teams), ring_most<R, S>, stream, A);
}

// The shape goes by type, alignment and width, never by the number of rows: a row's
// result is the same bits in a call of one row and of many.  The smallest that holds
// the row is taken; 640 threads with four units of each of four streams would leave
// room for one stage only.
template <typename T, int kVec, bool kCollapse>
hcmix_status launch_norm(const NormArgs& A, cudaStream_t stream) {
  constexpr int kNarrow = 4096;  // bytes
  using S1 = Shape<2, 256, 3, 0>;
  // 16384 rows of 5120 bf16: two blocks 64.5 us, three 80 us (too few registers); 3001 of
  // 2051 fp32: 15.3 us and 14.2 us
  using S2 = Shape<2, 320, sizeof(T) == 4 && !kCollapse ? 3 : 2, kNarrow>;
  using S3 = Shape<2, 640, 1, S2::kRowBytes>;
  using S4 = Shape<4, 640, 1, S3::kRowBytes>;
  using S5 = Shape<8, 640, 1, S4::kRowBytes>;  // of fp32, as many values a thread as S4's of 16 bits
  const int64_t bytes = A.N * (int64_t)sizeof(T);
  if (bytes <= kNarrow) return launch_norm_ring<T, kVec, S1, kCollapse>(A, stream);
  if (bytes <= S2::kRowBytes) return launch_norm_ring<T, kVec, S2, kCollapse>(A, stream);
  if (bytes <= S3::kRowBytes) return launch_norm_ring<T, kVec, S3, kCollapse>(A, stream);
  if constexpr (!kCollapse) {
    if (bytes <= S4::kRowBytes) return launch_norm_ring<T, kVec, S4, false>(A, stream);
    if constexpr (sizeof(T) == 4)
      if (bytes <= S5::kRowBytes) return launch_norm_ring<T, kVec, S5, false>(A, stream);
  }
  return launch(hcmix_norm_wide_kernel<T, kVec, kCollapse>, dim3((unsigned)A.M), dim3(512), 0, 0,
                stream, A);
}

inline hcmix_status run_norm(const NormArgs& A, hcmix_type type, bool collapse,
                             cudaStream_t stream) {
  // a row's streams start N apart, whatever its stride
  const int bytes = vector_bytes(size_of(type), {{A.x, A.x_stride}, {A.y, A.N}, {A.h, A.N}});
  return with_vector(type, bytes, [&](auto t, auto vec, auto) {
    using T = decltype(t);
    constexpr int kVec = decltype(vec)::value;
    return collapse ? launch_norm<T, kVec, true>(A, stream) : launch_norm<T, kVec, false>(A, stream);
  });
}

// ---------------------------------------------------------------- backward

// dx on its own, one block a row, the row passed over twice: 4096 x 5120 bf16 34.5 us, fp32
// 4096 x 4096 49 us (with the other gradients, through the ring, 29.5 and 40 us).
template <typename T, int kVec>
__global__ void __launch_bounds__(512) hcmix_norm_dx_kernel(const NormArgs A) {
  begin_kernel();
  __shared__ float part[2 * 32];
  const int64_t row = blockIdx.x;
  const T* x = static_cast<const T*>(A.x) + row * A.x_stride;
  const T* dy = static_cast<const T*>(A.dy) + row * A.dy_stride;
  const float mean = A.mean[row], rstd = A.rstd[row];
  const int64_t step = (int64_t)blockDim.x * kVec, c0 = (int64_t)threadIdx.x * kVec;
  float xh[kVec], t[kVec], w[kVec];
  const auto load = [&](int64_t c) {
    load_vec<T, kVec>(x + c).unpack(xh);
    load_vec<T, kVec>(dy + c).unpack(t);
    load_param<T, kVec>(A.weight, A.p32, c, 1.f, w);
    vadd(xh, -mean, xh);
    vmul(xh, rstd, xh);
    vmul(t, t, w);
  };
  Acc acc[2];
#pragma unroll 4
  for (int64_t c = c0; c < A.N; c += step) {
    load(c);
    acc[0].add(t);
    acc[1].add(t, xh);
  }
  float sum[2] = {acc[0].sum(), acc[1].sum()};
  team_sums<2>(sum, part);
  const float inv = 1.f / (float)A.N;
  const float c1 = sum[0] * inv, c2 = sum[1] * inv;
#pragma unroll 4
  for (int64_t c = c0; c < A.N; c += step) {
    load(c);
    vadd(t, -c1, t);
    vfma(t, -c2, xh, t);
    vmul(t, rstd, t);
    store_f32<T, kVec>(static_cast<T*>(A.dx) + row * A.N + c, t);
  }
}

// A thread's vector of the partial sums of the weight's and bias's gradient: on 16
// bytes in the workspace too where the vectors are 16 bytes.
template <typename T, int kVec>
__device__ __forceinline__ void store_partial(float* out, const float (&v)[kVec]) {
  constexpr int kQuad = kVec % 4 == 0 ? 4 : 1;
#pragma unroll
  for (int e = 0; e < kVec; e += kQuad) {
    float q[kQuad];
#pragma unroll
    for (int i = 0; i < kQuad; ++i) q[i] = v[e + i];
    store_f32<float, kQuad>(out + e, q);
  }
}

constexpr int kColumnThreads = 128, kColumnSlabs = 64;

// Partial sums of the weight's and bias's gradient on their own: block (b, s) takes
// columns from b * kColumnThreads * kVec and rows s, s + slabs, ...
template <typename T, int kVec>
__global__ void __launch_bounds__(kColumnThreads) hcmix_norm_columns_kernel(const NormArgs A) {
  begin_kernel();
  const int64_t c = ((int64_t)blockIdx.x * kColumnThreads + threadIdx.x) * kVec;
  if (c >= A.N) return;
  float dw[kVec] = {}, db[kVec] = {};
#pragma unroll 4
  for (int64_t row = blockIdx.y; row < A.M; row += gridDim.y) {
    float v[kVec], g[kVec];
    load_vec<T, kVec>(static_cast<const T*>(A.x) + row * A.x_stride + c).unpack(v);
    load_vec<T, kVec>(static_cast<const T*>(A.dy) + row * A.dy_stride + c).unpack(g);
    vadd(v, -A.mean[row], v);
    vmul(v, A.rstd[row], v);
    vfma(dw, g, v, dw);
    vadd(db, g, db);
  }
  float* out = A.part + (int64_t)blockIdx.y * 2 * A.N + c;
  store_partial<T, kVec>(out, dw);
  store_partial<T, kVec>(out + A.N, db);
}

// dx and the partial sums of the weight's and bias's gradient in one pass over x
// and dy, through the ring; a team works on kGroup rows at a time, with one barrier
// for all their sums.  A thread keeps dweight and dbias of its columns in registers,
// and the weight where they leave room (two units a thread); after the barrier x and
// dy are read from the stage again.
template <typename T, int kVec, typename S, int kGroup>
__global__ void __launch_bounds__(S::kThreads, S::kBlocks) hcmix_norm_backward_kernel(
    const NormArgs A) {
  begin_kernel();
  extern __shared__ __align__(16) unsigned char smem[];
  __shared__ float parts[8][2][2 * kGroup * 32];  // of each team
  float(&part)[2][2 * kGroup * 32] = parts[threadIdx.y];
  constexpr int kPer = S::kUnits * 16 / (kVec * (int)sizeof(T));
  constexpr int kStages = kStagesOf<S, 2 * kGroup>;
  using R = Ring<T, kVec, kPer, 2 * kGroup, kStages, S::template kFull<kPer>>;
  constexpr bool kKeepWeight = S::kUnits <= 2;
  constexpr int kKept = kKeepWeight ? kPer : 16 / kVec < kPer ? 16 / kVec : kPer;  // or at a time
  R ring(smem, A.N);
  const Matrix all_x = Matrix::of<T>(A.x, A.M, A.x_stride, A.N);
  const Matrix all_dy = Matrix::of<T>(A.dy, A.M, A.dy_stride, A.N);
  const uint32_t M = (uint32_t)A.M, jump = gridDim.x * blockDim.y * kGroup;
  const uint32_t first = (blockIdx.x * blockDim.y + threadIdx.y) * kGroup;
  const T* x = static_cast<const T*>(A.x) + first * A.x_stride;
  const T* dy = static_cast<const T*>(A.dy) + first * A.dy_stride;
  const int64_t x_jump = jump * A.x_stride, dy_jump = jump * A.dy_stride;
  uint32_t next = first;
  const auto fetch = [&](int to) {
#pragma unroll
    for (int r = 0; r < kGroup; ++r) {
      if (next + r < M) {
        ring.copy(to, 2 * r, x + r * A.x_stride, all_x);
        ring.copy(to, 2 * r + 1, dy + r * A.dy_stride, all_dy);
      }
    }
    async_commit();  // an empty group past the last row keeps the count
    next += jump;
    x += x_jump;
    dy += dy_jump;
  };
#pragma unroll
  for (int s = 0; s < kStages - 1; ++s) fetch(s * ring.group());
  float dw[kPer][kVec] = {}, db[kPer][kVec] = {}, w[kKept][kVec];
  const auto load_weights = [&](int from) {  // of vectors from .. from + kKept - 1
#pragma unroll
    for (int i = 0; i < kKept; ++i)
      if (ring.has(from + i))
        load_param<T, kVec>(A.weight, A.p32, ring.column(from + i), 1.f, w[i]);
  };
  if constexpr (kKeepWeight) load_weights(0);
  const float inv = 1.f / (float)A.N;
  int odd = 0;
  float next_mean[kGroup], next_rstd[kGroup];
  const auto fetch_stats = [&](uint32_t row) {
#pragma unroll
    for (int r = 0; r < kGroup; ++r) {
      if (row + r < M) {
        next_mean[r] = A.mean[row + r];
        next_rstd[r] = A.rstd[row + r];
      }
    }
  };
  fetch_stats(first);
  for (uint32_t row = first; row < M; row += jump, odd ^= 1) {
    float mean[kGroup], rstd[kGroup];
#pragma unroll
    for (int r = 0; r < kGroup; ++r) mean[r] = next_mean[r], rstd[r] = next_rstd[r];
    fetch_stats(row + jump);
    ring.turn(fetch);
    float xh[kVec], t[kVec], g[kVec];
    const auto load_row = [&](int r, int k) {
      int mx = 0, my = 0;
      if constexpr (!R::kOwn) mx = all_x.misalignment(row + r), my = all_dy.misalignment(row + r);
      ring.read(2 * r, k, mx).unpack(xh);
      ring.read(2 * r + 1, k, my).unpack(g);
      vadd(xh, -mean[r], xh);
      vmul(xh, rstd[r], xh);
      vmul(t, g, w[k % kKept]);
    };
    float sums[2 * kGroup];
#pragma unroll
    for (int r = 0; r < kGroup; ++r) {
      Acc acc[2];
#pragma unroll
      for (int k = 0; k < kPer; ++k) {
        if (!kKeepWeight && k % kKept == 0) load_weights(k);
        if (ring.has(k) && row + r < M) {
          load_row(r, k);
          vfma(dw[k], g, xh, dw[k]);
          vadd(db[k], g, db[k]);
          acc[0].add(t);
          acc[1].add(t, xh);
        }
      }
      sums[2 * r] = acc[0].sum();
      sums[2 * r + 1] = acc[1].sum();
    }
    // two groups apart, a barrier lies between the uses of `part`
    team_sums<2 * kGroup>(sums, part[odd]);
#pragma unroll
    for (int r = 0; r < kGroup; ++r) {
      // dx = rstd t - rstd c1 - rstd c2 xh, c1 and c2 the means of t and t xh
      const float s1 = -rstd[r] * (sums[2 * r] * inv), s2 = -rstd[r] * (sums[2 * r + 1] * inv);
      T* dx = static_cast<T*>(A.dx) + (int64_t)(row + r) * A.N;
#pragma unroll
      for (int k = 0; k < kPer; ++k) {
        if (!kKeepWeight && k % kKept == 0) load_weights(k);
        if (ring.has(k) && row + r < M) {
          load_row(r, k);
          vfma(xh, s2, xh, s1);
          vfma(xh, rstd[r], t, xh);
          store_f32<T, kVec>(dx + ring.column(k), xh);
        }
      }
    }
    ring.advance();
  }
  float* out = A.part + (int64_t)blockIdx.x * 2 * A.N;
  if (blockDim.y == 1) {
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
      if (ring.has(k)) {
        store_partial<T, kVec>(out + ring.column(k), dw[k]);
        store_partial<T, kVec>(out + A.N + ring.column(k), db[k]);
      }
    }
    return;
  }
  // the teams' sums added up in order, through the rings' memory
  __syncthreads();
  float* sums = reinterpret_cast<float*>(smem);
  float* own = sums + threadIdx.y * 2 * ring.columns;
#pragma unroll
  for (int k = 0; k < kPer; ++k) {
    if (ring.has(k)) {
#pragma unroll
      for (int e = 0; e < kVec; ++e) {
        own[ring.column(k) + e] = dw[k][e];
        own[ring.columns + ring.column(k) + e] = db[k][e];
      }
    }
  }
  __syncthreads();
  for (int i = threadIdx.y * blockDim.x + threadIdx.x; i < 2 * ring.columns;
       i += blockDim.x * blockDim.y) {
    float s = 0.f;
    for (int team = 0; team < (int)blockDim.y; ++team) s += sums[team * 2 * ring.columns + i];
    out[i] = s;
  }
}

// The partial rows added up: 32 columns a block, 16 groups of rows, each group's
// rows and then the groups in order.  Up to 320 partial rows (two blocks a
// multiprocessor leave 304) are one round of loads.
constexpr int kJoinGroups = 16, kJoinRound = 20;

__global__ void __launch_bounds__(32 * kJoinGroups) hcmix_norm_join_kernel(const NormArgs A) {
  begin_kernel();
  __shared__ float part[kJoinGroups][32];
  const int lane = threadIdx.x % 32, group = threadIdx.x / 32;
  const int64_t c = (int64_t)blockIdx.x * 32 + lane;
  float s = 0.f;
  if (c < 2 * A.N) {
    for (int b = group; b < A.blocks; b += kJoinGroups * kJoinRound) {
      float v[kJoinRound];
#pragma unroll
      for (int q = 0; q < kJoinRound; ++q) {
        const int r = b + q * kJoinGroups;
        v[q] = r < A.blocks ? A.part[(int64_t)r * 2 * A.N + c] : 0.f;
      }
#pragma unroll
      for (int q = 0; q < kJoinRound; ++q) s += v[q];
    }
  }
  part[group][lane] = s;
  __syncthreads();
  if (group != 0 || c >= 2 * A.N) return;
  for (int i = 1; i < kJoinGroups; ++i) s += part[i][lane];
  (c < A.N ? A.dweight[c] : A.dbias[c - A.N]) = s;
}

// Rows of up to kBackNarrow bytes, then of what a shape holds.  The last shape keeps the
// gradients of 32 columns of 16 bits a thread and spills, up to 1528 bytes of loads for single
// elements.  With its rows passed over by two kernels instead (us, ring / two kernels):
// 2048 x 20480 bf16 109 / 115, x 20478 148 / 220, x 20479 275 / 280; 4096 x 10248 116 / 127,
// x 10246 176 / 194, x 10247 256 / 249; 256 x 20480 29.5 / 28.4, x 20479 62 / 68; fp32 2048 x
// 10240 60 / 109, x 10239 76 / 201.
constexpr int kBackNarrow = 4096;
using Back1 = Shape<2, 256, 2, 0>;
using Back2 = Shape<2, 320, 2, kBackNarrow>;
using Back3 = Shape<2, 640, 1, Back2::kRowBytes>;
using Back4 = Shape<4, 640, 1, Back3::kRowBytes>;

// How a backward call runs: its shape (1 to 4; 0: dx and the column sums by separate
// kernels) and its blocks.  Rows of 16-byte vectors (`own`) go two at a time in the first two
// shapes; narrower vectors have no registers for that (4096 x 5119 bf16: two at a time 99 us,
// one 56 us).
struct NormPlan {
  int shape;
  RingPlan ring;
};

inline NormPlan norm_plan(int size, bool own, int64_t M, int64_t N) {
  NormPlan p = {};
  const int64_t row = N * size, groups = own ? (M + 1) / 2 : M;
  if (M == 0) return p;
  if (row <= kBackNarrow) p.shape = 1, p.ring = ring_plan<Back1>(row, groups);
  else if (row <= Back2::kRowBytes) p.shape = 2, p.ring = ring_plan<Back2>(row, groups);
  else if (row <= Back3::kRowBytes) p.shape = 3, p.ring = ring_plan<Back3>(row, M);
  else if (row <= Back4::kRowBytes) p.shape = 4, p.ring = ring_plan<Back4>(row, M);
  else p.ring.blocks = (int)(M < kColumnSlabs ? M : kColumnSlabs);
  return p;
}

// The workspace is sized before the operands' alignment is known, and one for many rows does
// for fewer: a partial row for each block that the shape can have.
inline size_t norm_workspace(int size, int64_t M, int64_t N) {
  const NormPlan p = norm_plan(size, true, M, N);
  const int64_t most = p.shape == 0   ? kColumnSlabs
                       : p.shape <= 2 ? kSms * Back1::kBlocks
                                      : kSms * Back3::kBlocks;
  static_assert(Back1::kBlocks == Back2::kBlocks && Back3::kBlocks == Back4::kBlocks, "");
  return ((size_t)(M < most ? M : most) * 2 * (size_t)N * 4 + 255) / 256 * 256;
}

template <typename T, int kVec, typename S, int kGroup>
hcmix_status launch_norm_backward_ring(const NormArgs& A, const RingPlan& p, cudaStream_t stream) {
  using R = Ring<T, kVec, S::kUnits * 16 / (kVec * (int)sizeof(T)), 2 * kGroup,
                 kStagesOf<S, 2 * kGroup>, 0>;
  return launch(hcmix_norm_backward_kernel<T, kVec, S, kGroup>, dim3(p.blocks),
                dim3(p.threads, p.teams), R::bytes(p.threads, p.teams), ring_most<R, S>, stream, A);
}

template <typename T, int kVec>
hcmix_status launch_norm_backward(NormArgs A, cudaStream_t stream) {
  constexpr bool kOwn = kVec * sizeof(T) == 16;
  constexpr int kGroup = kOwn ? 2 : 1;
  const NormPlan p = norm_plan(sizeof(T), kOwn, A.M, A.N);
  A.blocks = p.ring.blocks;
  hcmix_status st = HCMIX_OK;
  if (A.dweight == nullptr || p.shape == 0) {
    const int64_t vecs = (A.N + kVec - 1) / kVec;
    const unsigned threads = vecs >= 256 ? 256 : (unsigned)(vecs + 31) / 32 * 32;
    if (A.M > 0)
      st = launch(hcmix_norm_dx_kernel<T, kVec>, dim3((unsigned)A.M), dim3(threads), 0, 0, stream, A);
    if (st != HCMIX_OK || A.dweight == nullptr) return st;
    const int64_t per = (int64_t)kColumnThreads * kVec;
    if (A.blocks > 0)
      st = launch(hcmix_norm_columns_kernel<T, kVec>,
                  dim3((unsigned)((A.N + per - 1) / per), A.blocks), dim3(kColumnThreads), 0, 0,
                  stream, A);
  } else {
    switch (p.shape) {
      case 1: st = launch_norm_backward_ring<T, kVec, Back1, kGroup>(A, p.ring, stream); break;
      case 2: st = launch_norm_backward_ring<T, kVec, Back2, kGroup>(A, p.ring, stream); break;
      case 3: st = launch_norm_backward_ring<T, kVec, Back3, 1>(A, p.ring, stream); break;
      default: st = launch_norm_backward_ring<T, kVec, Back4, 1>(A, p.ring, stream);
    }
  }
  if (st != HCMIX_OK) return st;
  return launch(hcmix_norm_join_kernel, dim3((unsigned)((2 * A.N + 31) / 32)),
                dim3(32 * kJoinGroups), 0, 0, stream, A);
}

inline hcmix_status run_norm_backward(const NormArgs& A, hcmix_type type, cudaStream_t stream) {
  const int bytes =
      vector_bytes(size_of(type), {{A.x, A.x_stride}, {A.dy, A.dy_stride}, {A.dx, A.N}});
  return with_vector(type, bytes, [&](auto t, auto vec, auto) {
    return launch_norm_backward<decltype(t), decltype(vec)::value>(A, stream);
  });
}

}  // namespace sublayer
}  // namespace hcmix
