// Loads, stores, conversions and reductions shared by the sublayer kernels.
//
// A kernel handles a row in vectors of kVec consecutive elements per thread: 16
// bytes where every row of every operand starts on 16 bytes, else 4 bytes where all
// start on 4, else one element.  Values are unpacked to fp32, and a result is rounded
// once, here, when it is packed for its store.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>
#include <initializer_list>

#include "hcmix_sublayer.h"

namespace hcmix {
namespace sublayer {

constexpr int kStreams = 4;

__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float to_f32(__half v) { return __half2float(v); }

template <typename T>
__device__ __forceinline__ T from_f32(float v);
template <>
__device__ __forceinline__ float from_f32<float>(float v) {
  return v;
}
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v) {
  return __float2bfloat16_rn(v);
}
template <>
__device__ __forceinline__ __half from_f32<__half>(float v) {
  return __float2half_rn(v);
}

// Elements of a 16-byte vector.
template <typename T>
constexpr int kWide = 16 / (int)sizeof(T);

// Two elements of a 16-bit type and their values.
__device__ __forceinline__ float2 pair_to_f32(__nv_bfloat162 v) {
  // a bf16's bits are the upper half of its fp32's
  const uint32_t w = *reinterpret_cast<const uint32_t*>(&v);
  return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}
__device__ __forceinline__ float2 pair_to_f32(__half2 v) { return __half22float2(v); }
__device__ __forceinline__ void pair_from_f32(__nv_bfloat162& p, float a, float b) {
  p = __floats2bfloat162_rn(a, b);
}
__device__ __forceinline__ void pair_from_f32(__half2& p, float a, float b) {
  p = __floats2half2_rn(a, b);
}
template <typename T>
struct PairOf;
template <>
struct PairOf<__nv_bfloat16> {
  using type = __nv_bfloat162;
};
template <>
struct PairOf<__half> {
  using type = __half2;
};

// kVec elements as they lie in memory, and their values.
template <typename T, int kVec>
struct alignas(kVec * sizeof(T)) Packed {
  T e[kVec];
  __device__ __forceinline__ void unpack(float (&v)[kVec]) const {
    if constexpr (sizeof(T) == 2 && kVec % 2 == 0) {
      using P = typename PairOf<T>::type;
#pragma unroll
      for (int i = 0; i < kVec; i += 2) {
        const float2 f = pair_to_f32(reinterpret_cast<const P*>(e)[i / 2]);
        v[i] = f.x;
        v[i + 1] = f.y;
      }
    } else {
#pragma unroll
      for (int i = 0; i < kVec; ++i) v[i] = to_f32(e[i]);
    }
  }
  __device__ __forceinline__ void pack(const float (&v)[kVec]) {
    if constexpr (sizeof(T) == 2 && kVec % 2 == 0) {
      using P = typename PairOf<T>::type;
#pragma unroll
      for (int i = 0; i < kVec; i += 2)
        pair_from_f32(reinterpret_cast<P*>(e)[i / 2], v[i], v[i + 1]);
    } else {
#pragma unroll
      for (int i = 0; i < kVec; ++i) e[i] = from_f32<T>(v[i]);
    }
  }
};

// Elementwise arithmetic on vectors, two fp32 at a time where there are two.
template <int N>
__device__ __forceinline__ void vfma(float (&d)[N], const float (&a)[N], const float (&b)[N],
                                     const float (&c)[N]) {
  if constexpr (N % 2 == 0) {
#pragma unroll
    for (int i = 0; i < N; i += 2) {
      const float2 r = __ffma2_rn(make_float2(a[i], a[i + 1]), make_float2(b[i], b[i + 1]),
                                  make_float2(c[i], c[i + 1]));
      d[i] = r.x;
      d[i + 1] = r.y;
    }
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) d[i] = fmaf(a[i], b[i], c[i]);
  }
}

template <int N>
__device__ __forceinline__ void vfma(float (&d)[N], float a, const float (&b)[N],
                                     const float (&c)[N]) {
  if constexpr (N % 2 == 0) {
#pragma unroll
    for (int i = 0; i < N; i += 2) {
      const float2 r = __ffma2_rn(make_float2(a, a), make_float2(b[i], b[i + 1]),
                                  make_float2(c[i], c[i + 1]));
      d[i] = r.x;
      d[i + 1] = r.y;
    }
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) d[i] = fmaf(a, b[i], c[i]);
  }
}

template <int N>
__device__ __forceinline__ void vfma(float (&d)[N], float a, const float (&b)[N], float c) {
  if constexpr (N % 2 == 0) {
#pragma unroll
    for (int i = 0; i < N; i += 2) {
      const float2 r =
          __ffma2_rn(make_float2(a, a), make_float2(b[i], b[i + 1]), make_float2(c, c));
      d[i] = r.x;
      d[i + 1] = r.y;
    }
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) d[i] = fmaf(a, b[i], c);
  }
}

template <int N>
__device__ __forceinline__ void vmul(float (&d)[N], const float (&a)[N], const float (&b)[N]) {
  if constexpr (N % 2 == 0) {
#pragma unroll
    for (int i = 0; i < N; i += 2) {
      const float2 r = __fmul2_rn(make_float2(a[i], a[i + 1]), make_float2(b[i], b[i + 1]));
      d[i] = r.x;
      d[i + 1] = r.y;
    }
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) d[i] = a[i] * b[i];
  }
}

template <int N>
__device__ __forceinline__ void vmul(float (&d)[N], float a, const float (&b)[N]) {
  if constexpr (N % 2 == 0) {
#pragma unroll
    for (int i = 0; i < N; i += 2) {
      const float2 r = __fmul2_rn(make_float2(a, a), make_float2(b[i], b[i + 1]));
      d[i] = r.x;
      d[i + 1] = r.y;
    }
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) d[i] = a * b[i];
  }
}

template <int N>
__device__ __forceinline__ void vadd(float (&d)[N], const float (&a)[N], const float (&b)[N]) {
  if constexpr (N % 2 == 0) {
#pragma unroll
    for (int i = 0; i < N; i += 2) {
      const float2 r = __fadd2_rn(make_float2(a[i], a[i + 1]), make_float2(b[i], b[i + 1]));
      d[i] = r.x;
      d[i + 1] = r.y;
    }
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) d[i] = a[i] + b[i];
  }
}

template <int N>
__device__ __forceinline__ void vadd(float (&d)[N], float a, const float (&b)[N]) {
  if constexpr (N % 2 == 0) {
#pragma unroll
    for (int i = 0; i < N; i += 2) {
      const float2 r = __fadd2_rn(make_float2(a, a), make_float2(b[i], b[i + 1]));
      d[i] = r.x;
      d[i + 1] = r.y;
    }
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) d[i] = a + b[i];
  }
}

// Sums over vectors run in two chains, the elements' parities.
struct Acc {
  float v[2] = {0.f, 0.f};
  template <int N>
  __device__ __forceinline__ void add(const float (&a)[N]) {
    if constexpr (N % 2 == 0) {
#pragma unroll
      for (int i = 0; i < N; i += 2) {
        const float2 r = __fadd2_rn(make_float2(v[0], v[1]), make_float2(a[i], a[i + 1]));
        v[0] = r.x;
        v[1] = r.y;
      }
    } else {
#pragma unroll
      for (int i = 0; i < N; ++i) v[0] += a[i];
    }
  }
  template <int N>
  __device__ __forceinline__ void add(const float (&a)[N], const float (&b)[N]) {
    if constexpr (N % 2 == 0) {
#pragma unroll
      for (int i = 0; i < N; i += 2) {
        const float2 r = __ffma2_rn(make_float2(a[i], a[i + 1]), make_float2(b[i], b[i + 1]),
                                    make_float2(v[0], v[1]));
        v[0] = r.x;
        v[1] = r.y;
      }
    } else {
#pragma unroll
      for (int i = 0; i < N; ++i) v[0] = fmaf(a[i], b[i], v[0]);
    }
  }
  __device__ __forceinline__ float sum() const { return v[0] + v[1]; }
};

// ---- rows in global memory, in vectors of 16 bytes where every row of every operand
// starts on 16 bytes, else of 4 bytes or of one element.
//
// Streamed operands are read once and not kept in L1, which is left to what every
// row uses (weights, coefficients).
template <typename T, int kVec>
__device__ __forceinline__ Packed<T, kVec> load_vec(const T* p) {
  Packed<T, kVec> r;
  if constexpr (sizeof(r) == 16) {
    uint4 v;
    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p));
    *reinterpret_cast<uint4*>(&r) = v;
  } else if constexpr (sizeof(r) == 4) {
    uint32_t v;
    asm volatile("ld.global.L1::no_allocate.u32 %0, [%1];" : "=r"(v) : "l"(p));
    *reinterpret_cast<uint32_t*>(&r) = v;
  } else {
    r = *reinterpret_cast<const Packed<T, kVec>*>(p);
  }
  return r;
}

// The same for what other warps of the block read too: kept in L1.
template <typename T, int kVec>
__device__ __forceinline__ Packed<T, kVec> load_cached_vec(const T* p) {
  Packed<T, kVec> r;
  if constexpr (sizeof(r) == 16)
    *reinterpret_cast<uint4*>(&r) = *reinterpret_cast<const uint4*>(p);
  else
    r = *reinterpret_cast<const Packed<T, kVec>*>(p);
  return r;
}

template <typename T, int kVec>
__device__ __forceinline__ void store_vec(T* p, const Packed<T, kVec>& v) {
  if constexpr (sizeof(v) == 16)
    *reinterpret_cast<uint4*>(p) = *reinterpret_cast<const uint4*>(&v);
  else
    *reinterpret_cast<Packed<T, kVec>*>(p) = v;
}

template <typename T, int kVec>
__device__ __forceinline__ void store_f32(T* p, const float (&v)[kVec]) {
  Packed<T, kVec> r;
  r.pack(v);
  store_vec<T, kVec>(p, r);
}

// A thread's share of a row: kU vectors of kVec elements, `step` apart, from column
// c on.  Rows of 16-byte vectors take one each; narrower vectors take several, so
// that as many bytes are under way.  Past the row's end the first vector is loaded
// again (column c is in the row) and zeros take its place: no branch parts the loads.
template <typename T, int kVec, int kU>
struct Cols {
  Packed<T, kVec> q[kU];
  __device__ __forceinline__ void load(const T* row, int64_t c, int step, int64_t width) {
#pragma unroll
    for (int u = 0; u < kU; ++u) q[u] = load_vec<T, kVec>(row + place(c, u, step, width));
    zero_past(c, step, width);
  }
  __device__ __forceinline__ void load_cached(const T* row, int64_t c, int step, int64_t width) {
#pragma unroll
    for (int u = 0; u < kU; ++u) q[u] = load_cached_vec<T, kVec>(row + place(c, u, step, width));
    zero_past(c, step, width);
  }
  __device__ __forceinline__ void store(T* row, int64_t c, int step, int64_t width) const {
#pragma unroll
    for (int u = 0; u < kU; ++u)
      if (u == 0 || c + u * step < width) store_vec<T, kVec>(row + c + u * step, q[u]);
  }
  __device__ __forceinline__ void unpack(float (&v)[kU * kVec]) const {
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      float t[kVec];
      q[u].unpack(t);
#pragma unroll
      for (int e = 0; e < kVec; ++e) v[u * kVec + e] = t[e];
    }
  }
  __device__ __forceinline__ void pack(const float (&v)[kU * kVec]) {
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      float t[kVec];
#pragma unroll
      for (int e = 0; e < kVec; ++e) t[e] = v[u * kVec + e];
      q[u].pack(t);
    }
  }

 private:
  static __device__ __forceinline__ int64_t place(int64_t c, int u, int step, int64_t width) {
    return u == 0 || c + u * step >= width ? c : c + u * step;
  }
  __device__ __forceinline__ void zero_past(int64_t c, int step, int64_t width) {
#pragma unroll
    for (int u = 1; u < kU; ++u) {
#pragma unroll
      for (int e = 0; e < kVec; ++e)
        if (c + u * step >= width) q[u].e[e] = from_f32<T>(0.f);
    }
  }
};

template <typename T, int kVec, int kU>
__device__ __forceinline__ void store_cols(T* row, int64_t c, int step, int64_t width,
                                           const float (&v)[kU * kVec]) {
  Cols<T, kVec, kU> q;
  q.pack(v);
  q.store(row, c, step, width);
}

// kVec values from column c on of a norm's weight or bias, fp32 (p32) or of type T;
// `other` where there is none.
template <typename T, int kVec>
__device__ __forceinline__ void load_param(const void* p, bool p32, int64_t c, float other,
                                           float (&v)[kVec]) {
  if (p == nullptr) {
#pragma unroll
    for (int e = 0; e < kVec; ++e) v[e] = other;
  } else if (p32) {
    const float* f = static_cast<const float*>(p) + c;
    if (kVec % 4 == 0 && reinterpret_cast<uintptr_t>(f) % 16 == 0) {
      if constexpr (kVec % 4 == 0) {
#pragma unroll
        for (int i = 0; i < kVec; i += 4) {
          const float4 q = *reinterpret_cast<const float4*>(f + i);
          v[i] = q.x, v[i + 1] = q.y, v[i + 2] = q.z, v[i + 3] = q.w;
        }
      }
    } else {
#pragma unroll
      for (int e = 0; e < kVec; ++e) v[e] = f[e];
    }
  } else {
    const T* t = static_cast<const T*>(p) + c;
    if (reinterpret_cast<uintptr_t>(t) % sizeof(Packed<T, kVec>) == 0) {
      load_cached_vec<T, kVec>(t).unpack(v);
    } else {
#pragma unroll
      for (int e = 0; e < kVec; ++e) v[e] = to_f32(t[e]);
    }
  }
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// Warp sums of kN <= 32 values at once.  At each step a lane keeps one half of
// the values, adding the other lane's, and gives the other half away, so kN values
// take about kN shuffles instead of 5 kN.  Lane l ends with the sum of value
// warp_sums_index(l); kN is padded to the next power of two.
template <int kN>
constexpr int kPadded = kN <= 1 ? 1 : 2 * kPadded<(kN + 1) / 2>;
template <>
constexpr int kPadded<1> = 1;

template <int kN>
__device__ __forceinline__ float warp_sums(const float (&in)[kN]) {
  constexpr int kP = kPadded<kN>;
  float v[kP];
#pragma unroll
  for (int i = 0; i < kP; ++i) v[i] = i < kN ? in[i] : 0.f;
  const int lane = threadIdx.x % 32;
  int o = 16;
#pragma unroll
  for (int n = kP / 2; n > 0; n /= 2, o /= 2) {
#pragma unroll
    for (int i = 0; i < n; ++i) {
      const bool upper = lane & o;
      const float keep = upper ? v[i + n] : v[i], give = upper ? v[i] : v[i + n];
      v[i] = keep + __shfl_xor_sync(0xffffffffu, give, o);
    }
  }
#pragma unroll
  for (; o > 0; o /= 2) v[0] += __shfl_xor_sync(0xffffffffu, v[0], o);
  return v[0];
}

// The value whose sum lane l holds: its top log2(kP) bits, the first step's bit
// the value's highest.
template <int kN>
__device__ __forceinline__ int warp_sums_index(int lane) {
  constexpr int kP = kPadded<kN>;
  return lane / (32 / kP);
}

// Sums of kN values over the block: thread i < kN returns value i's (the others
// nothing of use).  The block is whole warps; `part` holds 32 * kN floats.
template <int kN>
__device__ __forceinline__ float block_sums(const float (&v)[kN], float* part) {
  const int warps = blockDim.x / 32, warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  constexpr int kEach = 32 / kPadded<kN>;  // lanes that hold the same sum
  const float s = warp_sums<kN>(v);
  const int i = warp_sums_index<kN>(lane);
  if (lane % kEach == 0 && i < kN) part[warp * kN + i] = s;
  __syncthreads();
  float t = 0.f;
  if (threadIdx.x < kN)
    for (int w = 0; w < warps; ++w) t += part[w * kN + threadIdx.x];
  return t;
}

// Barrier of the `warps` warps of one of a block's teams (threads of one
// threadIdx.y); a block of one team is a team of its own.
__device__ __forceinline__ void team_sync(int warps) {
  if (blockDim.y == 1)
    __syncthreads();
  else if (warps > 1)
    asm volatile("bar.sync %0, %1;" ::"r"(threadIdx.y + 1), "r"(warps * 32) : "memory");
  else
    __syncwarp();
}

// Sums of kN values over a team (blockDim.x threads), in every thread, by
// warp_sums twice: `part`, the team's own, holds 32 * kN floats and is free again at
// the next barrier.
template <int kN>
__device__ __forceinline__ void team_sums(float (&v)[kN], float* part) {
  static_assert(kPadded<kN> == kN && kN <= 32, "");
  const int warps = blockDim.x / 32, warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  constexpr int kEach = 32 / kN;  // lanes that hold the same sum
  float s = warp_sums<kN>(v);
  if (warps > 1) {
    if (lane % kEach == 0) part[warp * kN + lane / kEach] = s;
    team_sync(warps);
    // kEach lanes share a value's partials, value i's lanes from i * kEach on
    const int i = lane / kEach;
    s = 0.f;
    for (int w = lane % kEach; w < warps; w += kEach) s += part[w * kN + i];
#pragma unroll
    for (int o = kEach / 2; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  }
#pragma unroll
  for (int i = 0; i < kN; ++i) v[i] = __shfl_sync(0xffffffffu, s, i * kEach);
}

// ---- asynchronous copies into shared memory, completed for the copying thread
// by async_wait; 16 bytes each

__device__ __forceinline__ void async_copy16(void* dst, const void* src) {
  const uint32_t to = static_cast<uint32_t>(__cvta_generic_to_shared(dst));
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to), "l"(src) : "memory");
}

__device__ __forceinline__ void async_commit() {
  asm volatile("cp.async.commit_group;" ::: "memory");
}

// Waits until at most kLeft of the thread's newest groups are in flight.
template <int kLeft>
__device__ __forceinline__ void async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(kLeft) : "memory");
}

// ---- programmatic dependent launch.  Every sublayer kernel is launched so that
// its blocks may be set up while the grid before it in the stream still runs, and
// begins with this: the next grid may be set up, and nothing is read or written
// before the grid before this one has ended and its memory can be seen.
__device__ __forceinline__ void begin_kernel() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
}

// ---- host side

// The widest vector that every row of the operands allows: 16 bytes, 4 or one
// element of `size` bytes.  A null operand allows all.
struct Operand {
  const void* p;
  int64_t stride;  // elements
};
inline int vector_bytes(int size, std::initializer_list<Operand> operands) {
  for (int to : {16, 4}) {
    bool all = to >= size;
    for (const Operand& o : operands)
      all = all && (o.p == nullptr || (reinterpret_cast<uintptr_t>(o.p) % to == 0 &&
                                       o.stride * size % to == 0));
    if (all) return to;
  }
  return size;
}

inline int size_of(hcmix_type t) { return t == HCMIX_F32 ? 4 : 2; }

// Calls f(T{}) for the element type of `t`.
template <typename F>
inline hcmix_status with_type(hcmix_type t, F&& f) {
  switch (t) {
    case HCMIX_BF16: return f(__nv_bfloat16{});
    case HCMIX_F16: return f(__half{});
    case HCMIX_F32: return f(float{});
  }
  return HCMIX_ERR_INVALID_ARG;
}

// Calls f(T{}, vec, u) with the type, the elements of a vector and the vectors of a
// thread's share of a row, as constants.
template <int kN>
struct Int {
  static constexpr int value = kN;
};
template <typename F>
inline hcmix_status with_vector(hcmix_type t, int bytes, F&& f) {
  return with_type(t, [&](auto z) {
    using T = decltype(z);
    if (bytes == 16) return f(z, Int<kWide<T>>{}, Int<1>{});
    if (bytes == (int)sizeof(T)) return f(z, Int<1>{}, Int<4>{});
    return f(z, Int<4 / (int)sizeof(T)>{}, Int<4>{});
  });
}

// HCMIX_OK, or HCMIX_ERR_CUDA with the error taken from the runtime, where a later call of
// the process that asks for the last error would take it for its own.
inline hcmix_status checked(cudaError_t e) {
  if (e == cudaSuccess) return HCMIX_OK;
  cudaGetLastError();
  return HCMIX_ERR_CUDA;
}

// Launches a kernel that starts with begin_kernel(); `cluster` blocks a cluster.  The kernel's
// limit of dynamic shared memory is one for all threads of the process: it is set to `most`, the
// most that any call of the kernel takes, so that no call lowers it under another's launch.
template <typename Args>
inline hcmix_status launch(void (*kernel)(const Args), dim3 grid, dim3 threads, size_t smem,
                           size_t most, cudaStream_t stream, const Args& args,
                           unsigned cluster = 1) {
  if (smem > most) return HCMIX_ERR_UNSUPPORTED;
  // with its static shared memory a kernel may pass the default 48 KB sooner
  if (smem > 32 * 1024) {
    const hcmix_status st = checked(
        cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)most));
    if (st != HCMIX_OK) return st;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = threads;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = cluster;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  return checked(cudaLaunchKernelEx(&cfg, kernel, args));
}

}  // namespace sublayer
}  // namespace hcmix
