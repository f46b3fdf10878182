// Loads, stores, conversions and reductions shared by the sublayer kernels.
//
// A kernel handles a row in vectors of kVec consecutive elements per thread:
// 16 bytes where every row of every operand starts on 16 bytes, else one
// element.  Values are unpacked to fp32, and a result is rounded once, here,
// when it is packed for its store.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>

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

// kVec elements as they lie in memory, and their values.
template <typename T, int kVec>
struct alignas(kVec * sizeof(T)) Packed {
  T e[kVec];
  __device__ __forceinline__ void unpack(float (&v)[kVec]) const {
#pragma unroll
    for (int i = 0; i < kVec; ++i) v[i] = to_f32(e[i]);
  }
  __device__ __forceinline__ void pack(const float (&v)[kVec]) {
#pragma unroll
    for (int i = 0; i < kVec; ++i) e[i] = from_f32<T>(v[i]);
  }
};

template <typename T, int kVec>
__device__ __forceinline__ Packed<T, kVec> load_vec(const T* p) {
  Packed<T, kVec> r;
  if constexpr (sizeof(T) * kVec == 16) {
    *reinterpret_cast<uint4*>(&r) = *reinterpret_cast<const uint4*>(p);
  } else {
    r = *reinterpret_cast<const Packed<T, kVec>*>(p);
  }
  return r;
}

template <typename T, int kVec>
__device__ __forceinline__ void store_vec(T* p, const Packed<T, kVec>& v) {
  if constexpr (sizeof(T) * kVec == 16) {
    *reinterpret_cast<uint4*>(p) = *reinterpret_cast<const uint4*>(&v);
  } else {
    *reinterpret_cast<Packed<T, kVec>*>(p) = v;
  }
}

template <typename T, int kVec>
__device__ __forceinline__ void load_f32(const T* p, float (&v)[kVec]) {
  load_vec<T, kVec>(p).unpack(v);
}

template <typename T, int kVec>
__device__ __forceinline__ void store_f32(T* p, const float (&v)[kVec]) {
  Packed<T, kVec> r;
  r.pack(v);
  store_vec<T, kVec>(p, r);
}

// kVec values of a norm's weight or bias, fp32 (p32) or of type T.
template <typename T, int kVec>
__device__ __forceinline__ void load_param(const void* p, bool p32, int64_t at, float (&v)[kVec]) {
  if (p32) {
#pragma unroll
    for (int i = 0; i < kVec; ++i) v[i] = static_cast<const float*>(p)[at + i];
  } else {
#pragma unroll
    for (int i = 0; i < kVec; ++i) v[i] = to_f32(static_cast<const T*>(p)[at + i]);
  }
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// Sums of kN values over the block, in every thread.  The block is whole
// warps; `part` holds kN * 32 floats and is free again at the next barrier.
template <int kN>
__device__ __forceinline__ void block_sum(float (&v)[kN], float* part) {
#pragma unroll
  for (int i = 0; i < kN; ++i) v[i] = warp_sum(v[i]);
  const int warps = blockDim.x / 32, warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  if (warps == 1) return;
  if (lane == 0) {
#pragma unroll
    for (int i = 0; i < kN; ++i) part[i * 32 + warp] = v[i];
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kN; ++i) v[i] = warp_sum(lane < warps ? part[i * 32 + lane] : 0.f);
}

// ---- host side

inline bool aligned_rows(const void* p, int64_t stride, int size) {
  return p == nullptr || (reinterpret_cast<uintptr_t>(p) % 16 == 0 && stride * size % 16 == 0);
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

inline hcmix_status launched() {
  return cudaGetLastError() == cudaSuccess ? HCMIX_OK : HCMIX_ERR_CUDA;
}

}  // namespace sublayer
}  // namespace hcmix
