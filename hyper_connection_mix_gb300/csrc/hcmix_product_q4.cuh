// Products of few rows with experts' weights of 4 bits: w = (code - 8) scale, a scale for
// each group of 32 to 256 along k.  Bound by reading the codes of the experts that have rows.
//
// A warp takes 16 features of W (16 of g and of u where the product is gated) and 8 rows
// as mma.m16n8k16 tiles, features as M.  The order of k within a tile is free as long as
// both operands have it: a thread's word of 8 codes of one feature, k = 8 t .. 8 t + 7 of a
// block of 32, gives its registers of two tiles, and one 16-byte load of a row the same k.
// A code becomes 1 + code / 16 by two bit operations; 1.5 taken off (exact), it is
// (code - 8) / 16.  Sums of a group are fp32, and are scaled and added in fp32.
#pragma once

#include "hcmix_vec.cuh"

namespace hcmix {
namespace sublayer {

struct Q4Args {
  const void* xs;
  int64_t xs_stride, R;
  const uint8_t* codes;  // [E, N, K / 2], the lower half of a byte is the even k
  const void* scales;    // [E, N, K / group]
  const int32_t* offsets;
  int E, K, N, group;
  int gated;  // features N / 2 .. N - 1 are u's
  void* out;  // [R, N], or [R, N / 2]
  int vec;    // rows of xs start on 16 bytes
};

template <typename T>
struct Codes;
template <>
struct Codes<__nv_bfloat16> {
  // codes i and i + 4 of a word, as bits 3..6 of 1.0's fraction
  static __device__ __forceinline__ uint32_t pair(uint32_t w, int i) {
    const uint32_t s = i == 0 ? w << 3 : w >> (4 * i - 3);
    uint32_t v = (s & 0x00780078u) | 0x3F803F80u;
    __nv_bfloat162 h = *reinterpret_cast<__nv_bfloat162*>(&v);
    h = __hsub2(h, __nv_bfloat162(__ushort_as_bfloat16(0x3FC0), __ushort_as_bfloat16(0x3FC0)));
    return *reinterpret_cast<uint32_t*>(&h);
  }
  static __device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                             uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
        "{%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  }
};
template <>
struct Codes<__half> {
  static __device__ __forceinline__ uint32_t pair(uint32_t w, int i) {
    const uint32_t s = i < 2 ? w << (6 - 4 * i) : w >> (4 * i - 6);
    uint32_t v = (s & 0x03C003C0u) | 0x3C003C00u;
    __half2 h = *reinterpret_cast<__half2*>(&v);
    h = __hsub2(h, __half2(__ushort_as_half(0x3E00), __ushort_as_half(0x3E00)));
    return *reinterpret_cast<uint32_t*>(&h);
  }
  static __device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                             uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
        "{%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  }
};

constexpr int kQ4Warps = 4;  // they share out k

__device__ __forceinline__ int q4_offset(int v, int64_t R) {
  return v < 0 ? 0 : v > R ? (int)R : v;
}

template <typename T, bool kGated>
__global__ void __launch_bounds__(kQ4Warps * 32) hcmix_product_q4_kernel(const Q4Args A) {
  begin_kernel();
  constexpr int kHalves = kGated ? 2 : 1;
  __shared__ float part[kQ4Warps][kHalves][4][32];
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, g = lane / 4, t = lane % 4;
  const int F = kGated ? A.N / 2 : A.N;
  const int64_t ft = (F + 15) / 16, tiles = ft * A.E;
  for (int64_t tile = blockIdx.x; tile < tiles; tile += gridDim.x) {
    const int e = (int)(tile / ft), f0 = (int)(tile - e * ft) * 16;
    const int first = q4_offset(A.offsets[e], A.R), last = q4_offset(A.offsets[e + 1], A.R);
    for (int r0 = first; r0 < last; r0 += 8) {
      const T* x = static_cast<const T*>(A.xs) + (int64_t)(r0 + g) * A.xs_stride;
      const bool has = r0 + g < last;
      float total[kHalves][4] = {};
      const int groups = A.K / A.group;
      for (int q = warp; q < groups; q += kQ4Warps) {
        float acc[kHalves][4] = {};
        for (int k = q * A.group; k < (q + 1) * A.group; k += 32) {
          uint32_t xw[4] = {};
          const T* xk = x + k + 8 * t;
          if (has) {
            if (A.vec) {
              const uint4 v = *reinterpret_cast<const uint4*>(xk);
              xw[0] = v.x, xw[1] = v.y, xw[2] = v.z, xw[3] = v.w;
            } else {
              const uint16_t* p = reinterpret_cast<const uint16_t*>(xk);
#pragma unroll
              for (int i = 0; i < 4; ++i) xw[i] = p[2 * i] | (uint32_t)p[2 * i + 1] << 16;
            }
          }
#pragma unroll
          for (int h = 0; h < kHalves; ++h) {
            uint32_t w[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              int f = f0 + g + 8 * i;
              f = (f < F ? f : F - 1) + h * F;
              w[i] = *reinterpret_cast<const uint32_t*>(
                  A.codes + ((int64_t)e * A.N + f) * (A.K / 2) + k / 2 + 4 * t);
            }
#pragma unroll
            for (int s = 0; s < 2; ++s) {
              const uint32_t a[4] = {Codes<T>::pair(w[0], 2 * s), Codes<T>::pair(w[1], 2 * s),
                                     Codes<T>::pair(w[0], 2 * s + 1),
                                     Codes<T>::pair(w[1], 2 * s + 1)};
              Codes<T>::mma(acc[h], a, __byte_perm(xw[s], xw[s + 2], 0x5410),
                            __byte_perm(xw[s], xw[s + 2], 0x7632));
            }
          }
        }
#pragma unroll
        for (int h = 0; h < kHalves; ++h)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            int f = f0 + g + 8 * i;
            f = (f < F ? f : F - 1) + h * F;
            const float s = 16.0f * to_f32(static_cast<const T*>(
                                        A.scales)[((int64_t)e * A.N + f) * groups + q]);
            total[h][2 * i] = fmaf(s, acc[h][2 * i], total[h][2 * i]);
            total[h][2 * i + 1] = fmaf(s, acc[h][2 * i + 1], total[h][2 * i + 1]);
          }
      }
      __syncthreads();
#pragma unroll
      for (int h = 0; h < kHalves; ++h)
#pragma unroll
        for (int i = 0; i < 4; ++i) part[warp][h][i][lane] = total[h][i];
      __syncthreads();
      // value i of a lane: feature g + 8 (i / 2), row 2 t + i % 2
      const int i = warp;
      static_assert(kQ4Warps == 4, "a warp for each value");
      float v[kHalves];
#pragma unroll
      for (int h = 0; h < kHalves; ++h)
        v[h] = (part[0][h][i][lane] + part[1][h][i][lane]) +
               (part[2][h][i][lane] + part[3][h][i][lane]);
      const int f = f0 + g + 8 * (i / 2), r = r0 + 2 * t + i % 2;
      if (f < F && r < last) {
        float o = v[0];
        if (kGated) o = __fdividef(v[0], 1.0f + __expf(-v[0])) * v[kHalves - 1];
        static_cast<T*>(A.out)[(int64_t)r * F + f] = from_f32<T>(o);
      }
    }
  }
  const int64_t end = q4_offset(A.offsets[A.E], A.R), step = (int64_t)gridDim.x * blockDim.x;
  for (int64_t i = end * F + (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < A.R * F; i += step)
    static_cast<T*>(A.out)[i] = from_f32<T>(0.0f);
}

inline hcmix_status run_product_q4(const Q4Args& A, hcmix_type type, cudaStream_t stream) {
  const int64_t F = A.gated ? A.N / 2 : A.N;
  const int64_t tiles = (F + 15) / 16 * A.E;
  const dim3 grid((unsigned)(tiles < (1 << 30) ? tiles : (1 << 30)));
  const auto go = [&](auto z) {
    using T = decltype(z);
    return A.gated ? launch(hcmix_product_q4_kernel<T, true>, grid, dim3(kQ4Warps * 32), 0, 0,
                            stream, A)
                   : launch(hcmix_product_q4_kernel<T, false>, grid, dim3(kQ4Warps * 32), 0, 0,
                            stream, A);
  };
  return type == HCMIX_BF16 ? go(__nv_bfloat16{}) : go(__half{});
}

}  // namespace sublayer
}  // namespace hcmix
