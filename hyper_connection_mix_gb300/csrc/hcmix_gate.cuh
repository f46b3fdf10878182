// The gate of an expert's feed-forward network: h = g q u with q = 1 / (1 + exp(-g)), for the
// products' epilogues, and its gradient: with (g, u) the halves of a row of gu,
//   dg = dh u q (1 + g (1 - q)),  du = dh g q.
// Elementwise, bound by HBM: dh, g and u are read once, dg and du written once (32768 x 2048 bf16
// 99 us, 6.7 TB/s; 3001 x 1001 fp32, whose rows are read element by element, 14.1 us).
#pragma once

#include "hcmix_vec.cuh"

namespace hcmix {
namespace sublayer {

// g q u.  With e = exp(-|g|), q is 1 / (1 + e), or e / (1 + e) for a negative g: 1 + e, from 1 to
// 2, is a divisor that the fast division takes (from 2^126 up, g below -87.3, it gives 0 or NaN).
// For a negative g both factors take half of e: what is small by g and large by u stays in range.
__device__ __forceinline__ float gate(float g, float u) {
  const float half = __expf(-0.5f * fabsf(g));
  const float w = g < 0.0f ? half : 1.0f;
  return __fdividef(g * w, fmaf(half, half, 1.0f)) * (u * w);
}

struct GateArgs {
  const void *dh, *gu;
  int64_t dh_stride, gu_stride;
  void* dgu;
  int64_t R, F;
  int across;  // log2 of a block's threads along a row
};

// A block is across x down threads, so that none divides by the width: `across` a power of two
// as large as a row's vectors, at most the block's threads.  A thread takes kRows rows' vectors at
// a time, one of 16 bytes or four smaller ones, and loads all of them first.
constexpr int kGateThreads = 256;
template <typename T, int kVec>
constexpr int kGateRows = kVec * sizeof(T) == 16 ? 1 : 4;

template <typename T, int kVec>
__global__ void __launch_bounds__(kGateThreads) hcmix_gate_backward_kernel(const GateArgs A) {
  begin_kernel();
  using V = Packed<T, kVec>;
  constexpr int kRows = kGateRows<T, kVec>;
  const int down = kGateThreads >> A.across;
  const int64_t column = ((int64_t)blockIdx.x << A.across) + (threadIdx.x & ((1 << A.across) - 1));
  const int64_t f = column * kVec;
  if (f >= A.F) return;
  for (int64_t r0 = (int64_t)blockIdx.y * kRows * down + (threadIdx.x >> A.across); r0 < A.R;
       r0 += (int64_t)gridDim.y * kRows * down) {
    V in[kRows][3];
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      const int64_t r = r0 + i * down;
      if (r >= A.R) continue;
      const T* gu = static_cast<const T*>(A.gu) + r * A.gu_stride + f;
      in[i][0] = *reinterpret_cast<const V*>(static_cast<const T*>(A.dh) + r * A.dh_stride + f);
      in[i][1] = *reinterpret_cast<const V*>(gu);
      in[i][2] = *reinterpret_cast<const V*>(gu + A.F);
    }
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      const int64_t r = r0 + i * down;
      if (r >= A.R) continue;
      float dh[kVec], g[kVec], u[kVec];
      in[i][0].unpack(dh);
      in[i][1].unpack(g);
      in[i][2].unpack(u);
#pragma unroll
      for (int k = 0; k < kVec; ++k) {
        // e by halves, as in gate(): exp(-g) is past the largest fp32 from g = -88.7 down, where q
        // times a large dh or u is not
        const float half = expf(-0.5f * fabsf(g[k])), e = half * half;
        const float r = __fdividef(1.0f, 1.0f + e), w = g[k] < 0.0f ? half : 1.0f;  // q = w w r
        const float s = dh[k] * w * r;
        u[k] = s * (1.0f + g[k] * (g[k] < 0.0f ? r : e * r)) * (u[k] * w);
        g[k] = s * (g[k] * w);
      }
      V dg, du;
      dg.pack(u);
      du.pack(g);
      T* out = static_cast<T*>(A.dgu) + r * 2 * A.F + f;
      *reinterpret_cast<V*>(out) = dg;
      *reinterpret_cast<V*>(out + A.F) = du;
    }
  }
}

inline hcmix_status run_gate_backward(GateArgs A, hcmix_type type, cudaStream_t stream) {
  const int size = size_of(type);
  // a vector lies in one half of a row, and both halves start on one
  int bytes = vector_bytes(size, {{A.dh, A.dh_stride}, {A.gu, A.gu_stride}, {A.dgu, A.F}});
  while (bytes > size && A.F * size % bytes != 0) bytes = bytes == 16 && size < 4 ? 4 : size;
  return with_vector(type, bytes, [&](auto z, auto vec, auto) {
    constexpr int kVec = decltype(vec)::value;
    const int64_t per = (A.F + kVec - 1) / kVec;
    A.across = 0;
    while ((1 << A.across) < per && (1 << A.across) < kGateThreads) ++A.across;
    const int64_t down = (kGateThreads >> A.across) * kGateRows<decltype(z), kVec>;
    const int64_t rows = (A.R + down - 1) / down;
    const dim3 grid((unsigned)((per + (1 << A.across) - 1) >> A.across),
                    (unsigned)(rows < 65535 ? rows : 65535));
    return launch(hcmix_gate_backward_kernel<decltype(z), kVec>, grid, dim3(kGateThreads), 0, 0,
                  stream, A);
  });
}

}  // namespace sublayer
}  // namespace hcmix
