// The gate of an expert's feed-forward network, backward: with (g, u) the halves of a
// row of gu and q = 1 / (1 + exp(-g)),
//   dg = dh u q (1 + g (1 - q)),  du = dh g q.
// Elementwise, bound by HBM: dh, g and u are read once, dg and du written once.
#pragma once

#include "hcmix_vec.cuh"

namespace hcmix {
namespace sublayer {

struct GateArgs {
  const void *dh, *gu;
  int64_t dh_stride, gu_stride;
  void* dgu;
  int64_t R, F;
  int across;  // log2 of a block's threads along a row
};

template <typename T, int kVec>
__device__ __forceinline__ void gate_vector(const GateArgs& A, int64_t r, int64_t f) {
  using V = Packed<T, kVec>;
  const T* gu = static_cast<const T*>(A.gu) + r * A.gu_stride + f;
  float dh[kVec], g[kVec], u[kVec];
  reinterpret_cast<const V*>(static_cast<const T*>(A.dh) + r * A.dh_stride + f)->unpack(dh);
  reinterpret_cast<const V*>(gu)->unpack(g);
  reinterpret_cast<const V*>(gu + A.F)->unpack(u);
#pragma unroll
  for (int k = 0; k < kVec; ++k) {
    const float q = 1.0f / (1.0f + expf(-g[k]));
    const float s = dh[k] * q;
    u[k] *= s * (1.0f + g[k] * (1.0f - q));
    g[k] *= s;
  }
  V dg, du;
  dg.pack(u);
  du.pack(g);
  T* out = static_cast<T*>(A.dgu) + r * 2 * A.F + f;
  *reinterpret_cast<V*>(out) = dg;
  *reinterpret_cast<V*>(out + A.F) = du;
}

// A vector a thread.  A block is across x down of them, so that no thread divides by the
// width: `across` a power of two as large as a row's vectors, at most the block's threads.
constexpr int kGateThreads = 256;
template <typename T, int kVec>
__global__ void __launch_bounds__(kGateThreads) hcmix_gate_backward_kernel(const GateArgs A) {
  begin_kernel();
  const int down = kGateThreads >> A.across;
  const int64_t f = ((int64_t)blockIdx.x << A.across) + (threadIdx.x & ((1 << A.across) - 1));
  if (f * kVec >= A.F) return;
  for (int64_t r = (int64_t)blockIdx.y * down + (threadIdx.x >> A.across); r < A.R;
       r += (int64_t)gridDim.y * down)
    gate_vector<T, kVec>(A, r, f * kVec);
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
    const int64_t down = kGateThreads >> A.across, rows = (A.R + down - 1) / down;
    const dim3 grid((unsigned)((per + (1 << A.across) - 1) >> A.across),
                    (unsigned)(rows < 65535 ? rows : 65535));
    return launch(hcmix_gate_backward_kernel<decltype(z), kVec>, grid, dim3(kGateThreads), 0, 0,
                  stream, A);
  });
}

}  // namespace sublayer
}  // namespace hcmix
