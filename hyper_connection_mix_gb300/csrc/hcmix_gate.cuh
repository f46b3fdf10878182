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
};

template <typename T, int kVec>
__global__ void __launch_bounds__(256) hcmix_gate_backward_kernel(const GateArgs A) {
  begin_kernel();
  using V = Packed<T, kVec>;
  const int64_t per = (A.F + kVec - 1) / kVec, all = A.R * per;
  const int64_t step = (int64_t)gridDim.x * blockDim.x;
  for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < all; i += step) {
    const int64_t r = i / per, f = (i - r * per) * kVec;
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
}

inline hcmix_status run_gate_backward(const GateArgs& A, hcmix_type type, cudaStream_t stream) {
  const int size = size_of(type);
  // a vector lies in one half of a row, and both halves start on one
  int bytes = vector_bytes(size, {{A.dh, A.dh_stride}, {A.gu, A.gu_stride}, {A.dgu, A.F}});
  while (bytes > size && A.F * size % bytes != 0) bytes = bytes == 16 && size < 4 ? 4 : size;
  return with_vector(type, bytes, [&](auto z, auto vec, auto) {
    constexpr int kVec = decltype(vec)::value;
    const int64_t all = A.R * ((A.F + kVec - 1) / kVec), blocks = (all + 255) / 256;
    return launch(hcmix_gate_backward_kernel<decltype(z), kVec>,
                  dim3((unsigned)(blocks < (1 << 30) ? blocks : (1 << 30))), dim3(256), 0, 0,
                  stream, A);
  });
}

}  // namespace sublayer
}  // namespace hcmix
