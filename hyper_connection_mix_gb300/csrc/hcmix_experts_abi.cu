// C ABI of the experts' feed-forward network (declared in include/hcmix_experts.h).
//
// Host side only: argument checks and dispatch.  Every step of the computation runs in
// the kernels included below.
#include <cuda_runtime.h>

#include <cstdint>

#include "hcmix_experts.h"
#include "hcmix_gate.cuh"
#include "hcmix_product.cuh"
#include "hcmix_product_q4.cuh"

using namespace hcmix::sublayer;

namespace {

// a tile's rows behind the last are counted in 32 bits too
constexpr int64_t kMaxRows = ((int64_t)1 << 31) - 4096;
constexpr int64_t kMaxWidth = (int64_t)1 << 24;

#define HCMIX_TRY(expr)                                  \
  do {                                                   \
    const hcmix_status status_ = (expr);                 \
    if (status_ != HCMIX_OK) return status_;             \
  } while (0)

bool aligned(const void* p, int size) { return reinterpret_cast<uintptr_t>(p) % size == 0; }

cudaStream_t as_stream(void* s) { return static_cast<cudaStream_t>(s); }

hcmix_status check_extent(int64_t rows, int64_t width) {
  if (rows < 0 || width <= 0) return HCMIX_ERR_INVALID_ARG;
  return rows > kMaxRows || width > kMaxWidth ? HCMIX_ERR_UNSUPPORTED : HCMIX_OK;
}

hcmix_status check_type(hcmix_type type) {
  if (type == HCMIX_F32) return HCMIX_ERR_UNSUPPORTED;
  return type == HCMIX_BF16 || type == HCMIX_F16 ? HCMIX_OK : HCMIX_ERR_INVALID_ARG;
}

hcmix_status check_matrix(const void* p, int64_t stride, int64_t width, int size) {
  if (p == nullptr || stride < width) return HCMIX_ERR_INVALID_ARG;
  return aligned(p, size) ? HCMIX_OK : HCMIX_ERR_ALIGNMENT;
}

hcmix_status check_offsets(const int32_t* offsets, int64_t E) {
  if (E <= 0 || offsets == nullptr) return HCMIX_ERR_INVALID_ARG;
  if (E > kProductExperts) return HCMIX_ERR_UNSUPPORTED;
  return aligned(offsets, 4) ? HCMIX_OK : HCMIX_ERR_ALIGNMENT;
}

// W[E, outer, inner]
hcmix_status check_weight(const void* w, int64_t stride, int64_t expert, int64_t E, int64_t inner,
                          int64_t outer) {
  HCMIX_TRY(check_matrix(w, stride, inner, 2));
  return E > 1 && expert < (outer - 1) * stride + inner ? HCMIX_ERR_INVALID_ARG : HCMIX_OK;
}

Matrix3 matrix(const void* p, int64_t row, int64_t expert, int64_t inner, int64_t outer) {
  return Matrix3{p, row, expert, (int)inner, (int)outer};
}

// A product onto M features, of weights with M or 2 M of them.
hcmix_status product(const void* xs, int64_t xs_stride, hcmix_type type, int64_t R, int64_t K,
                     int64_t M, bool gated, const void* weight, int64_t w_stride,
                     int64_t w_expert_stride, int transposed, const int32_t* offsets, int64_t E,
                     void* out, void* saved, void* stream) {
  const int64_t features = gated ? 2 * M : M;
  HCMIX_TRY(check_extent(R, K));
  HCMIX_TRY(check_extent(R, M));
  HCMIX_TRY(check_extent(R, features));
  HCMIX_TRY(check_type(type));
  HCMIX_TRY(check_offsets(offsets, E));
  const int64_t inner = transposed ? features : K, outer = transposed ? K : features;
  HCMIX_TRY(check_weight(weight, w_stride, w_expert_stride, E, inner, outer));
  if (R == 0) return HCMIX_OK;
  HCMIX_TRY(check_matrix(xs, xs_stride, K, 2));
  HCMIX_TRY(check_matrix(out, M, M, 2));
  if (!aligned(saved, 2)) return HCMIX_ERR_ALIGNMENT;
  ProductArgs A = {};
  A.a = matrix(weight, w_stride, w_expert_stride, inner, outer);
  A.b = matrix(xs, xs_stride, 0, K, R);
  A.offsets = offsets, A.R = R, A.E = (int)E;
  A.M = (int)M, A.K = (int)K, A.gated = gated;
  A.out = out, A.saved = saved, A.f16 = type == HCMIX_F16;
  return transposed ? run_product<ProductMode::kRowsM>(A, as_stream(stream))
                    : run_product<ProductMode::kRowsK>(A, as_stream(stream));
}

}  // namespace

extern "C" {

hcmix_status hc_mix_expert_product(const void* xs, int64_t xs_stride, hcmix_type type, int64_t R,
                                   int64_t K, int64_t N, const void* weight, int64_t w_stride,
                                   int64_t w_expert_stride, int transposed,
                                   const int32_t* offsets, int64_t E, void* ys, void* stream) {
  return product(xs, xs_stride, type, R, K, N, false, weight, w_stride, w_expert_stride, transposed,
                 offsets, E, ys, nullptr, stream);
}

hcmix_status hc_mix_expert_product_gated(const void* xs, int64_t xs_stride, hcmix_type type,
                                         int64_t R, int64_t K, int64_t F, const void* weight,
                                         int64_t w_stride, int64_t w_expert_stride,
                                         int transposed, const int32_t* offsets, int64_t E,
                                         void* h, void* gu, void* stream) {
  return product(xs, xs_stride, type, R, K, F, true, weight, w_stride, w_expert_stride, transposed,
                 offsets, E, h, gu, stream);
}

hcmix_status hc_mix_expert_product_weight_backward(const void* dys, int64_t dys_stride,
                                                   const void* xs, int64_t xs_stride,
                                                   hcmix_type type, int64_t R, int64_t K,
                                                   int64_t N, int transposed,
                                                   const int32_t* offsets, int64_t E,
                                                   void* dweight, hcmix_type grad_type,
                                                   void* stream) {
  HCMIX_TRY(check_extent(R, K));
  HCMIX_TRY(check_extent(R, N));
  HCMIX_TRY(check_type(type));
  if (grad_type != type && grad_type != HCMIX_F32) return HCMIX_ERR_INVALID_ARG;
  HCMIX_TRY(check_offsets(offsets, E));
  HCMIX_TRY(check_matrix(dweight, 0, 0, size_of(grad_type)));
  if (R > 0) {
    HCMIX_TRY(check_matrix(dys, dys_stride, N, 2));
    HCMIX_TRY(check_matrix(xs, xs_stride, K, 2));
  }
  // the result's outer index is the lanes': n, or k where dweight is transposed
  const Matrix3 x = matrix(xs, xs_stride, 0, K, R), dy = matrix(dys, dys_stride, 0, N, R);
  ProductArgs A = {};
  A.a = transposed ? x : dy, A.b = transposed ? dy : x;
  A.offsets = offsets, A.R = R, A.E = (int)E;
  A.M = A.a.inner, A.N = A.b.inner;
  A.out = dweight, A.f16 = type == HCMIX_F16, A.out_f32 = grad_type == HCMIX_F32;
  return run_product<ProductMode::kWeight>(A, as_stream(stream));
}

hcmix_status hc_mix_expert_gate_backward(const void* dh, int64_t dh_stride, const void* gu,
                                         int64_t gu_stride, hcmix_type type, int64_t R, int64_t F,
                                         void* dgu, void* stream) {
  HCMIX_TRY(check_extent(R, F));
  HCMIX_TRY(check_extent(R, 2 * F));
  if (type != HCMIX_F32) HCMIX_TRY(check_type(type));
  if (R == 0) return HCMIX_OK;
  const int size = size_of(type);
  HCMIX_TRY(check_matrix(dh, dh_stride, F, size));
  HCMIX_TRY(check_matrix(gu, gu_stride, 2 * F, size));
  HCMIX_TRY(check_matrix(dgu, 2 * F, 2 * F, size));
  return run_gate_backward(GateArgs{dh, gu, dh_stride, gu_stride, dgu, R, F, 0}, type,
                           as_stream(stream));
}

hcmix_status hc_mix_expert_product_q4(const void* xs, int64_t xs_stride, hcmix_type type,
                                      int64_t R, int64_t K, int64_t N, const void* codes,
                                      const void* scales, int64_t group, int gated,
                                      const int32_t* offsets, int64_t E, void* out, void* stream) {
  HCMIX_TRY(check_extent(R, K));
  HCMIX_TRY(check_extent(R, N));
  HCMIX_TRY(check_type(type));
  HCMIX_TRY(check_offsets(offsets, E));
  if ((gated && N % 2 != 0) || group <= 0 || K % group != 0) return HCMIX_ERR_INVALID_ARG;
  if (group != 32 && group != 64 && group != 128 && group != 256) return HCMIX_ERR_UNSUPPORTED;
  HCMIX_TRY(check_matrix(codes, 0, 0, 16));
  HCMIX_TRY(check_matrix(scales, 0, 0, 2));
  if (R == 0) return HCMIX_OK;
  HCMIX_TRY(check_matrix(xs, xs_stride, K, 2));
  HCMIX_TRY(check_matrix(out, 0, 0, 2));
  Q4Args A = {};
  A.xs = xs, A.xs_stride = xs_stride, A.R = R;
  A.codes = static_cast<const uint8_t*>(codes), A.scales = scales, A.offsets = offsets;
  A.E = (int)E, A.K = (int)K, A.N = (int)N, A.group = (int)group, A.gated = gated != 0;
  A.out = out, A.vec = vector_bytes(2, {{xs, xs_stride}}) == 16;
  return run_product_q4(A, type, as_stream(stream));
}

hcmix_status hc_mix_expert_device_status(void* stream) {
  uint32_t word = 0;
  HCMIX_TRY(checked(cudaStreamSynchronize(as_stream(stream))));
  HCMIX_TRY(checked(cudaMemcpyFromSymbol(&word, g_product_error, sizeof word)));
  if (word == 0) return HCMIX_OK;
  word = 0;
  HCMIX_TRY(checked(cudaMemcpyToSymbol(g_product_error, &word, sizeof word)));
  return HCMIX_ERR_DEVICE;
}

}  // extern "C"
