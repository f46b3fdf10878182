// C ABI of the sublayer operators (declared in include/hcmix_sublayer.h).
//
// Host side only: argument checks, workspace size and dispatch.  Every step of
// the computation runs in the kernels included below.
#include <cuda_runtime.h>

#include <cstdint>

#include "hcmix_experts.cuh"
#include "hcmix_norm.cuh"
#include "hcmix_streams.cuh"
#include "hcmix_sublayer.h"

using namespace hcmix::sublayer;

namespace {

constexpr int64_t kMaxRows = ((int64_t)1 << 31) - 1;
constexpr int64_t kMaxWidth = (int64_t)1 << 24;

hcmix_status check_shape(int64_t M, int64_t N) {
  if (M < 0 || N <= 0) return HCMIX_ERR_INVALID_ARG;
  if (M > kMaxRows || N > kMaxWidth) return HCMIX_ERR_UNSUPPORTED;
  return HCMIX_OK;
}

bool valid_type(hcmix_type t) { return t == HCMIX_BF16 || t == HCMIX_F16 || t == HCMIX_F32; }

bool valid_param(hcmix_type param, hcmix_type type) { return param == HCMIX_F32 || param == type; }

// A pointer of a type of `size` bytes that may be null (checked elsewhere).
bool aligned(const void* p, int size) { return reinterpret_cast<uintptr_t>(p) % size == 0; }

// Matrices: each present, its rows at least `width` apart, aligned to its type.
hcmix_status check_matrix(const void* p, int64_t stride, int64_t width, hcmix_type type) {
  if (p == nullptr || stride < width) return HCMIX_ERR_INVALID_ARG;
  return aligned(p, size_of(type)) ? HCMIX_OK : HCMIX_ERR_ALIGNMENT;
}

#define HCMIX_TRY(expr)                                  \
  do {                                                   \
    const hcmix_status status_ = (expr);                 \
    if (status_ != HCMIX_OK) return status_;             \
  } while (0)

hcmix_status check_floats(const float* p) {
  if (p == nullptr) return HCMIX_ERR_INVALID_ARG;
  return aligned(p, 4) ? HCMIX_OK : HCMIX_ERR_ALIGNMENT;
}

hcmix_status check_streams(int64_t M, int64_t D, int hc, hcmix_type type) {
  HCMIX_TRY(check_shape(M, D));
  if (!valid_type(type)) return HCMIX_ERR_INVALID_ARG;
  if (hc != kStreams || D > kMaxWidth / kStreams) return HCMIX_ERR_UNSUPPORTED;
  return HCMIX_OK;
}

hcmix_status check_params(const void* weight, const void* bias, hcmix_type param,
                          hcmix_type type) {
  if (!valid_param(param, type)) return HCMIX_ERR_INVALID_ARG;
  const int n = size_of(param);
  return aligned(weight, n) && aligned(bias, n) ? HCMIX_OK : HCMIX_ERR_ALIGNMENT;
}

hcmix_status check_pairs(int64_t T, int64_t k) {
  if (T < 0 || k < 0) return HCMIX_ERR_INVALID_ARG;
  if (T > kMaxRows || k > kMaxRows || (k > 0 && T > kMaxRows / k)) return HCMIX_ERR_UNSUPPORTED;
  return HCMIX_OK;
}

hcmix_status check_rows(int64_t T, int64_t k, int64_t D, hcmix_type type, const int32_t* slots,
                        const int32_t* offsets, int64_t E) {
  HCMIX_TRY(check_shape(T, D));
  HCMIX_TRY(check_pairs(T, k));
  if (!valid_type(type) || (offsets != nullptr && E < 0)) return HCMIX_ERR_INVALID_ARG;
  if (T * k > 0 && slots == nullptr) return HCMIX_ERR_INVALID_ARG;
  return aligned(slots, 4) && aligned(offsets, 4) ? HCMIX_OK : HCMIX_ERR_ALIGNMENT;
}

cudaStream_t as_stream(void* s) { return static_cast<cudaStream_t>(s); }

}  // namespace

extern "C" {

hcmix_status hc_mix_layer_norm(const void* x, int64_t x_stride, hcmix_type type, int64_t M,
                               int64_t N, const void* weight, const void* bias,
                               hcmix_type param_type, float eps, void* y, float* mean,
                               float* rstd, void* stream) {
  HCMIX_TRY(check_shape(M, N));
  if (!valid_type(type)) return HCMIX_ERR_INVALID_ARG;
  HCMIX_TRY(check_params(weight, bias, param_type, type));
  if (M == 0) return HCMIX_OK;
  HCMIX_TRY(check_matrix(x, x_stride, N, type));
  HCMIX_TRY(check_matrix(y, N, N, type));
  if (!aligned(mean, 4) || !aligned(rstd, 4)) return HCMIX_ERR_ALIGNMENT;
  NormArgs A = {};
  A.x = x, A.x_stride = x_stride, A.M = M, A.N = N;
  A.weight = weight, A.bias = bias, A.p32 = param_type == HCMIX_F32, A.eps = eps;
  A.y = y, A.mean = mean, A.rstd = rstd;
  return run_norm(A, type, false, as_stream(stream));
}

size_t hc_mix_layer_norm_workspace_bytes(hcmix_type type, int64_t M, int64_t N) {
  if (check_shape(M, N) != HCMIX_OK || !valid_type(type)) return 0;
  return norm_workspace(size_of(type), M, N);
}

hcmix_status hc_mix_layer_norm_backward(const void* dy, int64_t dy_stride, const void* x,
                                        int64_t x_stride, hcmix_type type, int64_t M, int64_t N,
                                        const float* mean, const float* rstd, const void* weight,
                                        hcmix_type param_type, void* dx, float* dweight,
                                        float* dbias, void* workspace, size_t workspace_bytes,
                                        void* stream) {
  HCMIX_TRY(check_shape(M, N));
  if (!valid_type(type) || (dweight == nullptr) != (dbias == nullptr)) return HCMIX_ERR_INVALID_ARG;
  HCMIX_TRY(check_params(weight, nullptr, param_type, type));
  if (M > 0) {
    HCMIX_TRY(check_matrix(dy, dy_stride, N, type));
    HCMIX_TRY(check_matrix(x, x_stride, N, type));
    HCMIX_TRY(check_matrix(dx, N, N, type));
    HCMIX_TRY(check_floats(mean));
    HCMIX_TRY(check_floats(rstd));
  } else if (dweight == nullptr) {
    return HCMIX_OK;
  }
  if (dweight != nullptr) {
    if (!aligned(dweight, 4) || !aligned(dbias, 4)) return HCMIX_ERR_ALIGNMENT;
    const size_t need = norm_workspace(size_of(type), M, N);
    if (need > 0) {
      if (workspace == nullptr) return HCMIX_ERR_INVALID_ARG;
      if (!aligned(workspace, 256)) return HCMIX_ERR_ALIGNMENT;
      if (workspace_bytes < need) return HCMIX_ERR_WORKSPACE;
    }
  }
  NormArgs A = {};
  A.x = x, A.x_stride = x_stride, A.M = M, A.N = N;
  A.dy = dy, A.dy_stride = dy_stride;
  A.mean = const_cast<float*>(mean), A.rstd = const_cast<float*>(rstd);
  A.weight = weight, A.p32 = param_type == HCMIX_F32;
  A.dx = dx, A.dweight = dweight, A.dbias = dbias, A.part = static_cast<float*>(workspace);
  return run_norm_backward(A, type, as_stream(stream));
}

hcmix_status hc_mix_collapse(const void* x, int64_t x_stride, hcmix_type type, int64_t M,
                             int64_t D, int hc, const float* pre, void* h, void* stream) {
  HCMIX_TRY(check_streams(M, D, hc, type));
  if (M == 0) return HCMIX_OK;
  HCMIX_TRY(check_matrix(x, x_stride, hc * D, type));
  HCMIX_TRY(check_matrix(h, D, D, type));
  HCMIX_TRY(check_floats(pre));
  StreamsArgs A = {};
  A.x = x, A.x_stride = x_stride, A.pre = pre, A.out = h, A.M = M, A.D = D;
  return run_streams(StreamsOp::kCollapse, A, type, as_stream(stream));
}

hcmix_status hc_mix_collapse_norm(const void* x, int64_t x_stride, hcmix_type type, int64_t M,
                                  int64_t D, int hc, const float* pre, const void* weight,
                                  const void* bias, hcmix_type param_type, float eps, void* y,
                                  void* h, float* mean, float* rstd, void* stream) {
  HCMIX_TRY(check_streams(M, D, hc, type));
  HCMIX_TRY(check_params(weight, bias, param_type, type));
  if (M == 0) return HCMIX_OK;
  HCMIX_TRY(check_matrix(x, x_stride, hc * D, type));
  HCMIX_TRY(check_matrix(y, D, D, type));
  if (h != nullptr) HCMIX_TRY(check_matrix(h, D, D, type));
  HCMIX_TRY(check_floats(pre));
  if (!aligned(mean, 4) || !aligned(rstd, 4)) return HCMIX_ERR_ALIGNMENT;
  NormArgs A = {};
  A.x = x, A.x_stride = x_stride, A.pre = pre, A.M = M, A.N = D;
  A.weight = weight, A.bias = bias, A.p32 = param_type == HCMIX_F32, A.eps = eps;
  A.y = y, A.h = h, A.mean = mean, A.rstd = rstd;
  return run_norm(A, type, true, as_stream(stream));
}

hcmix_status hc_mix_collapse_backward(const void* dh, int64_t dh_stride, const void* x,
                                      int64_t x_stride, const void* dx_add, int64_t add_stride,
                                      hcmix_type type, int64_t M, int64_t D, int hc,
                                      const float* pre, void* dx, float* dpre, void* stream) {
  HCMIX_TRY(check_streams(M, D, hc, type));
  if (M == 0) return HCMIX_OK;
  HCMIX_TRY(check_matrix(dh, dh_stride, D, type));
  HCMIX_TRY(check_matrix(x, x_stride, hc * D, type));
  if (dx_add != nullptr) HCMIX_TRY(check_matrix(dx_add, add_stride, hc * D, type));
  HCMIX_TRY(check_matrix(dx, hc * D, hc * D, type));
  HCMIX_TRY(check_floats(pre));
  HCMIX_TRY(check_floats(dpre));
  StreamsArgs A = {};
  A.x = x, A.x_stride = x_stride, A.g = dh, A.g_stride = dh_stride;
  A.add = dx_add, A.add_stride = add_stride;
  A.pre = pre, A.out = dx, A.dpre = dpre, A.M = M, A.D = D;
  return run_streams(StreamsOp::kCollapseBackward, A, type, as_stream(stream));
}

hcmix_status hc_mix_expand(const void* x, int64_t x_stride, const void* y, int64_t y_stride,
                           hcmix_type type, int64_t M, int64_t D, int hc, const float* post,
                           const float* comb, void* out, void* stream) {
  HCMIX_TRY(check_streams(M, D, hc, type));
  if (M == 0) return HCMIX_OK;
  HCMIX_TRY(check_matrix(x, x_stride, hc * D, type));
  HCMIX_TRY(check_matrix(y, y_stride, D, type));
  HCMIX_TRY(check_matrix(out, hc * D, hc * D, type));
  HCMIX_TRY(check_floats(post));
  HCMIX_TRY(check_floats(comb));
  StreamsArgs A = {};
  A.x = x, A.x_stride = x_stride, A.y = y, A.y_stride = y_stride;
  A.post = post, A.comb = comb, A.out = out, A.M = M, A.D = D;
  return run_streams(StreamsOp::kExpand, A, type, as_stream(stream));
}

hcmix_status hc_mix_expand_backward(const void* dout, int64_t dout_stride, const void* x,
                                    int64_t x_stride, const void* y, int64_t y_stride,
                                    hcmix_type type, int64_t M, int64_t D, int hc,
                                    const float* post, const float* comb, void* dx, void* dy,
                                    float* dpost, float* dcomb, void* stream) {
  HCMIX_TRY(check_streams(M, D, hc, type));
  if (M == 0) return HCMIX_OK;
  HCMIX_TRY(check_matrix(dout, dout_stride, hc * D, type));
  HCMIX_TRY(check_matrix(x, x_stride, hc * D, type));
  HCMIX_TRY(check_matrix(y, y_stride, D, type));
  HCMIX_TRY(check_matrix(dx, hc * D, hc * D, type));
  HCMIX_TRY(check_matrix(dy, D, D, type));
  HCMIX_TRY(check_floats(post));
  HCMIX_TRY(check_floats(comb));
  HCMIX_TRY(check_floats(dpost));
  HCMIX_TRY(check_floats(dcomb));
  StreamsArgs A = {};
  A.x = x, A.x_stride = x_stride, A.y = y, A.y_stride = y_stride;
  A.g = dout, A.g_stride = dout_stride, A.post = post, A.comb = comb;
  A.out = dx, A.dy = dy, A.dpost = dpost, A.dcomb = dcomb, A.M = M, A.D = D;
  return run_streams(StreamsOp::kExpandBackward, A, type, as_stream(stream));
}

hcmix_status hc_mix_expert_sort(const void* ids, int id_bytes, int64_t T, int64_t k, int64_t E,
                                int32_t* offsets, int32_t* slots, int32_t* source, void* stream) {
  HCMIX_TRY(check_pairs(T, k));
  if ((id_bytes != 4 && id_bytes != 8) || E <= 0 || offsets == nullptr)
    return HCMIX_ERR_INVALID_ARG;
  if (E > kMostExperts) return HCMIX_ERR_UNSUPPORTED;
  if (T * k > 0 && (ids == nullptr || slots == nullptr || source == nullptr))
    return HCMIX_ERR_INVALID_ARG;
  if (!aligned(ids, id_bytes) || !aligned(offsets, 4) || !aligned(slots, 4) || !aligned(source, 4))
    return HCMIX_ERR_ALIGNMENT;
  SortArgs A = {ids, T * k, (int)E, offsets, slots, source};
  return run_sort(A, id_bytes == 8, as_stream(stream));
}

hcmix_status hc_mix_expert_dispatch(const void* x, int64_t x_stride, hcmix_type type, int64_t T,
                                    int64_t k, int64_t D, const int32_t* slots,
                                    const int32_t* offsets, int64_t E, void* xs, void* stream) {
  HCMIX_TRY(check_rows(T, k, D, type, slots, offsets, E));
  if (T * k == 0) return HCMIX_OK;
  HCMIX_TRY(check_matrix(x, x_stride, D, type));
  HCMIX_TRY(check_matrix(xs, D, D, type));
  RowsArgs A = {};
  A.x = x, A.x_stride = x_stride, A.T = T, A.k = k, A.D = D, A.rows = T * k;
  A.slots = slots, A.offsets = offsets, A.E = E, A.out = xs;
  return run_rows(RowsOp::kDispatch, A, type, as_stream(stream));
}

hcmix_status hc_mix_expert_combine(const void* ys, int64_t ys_stride, hcmix_type type,
                                   int64_t rows, int64_t T, int64_t k, int64_t D,
                                   const int32_t* slots, const float* weights, void* y,
                                   void* stream) {
  HCMIX_TRY(check_rows(T, k, D, type, slots, nullptr, 0));
  HCMIX_TRY(check_shape(rows, D));
  if (T == 0) return HCMIX_OK;
  if (rows > 0) HCMIX_TRY(check_matrix(ys, ys_stride, D, type));
  HCMIX_TRY(check_matrix(y, D, D, type));
  if (!aligned(weights, 4)) return HCMIX_ERR_ALIGNMENT;
  RowsArgs A = {};
  A.ys = ys, A.ys_stride = ys_stride, A.T = T, A.k = k, A.D = D, A.rows = rows;
  A.slots = slots, A.weights = weights, A.out = y;
  return run_rows(RowsOp::kCombine, A, type, as_stream(stream));
}

hcmix_status hc_mix_expert_combine_backward(const void* dy, int64_t dy_stride, const void* ys,
                                            int64_t ys_stride, hcmix_type type, int64_t rows,
                                            int64_t T, int64_t k, int64_t D, const int32_t* slots,
                                            const int32_t* offsets, int64_t E,
                                            const float* weights, void* dys, float* dweights,
                                            void* stream) {
  HCMIX_TRY(check_rows(T, k, D, type, slots, offsets, E));
  HCMIX_TRY(check_shape(rows, D));
  if (T * k == 0 && (rows == 0 || offsets == nullptr)) return HCMIX_OK;
  // with no pairs there is still a tail to zero
  if (T * k > 0) {
    HCMIX_TRY(check_matrix(dy, dy_stride, D, type));
    HCMIX_TRY(check_floats(weights));
    HCMIX_TRY(check_floats(dweights));
  }
  if (rows > 0) {
    HCMIX_TRY(check_matrix(ys, ys_stride, D, type));
    HCMIX_TRY(check_matrix(dys, D, D, type));
  }
  RowsArgs A = {};
  A.x = dy, A.x_stride = dy_stride, A.ys = ys, A.ys_stride = ys_stride;
  A.T = T, A.k = k, A.D = D, A.rows = rows, A.slots = slots, A.offsets = offsets, A.E = E;
  A.weights = weights, A.out = dys, A.dweights = dweights;
  return run_rows(RowsOp::kCombineBackward, A, type, as_stream(stream));
}

}  // extern "C"
