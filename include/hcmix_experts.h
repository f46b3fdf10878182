/*
 * hcmix_experts.h -- C ABI of libhcmix.so: the experts' feed-forward network on
 * sm_103a, between hc_mix_expert_dispatch and hc_mix_expert_combine (hcmix_sublayer.h).
 *
 * The rows of xs[R, K] are sorted by expert: expert e has rows offsets[e] ..
 * offsets[e + 1] - 1, as hc_mix_expert_sort gives them.
 *
 *   product      ys[r] = W[e] xs[r]                     and its gradients
 *   gated        h[r] = silu(g) u, (g, u) = W[e] xs[r]  silu(g) = g / (1 + exp(-g))
 *   product_q4   both with weights of 4 bits, for few rows
 *
 * Conventions, with those of hcmix_sublayer.h (device pointers owned by the caller,
 * no allocation, no host synchronisation, asynchronous on `stream`, arguments checked
 * on the host before any launch, no trap):
 *   - `type` is the type of rows and weights.  The products take HCMIX_BF16 and
 *     HCMIX_F16 (HCMIX_F32 is refused: HCMIX_ERR_UNSUPPORTED), the gate's gradient
 *     all three.  Sums are fp32 (of the tensor cores, which drop what lies below a sum's
 *     last place; a sum of more than 16384 terms, or of more than 1024 for an fp32 result,
 *     is added up of such parts); a result of a 16-bit type is rounded once.
 *   - Matrices are row-major with inner stride 1.  Inputs have a row stride in
 *     elements, at least their width, weights a stride between experts too; outputs
 *     are contiguous.  Any width from 1 to 2^24 and any alignment of the type itself
 *     is accepted; operands whose rows (and experts) all start on 16 bytes are
 *     copied by the tensor memory accelerator and run fastest.
 *   - offsets[E + 1] is int32, on the device, offsets[0] = 0, not falling, its last
 *     at most R; 1 <= E <= 4096, 0 <= R <= 2^31 - 4096.  Offsets outside 0 .. R are taken as
 *     0 or R: no access is out of bounds whatever they hold, but results are then
 *     unspecified.
 *   - Rows from offsets[E] on belong to no expert.  Their results are zero, and what
 *     they hold is not used.  An expert without rows reads no weights.
 *   - The same call gives the same bits every time (no atomics on values).  The order of
 *     a row's sums depends on k and the type alone, not on what other rows its expert has.
 *   - Outputs may not overlap inputs.
 */
#ifndef HCMIX_EXPERTS_H
#define HCMIX_EXPERTS_H

#include "hcmix_sublayer.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ys[R, N] of xs[R, K].  weight is W[E, N, K], or with `transposed` W[E, K, N]; rows of
 * an expert's matrix are w_stride elements apart and experts w_expert_stride.
 * dxs[R, K] of dys[R, N] is the same call with N and K exchanged and the other
 * `transposed`. */
hcmix_status hc_mix_expert_product(const void* xs, int64_t xs_stride, hcmix_type type, int64_t R,
                                   int64_t K, int64_t N, const void* weight, int64_t w_stride,
                                   int64_t w_expert_stride, int transposed,
                                   const int32_t* offsets, int64_t E, void* ys, void* stream);

/* h[R, F] = silu(g) u of (g, u) = W[e] xs[r]: W is [E, 2 F, K], or transposed
 * [E, K, 2 F], g's features first.  g and u enter as fp32.  gu[R, 2 F], for
 * hc_mix_expert_gate_backward, may be NULL. */
hcmix_status hc_mix_expert_product_gated(const void* xs, int64_t xs_stride, hcmix_type type,
                                         int64_t R, int64_t K, int64_t F, const void* weight,
                                         int64_t w_stride, int64_t w_expert_stride,
                                         int transposed, const int32_t* offsets, int64_t E,
                                         void* h, void* gu, void* stream);

/* dweight[E, N, K] (or transposed [E, K, N]) = sum over each expert's rows of
 * dys[r] xs[r]^T, of grad_type: HCMIX_F32 or `type`; zero for an expert without rows. */
hcmix_status hc_mix_expert_product_weight_backward(const void* dys, int64_t dys_stride,
                                                   const void* xs, int64_t xs_stride,
                                                   hcmix_type type, int64_t R, int64_t K,
                                                   int64_t N, int transposed,
                                                   const int32_t* offsets, int64_t E,
                                                   void* dweight, hcmix_type grad_type,
                                                   void* stream);

/* dgu[R, 2 F] = (dh u q (1 + g (1 - q)), dh g q) with q = 1 / (1 + exp(-g)), for
 * dh[R, F] and gu[R, 2 F] = (g, u).  Row by row: there are no experts in it. */
hcmix_status hc_mix_expert_gate_backward(const void* dh, int64_t dh_stride, const void* gu,
                                         int64_t gu_stride, hcmix_type type, int64_t R, int64_t F,
                                         void* dgu, void* stream);

/* hc_mix_expert_product with W[E, N, K] of 4 bits, w = (code - 8) scale:
 *   codes[E, N, K / 2]       two codes a byte, the lower four bits the even k;
 *   scales[E, N, K / group]  of `type`, one for `group` neighbouring k.
 * Both are contiguous, codes 16-byte aligned.  group is 32, 64, 128 or 256 and divides
 * K.  gated: N is 2 F, and the result h[R, F] = silu(g) u as above, else ys[R, N].
 * Meant for few rows (single tokens): the weights are unpacked again for every 32 rows of
 * an expert, and from nine rows an expert on hc_mix_expert_product with weights of 16
 * bits takes less time (one expert: from about 32).  A row's sums are of eight interleaved
 * shares of k, scaled a group at a time, added in fp32 in a fixed order. */
hcmix_status hc_mix_expert_product_q4(const void* xs, int64_t xs_stride, hcmix_type type,
                                      int64_t R, int64_t K, int64_t N, const void* codes,
                                      const void* scales, int64_t group, int gated,
                                      const int32_t* offsets, int64_t E, void* out, void* stream);

/* Waits for `stream` and reports, once, whether a kernel of this header gave up a wait
 * on the current device since the last call (HCMIX_ERR_DEVICE: its outputs are
 * incomplete).  Every wait inside the kernels is bounded: it is given up when its block has
 * copied nothing for about two seconds, however long a call takes. */
hcmix_status hc_mix_expert_device_status(void* stream);

#ifdef __cplusplus
}
#endif

#endif /* HCMIX_EXPERTS_H */
