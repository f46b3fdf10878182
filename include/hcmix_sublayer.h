/*
 * hcmix_sublayer.h -- C ABI of libhcmix.so: the operators around a
 * hyper-connection sublayer on sm_103a.
 *
 * hc_mix_fused (hcmix.h) turns the streams x[M, hc * D] of every row into
 * pre[M, hc], post[M, hc] and comb[M, hc, hc].  These entry points apply them
 * and move the rows through a sublayer:
 *
 *   collapse  h = sum_i pre[i] x_i, and its layer norm    the sublayer's input
 *   expert_*  the tokens' rows sorted by expert and back  a mixture of experts
 *   expand    x'_i = post[i] y + sum_j comb[i][j] x_j     the sublayer's output
 *
 * with the layer norm on its own too, and the gradient of each.  x_i is stream i
 * of a row: its columns i * D .. i * D + D - 1.
 *
 * Conventions, with those of hcmix.h (device pointers owned by the caller, no
 * allocation, no host synchronisation, asynchronous on `stream`, arguments
 * checked on the host before any launch, no trap):
 *   - `type` is the type of every matrix of a call (HCMIX_BF16, HCMIX_F16 or
 *     HCMIX_F32).  All arithmetic is in fp32; a result of a 16-bit type is
 *     rounded once, at its store, to nearest even.  Coefficients, statistics,
 *     weights' gradients and expert weights are fp32.
 *   - Matrices are row-major with inner stride 1.  Inputs have a row stride in
 *     elements, at least their width; outputs are contiguous.  Any width from 1
 *     to 2^24 and any alignment of the type itself is accepted; rows that all
 *     start on 16 bytes are read and written in 16-byte pieces and run fastest.
 *   - Zero rows are a valid call.  Outputs that sum over rows are then zero.
 *   - Results do not depend on the order in which thread blocks run: there
 *     are no atomics on values, and the same call gives the same bits every
 *     time.  What belongs to one row is the same bits whatever other rows its
 *     call has; dweight and dbias, sums over rows, are formed by their number.
 *   - Outputs may not overlap inputs, except where said.
 */
#ifndef HCMIX_SUBLAYER_H
#define HCMIX_SUBLAYER_H

#include "hcmix.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef enum { HCMIX_BF16 = 0, HCMIX_F16 = 1, HCMIX_F32 = 2 } hcmix_type;

/* ---- layer norm ---------------------------------------------------------
 * mean = sum x / N, rstd = 1 / sqrt(sum (x - mean)^2 / N + eps) and
 * y = (x - mean) rstd weight + bias, for every row of x[M, N].
 * weight[N] and bias[N] may each be NULL (ones, zeros); they are of
 * `param_type`: HCMIX_F32 or `type`.  mean[M] and rstd[M] may be NULL. */
hcmix_status hc_mix_layer_norm(const void* x, int64_t x_stride, hcmix_type type, int64_t M,
                               int64_t N, const void* weight, const void* bias,
                               hcmix_type param_type, float eps, void* y, float* mean,
                               float* rstd, void* stream);

/* With xh = (x - mean) rstd and g = dy weight:
 *   dx = rstd (g - sum g / N - xh sum(g xh) / N),
 *   dweight = sum over rows of dy xh,  dbias = sum over rows of dy  (fp32 [N]).
 * dweight and dbias are given together, or both NULL: then no workspace is
 * needed.  Else `workspace` holds hc_mix_layer_norm_workspace_bytes(type, M, N)
 * bytes, 256-byte aligned; it needs no initialising.  The size never falls as M
 * grows: a workspace for the largest call does for the others of its N and type. */
size_t hc_mix_layer_norm_workspace_bytes(hcmix_type type, int64_t M, int64_t N);
hcmix_status hc_mix_layer_norm_backward(const void* dy, int64_t dy_stride, const void* x,
                                        int64_t x_stride, hcmix_type type, int64_t M, int64_t N,
                                        const float* mean, const float* rstd, const void* weight,
                                        hcmix_type param_type, void* dx, float* dweight,
                                        float* dbias, void* workspace, size_t workspace_bytes,
                                        void* stream);

/* ---- streams (hc == 4) --------------------------------------------------
 * h[M, D] = sum_i pre[m, i] x_i. */
hcmix_status hc_mix_collapse(const void* x, int64_t x_stride, hcmix_type type, int64_t M,
                             int64_t D, int hc, const float* pre, void* h, void* stream);

/* The same h, and y[M, D] its layer norm, taken of the fp32 h.  h, mean and
 * rstd may be NULL; training keeps them for hc_mix_layer_norm_backward. */
hcmix_status hc_mix_collapse_norm(const void* x, int64_t x_stride, hcmix_type type, int64_t M,
                                  int64_t D, int hc, const float* pre, const void* weight,
                                  const void* bias, hcmix_type param_type, float eps, void* y,
                                  void* h, float* mean, float* rstd, void* stream);

/* dx_i = pre[i] dh + dx_add_i, dpre[i] = sum dh x_i.  dx_add[M, hc * D], the
 * gradient that reached x another way (through hc_mix_expand), may be NULL; dx
 * may be dx_add itself where its rows are contiguous. */
hcmix_status hc_mix_collapse_backward(const void* dh, int64_t dh_stride, const void* x,
                                      int64_t x_stride, const void* dx_add, int64_t add_stride,
                                      hcmix_type type, int64_t M, int64_t D, int hc,
                                      const float* pre, void* dx, float* dpre, void* stream);

/* out_i = post[i] y + sum_j comb[i][j] x_j.  out may be x itself where its rows
 * are contiguous.
 * The sum is over comb's second index: comb[i] holds the weights of the streams in
 * stream i of the result.  hc_mix_fused says how comb is made (its columns are
 * divided last), not how a model applies it.  One whose weights mean the sum over
 * the first index, out_j = post[j] y + sum_i comb[i][j] x_i, passes comb with these
 * two indices exchanged, here and to the gradient, whose dcomb is exchanged too. */
hcmix_status hc_mix_expand(const void* x, int64_t x_stride, const void* y, int64_t y_stride,
                           hcmix_type type, int64_t M, int64_t D, int hc, const float* post,
                           const float* comb, void* out, void* stream);

/* dx_j = sum_i comb[i][j] dout_i, dy = sum_i post[i] dout_i,
 * dpost[i] = sum dout_i y, dcomb[i][j] = sum dout_i x_j.  dx may be dout itself
 * where its rows are contiguous. */
hcmix_status hc_mix_expand_backward(const void* dout, int64_t dout_stride, const void* x,
                                    int64_t x_stride, const void* y, int64_t y_stride,
                                    hcmix_type type, int64_t M, int64_t D, int hc,
                                    const float* post, const float* comb, void* dx, void* dy,
                                    float* dpost, float* dcomb, void* stream);

/* ---- experts ------------------------------------------------------------
 * ids[T, k] names each token's experts (id_bytes 4 or 8: int32 or int64; an id
 * outside 0 .. E - 1 names none, and its pair is dropped).  The pairs are put in
 * the order of their experts, and among one expert's in the order of ids:
 *   offsets[E + 1]  expert e's rows are offsets[e] .. offsets[e + 1] - 1;
 *   slots[T, k]     the row of each pair, -1 for a dropped one;
 *   source[T * k]   the pair t * k + j of each row, -1 from offsets[E] on.
 * 1 <= E <= 4096 and T * k < 2^31. */
hcmix_status hc_mix_expert_sort(const void* ids, int id_bytes, int64_t T, int64_t k, int64_t E,
                                int32_t* offsets, int32_t* slots, int32_t* source, void* stream);

/* xs[slots[t, j]] = x[t] for xs[T * k, D]; rows from offsets[E] on are zero (with
 * offsets NULL they are left as they are).  Slots outside xs are dropped pairs. */
hcmix_status hc_mix_expert_dispatch(const void* x, int64_t x_stride, hcmix_type type, int64_t T,
                                    int64_t k, int64_t D, const int32_t* slots,
                                    const int32_t* offsets, int64_t E, void* xs, void* stream);

/* y[t] = sum_j weights[t, j] ys[slots[t, j]] in the order of j, for ys[rows, D];
 * weights NULL: of one (the gradient of hc_mix_expert_dispatch).  A dropped pair
 * adds nothing, and a token of dropped pairs gets zeros. */
hcmix_status hc_mix_expert_combine(const void* ys, int64_t ys_stride, hcmix_type type,
                                   int64_t rows, int64_t T, int64_t k, int64_t D,
                                   const int32_t* slots, const float* weights, void* y,
                                   void* stream);

/* dys[slots[t, j]] = weights[t, j] dy[t], dweights[t, j] = sum dy[t] ys[slots[t, j]],
 * for ys[rows, D] and dys[rows, D]; a dropped pair's dweights is zero.  Rows of
 * dys from offsets[E] on are zero (offsets NULL: left as they are). */
hcmix_status hc_mix_expert_combine_backward(const void* dy, int64_t dy_stride, const void* ys,
                                            int64_t ys_stride, hcmix_type type, int64_t rows,
                                            int64_t T, int64_t k, int64_t D, const int32_t* slots,
                                            const int32_t* offsets, int64_t E,
                                            const float* weights, void* dys, float* dweights,
                                            void* stream);

#ifdef __cplusplus
}
#endif

#endif /* HCMIX_SUBLAYER_H */
