/*
 * fp8bg_tokens.h -- operators by which every token picks its weights: routing
 * to experts, the way into expert order and back, which the grouped products of
 * fp8bg.h stand between, and low-rank adapters of many requests beside a
 * shared projection.
 *
 * Tensors, sizes, statuses, streams and ownership are as in the second part of
 * fp8bg.h: row-major, unit column stride, a row pitch `ld*` in ELEMENTS, any
 * size >= 0, nothing thrown, allocated or kept, each call asynchronous on
 * `stream` and capturable in a HIP graph.  Index arrays are int32 on the
 * device and never read by the host; whatever they hold, no kernel addresses
 * outside the operands.  Every call is deterministic, bit for bit.
 */
#ifndef FP8BG_TOKENS_H
#define FP8BG_TOKENS_H

#include "fp8bg.h"

#ifdef __cplusplus
extern "C" {
#endif

/* How fbg_route_experts makes scores of logits, and a group's of its experts'. */
enum { FBG_SCORE_SOFTMAX = 0, FBG_SCORE_SIGMOID = 1 };
enum { FBG_GROUP_MAX = 0, FBG_GROUP_TOP2 = 1 };

/*
 * fbg_route_experts -- for each token (row of logits [T,E], of `dtype`, an
 * FBG_OUT_* code) the `topk` experts and their weights:
 *
 *     s[e] = softmax(logits)[e]  or  1 / (1 + exp(-logits[e]))
 *     c[e] = s[e] + bias[e]                      (logits[e] where bias is NULL)
 *     groups of E / groups experts in a row; the topk_groups groups of largest
 *         value stay: the largest c of a group (FBG_GROUP_MAX) or the sum of its
 *         two largest s[e] + bias[e] (FBG_GROUP_TOP2; of one expert, its own)
 *     experts[t,j]: the j-th largest c among them
 *     weights[t,j] = scale * s / max(sum of the chosen s, 1e-20)   (renormalize)
 *                    scale * s                                     (else)
 *
 * Of equal values the lowest index comes first.  What is compared is exact for
 * logits and in 64 bits where a bias is added or scores are summed, so the
 * choice does not hang on a rounding of the scores.  Weights are fp32, off by at most
 * 2^-24 (|largest logit - logit| + topk + 48) of themselves (sigmoid: |logit|) where the
 * scores are normal numbers.
 * bias [E] fp32 or NULL; mask [T] bytes or NULL: a token whose byte is not zero
 * gets experts -1 and weights 0.  A row that holds a NaN or +infinity (or with
 * a bias that does), or a softmax of nothing but -infinity, has no routing: its
 * weights are NaN and its experts 0 .. topk-1.  A -infinity in a logit without a
 * bias, or in a bias, otherwise leaves its expert to be chosen last.
 *
 * weights [T,topk] fp32 and experts [T,topk] int32, contiguous, 4-byte aligned,
 * overlapping nothing.  E <= 1024, topk <= 64, topk <= topk_groups * E / groups,
 * groups <= 64 dividing E: beyond -> UNSUPPORTED for the limits, INVALID_VALUE
 * for what cannot be.  T == 0 or topk == 0: nothing launched.
 */
int fbg_route_experts(const void *logits, int64_t ld, int dtype, int64_t T, int64_t E, int64_t topk, int score,
                      const float *bias, int64_t groups, int64_t topk_groups, int group_score, int renormalize,
                      float scale, const uint8_t *mask, float *weights, int32_t *experts, void *stream);

/*
 * fbg_dispatch_tokens -- rows in the order of their experts: A, a_s and offsets
 * of the grouped products.  Choice j of token t picks expert
 * e = experts[t,j] - first_expert; it gets a row where 0 <= e < E (the experts
 * that are held here), and those rows lie expert by expert, in one by token and
 * then by j:
 *
 *     offsets[e]  = choices of experts below e                  (e = 0 .. E)
 *     slots[t,j]  = offsets[e] + earlier choices of e, or -1 for a choice without a row
 *     rows[slots[t,j]] = x[t],  row_scale[slots[t,j]] = x_scale[t]
 *
 * x [T,K] of elements of `size` bytes (1, 2 or 4), x_scale [T,S] fp32
 * contiguous, or NULL (then S and row_scale mean nothing).  rows [T*topk, K] and
 * row_scale [T*topk, S] contiguous: those behind offsets[E] are left as they
 * are.  experts and slots [T,topk], offsets [E+1].  x and rows aligned to
 * `size`, the others to 4 bytes.  E <= 1024, topk <= 64, T * topk and
 * first_expert <= INT32_MAX - 1024.
 */
int fbg_dispatch_tokens(const int32_t *experts, int64_t T, int64_t topk, int64_t first_expert, int64_t E,
                        const void *x, int64_t ldx, int64_t K, int size, const float *x_scale, int64_t S, void *rows,
                        int64_t ldrows, float *row_scale, int32_t *offsets, int32_t *slots, void *stream);

/*
 * fbg_combine_experts -- the way back, each token's rows summed by weight:
 *
 *     out[t] = base[t] + sum over j of weights[t,j] * rows[slots[t,j]]
 *
 * in fp32, base first and then by j, one rounding at the end.  A slot outside
 * 0 .. R-1 adds nothing, whatever its weight (the -1 of a choice without a row).
 * rows [R,D] of `dtype`; base [T,D] of base_dtype (`dtype` or out_dtype), or NULL;
 * out [T,D] of out_dtype; weights and slots [T,topk] contiguous.  topk <= 64.
 * out overlaps nothing, but may be base itself (same address, pitch and type).
 */
int fbg_combine_experts(const void *rows, int64_t ldrows, int dtype, int64_t R, const int32_t *slots,
                        const float *weights, const void *base, int64_t ldbase, int base_dtype, void *out,
                        int64_t ldout, int out_dtype, int64_t T, int64_t topk, int64_t D, void *stream);

/*
 * fbg_add_adapters -- low-rank adapters of many requests at once, added to the
 * output of the projection that they share.  With a = adapters[m]:
 *
 *     out[m] = y[m] + scales[a] * B[a] (A[a] x[m])      where 0 <= a < L
 *     out[m] = y[m]                                     elsewhere
 *
 * x [M,K], A [L,R,K] and B [L,N,R] contiguous, of `dtype` (bf16 or fp16); y and
 * out [M,N] of out_dtype; adapters [M] int32; scales [L] fp32, or NULL for ones.
 * Adapters of a lower rank than R are padded with zeros.  Sums are fp32 and out is
 * rounded once.  Between the two products the R values are summed and kept in fp32;
 * the second takes each as a sum of 16-bit terms, which is the value itself for bf16
 * weights and an fp32 out, off by at most 2^-17 of it for bf16 weights and a 16-bit out, and
 * for fp16 weights by 2^-22 of the largest of its token's ranks 32 i .. 32 i + 31.
 * Infinities and NaN go where the formula takes them.  out may be
 * y itself (same address and pitch: rows without an adapter are then not touched),
 * and otherwise overlaps nothing.  R <= 256, K <= 2^24 - 128.  x, A, B, y and out
 * aligned to their elements.  K, R or L of 0: out is y.  workspace: 16-byte aligned
 * device memory of at least fbg_add_adapters_workspace_size(M, N, K, R) bytes, of any content; too
 * small -> OUT_OF_MEMORY.  Calls that overlap in time must not share one.
 */
int fbg_add_adapters(const void *y, int64_t ldy, const void *x, int64_t ldx, const void *A, const void *B,
                     const int32_t *adapters, const float *scales, void *out, int64_t ldout, int64_t M, int64_t N,
                     int64_t K, int64_t R, int64_t L, int dtype, int out_dtype, void *workspace,
                     size_t workspace_bytes, void *stream);
size_t fbg_add_adapters_workspace_size(int64_t M, int64_t N, int64_t K, int64_t R);

#ifdef __cplusplus
}
#endif

#endif /* FP8BG_TOKENS_H */
