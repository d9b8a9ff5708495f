/*
 * gemm_ws_lm.h — operators of language models around the matrix product
 *
 * What surrounds the last products of a training or scoring step, on the
 * same handle and library as gemm_ws.h:
 *
 *   gemm_ws_dropout                 y = keep * x / (1 - p)
 *   gemm_ws_add_rms_norm            h = residual + dropout(x); y = weight * h / rms(h),
 *                                   also in 8 bits with scales
 *   gemm_ws_add_rms_norm_backward   its gradients
 *   gemm_ws_linear_ce               softmax cross entropy of x * weight^T over a
 *                                   vocabulary, the logits never held
 *   gemm_ws_linear_ce_backward      its gradients
 *   gemm_ws_block_norm              the norms after and before a block, with its gate
 *                                   and the scaled residual, also in 8 bits with scales
 *   gemm_ws_block_norm_backward     its gradients
 *   gemm_ws_quantize_rows           rows to 8-bit integers with a scale for each
 *   gemm_ws_int8_matmul             the product of 8-bit integers with a scale for each
 *                                   token and each channel
 *   gemm_ws_adjust_logits           penalties for repeated tokens, biases, masks
 *
 * Everything that gemm_ws.h says of handles, threads, streams, ownership and
 * errors holds here: calls are asynchronous on `stream`, allocate nothing,
 * can be captured in CUDA graphs, and calls on one handle must not overlap on
 * the GPU. A call that returns an error other than GEMM_WS_ERR_CUDA launched
 * nothing. Results have the same bits on every run.
 *
 * A matrix is `rows` rows of `cols` contiguous elements, `ld` elements from
 * one row to the next (cols <= ld <= 2^40). What lies between two rows of an input may be
 * read, and plays no part; between two rows of an output nothing is written. An
 * output may be exactly one of the call's inputs where that is said; any other
 * overlap of an output with another argument (first to last element, what lies
 * between the rows included) is refused.
 */
#ifndef GEMM_WS_LM_H_
#define GEMM_WS_LM_H_

#include <stdint.h>

#include "gemm_ws.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef enum gemm_ws_dtype {
  GEMM_WS_BF16 = 0,
  GEMM_WS_F16 = 1,
  GEMM_WS_F32 = 2
} gemm_ws_dtype;

typedef enum gemm_ws_norm_output {
  GEMM_WS_NORM_SAME = 0,        /* y has the type of x */
  GEMM_WS_NORM_E4M3_ROW = 1,    /* y is e4m3, one fp32 scale a row */
  GEMM_WS_NORM_E4M3_GROUP = 2,  /* y is e4m3, one fp32 scale for each 128 columns */
  GEMM_WS_NORM_INT8_ROW = 3     /* gemm_ws_block_norm: y is 8-bit integers, one fp32 scale a row */
} gemm_ws_norm_output;

/* Dropout (here and in the norm). `rng` is a device pointer to two uint64:
 * a seed and the first counter; it is read when the kernel runs, so a captured
 * graph draws new numbers once the words it points to are changed. Column c
 * of row r is dropped iff its 16-bit word is below round(65536 * p), where
 * the word is number c % 8 of the 128 bits (lowest first) of Philox4x32-10
 * with key seed and counter first + r * ceil(cols / 8) + c / 8 (modulo 2^64);
 * what is kept is multiplied by 65536 / (65536 - round(65536 * p)). A call
 * uses rows * ceil(cols / 8) counters: the next one should start after them.
 * The mask is never stored: the backward pass is the same call with the same
 * rng words on the gradient. 0 <= p <= 1; with p == 0 nothing is dropped and
 * rng is not read (it may be NULL); with p == 1 all is 0. A dropped value
 * gives 0 whatever it was, an infinity or a NaN too.
 *  - x, y: rows x cols of `dtype` (a gemm_ws_dtype); y may be x.
 *  - 0 <= rows, cols < 2^31 (an empty call launches nothing). */
int gemm_ws_dropout(gemm_ws_t* h, int dtype, const void* x, int64_t ldx, void* y, int64_t ldy,
                    int64_t rows, int64_t cols, double p, const uint64_t* rng, void* stream);

/* hidden = residual + dropout(x); y = weight * hidden / sqrt(mean(hidden^2) + eps).
 * In 32 bits from the inputs to each output's one rounding: y is computed
 * from the unrounded sum.
 *  - x, residual (NULL: zero), hidden (NULL: not written), y: rows x cols;
 *    weight: cols; all of `dtype`, but y e4m3 bytes where `output` says so.
 *    hidden may be x or residual, and y may be x.
 *  - output: a gemm_ws_norm_output. The scale of a row (or of 128 columns, the
 *    last ones fewer) is max |y| / 448, at least 2^-126, and y holds the
 *    e4m3 roundings of y / scale. scales: rows (or rows x ceil(cols / 128)) fp32. (A row's
 *    largest |y| is taken from hidden * weight, whose products have to lie in the range of normal fp32.)
 *  - rstd: rows fp32, 1 / sqrt(mean(hidden^2) + eps), for the backward pass; or NULL.
 *  - 1 <= cols <= 32768; 0 <= rows < 2^31; p and rng as in gemm_ws_dropout. */
int gemm_ws_add_rms_norm(gemm_ws_t* h, int dtype, const void* x, int64_t ldx,
                         const void* residual, int64_t ldr, const void* weight, void* hidden,
                         int64_t ldh, void* y, int64_t ldy, int output, float* scales,
                         float* rstd, int64_t rows, int64_t cols, float eps, double p,
                         const uint64_t* rng, void* stream);

/* The gradients of gemm_ws_add_rms_norm with output GEMM_WS_NORM_SAME.
 *  - dy: of y; dhidden: what reaches hidden from its other uses (NULL: zero);
 *    hidden and rstd: what the forward call wrote.
 *  - dresidual: of residual (NULL: not written); dx: of x, which without
 *    dropout is the same. dx and dresidual may each be dy or dhidden.
 *  - dweight: cols, the sum over rows in 32 bits rounded once to `dtype`;
 *    NULL: not computed. With rows == 0 it is zero.
 *  - p and rng: those of the forward call.
 * Launches one kernel, two with dweight. */
int gemm_ws_add_rms_norm_backward(gemm_ws_t* h, int dtype, const void* dy, int64_t lddy,
                                  const void* dhidden, int64_t lddh, const void* hidden,
                                  int64_t ldh, const void* weight, const float* rstd, void* dx,
                                  int64_t lddx, void* dresidual, int64_t lddr, void* dweight,
                                  int64_t rows, int64_t cols, double p, const uint64_t* rng,
                                  void* stream);

/* Softmax cross entropy of z = x * weight^T over a vocabulary, in pieces of the
 * vocabulary, the logits z never held:
 *   lse[t] = log sum_j exp(z[t][j]);  loss[t] = lse[t] - z[t][target[t]].
 *  - x: tokens x hidden bf16; weight: vocab x hidden bf16; target: tokens
 *    int64 (target_bytes 8) or int32 (4).
 *  - A token whose target is `ignore` is not counted: its loss and lse are 0
 *    and its row of x plays no part (it may hold anything). A counted token
 *    whose target is outside [0, vocab) has loss NaN, and no gradient.
 *  - A logit of -inf is a word of no probability: nothing to lse, loss +inf
 *    where it is the target. A logit of +inf or NaN makes the token's lse and
 *    loss NaN.
 *  - loss, lse: tokens fp32; mean: two fp32, the mean loss over the counted
 *    tokens and 1 / their number (both 0 with none), or NULL.
 *  - workspace: gemm_ws_linear_ce_workspace bytes on the device, 256-byte
 *    aligned, for this call alone (its contents mean nothing before or after).
 *  - hidden: a multiple of 8; weight 16-byte aligned, ldw a multiple of 8 (x
 *    may lie anywhere). 0 <= tokens, 1 <= vocab, 8 <= hidden, each at most
 *    2^31 - 4096; tokens * hidden, vocab * hidden and tokens * vocab at most 2^40.
 * Products in bf16 with fp32 sums in tensor memory; everything after them in
 * fp32. Launches three kernels; two where x's rows lie on 16-byte boundaries and
 * there are up to 128 of them or no more tiles than run at once, one for up to
 * 8 of them. */
int gemm_ws_linear_ce(gemm_ws_t* h, const uint16_t* x, int64_t ldx, const uint16_t* weight,
                      int64_t ldw, const void* target, int target_bytes, int64_t ignore,
                      float* loss, float* lse, float* mean, int64_t tokens, int64_t hidden,
                      int64_t vocab, void* workspace, int64_t workspace_bytes, void* stream);

/* The gradients of sum_t grad[t] * loss[t].
 *  - x, weight, target, ignore: as given to gemm_ws_linear_ce; lse: what it wrote.
 *  - grad: fp32, one for each token (grad_step 1) or one for all (grad_step
 *    0; with &mean[1] the gradient of the mean loss).
 *  - dx: tokens x hidden bf16, zero for uncounted tokens; dweight: vocab x
 *    hidden bf16; either may be NULL. 16-byte aligned, lddx and lddw multiples
 *    of 8.
 * (softmax - [target]) * grad / max |grad| is rounded to bf16; the sums over the
 * vocabulary (dx) and the tokens (dweight) are fp32, multiplied by max |grad| and
 * rounded once. */
int gemm_ws_linear_ce_backward(gemm_ws_t* h, const uint16_t* x, int64_t ldx,
                               const uint16_t* weight, int64_t ldw, const void* target,
                               int target_bytes, int64_t ignore, const float* lse,
                               const float* grad, int grad_step, uint16_t* dx, int64_t lddx,
                               uint16_t* dweight, int64_t lddw, int64_t tokens, int64_t hidden,
                               int64_t vocab, void* workspace, int64_t workspace_bytes,
                               void* stream);

/* Workspace bytes of gemm_ws_linear_ce (backward 0) or its backward (nonzero)
 * for these sizes on this handle; negative (a gemm_ws_status, negated) for
 * sizes that they refuse. Host arithmetic only. */
int64_t gemm_ws_linear_ce_workspace(gemm_ws_t* h, int64_t tokens, int64_t hidden, int64_t vocab,
                                    int backward);

/* What lies between one block of a model and the next:
 *   n = x / sqrt(mean(x^2) + eps);  b = post_weight * n
 *   hidden = alpha * residual + gate * b
 *   y = weight * hidden / sqrt(mean(hidden^2) + eps)
 * In 32 bits from the inputs to each output's one rounding: y is computed from the
 * unrounded hidden.
 *  - x (the block's output), residual, hidden (NULL: not written), y: rows x cols;
 *    post_weight (NULL: no norm after the block, b = x), weight: cols; all of
 *    `dtype`, but y bytes where `output` says so. hidden may be x or
 *    residual, and y may be x.
 *  - gate: NULL (1), cols with ldg 0 (one for each channel), or rows x cols.
 *  - output: a gemm_ws_norm_output, and scales, as in gemm_ws_add_rms_norm. With
 *    GEMM_WS_NORM_INT8_ROW the scale of a row is max |y| / 127, at least 2^-126, and y
 *    holds the integers nearest to the fp32 quotients y / scale (halves to even). A row of y with an
 *    infinity or a NaN has scale NaN and zeros.
 *  - post_rstd (only with post_weight), rstd: rows fp32, 1 / sqrt(mean + eps) of the
 *    two norms, for the backward pass; or NULL.
 *  - alpha: finite. 1 <= cols <= 16384; 0 <= rows < 2^31.
 * Launches one kernel. */
int gemm_ws_block_norm(gemm_ws_t* h, int dtype, const void* x, int64_t ldx, const void* residual,
                       int64_t ldr, const void* gate, int64_t ldg, const void* post_weight,
                       const void* weight, void* hidden, int64_t ldh, void* y, int64_t ldy,
                       int output, float* scales, float* post_rstd, float* rstd, int64_t rows,
                       int64_t cols, float alpha, float eps, void* stream);

/* The gradients of gemm_ws_block_norm with output GEMM_WS_NORM_SAME.
 *  - dy: of y; dhidden: what reaches hidden from its other uses (NULL: zero); x, gate,
 *    post_weight, weight, alpha: as given to the forward call; hidden, post_rstd (with
 *    post_weight) and rstd: what it wrote.
 *  - dx: of x; dresidual: of residual (NULL: not written). Each may be dy or dhidden.
 *  - dgate: of gate, laid out like it (lddg elements between rows; not read for a gate of
 *    each channel); dpost_weight, dweight: cols. Sums over rows are in 32 bits and rounded once;
 *    each may be NULL, and with rows == 0 they are zero.
 * Launches one kernel, two with a sum over rows. */
int gemm_ws_block_norm_backward(gemm_ws_t* h, int dtype, const void* dy, int64_t lddy,
                                const void* dhidden, int64_t lddh, const void* x, int64_t ldx,
                                const void* hidden, int64_t ldh, const void* gate, int64_t ldg,
                                const void* post_weight, const void* weight,
                                const float* post_rstd, const float* rstd, void* dx, int64_t lddx,
                                void* dresidual, int64_t lddr, void* dgate, int64_t lddg,
                                void* dpost_weight, void* dweight, int64_t rows, int64_t cols,
                                float alpha, void* stream);

/* Rows in 8-bit integers: scales[r] = max_c |x[r][c]| / 127, at least 2^-126, and y the
 * integers nearest to the fp32 quotients x / scale (halves to even), -127 to 127. A row with an infinity or
 * a NaN has scale NaN and zeros.
 *  - x: rows x cols of `dtype`; y: rows x cols; scales: rows.
 *  - 1 <= cols <= 32768; 0 <= rows < 2^31. */
int gemm_ws_quantize_rows(gemm_ws_t* h, int dtype, const void* x, int64_t ldx, int8_t* y,
                          int64_t ldy, float* scales, int64_t rows, int64_t cols, void* stream);

/* d[m][n] = (sum_k a[m][k] * w[n][k]) * a_scales[m] * w_scales[n] + bias[n]. The sums are
 * exact in 32-bit integers; what follows is fp32, rounded once to `dtype`.
 *  - a: tokens x k, w: channels x k, 8-bit integers, -128 included; a_scales: tokens,
 *    w_scales: channels, bias: channels (NULL: none), fp32; d: tokens x channels of `dtype`.
 *  - w 16-byte aligned, ldw a multiple of 16, channels * ldw at most 2^40 (a, d and k are free).
 *  - workspace: gemm_ws_int8_matmul_workspace bytes on the device, 256-byte aligned,
 *    for this call alone (its contents mean nothing before or after); NULL where it is 0.
 *  - 0 <= tokens, 1 <= channels, each at most 2^31 - 4096; 1 <= k < 2^17;
 *    tokens * k, channels * k and tokens * channels at most 2^40.
 * GEMM_WS_ERR_BUILD for more than a few tokens where the compiler gave the kernel other registers than
 * its warps share out, with which they would wait for each other (the build checks it). */
int gemm_ws_int8_matmul(gemm_ws_t* h, const int8_t* a, int64_t lda, const float* a_scales,
                        const int8_t* w, int64_t ldw, const float* w_scales, const float* bias,
                        void* d, int64_t ldd, int dtype, int64_t tokens, int64_t channels,
                        int64_t k, void* workspace, int64_t workspace_bytes, void* stream);

/* Workspace bytes of gemm_ws_int8_matmul for these sizes on this handle; negative (a
 * gemm_ws_status, negated) for sizes that it refuses. Host arithmetic only. */
int64_t gemm_ws_int8_matmul_workspace(gemm_ws_t* h, int64_t tokens, int64_t channels, int64_t k);

/* Logits as a sampler takes them. For token v of a row, with c = how often it stands in
 * the generated part of the row's history:
 *   z = logits[v]
 *   z = z > 0 ? z / repetition : z * repetition     if v stands in the history at all
 *   z = z - (frequency * c + presence)               if c > 0
 *   z = z + the sum of v's biases
 *   z = -inf                                         if v is not allowed
 * In fp32, rounded once.
 *  - logits: rows x vocab of `dtype`; out: rows x vocab of `dtype` or fp32
 *    (out_dtype); out may be the logits.
 *  - tokens: rows x history, int64 (token_bytes 8) or int32 (4), ldt elements between
 *    rows; the first lengths[r] (NULL: history; taken as at least 0 and at most history) of
 *    row r count, of which the first prompt_lengths[r] (NULL: 0) are the prompt and the rest
 *    generated. A token outside [0, vocab) counts for nothing. history 0: no history.
 *  - repetition (not 0), frequency, presence: rows fp32, or NULL: 1, 0, 0.
 *  - bias_tokens (int64 or int32), bias_values (fp32): rows x biases, at most 1024; a
 *    token outside [0, vocab) is left out, one given twice gets both, added in their order.
 *  - allowed: rows x ceil(vocab / 32) words, lda words between rows; token v is allowed iff
 *    bit v % 32 of word v / 32 is set. NULL: all are. A row may allow nothing.
 *  - 0 <= rows < 2^31; 1 <= vocab < 2^31 - 4096; 0 <= history < 2^31 - 8192. */
int gemm_ws_adjust_logits(gemm_ws_t* h, int dtype, const void* logits, int64_t ldl, int out_dtype,
                          void* out, int64_t ldo, const void* tokens, int token_bytes, int64_t ldt,
                          int64_t history, const int32_t* lengths, const int32_t* prompt_lengths,
                          const float* repetition, const float* frequency, const float* presence,
                          const void* bias_tokens, int bias_token_bytes, int64_t ldb,
                          const float* bias_values, int64_t ldv, int64_t biases,
                          const uint32_t* allowed, int64_t lda, int64_t rows, int64_t vocab,
                          void* stream);

#ifdef __cplusplus
}
#endif

#endif /* GEMM_WS_LM_H_ */
