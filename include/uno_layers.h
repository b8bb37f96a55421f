/*
 * uno_layers.h — C ABI of the operators around the Uno hot path on NVIDIA B200 (sm_100a):
 * an 8-bit frozen base under the gated LoRA projections, and what a step reports about its
 * tokens or trains on. Same library (libuno.so), conventions, status codes and error string
 * as uno.h.
 *
 *   uno_rms_norm_fp8           residual addition, RMS norm, e4m3 values with block scales
 *   uno_fp8_quantize           e4m3 values with block scales of weights and activations
 *   uno_fp8_gated_lora_linear  the row-gated LoRA projection on an e4m3 base weight
 *   uno_token_logprobs         log probabilities of given tokens, entropy, top alternatives
 *   uno_token_logprobs_grad    their gradient with respect to the logits
 *
 * The 8-bit format. A value is e4m3 (1-4-3, finite, largest 448; one byte). Scales are
 * float32. A matrix [rows, cols] held by 1 x 128 blocks has scales [rows, ceil(cols / 128)];
 * held by 128 x 128 blocks it has scales [ceil(rows / 128), ceil(cols / 128)]; the last
 * blocks may be short. An element stands for value * scale. With a = max |x| of a block:
 *   scale = max(a / 448, 2^-126)        (a float32)
 *   value = e4m3(448 x / a)             (one rounding to nearest, ties to even; with the
 *                                        smallest scale: x / scale)
 * A NaN stays a NaN; a block that holds an infinity comes out as NaN.
 *
 * All calls: device pointers 16-byte aligned, tensors contiguous; outputs may not overlap
 * inputs except where a comment says so. M = 0 or N = 0 launches nothing.
 */
#ifndef UNO_LAYERS_H
#define UNO_LAYERS_H

#include "uno.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ======================================================================================
 * RMS norm with the residual's addition and an 8-bit output
 *
 *   h = x + residual          (rounded to dtype; x itself without a residual)
 *   y = h * weight / sqrt(mean(h^2) + eps)                       per row
 *   out_q, out_scale = y by 1 x 128 blocks (the values from h * weight: a row's factor is
 *                      in its scales and cancels in its values)
 *
 *   x, residual [M, d] dtype (bf16 or f32); residual may be NULL
 *   weight      [d] dtype
 *   out_residual[M, d] dtype or NULL: h; may be x or residual itself
 *   out_q       [M, d] e4m3, out_scale [M, ceil(d/128)] float32; both or neither
 *   out_y       [M, d] dtype or NULL: y rounded to dtype (what an adapter reads)
 *
 * Sums of squares in float32; a row whose sum passes its range comes out as NaN. bf16 rows hold
 * the products h * weight in float32: one below 2^-126 in size keeps fewer bits, one above its
 * range is infinite (float32 rows hold them in float64).
 * Limits (else UNO_ERR_UNSUPPORTED): d a multiple of 16, d <= 32768, M < 2^31. eps positive and
 * finite; out_q or out_y has to be given; out_residual needs residual. No workspace.
 * ====================================================================================== */
uno_status uno_rms_norm_fp8(const void* x, const void* residual, const void* weight, uno_dtype dtype, int64_t M,
                            int64_t d, float eps, void* out_residual, void* out_q, float* out_scale, void* out_y,
                            uno_stream_t stream);

/* ======================================================================================
 * 8-bit values and block scales of a matrix
 *
 *   x          [rows, cols] dtype (bf16 or f32)
 *   block_rows 1 (activations) or 128 (weights): blocks of block_rows x 128
 *   out_q      [rows, cols] e4m3, out_scale [ceil(rows/block_rows), ceil(cols/128)] float32
 *
 * Limits (else UNO_ERR_UNSUPPORTED): cols a multiple of 16, rows and cols < 2^31.
 * No workspace.
 * ====================================================================================== */
uno_status uno_fp8_quantize(const void* x, uno_dtype dtype, int64_t rows, int64_t cols, int32_t block_rows,
                            void* out_q, float* out_scale, uno_stream_t stream);

/* ======================================================================================
 * Row-gated LoRA linear on an 8-bit base
 *
 *   Y = (x_q x_scale) (w_q w_scale)^T + scale * diag(g) (X A^T) B^T
 *
 * uno_gated_lora_linear with the frozen weight and the activations it multiplies held in
 * e4m3; the adapter reads the bf16 activations and stays bf16.
 *
 *   x_q     [M, d_in] e4m3, x_scale [M, ceil(d_in/128)] float32        (1 x 128 blocks)
 *   w_q     [d_out, d_in] e4m3, w_scale [ceil(d_out/128), ceil(d_in/128)]  (128 x 128)
 *   rank    0: no adapter (x, lora_a, lora_b, row_gate are not read and may be NULL)
 *   x       [M, d_in] bf16, lora_a [rank, d_in] bf16, lora_b [d_out, rank] bf16
 *   row_gate[M] float32; NULL means all zeros (base layer only)
 *   y       [M, d_out] y_dtype (bf16; or f32 without an adapter)
 *
 * Arithmetic: each block of 128 columns is one tensor-core product of e4m3 values with
 * float32 accumulation, multiplied by its two scales and summed in float32. (The product of the
 * two scales is a float32 too: below 2^-126 it keeps fewer bits, above the range it is
 * infinite.) The adapter's
 * X A^T is accumulated in float32 and rounded once to bf16; its product with B is
 * accumulated in float32 and multiplied by scale * g. A row whose scale * g is 0 gets no
 * adapter term. Y is rounded once to y_dtype. Sums are taken in an order fixed by the sizes.
 *
 * Limits (else UNO_ERR_UNSUPPORTED): d_in a multiple of 16, d_in <= 65536; d_out <= 2^20;
 * M <= 2^20; rank 0 or a multiple of 8 up to 256; y_dtype UNO_F32 only with rank 0; output tiles
 * of 128 x 256 (few rows: 128 x 128) times blocks of 128 columns below 2^31.
 * Workspace: uno_fp8_gated_lora_linear_workspace_size bytes (0 with rank 0: may be NULL).
 * ====================================================================================== */
size_t uno_fp8_gated_lora_linear_workspace_size(int64_t M, int64_t d_in, int64_t d_out, int64_t rank);

uno_status uno_fp8_gated_lora_linear(const void* x_q, const float* x_scale, const void* w_q, const float* w_scale,
                                     const void* x, const void* lora_a, const void* lora_b, const float* row_gate,
                                     float scale, int64_t M, int64_t d_in, int64_t d_out, int64_t rank, void* y,
                                     uno_dtype y_dtype, void* workspace, size_t workspace_bytes,
                                     uno_stream_t stream);

/* ======================================================================================
 * Log probabilities of given tokens, entropy and the most probable alternatives
 *
 *   l[n, v] = logits[n, v] / temperature - log sum_w exp(logits[n, w] / temperature)
 *   out_logprob[n]  = l[n, tokens[n]]
 *   out_entropy[n]  = - sum_v exp(l[n, v]) l[n, v]                   (nats)
 *   out_top_ids[n], out_top_logprobs[n] = the top_n most probable tokens, by value
 *                     descending, equal values by id ascending
 *   out_stats[n]    = (max_v logits[n, v], log sum_v exp((logits[n, v] - max) / temperature)),
 *                     what the gradient needs
 *
 *   logits  [N, V] dtype (bf16 or f32); -inf marks a token that cannot be produced
 *   tokens  [N] int32 or NULL. A row whose token is not in [0, V) is left out (padding,
 *           positions behind an accepted prefix): its logits are not read, its log
 *           probability, entropy and stats are 0, its alternatives (-1, -inf). With NULL
 *           every row is taken and out_logprob has to be NULL.
 *   top_n   0 to 32; places beyond the tokens that can be produced hold (-1, -inf)
 *   Every output but one may be NULL; out_top_ids and out_top_logprobs [N, top_n] are given
 *   exactly when top_n > 0. out_logprob, out_entropy [N], out_stats [N, 2] float32.
 *
 * A row of nothing but -inf has log probability -inf, entropy 0, stats (-inf, 0) and no
 * alternatives. NaN and +inf logits make their row's numbers unspecified (NaN as a rule).
 * Finite logits may be of any size; a log probability beyond float32 is -inf. No log
 * probability is above 0 and no entropy below.
 * Limits: 1 <= V < 2^31 - 4096, N * V < 2^40, N < 2^31; temperature finite and at least
 * 1e-30. No workspace.
 * ====================================================================================== */
uno_status uno_token_logprobs(const void* logits, uno_dtype dtype, int64_t N, int64_t V, float temperature,
                              const int32_t* tokens, int32_t top_n, float* out_logprob, float* out_entropy,
                              float* out_stats, int32_t* out_top_ids, float* out_top_logprobs, uno_stream_t stream);

/* ======================================================================================
 * Gradient of the log probabilities and entropies
 *
 *   grad_logits[n, v] = ( grad_logprob[n] (1[v = tokens[n]] - p_v)
 *                         - grad_entropy[n] p_v (l[n, v] + entropy[n]) ) / temperature
 *   with p = exp(l); 0 on rows that are left out and on rows of nothing but -inf. A p below
 *   2^-126 counts as 0.
 *
 *   logits, tokens, temperature: as given to uno_token_logprobs
 *   stats        [N, 2], entropy [N]: its out_stats and out_entropy
 *   grad_logprob [N] float32 or NULL (zeros); needs tokens
 *   grad_entropy [N] float32 or NULL (zeros); needs entropy. At least one of the two.
 *   grad_logits  [N, V] dtype; may be logits itself
 * Limits as for uno_token_logprobs; |grad_entropy| / temperature up to 1e36 (beyond it a token's
 * gradient may be NaN). No workspace.
 * ====================================================================================== */
uno_status uno_token_logprobs_grad(const void* logits, uno_dtype dtype, int64_t N, int64_t V, float temperature,
                                   const int32_t* tokens, const float* stats, const float* entropy,
                                   const float* grad_logprob, const float* grad_entropy, void* grad_logits,
                                   uno_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* UNO_LAYERS_H */
