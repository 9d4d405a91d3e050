/*
 * lp_head.h — C ABI of the operators a served model's head needs around the ragged
 * log-probability path of lp_ragged.h: the final norm (with the residual's addition and
 * an 8-bit output), the vocabulary projection with low-rank adapters, and the processing
 * of logits (repetition, frequency and presence penalties, biases, grammar masks).
 *
 *     hidden -> lp_head_norm -> lp_head_project -> lp_head_process -> lp_ragged_step
 *
 * Conventions are those of lp_ragged.h: the caller owns every buffer and the stream, the
 * library allocates nothing, LP_OK means "validated and enqueued", host-checked errors
 * leave nothing enqueued, and errors found on the device set bits of the workspace's
 * status word (bit c <=> code c; read it with lp_ragged_read_status) and never trap.
 * These entry points only ever add bits: lp_head_clear_status (or lp_ragged_plan on the
 * same workspace) clears the word. Workspaces are aligned to 256 bytes, every other pointer to
 * its type at least (else LP_ERR_SHAPE). Strides are in elements. Row counts, sizes and ids are
 * uint32; row strides and totals may pass 32 bits.
 */
#ifndef LP_HEAD_H
#define LP_HEAD_H

#include "lp_ragged.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef enum lp_dtype {
    LP_F32 = 0,
    LP_BF16 = 1,
    LP_F16 = 2,
    LP_E4M3 = 3 /* 8 bits: 4 exponent, 3 mantissa, largest value 448, no infinity */
} lp_dtype;

#define LP_MAX_HIDDEN 32768u /* widest row of lp_head_norm */
#define LP_MIN_REPETITION 9.5367432e-07f /* 2^-20 */
#define LP_MAX_REPETITION 1048576.0f     /* 2^20 */
#define LP_MAX_RANK 64u      /* largest adapter rank of lp_head_project */

/*
 * Bytes of scratch the calls below need: a 256-byte header with the status word, and for
 * lp_head_project with adapters, u of every row in f32 and as 16-bit parts, and a list of its
 * adapters for every 32 rows.
 * lp_head_norm only uses the header (T = rank = 0); lp_head_process has a size of its own.
 */
size_t lp_head_workspace_size(uint32_t T, uint32_t rank);

/* Enqueue the clearing of a workspace's status word. */
lp_status lp_head_clear_status(void *workspace, lp_stream_t stream);

/*
 * Final norm. For output row o, with i = rows ? rows[o] : o,
 *     h = x[i] + residual[i]                      (f32; h = x[i] without a residual)
 *     y = h / sqrt(mean(h^2) + eps) * weight      (f32)
 *     out[o] = y rounded to out_dtype, or for LP_E4M3
 *     out_scale[o] = max(max|y| / 448, 2^-126),  out[o] = e4m3(y / out_scale[o])
 *                    (y times the rounded reciprocal: a value next to the middle of two
 *                    codes may take the other one)
 *     residual_out[o] = h rounded to dtype        (optional)
 * The norm reads h before its rounding.
 *   x, residual     device, [T][H] of dtype (LP_F32, LP_BF16, LP_F16); residual may be NULL
 *   weight          device, [H] of weight_dtype (dtype or LP_F32)
 *   rows, n         device, uint32[n], the rows to take, or NULL (then n must equal T)
 *   out             device out, [n][H] of out_dtype (dtype, LP_F32 or LP_E4M3)
 *   out_scale       device out, float[n], for LP_E4M3 only
 *   residual_out    device out, [n][H] of dtype, or NULL. Without rows, out and
 *                   residual_out may be x or residual themselves (same type and stride);
 *                   otherwise outputs and inputs lie apart (LP_ERR_SHAPE where they begin
 *                   at one place)
 *   workspace       the status word; required with rows, else may be NULL
 * A row holding NaN or an infinity becomes NaN where the formula does (LP_E4M3: the row's
 * scale is NaN). Only h, y and out_scale have to fit f32, not h^2 or its sum. Device check: rows[o] < T (LP_ERR_OFFSETS; that output row gets NaN).
 * Host checks: H in 1..LP_MAX_HIDDEN, strides >= H, pointers aligned to their type.
 */
lp_status lp_head_norm(const void *x, const void *residual, const void *weight, uint32_t dtype,
                       uint32_t weight_dtype, uint32_t T, uint32_t H, uint64_t x_stride, uint64_t residual_stride,
                       const uint32_t *rows, uint32_t n, float eps, void *out, uint32_t out_dtype,
                       uint64_t out_stride, float *out_scale, void *residual_out, uint64_t residual_out_stride,
                       void *workspace, size_t workspace_bytes, lp_stream_t stream);

/*
 * Projection of hidden states to logits, with low-rank adapters of many requests at once:
 *     out[t, v] = sx[t] sw[v] sum_h x[t, h] W[v, h]  +  sum_j u[t, j] B_a[v, j]
 *     u[t, j]   = s_a sx[t] sum_h x[t, h] A_a[j, h]
 * with a = adapter_ids[b] for the request b of row t (rows as in lp_head_process); a
 * negative id means no adapter. Products are exact and sums f32: on the tensor cores, whose
 * f32 sums drop what is below their last place, for f32 logits of 16-bit inputs over 768
 * products at most at a time, which are added with rounding, else over all of H. u is a f32
 * sum that enters the second product with its 24 bits (or, LP_F16 adapters on the tensor
 * cores, to 2^-38 of the row's largest). The result is rounded once to out_dtype.
 *   x               device, [T][H] of dtype (LP_BF16, LP_F16, LP_E4M3)
 *   x_scale         device, float[T], sx, for LP_E4M3 only (else NULL, and sx = 1)
 *   weight          device, [V][H] of dtype; weight_scale: device, float[V], as x_scale
 *   lora_a, lora_b  device, [adapters][rank][H] and [adapters][V][rank], contiguous, of
 *                   lora_dtype: dtype, or LP_BF16 / LP_F16 where dtype is LP_E4M3
 *   adapters        0: no adapters (the lora arguments, ids and offsets are not read)
 *   adapter_scale   device, float[adapters], s_a, or NULL (1)
 *   adapter_ids     device, int32[B]
 *   row_offsets, B  device, uint32[B+1], or NULL (request t has row t, B == T)
 *   out             device out, [T][V] of out_dtype (LP_F32, LP_BF16, LP_F16)
 *   workspace       lp_head_workspace_size(T, rank) bytes (T = rank = 0 without adapters)
 * Requests may hold adapters in any order; rows of one adapter that stand together share
 * its B. Host checks: 1 <= rank <= LP_MAX_RANK; x, weight, lora_a, lora_b 16-byte aligned;
 * H and the strides of x and weight whole multiples of 16 bytes. Device checks: every row
 * in a request (LP_ERR_OFFSETS), ids below `adapters` (LP_ERR_ADAPTER); such a row's
 * logits are NaN. LP_ERR_TIMEOUT: a wait inside the kernel ran out (out is not complete).
 */
lp_status lp_head_project(const void *x, uint32_t dtype, uint32_t T, uint32_t H, uint64_t x_stride,
                          const float *x_scale, const void *weight, uint32_t V, uint64_t weight_stride,
                          const float *weight_scale, const void *lora_a, const void *lora_b, uint32_t lora_dtype,
                          uint32_t adapters, uint32_t rank, const float *adapter_scale, const int32_t *adapter_ids,
                          const uint32_t *row_offsets, uint32_t B, void *out, uint32_t out_dtype, uint64_t out_stride,
                          void *workspace, size_t workspace_bytes, lp_stream_t stream);

/*
 * How lp_head_project cuts a product of these sizes on a device of `sms` SMs (0: the current
 * one's), for diagnostics: *ctas = 1 or 2 (a pair) to a tile, *rows = rows of x in a tile,
 * *on_tensor_cores = 1 where the adapters of 32 neighbouring rows that have one or two are
 * multiplied there (0: all by the epilogue). adapters, rank: 0 without.
 */
lp_status lp_head_project_cut(uint32_t T, uint32_t H, uint32_t V, uint32_t dtype, uint32_t adapters, uint32_t rank,
                              uint32_t sms, uint32_t *ctas, uint32_t *rows, uint32_t *on_tensor_cores);

/*
 * Processing of logits. Logits row t belongs to the request b with
 * row_offsets[b] <= t < row_offsets[b+1] (row_offsets NULL: request t, B == T). With
 * `seen` = the token is in the request's history, `count` = how often it is in the
 * history's output part, every value becomes, in f32 and in this order,
 *     x = seen ? (x > 0 ? x / repetition[b] : x * repetition[b]) : x   (x / r as x times
 *                                                                       the rounded 1 / r)
 *     x = x - frequency[b] * count - (count > 0 ? presence[b] : 0)
 *     x = x + bias                                  (tokens of the request's bias list)
 *     x = -inf                                      (tokens whose mask bit is 0)
 *   logits          device, [T][V] of dtype (LP_F32, LP_BF16, LP_F16)
 *   out             device out, float[T][V]; may be logits itself for LP_F32 (same stride)
 *   history         device, uint32[history_total]; request b's part is
 *   history_offsets device, uint32[B+1]; its first prompt_lens[b] tokens are the prompt
 *   prompt_lens     device, uint32[B], or NULL (no prompt)
 *   repetition, frequency, presence   device, float[B] each, or NULL (1, 0, 0)
 *   bias_tokens, bias_values, bias_offsets   device, uint32[bias_total], float[bias_total],
 *                   uint32[B+1]: request b's biases, token ids strictly ascending; NULL: none
 *   mask            device, uint32[mask_rows][mask_stride], bit v % 32 of word v / 32 is 1
 *                   where token v is allowed; NULL: none
 *   mask_index      device, int32[T]: row t's mask row, negative: row t is not masked;
 *                   NULL: row t has mask row t (mask_rows >= T)
 *   workspace       lp_head_process_workspace_size(B, history_total) bytes: the status word
 *                   and, for histories of some thousand tokens, room to sort them. The size
 *                   grows with both, so that the largest call's workspace serves them all
 * A row whose mask allows nothing is all -inf. A masked value is -inf whatever it was.
 * The history of a request with repetition 1 and frequency = presence = 0 is not read.
 * Device checks: the row, history and bias offsets as a whole nondecreasing and within T and
 * their totals (LP_ERR_OFFSETS; a row gets NaN if it is in no request, or if its own request's
 * list of tokens or biases is wrong), mask_index < mask_rows (LP_ERR_OFFSETS, NaN); repetition within LP_MIN_REPETITION ... LP_MAX_REPETITION, frequency and
 * presence finite (LP_ERR_PENALTY, NaN). A history or bias token >= V is skipped (LP_ERR_TOKEN_RANGE), bias
 * ids not strictly ascending set LP_ERR_OFFSETS (that request's biases are unspecified).
 */
size_t lp_head_process_workspace_size(uint32_t B, uint32_t history_total);

lp_status lp_head_process(const void *logits, uint32_t dtype, uint32_t T, uint32_t V, uint64_t stride,
                          const uint32_t *row_offsets, uint32_t B, const uint32_t *history,
                          const uint32_t *history_offsets, uint32_t history_total, const uint32_t *prompt_lens,
                          const float *repetition, const float *frequency, const float *presence,
                          const uint32_t *bias_tokens, const float *bias_values, const uint32_t *bias_offsets,
                          uint32_t bias_total, const uint32_t *mask, uint64_t mask_stride, uint32_t mask_rows,
                          const int32_t *mask_index, float *out, uint64_t out_stride, void *workspace,
                          size_t workspace_bytes, lp_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* LP_HEAD_H */
