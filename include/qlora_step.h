/*
 * qlora_step.h -- C ABI of the operators that a decoder's training step and its step of an answer
 * need beside those of qlora_decoder.h: the norms around a block with its gate and residual
 * addition, the gradients' global norm and their clipping, attention over the paged cache with a
 * sliding window, and the penalties, biases and masks of logits.
 *
 * The library, its status codes, nf4_last_error() and the shared conventions (memory,
 * streams, errors before anything is enqueued, concurrency) are those of qlora_nf4.h.
 * No entry point throws, allocates device memory or synchronizes the host.
 */
#ifndef QLORA_STEP_H
#define QLORA_STEP_H

#include "qlora_decoder.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Rows in memory: [M][K], each row dense, `stride` values from one to the next.  What is only read may
 * repeat (a stride of 0 is one row for all); rows that are written may not share memory. */
typedef struct qlora_rows {
    void* data;
    int64_t stride;
} qlora_rows;

/* What lies between a block's output x and the next block's input y, on the stream h:
 *   n(a) = a / sqrt(mean(a^2) + eps)
 *   h' = h + scale * gate * (norm_post ? n(x) post : x)       y = n(h') pre
 * h' is rounded to the stream's type, and y is the norm of what was rounded.
 *   pre, post  device [K], or NULL for ones; pre only with norm_pre, post only with norm_post
 *   gate       device [gate_rows][K], or NULL for ones: row i belongs to the i-th M / gate_rows tokens (1: one gate for
 *              all; M: each token's own); gate_rows divides M
 *   dtype      of pre, post and gate
 *   scale      finite;  eps  2^-126 at least, and finite */
typedef struct qlora_block_norm {
    const void* pre;
    const void* post;
    const void* gate;
    int64_t gate_rows;
    int32_t norm_pre;
    int32_t norm_post;
    nf4_dtype dtype;
    float scale;
    float eps;
} qlora_block_norm;

/* Forward.  M tokens of width K, 0 <= M < 2^31, 1 <= K <= 32768.
 *   h       the stream, fp32 or bf16 (stream_dtype)
 *   x       bf16, the block's output; NULL: no block, and y = n(h) pre (norm_post, gate and h_out are then not given)
 *   h_out   with x: the stream after the block, of the stream's type; may be h itself (same pointer and stride)
 *   y       bf16, with norm_pre
 * Outputs may not share memory with anything else, which is refused (NF4_ERR_ARG); rows of several operands may lie side by
 * side in one buffer.  Any strides and alignments of whole values. */
nf4_status qlora_block_norm_fwd(const qlora_block_norm* norm, int64_t M, int64_t K, nf4_dtype stream_dtype,
                                const qlora_rows* h, const qlora_rows* x, const qlora_rows* h_out, const qlora_rows* y,
                                void* stream);

/* The gradient, from the operands of the forward pass alone.
 *   h       the stream after the block (the forward's h_out; h itself without a block); read with norm_pre
 *   x       the block's output, or NULL: no block (then no norm_post, gate or dx)
 *   dy      bf16, the gradient of y; with norm_pre
 *   dh      the gradient of the stream after the block from what comes later, of the stream's type, or NULL (zero)
 *   dh_out  out: the gradient of the stream before the block, of the stream's type; may be dh itself
 *   dx      out, with x: bf16, the gradient of the block's output
 *   dpre, dpost, dgate   out: fp32 [K], [K], [gate_rows][K], or NULL: sums over the tokens in a fixed order
 *   workspace  qlora_block_norm_bwd_workspace_bytes of the same sizes, 256-byte aligned: fp32 sums of up to 2048
 *              workers, each as long as the outputs asked for (of several gates two rows each)
 * Outputs and the workspace may not share memory with anything else, as in the forward call. */
size_t qlora_block_norm_bwd_workspace_bytes(int64_t M, int64_t K, int64_t gate_rows, int32_t need_dpre, int32_t need_dpost,
                                            int32_t need_dgate);
nf4_status qlora_block_norm_bwd(const qlora_block_norm* norm, int64_t M, int64_t K, nf4_dtype stream_dtype,
                                const qlora_rows* h, const qlora_rows* x, const qlora_rows* dy, const qlora_rows* dh,
                                const qlora_rows* dh_out, const qlora_rows* dx, float* dpre, float* dpost, float* dgate,
                                void* workspace, size_t workspace_bytes, void* stream);

/* A dense tensor of n values, fp32 or bf16, aligned to a value.  n of 0 is nothing (data may be NULL). */
typedef struct qlora_tensor {
    void* data;
    int64_t n;
    nf4_dtype dtype;
} qlora_tensor;

/* norm = sqrt(sum of the squares of all values), and the factor that clips it to max_norm:
 * factor = max_norm / norm if norm > max_norm, else 1 (a norm of infinity gives 0, of NaN NaN).  It is a fp32 number: norms of
 * more than 2^126 max_norm leave it fewer bits than a normal one has, and past 2^150 max_norm it is 0.
 * Squares are added in 64 bits in a fixed order.  A tensor given twice counts twice.
 *   norm, factor  device fp32; factor may be NULL (max_norm is not looked at then);  max_norm >= 0
 *   count         0 .. 2^24 (0: norm 0)
 *   workspace     qlora_grad_norm_workspace_bytes of the same tensors, 256-byte aligned */
size_t qlora_grad_norm_workspace_bytes(const qlora_tensor* grads, int64_t count);
nf4_status qlora_grad_norm(const qlora_tensor* grads, int64_t count, double max_norm, float* norm, float* factor,
                           void* workspace, size_t workspace_bytes, void* stream);

/* out[i] = factor * grads[i], each product rounded to the tensor's type, and the norm before.  out[i] may be grads[i]
 * itself (nothing is written then where the factor is 1); tensors that are written may not overlap any other.
 *   workspace     qlora_grad_clip_workspace_bytes of the same tensors, 256-byte aligned */
size_t qlora_grad_clip_workspace_bytes(const qlora_tensor* grads, int64_t count);
nf4_status qlora_grad_clip(const qlora_tensor* grads, const qlora_tensor* out, int64_t count, double max_norm, float* norm,
                           void* workspace, size_t workspace_bytes, void* stream);

/* nf4_adamw_step and nf4_adamw_step_paged with the gradient times a factor (device fp32, of qlora_grad_norm), which is
 * rounded to fp32 before the step; with a factor of 1 they give the same bits as those.  The factor lies apart from all
 * that is written (the state, p_bf16, the stage). */
nf4_status qlora_adamw_step_scaled(float* p, const float* g, float* m, float* v, uint16_t* p_bf16, int64_t n,
                                   float lr, float beta1, float beta2, float eps, float weight_decay,
                                   int64_t step, const float* factor, void* stream);
nf4_status qlora_adamw_step_paged_scaled(float* p_host, const float* g, float* m_host, float* v_host,
                                         uint16_t* p_bf16, int64_t n, float lr, float beta1, float beta2,
                                         float eps, float weight_decay, int64_t step, const float* factor, void* stage,
                                         size_t stage_bytes, void* stream);

/* qlora_kv_attention where a token at position p sees the keys j of 0 .. p with j > p - window or j < sinks.
 * Pages that none of the batch's tokens sees are not read: their table entries may be -1, and the pages given to others.
 * Precision, as for qlora_kv_attention: scores, maxima, sums and accumulators are fp32.  The weights of the softmax meet the
 * values in fp16, with 11 significant bits down to 2^-24 of a row's largest (outputs of the same inputs with weights of 22
 * bits differ by 7e-4 of their norm, most of it where the bf16 output rounds the other way).  Queries of sequences with many new
 * rows and heads of 128 and 256 meet the keys as the sum of two E4M3 numbers, exact down to 2^-14 of a query's largest value
 * and within 2^-23 of it below.
 *   window  1 .. 2^31 - 1;  sinks  0 .. 2^30;  everything else as for qlora_kv_attention (max_length is still the
 *           sequence's positions) */
size_t qlora_kv_attention_window_workspace_bytes(const qlora_kv_cache* cache, const qlora_kv_batch* batch, int32_t heads,
                                                 int64_t max_new, int64_t max_length, int64_t window, int64_t sinks);
nf4_status qlora_kv_attention_window(const qlora_kv_cache* cache, const qlora_kv_batch* batch, const qlora_heads* q,
                                     const qlora_heads* out, float scale, int64_t max_new, int64_t max_length,
                                     int64_t window, int64_t sinks, void* workspace, size_t workspace_bytes, void* stream);

/* What is done to logits before a token is chosen.  For row r and token v, in this order and in fp32:
 *   z / repetition if z > 0, else z * repetition   where v is among the row's tokens
 *   z - (frequency * count + presence)             where it is `count` > 0 times among those after the prompt
 *   z + bias                                       of the last entry of bias_ids that is v
 *   -inf                                           where bit v % 32 of word v / 32 of `allowed` is 0
 * Fields of NULL leave their step out.  What has a stride may be one row for all (a stride of 0).
 *   history       int32 [rows][history_width]: token i of a row counts for i < lengths[r] (NULL: all; held to
 *                 0 .. history_width), and as the prompt's for i < prompts[r] (NULL: none); tokens outside 0 .. V-1 are
 *                 passed over
 *   repetitions, presences, frequencies   fp32 [rows], or NULL: the one number beside them for all rows
 *   bias_ids, bias   int32 and fp32 [rows][biases]; ids outside 0 .. V-1 are unused
 *   allowed       int32 [rows][allowed_stride], at least ceil(V / 32) words a row */
typedef struct qlora_logit_rules {
    const int32_t* history;
    int64_t history_stride;
    int64_t history_width;
    const int32_t* lengths;
    const int32_t* prompts;
    float repetition;
    float presence;
    float frequency;
    const float* repetitions;
    const float* presences;
    const float* frequencies;
    const int32_t* bias_ids;
    int64_t bias_ids_stride;
    const float* bias;
    int64_t bias_stride;
    int64_t biases;
    const int32_t* allowed;
    int64_t allowed_stride;
} qlora_logit_rules;

/* logits and out: fp32 or bf16 [rows][V], rounded once; out may be the logits themselves (same pointer and stride),
 * and may share memory with nothing else (NF4_ERR_ARG).
 * 0 <= rows < 2^24, 1 <= V < 2^28; history_width and biases up to 2^31 - 2.  A repetition must be positive; one given as a
 * number is checked. */
nf4_status qlora_logits_shape(const qlora_logit_rules* rules, int64_t rows, int64_t V, nf4_dtype dtype,
                              const qlora_rows* logits, const qlora_rows* out, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* QLORA_STEP_H */
