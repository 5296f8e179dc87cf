/*
 * qlora_decoder.h -- C ABI of the operators around the QLoRA linears of a decoder:
 * rotary positions, a paged key/value cache of 8 bits with its append and its attention,
 * and the softmax cross entropy of the vocabulary head.
 *
 * The library, its status codes, nf4_last_error() and the shared conventions (memory,
 * streams, errors before anything is enqueued, concurrency) are those of qlora_nf4.h.
 * No entry point throws, allocates device memory or synchronizes the host.
 */
#ifndef QLORA_DECODER_H
#define QLORA_DECODER_H

#include "qlora_nf4.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Per-token heads in memory: [tokens][heads][head_dim], the last dimension dense, the
 * strides in elements (so that q, k and v may be slices of one projection's output).  What is
 * only read may repeat: a stride of 0 is one head, or token, for all.  Where a call writes them,
 * token follows token or head follows head without sharing memory. */
typedef struct qlora_heads {
    void* data;
    int64_t token_stride;
    int64_t head_stride;
    int32_t heads;
} qlora_heads;

/* A rotation: pair i of the first rotary_dim values of a head turns by
 * position * freq[i] / 2^64 whole turns (the product is taken modulo 2^64: whole turns
 * drop out, and a position of any size keeps its digits), and is multiplied by `magnitude`.
 *   pair i = (x[2i], x[2i+1]) if interleaved, else (x[i], x[i + rotary_dim/2])
 *   (a, b) -> magnitude * (a cos - b sin, a sin + b cos)
 * Values past rotary_dim stay as they are.  freq: device, rotary_dim / 2 entries. */
typedef struct qlora_rope {
    const int64_t* freq;
    int32_t rotary_dim;    /* even, 2 .. head_dim */
    int32_t interleaved;
    float magnitude;       /* finite */
} qlora_rope;

/* Rotates one or two tensors (the queries and the keys) of the same tokens in one launch,
 * in fp32 with one rounding at the end.  backward != 0 applies the transpose, which is the
 * gradient: the same pairs turned the other way, times the same magnitude.
 *   positions  device int32[M]
 *   in, out    `count` (1 or 2) tensors each; out[i] may be in[i] itself (same pointer and
 *              strides), and may not overlap it otherwise.  Any strides; 16-byte aligned
 *              rows take the fast path.
 *   head_dim   2 .. 512;  0 <= M < 2^24 (M == 0 enqueues nothing); up to 65536 heads in all */
nf4_status qlora_rope_apply(const qlora_rope* rope, int32_t backward, const int32_t* positions, int64_t M,
                            int32_t head_dim, nf4_dtype dtype, const qlora_heads* in, const qlora_heads* out,
                            int32_t count, void* stream);

/* A key/value cache in pages of `page_size` tokens, 8 bits a value:
 *   codes   [pages][2: key, value][kv_heads][page_size][head_dim] OCP E4M3 bytes, 16-byte aligned
 *   scales  [pages][2][kv_heads] fp32, each a power of two 2^e, -50 <= e <= 50;
 *           value = code * scale
 * head_dim 64, 128 or 256; page_size 16, 32, 64, 128 or 256; pages * kv_heads * 2 < 2^31. */
typedef struct qlora_kv_cache {
    uint8_t* codes;
    float* scales;
    int64_t pages;
    int32_t kv_heads;
    int32_t page_size;
    int32_t head_dim;
} qlora_kv_cache;

/* New tokens of `seqs` sequences, packed one sequence after the other.
 *   starts   device int32[seqs + 1], ascending: sequence b has tokens starts[b] ..
 *            starts[b+1] - 1 of the `tokens` packed ones (possibly none)
 *   lengths  device int32[seqs]: tokens of the sequence before these; token j of the
 *            sequence's new ones has position lengths[b] + j
 *   table    device int32[seqs][table_stride]: page of each page_size positions
 * starts[0] is 0 and starts[seqs] is `tokens` (starts that say otherwise give rows of no meaning,
 * but nothing outside the batch's tokens is read or written).  A token whose position is negative or past
 * the table's table_width pages is left out: not appended, and its attention is zero (a
 * negative length marks an unused row of a fixed batch).  An entry of the table outside the
 * pool (such as -1) is never followed: tokens there are not appended, and attention passes
 * over them.  tokens < 2^23, seqs < 65536. */
typedef struct qlora_kv_batch {
    const int32_t* starts;
    const int32_t* lengths;
    const int32_t* table;
    int64_t table_stride;
    int64_t tokens;
    int32_t seqs;
    int32_t table_width;
} qlora_kv_batch;

/* Appends keys and values to the cache, the keys rotated to their positions on the way
 * (rope == NULL: as they are), and rotates the queries of the same tokens in the same launch
 * (q_in == NULL: none).
 * Per page, head and kind, e is the smallest exponent of -50 .. 50 for which no new value
 * there, at any position, leaves +-448 * 2^e: the largest pair norm (of a rotated pair,
 * after the magnitude) or magnitude (else) decides, so the scale does not depend on the
 * positions.  A page that holds earlier tokens keeps max(e, its exponent), and if that
 * grows, its earlier codes are written again, rounded to nearest even, at the new scale.
 * Codes are the values divided by the scale, clamped to +-448, rounded to nearest even.
 * A token with a non-finite key or value in a head is stored there with NaN key codes and
 * zero value codes (whoever attends to it gets NaN, nobody else does) and has no part in
 * the scale.
 *   k, v    bf16 [tokens][kv_heads][head_dim], rows 16-byte aligned
 *   q_in, q_out  bf16 [tokens][heads][head_dim]; q_out may be q_in
 * The pages of these tokens must not be shared with another sequence. */
nf4_status qlora_kv_append(const qlora_kv_cache* cache, const qlora_kv_batch* batch, const qlora_heads* k,
                           const qlora_heads* v, const qlora_rope* rope, const qlora_heads* q_in,
                           const qlora_heads* q_out, void* stream);

/* Causal attention of the batch's tokens over the cache, which already holds them:
 *   out[t] = sum_j p_j v_j,  p = softmax_j(scale * q[t] . k_j),  j = 0 .. position of t
 * Head h of the queries reads kv head h / (heads / kv_heads).
 * Sums of queries times codes are held in fp32 before any scale is applied to them: queries up
 * to 2^110 in magnitude stay within it at any head size.
 * A query with a non-finite value that sees any key gives NaN.
 *   q, out      bf16 [tokens][heads][head_dim], rows 16-byte aligned; heads a multiple of kv_heads
 *   scale       of any sign, below 2^127 in magnitude (0: every key that is seen weighs the same)
 *   max_new     the most new tokens of one sequence (at least 1; more than `tokens` count as that), and
 *   max_length  the most positions of one sequence, new tokens included: they size the launch.
 *               Larger batches than they say are still computed, only slower; smaller ones than a
 *               max_length says cost workgroups without keys.
 *   seqs times kv_heads is 2^25 at most
 *   workspace   qlora_kv_attention_workspace_bytes of the same sizes, 256-byte aligned */
size_t qlora_kv_attention_workspace_bytes(const qlora_kv_cache* cache, const qlora_kv_batch* batch, int32_t heads,
                                          int64_t max_new, int64_t max_length);
nf4_status qlora_kv_attention(const qlora_kv_cache* cache, const qlora_kv_batch* batch, const qlora_heads* q,
                              const qlora_heads* out, float scale, int64_t max_new, int64_t max_length,
                              void* workspace, size_t workspace_bytes, void* stream);

/* Softmax cross entropy of a vocabulary head, z = X W^T, without fp32 logits in memory:
 *   loss[m] = log sum_v exp(z[m][v]) - z[m][targets[m]]
 *   dX = G W,  dW = G^T X,  G[m][v] = dloss[m] (softmax(z[m])[v] - [v == targets[m]])
 * A row whose target is ignore_index or lies outside 0 .. V-1 has loss 0 and no gradient, whatever
 * X, dloss (and, for its row of dX, W) hold: its row of dX is zero, and dW takes nothing from it.
 * A target's logit of -inf (an fp32 sum that overflows) has loss +inf; one of +inf, and any
 * logit of +inf or NaN, has loss NaN; the same with and without gradients.
 *   X        bf16 M x K, W bf16 V x K, both dense; K a multiple of 64, K < 2^20;
 *            0 <= M < 2^22, 1 <= V < 2^23, ceil(M/256) * ceil(V/256) < 2^23 - 8
 *   targets  device int64[M]
 *   dloss    device fp32[M], the gradient of each row's loss; only read when dX or dW is given
 *   loss     out: fp32[M], or NULL
 *   dX       out: bf16 M x K, or NULL;  dW  out: bf16 V x K, or NULL
 *   workspace  qlora_head_loss_workspace_bytes(M, K, V, dX != NULL, dW != NULL), 256-byte aligned.  With
 *              m = M up to a multiple of 512, and pieces of the vocabulary of v entries each (multiples of
 *              512, as many as 2 m v <= 2^27 holds, one at least, and no more than V asks for), it holds
 *                2 m K                     X in the order of the products,
 *                8 m ceil(v / 32) or less  statistics of the logits' tiles (without gradients v is V),
 *                2 m v                     exponentials of a piece, with dX or dW,
 *                4 M K c                   with dX, fp32 sums: c is 1, or up to 64 where the tiles of dX are so few that
 *                                          its contraction is cut into as many parts (and 0 where one piece and
 *                                          one part need none),
 *                2 M K                     with dW, X with its ignored rows zero,
 *              and with dW, where 2 m V (whole pieces) is 2^30 at most, every exponential in three bytes and a
 *              piece of G^T (3 m V + 2 m v in place of 2 m v): more than bf16 logits take.  Beyond, each
 *              piece's logits are computed a second time instead. */
size_t qlora_head_loss_workspace_bytes(int64_t M, int64_t K, int64_t V, int32_t need_dx, int32_t need_dw);
nf4_status qlora_head_loss(const void* X, int64_t M, int64_t K, const void* W, int64_t V, const int64_t* targets,
                           int64_t ignore_index, const float* dloss, float* loss, void* dX, void* dW,
                           void* workspace, size_t workspace_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* QLORA_DECODER_H */
