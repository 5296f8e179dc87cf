// decoder_api.hip -- the extern "C" entry points declared in include/qlora_decoder.h.
//
// Host side only: arguments are checked before any HIP call, then the kernels of rope.hip,
// kv_append.hip, kv_attention.hip and head_loss.hip are launched.
#include <math.h>

#include "../../include/qlora_decoder.h"
#include "decoder.h"
#include "attend_plan.h"
#include "status.h"

using nf4::aligned;
using nf4::BatchView;
using nf4::CacheView;
using nf4::fail;
using nf4::HeadsView;
using nf4::hip_status;
using nf4::RopeView;

namespace {

// Nothing may leave a C entry point but a status.
template <typename F>
nf4_status guarded(F&& f) noexcept {
    try {
        return f();
    } catch (...) {
        return NF4_ERR_HIP;   // out of host memory, for a message
    }
}

constexpr int64_t MAX_TOKENS = (int64_t)1 << 23;

nf4_status check_heads(const qlora_heads* x, const char* name, int32_t head_dim, int elem, bool rows16, HeadsView& v) {
    const std::string n(name);
    if (!x || !x->data) return fail(NF4_ERR_ARG, n + " is NULL");
    if (x->heads < 1 || x->heads > 65536) return fail(NF4_ERR_ARG, n + ": heads must be 1 .. 65536");
    if (x->token_stride < 0 || x->head_stride < 0) return fail(NF4_ERR_ARG, n + ": negative stride");
    if (x->heads > 1 && x->head_stride != 0 && x->head_stride < head_dim) return fail(NF4_ERR_ARG, n + ": heads overlap");
    if (!aligned(x->data, elem)) return fail(NF4_ERR_ARG, n + " is misaligned");
    if (rows16 && (!aligned(x->data, 16) || x->token_stride % 8 || x->head_stride % 8))
        return fail(NF4_ERR_ARG, n + ": rows must be 16-byte aligned");
    v = HeadsView{x->data, x->token_stride, x->head_stride, x->heads};
    return NF4_OK;
}

// Heads that a call writes: rows of different tokens or heads may not share memory.
nf4_status check_written(const qlora_heads* x, const char* name, int32_t head_dim, int64_t tokens) {
    const int64_t token = (x->heads - 1) * x->head_stride + head_dim, head = (tokens - 1) * x->token_stride + head_dim;
    const bool apart = tokens <= 1 || x->token_stride >= token ||                                    // token after token, or
                       (x->token_stride >= head_dim && (x->heads == 1 || x->head_stride >= head));   // head after head
    return apart && (x->heads == 1 || x->head_stride >= head_dim) ? NF4_OK : fail(NF4_ERR_ARG, std::string(name) + ": rows that are written overlap");
}

nf4_status check_rope(const qlora_rope* r, int32_t head_dim, RopeView& v) {
    if (!r) return fail(NF4_ERR_ARG, "rope is NULL");
    if (!r->freq || !aligned(r->freq, 8)) return fail(NF4_ERR_ARG, "freq is NULL or misaligned");
    if (r->rotary_dim < 2 || r->rotary_dim % 2 || r->rotary_dim > head_dim)
        return fail(NF4_ERR_ARG, "rotary_dim must be even, 2 .. head_dim");
    if (!isfinite(r->magnitude)) return fail(NF4_ERR_ARG, "magnitude must be finite");
    v = RopeView{r->freq, r->rotary_dim, r->interleaved ? 1 : 0, r->magnitude, 1.0f};
    return NF4_OK;
}

nf4_status check_cache(const qlora_kv_cache* c, CacheView& v) {
    if (!c) return fail(NF4_ERR_ARG, "cache is NULL");
    if (c->head_dim != 64 && c->head_dim != 128 && c->head_dim != 256)
        return fail(NF4_ERR_UNSUPPORTED, "head_dim must be 64, 128 or 256");
    int log2 = 4;
    while (log2 < 8 && (1 << log2) != c->page_size) ++log2;
    if ((1 << log2) != c->page_size) return fail(NF4_ERR_UNSUPPORTED, "page_size must be 16, 32, 64, 128 or 256");
    if (c->kv_heads < 1 || c->kv_heads > 4096) return fail(NF4_ERR_ARG, "kv_heads must be 1 .. 4096");
    if (c->pages < 1 || c->pages > (int64_t)0x7FFFFFFF / 2 / c->kv_heads)
        return fail(NF4_ERR_UNSUPPORTED, "pages must be at least 1, and pages * kv_heads * 2 below 2^31");
    if (!c->codes || !aligned(c->codes, 16)) return fail(NF4_ERR_ARG, "codes is NULL or not 16-byte aligned");
    if (!c->scales || !aligned(c->scales, 4)) return fail(NF4_ERR_ARG, "scales is NULL or misaligned");
    v = CacheView{c->codes, c->scales, c->pages, c->kv_heads, log2, c->head_dim};
    return NF4_OK;
}

nf4_status check_batch(const qlora_kv_batch* b, const CacheView& c, BatchView& v) {
    if (!b) return fail(NF4_ERR_ARG, "batch is NULL");
    if (b->tokens < 0 || b->tokens >= MAX_TOKENS) return fail(NF4_ERR_UNSUPPORTED, "tokens must be 0 .. 2^23 - 1");
    if (b->seqs < 0 || b->seqs > 65535) return fail(NF4_ERR_UNSUPPORTED, "seqs must be 0 .. 65535");
    if (b->tokens > 0 && b->seqs == 0) return fail(NF4_ERR_ARG, "tokens without sequences");
    if (b->table_width < 0 || b->table_stride < b->table_width) return fail(NF4_ERR_ARG, "table_stride below table_width");
    if (b->table_width > (0x7FFFFFFF >> c.page_log2)) return fail(NF4_ERR_UNSUPPORTED, "a sequence holds 2^31 positions or more");
    if (b->tokens > 0 && (!b->starts || !b->lengths || (!b->table && b->table_width > 0)))
        return fail(NF4_ERR_ARG, "starts, lengths or table is NULL");
    if (!aligned(b->starts, 4) || !aligned(b->lengths, 4) || !aligned(b->table, 4))
        return fail(NF4_ERR_ARG, "starts, lengths or table is misaligned");
    v = BatchView{b->starts, b->lengths, b->table, b->table_stride, (int)b->tokens, b->seqs, b->table_width};
    return NF4_OK;
}

}  // namespace

extern "C" {

nf4_status qlora_rope_apply(const qlora_rope* rope, int32_t backward, const int32_t* positions, int64_t M,
                            int32_t head_dim, nf4_dtype dtype, const qlora_heads* in, const qlora_heads* out,
                            int32_t count, void* stream) {
    return guarded([&]() -> nf4_status {
        if (dtype != NF4_F32 && dtype != NF4_BF16) return fail(NF4_ERR_ARG, "dtype must be NF4_F32 or NF4_BF16");
        if (head_dim < 2 || head_dim > nf4::ROPE_MAX_DIM) return fail(NF4_ERR_UNSUPPORTED, "head_dim must be 2 .. 512");
        if (count < 1 || count > 2) return fail(NF4_ERR_ARG, "count must be 1 or 2");
        if (M < 0 || M >= ((int64_t)1 << 24)) return fail(NF4_ERR_UNSUPPORTED, "M must be 0 .. 2^24 - 1");
        RopeView r;
        if (nf4_status st = check_rope(rope, head_dim, r)) return st;
        if (backward) r.sign = -1.0f;
        if (!in || !out) return fail(NF4_ERR_ARG, "in or out is NULL");
        if (M == 0) return NF4_OK;
        if (!positions || !aligned(positions, 4)) return fail(NF4_ERR_ARG, "positions is NULL or misaligned");
        HeadsView x[2], y[2];
        int64_t heads = 0;
        for (int i = 0; i < count; ++i) {
            const int elem = dtype == NF4_BF16 ? 2 : 4;
            if (nf4_status st = check_heads(in + i, "in", head_dim, elem, false, x[i])) return st;
            if (nf4_status st = check_heads(out + i, "out", head_dim, elem, false, y[i])) return st;
            if (nf4_status st = check_written(out + i, "out", head_dim, M)) return st;
            if (x[i].heads != y[i].heads) return fail(NF4_ERR_ARG, "in and out have different heads");
            if (x[i].data == y[i].data && (x[i].token_stride != y[i].token_stride || x[i].head_stride != y[i].head_stride))
                return fail(NF4_ERR_ARG, "in place needs the same strides");
            heads += x[i].heads;
        }
        if (count == 2 && y[0].data == y[1].data) return fail(NF4_ERR_ARG, "out: both tensors are the same");
        if (heads > 65536) return fail(NF4_ERR_UNSUPPORTED, "more than 65536 heads");
        return hip_status(nf4::launch_rope(r, positions, M, head_dim, dtype == NF4_BF16, x, y, count, (hipStream_t)stream),
                          "qlora_rope_apply");
    });
}

nf4_status qlora_kv_append(const qlora_kv_cache* cache, const qlora_kv_batch* batch, const qlora_heads* k,
                           const qlora_heads* v, const qlora_rope* rope, const qlora_heads* q_in,
                           const qlora_heads* q_out, void* stream) {
    return guarded([&]() -> nf4_status {
        CacheView c;
        BatchView b;
        if (nf4_status st = check_cache(cache, c)) return st;
        if (nf4_status st = check_batch(batch, c, b)) return st;
        RopeView r{nullptr, 0, 0, 1.0f, 1.0f};
        if (rope)
            if (nf4_status st = check_rope(rope, c.dim, r)) return st;
        if (b.tokens == 0) return NF4_OK;
        HeadsView kv, vv, qi, qo;
        if (nf4_status st = check_heads(k, "k", c.dim, 2, true, kv)) return st;
        if (nf4_status st = check_heads(v, "v", c.dim, 2, true, vv)) return st;
        if (kv.heads != c.heads || vv.heads != c.heads) return fail(NF4_ERR_ARG, "k and v must have the cache's heads");
        if ((q_in != nullptr) != (q_out != nullptr)) return fail(NF4_ERR_ARG, "q_in and q_out go together");
        if (q_in) {
            if (nf4_status st = check_heads(q_in, "q_in", c.dim, 2, true, qi)) return st;
            if (nf4_status st = check_heads(q_out, "q_out", c.dim, 2, true, qo)) return st;
            if (nf4_status st = check_written(q_out, "q_out", c.dim, b.tokens)) return st;
            if (qi.heads != qo.heads) return fail(NF4_ERR_ARG, "q_in and q_out have different heads");
            if (qi.data == qo.data && (qi.token_stride != qo.token_stride || qi.head_stride != qo.head_stride))
                return fail(NF4_ERR_ARG, "in place needs the same strides");
        }
        // one launch of fewer than 2^24 workgroups
        const int64_t most = (int64_t)b.tokens * ((c.heads + 3) / 4) + (q_in ? ((int64_t)b.tokens + 4096) * ((qi.heads * (int64_t)c.dim + 2047) / 2048) : 0);
        if (most >= ((int64_t)1 << 24)) return fail(NF4_ERR_UNSUPPORTED, "too many tokens times heads for one call");
        return hip_status(nf4::launch_kv_append(c, b, kv, vv, r, q_in ? &qi : nullptr, q_in ? &qo : nullptr, (hipStream_t)stream),
                          "qlora_kv_append");
    });
}

static nf4_status check_attention(const qlora_kv_cache* cache, const qlora_kv_batch* batch, int32_t heads,
                                  int64_t max_new, int64_t max_length, CacheView& c, BatchView& b) {
    if (nf4_status st = check_cache(cache, c)) return st;
    if (nf4_status st = check_batch(batch, c, b)) return st;
    if (heads < 1 || heads > 65536 || heads % c.heads) return fail(NF4_ERR_ARG, "heads must be a multiple of the cache's, 65536 at most");
    if (max_new < 1 || max_length < 1) return fail(NF4_ERR_ARG, "max_new and max_length must be at least 1");
    if (max_new >= MAX_TOKENS || max_length > (int64_t)0x7FFFFFFF) return fail(NF4_ERR_UNSUPPORTED, "max_new or max_length too large");
    if ((int64_t)b.seqs * c.heads > nf4::ATTEND_PAIRS) return fail(NF4_ERR_UNSUPPORTED, "seqs times kv_heads must not pass 2^25");
    if (max_new * (heads / c.heads) >= ((int64_t)1 << 30)) return fail(NF4_ERR_UNSUPPORTED, "max_new times heads per key head too large");
    return NF4_OK;
}

size_t qlora_kv_attention_workspace_bytes(const qlora_kv_cache* cache, const qlora_kv_batch* batch, int32_t heads,
                                          int64_t max_new, int64_t max_length) {
    size_t bytes = 0;
    guarded([&]() -> nf4_status {
        CacheView c;
        BatchView b;
        if (nf4_status st = check_attention(cache, batch, heads, max_new, max_length, c, b)) return st;
        bytes = b.tokens > 0 ? nf4::kv_attention_ws_bytes(c, b, heads, max_new, max_length) : 0;
        return NF4_OK;
    });
    return bytes;
}

nf4_status qlora_kv_attention(const qlora_kv_cache* cache, const qlora_kv_batch* batch, const qlora_heads* q,
                              const qlora_heads* out, float scale, int64_t max_new, int64_t max_length,
                              void* workspace, size_t workspace_bytes, void* stream) {
    return guarded([&]() -> nf4_status {
        CacheView c;
        BatchView b;
        if (!q || !out) return fail(NF4_ERR_ARG, "q or out is NULL");
        if (nf4_status st = check_attention(cache, batch, q->heads, max_new, max_length, c, b)) return st;
        if (!(fabsf(scale) < 0x1p127f)) return fail(NF4_ERR_ARG, "scale must be below 2^127");
        if (b.tokens == 0) return NF4_OK;
        HeadsView qv, ov;
        if (nf4_status st = check_heads(q, "q", c.dim, 2, true, qv)) return st;
        if (nf4_status st = check_heads(out, "out", c.dim, 2, true, ov)) return st;
        if (nf4_status st = check_written(out, "out", c.dim, b.tokens)) return st;
        if (qv.heads != ov.heads) return fail(NF4_ERR_ARG, "q and out have different heads");
        if ((int64_t)b.tokens * qv.heads >= ((int64_t)1 << 26)) return fail(NF4_ERR_UNSUPPORTED, "tokens times heads must be below 2^26");
        const size_t need = nf4::kv_attention_ws_bytes(c, b, qv.heads, max_new, max_length);
        if (need > 0 && (!workspace || workspace_bytes < need)) return fail(NF4_ERR_WORKSPACE, "workspace missing or too small");
        if (need > 0 && !aligned(workspace, 256)) return fail(NF4_ERR_ARG, "workspace must be 256-byte aligned");
        return hip_status(nf4::launch_kv_attention(c, b, qv, ov, scale, max_new, max_length, workspace, (hipStream_t)stream),
                          "qlora_kv_attention");
    });
}

static nf4_status check_head(int64_t M, int64_t K, int64_t V) {
    if (M < 0 || K < 1 || V < 1) return fail(NF4_ERR_ARG, "M must be >= 0, K and V at least 1");
    if (K % 64 || K >= ((int64_t)1 << 20)) return fail(NF4_ERR_UNSUPPORTED, "K must be a multiple of 64 below 2^20");
    if (M >= ((int64_t)1 << 22) || V >= ((int64_t)1 << 23) || ((M + 255) / 256) * ((V + 255) / 256) >= ((int64_t)1 << 23) - 8)
        return fail(NF4_ERR_UNSUPPORTED, "M must be below 2^22, V below 2^23, ceil(M/256) * ceil(V/256) below 2^23 - 8");
    return NF4_OK;
}

size_t qlora_head_loss_workspace_bytes(int64_t M, int64_t K, int64_t V, int32_t need_dx, int32_t need_dw) {
    size_t bytes = 0;
    guarded([&]() -> nf4_status {
        if (nf4_status st = check_head(M, K, V)) return st;
        bytes = M > 0 ? nf4::head_loss_ws_bytes(M, K, V, need_dx != 0, need_dw != 0) : 0;
        return NF4_OK;
    });
    return bytes;
}

nf4_status qlora_head_loss(const void* X, int64_t M, int64_t K, const void* W, int64_t V, const int64_t* targets,
                           int64_t ignore_index, const float* dloss, float* loss, void* dX, void* dW,
                           void* workspace, size_t workspace_bytes, void* stream) {
    return guarded([&]() -> nf4_status {
        if (nf4_status st = check_head(M, K, V)) return st;
        if (dW && !aligned(dW, 16)) return fail(NF4_ERR_ARG, "dW must be 16-byte aligned");
        if (M == 0) {
            if (!dW) return NF4_OK;   // no tokens: no gradient
            return hip_status(nf4::launch_head_zero((uint16_t*)dW, V * K, (hipStream_t)stream), "qlora_head_loss");
        }
        if (!X || !W || !targets) return fail(NF4_ERR_ARG, "X, W or targets is NULL");
        if (!loss && !dX && !dW) return fail(NF4_ERR_ARG, "nothing to compute: loss, dX and dW are NULL");
        if ((dX || dW) && !dloss) return fail(NF4_ERR_ARG, "dX and dW need dloss");
        if (!aligned(X, 16) || !aligned(W, 16) || !aligned(dX, 16)) return fail(NF4_ERR_ARG, "X, W and dX must be 16-byte aligned");
        if (!aligned(targets, 8) || !aligned(dloss, 4) || !aligned(loss, 4))
            return fail(NF4_ERR_ARG, "targets, dloss or loss is misaligned");
        const size_t need = nf4::head_loss_ws_bytes(M, K, V, dX != nullptr, dW != nullptr);
        if (!workspace || workspace_bytes < need) return fail(NF4_ERR_WORKSPACE, "workspace missing or too small");
        if (!aligned(workspace, 256)) return fail(NF4_ERR_ARG, "workspace must be 256-byte aligned");
        return hip_status(nf4::launch_head_loss((const uint16_t*)X, M, K, (const uint16_t*)W, V, targets, ignore_index, dloss,
                                                loss, (uint16_t*)dX, (uint16_t*)dW, workspace, (hipStream_t)stream),
                          "qlora_head_loss");
    });
}

}  // extern "C"
