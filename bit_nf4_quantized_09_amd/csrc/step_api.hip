// step_api.hip -- the extern "C" entry points declared in include/qlora_step.h, but for those whose kernels
// serve another header's entry too (attention: decoder_api.hip, AdamW: api.hip).
//
// Host side only: arguments are checked before any HIP call, then the kernels of block_norm.hip, gradients.hip and
// logits.hip are launched.
#include <math.h>

#include <algorithm>
#include <initializer_list>
#include <string>
#include <vector>

#include "../../include/qlora_step.h"
#include "overlap.h"
#include "status.h"
#include "step.h"

using nf4::aligned;
using nf4::BlockNorm;
using nf4::fail;
using nf4::guarded;
using nf4::Gradient;
using nf4::hip_status;
using nf4::Memory;
using nf4::RowsView;

namespace {

int size_of(nf4_dtype t) { return t == NF4_BF16 ? 2 : 4; }
bool known(nf4_dtype t) { return t == NF4_F32 || t == NF4_BF16; }

// Rows of M x K; NULL where `wanted` says that there are none.
nf4_status check_rows(const qlora_rows* r, const char* name, bool wanted, bool written, int64_t M, int64_t K, int elem, RowsView& v) {
    const std::string n(name);
    v = RowsView{nullptr, 0};
    if (!wanted) return r ? fail(NF4_ERR_ARG, n + " is given where nothing takes it") : NF4_OK;
    if (!r || !r->data) return fail(NF4_ERR_ARG, n + " is NULL");
    if (!aligned(r->data, elem)) return fail(NF4_ERR_ARG, n + " is misaligned");
    if (r->stride < 0 || (r->stride != 0 && r->stride < K)) return fail(NF4_ERR_ARG, n + ": rows overlap");
    if (written && M > 1 && r->stride < K) return fail(NF4_ERR_ARG, n + ": rows that are written overlap");
    if (r->stride > ((int64_t)1 << 40)) return fail(NF4_ERR_ARG, n + ": stride too large");
    v = RowsView{r->data, r->stride};
    return NF4_OK;
}

nf4_status check_norm(const qlora_block_norm* n, int64_t M, int64_t K, nf4_dtype stream_dtype, bool block, BlockNorm& v) {
    if (!n) return fail(NF4_ERR_ARG, "norm is NULL");
    if (!known(stream_dtype) || !known(n->dtype)) return fail(NF4_ERR_ARG, "types must be NF4_F32 or NF4_BF16");
    if (M < 0 || M > (int64_t)0x7FFFFFFF) return fail(NF4_ERR_UNSUPPORTED, "M must be 0 .. 2^31 - 1");
    if (K < 1 || K > nf4::NORM_MAX_WIDTH) return fail(NF4_ERR_UNSUPPORTED, "K must be 1 .. 32768");
    if (!(n->eps >= 0x1p-126f) || !isfinite(n->eps)) return fail(NF4_ERR_ARG, "eps must be at least 2^-126 and finite");
    if (!isfinite(n->scale)) return fail(NF4_ERR_ARG, "scale must be finite");
    if (n->pre && !n->norm_pre) return fail(NF4_ERR_ARG, "pre is given without a norm before the next block");
    if (n->post && !n->norm_post) return fail(NF4_ERR_ARG, "post is given without a norm after the block");
    if (!block && (n->norm_post || n->gate)) return fail(NF4_ERR_ARG, "norm_post and gate need x");
    const int elem = size_of(n->dtype);
    if (!aligned(n->pre, elem) || !aligned(n->post, elem) || !aligned(n->gate, elem)) return fail(NF4_ERR_ARG, "pre, post or gate is misaligned");
    if (n->gate && (n->gate_rows < 1 || n->gate_rows > (int64_t)0x7FFFFFFF || M % n->gate_rows))
        return fail(NF4_ERR_ARG, "gate_rows must divide M");
    v = BlockNorm{n->pre, n->post, n->gate, n->gate ? n->gate_rows : 1, n->norm_pre != 0, n->norm_post != 0, n->dtype == NF4_BF16,
                  stream_dtype == NF4_BF16, n->scale, n->eps};
    return NF4_OK;
}

bool same_rows(const RowsView& a, const RowsView& b, int64_t M) { return a.data == b.data && (M <= 1 || a.stride == b.stride); }
Memory memory_of(const RowsView& r, int64_t M, int64_t K, int elem) { return Memory(r.data, M, r.stride, K, elem); }
// What is written may share memory with nothing else: other workgroups read or write that, whenever they come to it.
nf4_status check_apart(const Memory& out, const char* name, std::initializer_list<Memory> others) {
    for (const Memory& m : others)
        if (share_memory(out, m)) return fail(NF4_ERR_ARG, std::string(name) + " shares memory with another operand");
    return NF4_OK;
}

nf4_status gradients_of(const qlora_tensor* g, int64_t count, const char* name, std::vector<Gradient>& v) {
    const std::string n(name);
    if (count < 0 || count > ((int64_t)1 << 24)) return fail(NF4_ERR_UNSUPPORTED, "count must be 0 .. 2^24");
    if (count > 0 && !g) return fail(NF4_ERR_ARG, n + " is NULL");
    v.resize((size_t)count);
    int64_t total = 0;
    for (int64_t i = 0; i < count; ++i) {
        if (!known(g[i].dtype)) return fail(NF4_ERR_ARG, n + ": types must be NF4_F32 or NF4_BF16");
        if (g[i].n < 0 || g[i].n > ((int64_t)1 << 40)) return fail(NF4_ERR_ARG, n + ": a tensor's size must be 0 .. 2^40");
        if (g[i].n > 0 && (!g[i].data || !aligned(g[i].data, size_of(g[i].dtype)))) return fail(NF4_ERR_ARG, n + ": a tensor is NULL or misaligned");
        total += g[i].n;
        if (total > ((int64_t)1 << 40)) return fail(NF4_ERR_UNSUPPORTED, n + ": more than 2^40 values");
        v[(size_t)i] = Gradient{g[i].data, g[i].n, g[i].dtype == NF4_BF16};
    }
    return NF4_OK;
}

// Whether a tensor that is written shares memory with another one, read or written (in[i] and out[i] may be the same).
// Lists that ascend in memory, as most do, are not sorted.
bool written_overlap(const std::vector<Gradient>& in, const std::vector<Gradient>& out) {
    struct Range {
        uintptr_t from, to;
    };
    std::vector<Range> written, read;
    written.reserve(out.size());
    auto add = [](std::vector<Range>& v, const Gradient& g) {
        const uintptr_t at = (uintptr_t)g.data;
        if (g.n > 0) v.push_back(Range{at, at + (size_t)g.n * (g.bf16 ? 2 : 4)});
    };
    for (size_t i = 0; i < in.size(); ++i) {
        add(written, out[i]);
        if (in[i].data != out[i].data) add(read, in[i]);
    }
    auto before = [](const Range& a, const Range& b) { return a.from < b.from; };
    for (std::vector<Range>* v : {&written, &read})
        if (!std::is_sorted(v->begin(), v->end(), before)) std::sort(v->begin(), v->end(), before);
    uintptr_t any = 0, end = 0;           // where all so far end, and those that are written
    size_t r = 0;
    for (const Range& w : written) {
        for (; r < read.size() && read[r].from <= w.from; ++r) {
            if (read[r].from < end) return true;
            any = std::max(any, read[r].to);
        }
        if (w.from < any) return true;
        any = std::max(any, w.to);
        end = std::max(end, w.to);
    }
    return r < read.size() && read[r].from < end;
}

}  // namespace

extern "C" {

nf4_status qlora_block_norm_fwd(const qlora_block_norm* norm, int64_t M, int64_t K, nf4_dtype stream_dtype,
                                const qlora_rows* h, const qlora_rows* x, const qlora_rows* h_out, const qlora_rows* y,
                                void* stream) {
    return guarded([&]() -> nf4_status {
        BlockNorm n;
        const bool block = x != nullptr;
        if (nf4_status st = check_norm(norm, M, K, stream_dtype, block, n)) return st;
        if (!block && !n.norm_pre) return fail(NF4_ERR_ARG, "nothing to compute: neither x nor norm_pre");
        if (M == 0) return NF4_OK;
        const int elem = size_of(stream_dtype);
        RowsView hv, xv, ov, yv;
        if (nf4_status st = check_rows(h, "h", true, false, M, K, elem, hv)) return st;
        if (nf4_status st = check_rows(x, "x", block, false, M, K, 2, xv)) return st;
        if (nf4_status st = check_rows(h_out, "h_out", block, true, M, K, elem, ov)) return st;
        if (nf4_status st = check_rows(y, "y", n.norm_pre, true, M, K, 2, yv)) return st;
        if (ov.data && ov.data == hv.data && !same_rows(ov, hv, M)) return fail(NF4_ERR_ARG, "in place needs the same stride");
        const int welem = size_of(norm->dtype);
        const Memory hm = memory_of(hv, M, K, elem), xm = memory_of(xv, M, K, 2), om = memory_of(ov, M, K, elem), ym = memory_of(yv, M, K, 2),
                     pre(n.pre, 1, 0, K, welem), post(n.post, 1, 0, K, welem), gate(n.gate, n.gate_rows, K, K, welem);
        if (nf4_status st = check_apart(om, "h_out", {ov.data == hv.data ? Memory() : hm, xm, ym, pre, post, gate})) return st;
        if (nf4_status st = check_apart(ym, "y", {hm, xm, pre, post, gate})) return st;
        return hip_status(nf4::launch_block_norm_fwd(n, M, K, hv, xv, ov, yv, (hipStream_t)stream), "qlora_block_norm_fwd");
    });
}

size_t qlora_block_norm_bwd_workspace_bytes(int64_t M, int64_t K, int64_t gate_rows, int32_t need_dpre, int32_t need_dpost,
                                            int32_t need_dgate) {
    if (M < 1 || M > (int64_t)0x7FFFFFFF || K < 1 || K > nf4::NORM_MAX_WIDTH) return 0;
    return nf4::block_norm_ws_bytes(M, K, gate_rows < 1 ? 1 : gate_rows, need_dpre != 0, need_dpost != 0, need_dgate != 0);
}

nf4_status qlora_block_norm_bwd(const qlora_block_norm* norm, int64_t M, int64_t K, nf4_dtype stream_dtype,
                                const qlora_rows* h, const qlora_rows* x, const qlora_rows* dy, const qlora_rows* dh,
                                const qlora_rows* dh_out, const qlora_rows* dx, float* dpre, float* dpost, float* dgate,
                                void* workspace, size_t workspace_bytes, void* stream) {
    return guarded([&]() -> nf4_status {
        BlockNorm n;
        const bool block = x != nullptr;
        if (nf4_status st = check_norm(norm, M, K, stream_dtype, block, n)) return st;
        if (!aligned(dpre, 4) || !aligned(dpost, 4) || !aligned(dgate, 4)) return fail(NF4_ERR_ARG, "dpre, dpost or dgate is misaligned");
        if ((dpre && !n.pre) || (dpost && !n.post) || (dgate && !n.gate)) return fail(NF4_ERR_ARG, "a gradient of a weight that is not given");
        RowsView hv{}, xv{}, yv{}, dv{}, ov{}, dxv{};
        if (M > 0) {
            const int elem = size_of(stream_dtype);
            const bool later = dh != nullptr;
            if (nf4_status st = check_rows(h, "h", n.norm_pre, false, M, K, elem, hv)) return st;
            if (nf4_status st = check_rows(x, "x", block, false, M, K, 2, xv)) return st;
            if (nf4_status st = check_rows(dy, "dy", n.norm_pre, false, M, K, 2, yv)) return st;
            if (nf4_status st = check_rows(dh, "dh", later, false, M, K, elem, dv)) return st;
            if (nf4_status st = check_rows(dh_out, "dh_out", true, true, M, K, elem, ov)) return st;
            if (nf4_status st = check_rows(dx, "dx", block, true, M, K, 2, dxv)) return st;
            if (ov.data == dv.data && !same_rows(ov, dv, M)) return fail(NF4_ERR_ARG, "in place needs the same stride");
            const size_t need = nf4::block_norm_ws_bytes(M, K, n.gate_rows, dpre, dpost, dgate);
            if (need > 0 && (!workspace || workspace_bytes < need)) return fail(NF4_ERR_WORKSPACE, "workspace missing or too small");
            if (need > 0 && !aligned(workspace, 256)) return fail(NF4_ERR_ARG, "workspace must be 256-byte aligned");
            const int welem = size_of(norm->dtype);
            const Memory hm = memory_of(hv, M, K, elem), xm = memory_of(xv, M, K, 2), ym = memory_of(yv, M, K, 2), dm = memory_of(dv, M, K, elem),
                         om = memory_of(ov, M, K, elem), dxm = memory_of(dxv, M, K, 2), pre(n.pre, 1, 0, K, welem), post(n.post, 1, 0, K, welem),
                         gate(n.gate, n.gate_rows, K, K, welem), ws(workspace, need), wpre(dpre, 1, 0, K, 4), wpost(dpost, 1, 0, K, 4),
                         wgate(dgate, n.gate_rows, K, K, 4);
            if (nf4_status st = check_apart(om, "dh_out", {ov.data == dv.data ? Memory() : dm, hm, xm, ym, dxm, pre, post, gate, wpre, wpost, wgate, ws})) return st;
            if (nf4_status st = check_apart(dxm, "dx", {dm, hm, xm, ym, pre, post, gate, wpre, wpost, wgate, ws})) return st;
            if (nf4_status st = check_apart(wpre, "dpre", {dm, hm, xm, ym, pre, post, gate, wpost, wgate, ws})) return st;
            if (nf4_status st = check_apart(wpost, "dpost", {dm, hm, xm, ym, pre, post, gate, wgate, ws})) return st;
            if (nf4_status st = check_apart(wgate, "dgate", {dm, hm, xm, ym, pre, post, gate, ws})) return st;
            if (nf4_status st = check_apart(ws, "workspace", {dm, hm, xm, ym, pre, post, gate})) return st;
        }
        return hip_status(nf4::launch_block_norm_bwd(n, M, K, hv, xv, yv, dv, ov, dxv, dpre, dpost, dgate, workspace, (hipStream_t)stream),
                          "qlora_block_norm_bwd");
    });
}

size_t qlora_grad_norm_workspace_bytes(const qlora_tensor* grads, int64_t count) {
    size_t bytes = 0;
    guarded([&]() -> nf4_status {
        std::vector<Gradient> g;
        if (nf4_status st = gradients_of(grads, count, "grads", g)) return st;
        bytes = nf4::grad_norm_ws_bytes(g.data(), count);
        return NF4_OK;
    });
    return bytes;
}

nf4_status qlora_grad_norm(const qlora_tensor* grads, int64_t count, double max_norm, float* norm, float* factor,
                           void* workspace, size_t workspace_bytes, void* stream) {
    return guarded([&]() -> nf4_status {
        std::vector<Gradient> g;
        if (nf4_status st = gradients_of(grads, count, "grads", g)) return st;
        if (!norm || !aligned(norm, 4) || !aligned(factor, 4)) return fail(NF4_ERR_ARG, "norm is NULL, or norm or factor misaligned");
        if (factor && !(max_norm >= 0.0)) return fail(NF4_ERR_ARG, "max_norm must not be negative");
        const size_t need = nf4::grad_norm_ws_bytes(g.data(), count);
        if (need > 0 && (!workspace || workspace_bytes < need)) return fail(NF4_ERR_WORKSPACE, "workspace missing or too small");
        if (need > 0 && !aligned(workspace, 256)) return fail(NF4_ERR_ARG, "workspace must be 256-byte aligned");
        return hip_status(nf4::launch_grad_norm(g.data(), count, max_norm, norm, factor, workspace, (hipStream_t)stream), "qlora_grad_norm");
    });
}

// (the norm's sums, and a place for the factor)
size_t qlora_grad_clip_workspace_bytes(const qlora_tensor* grads, int64_t count) {
    size_t bytes = 0;
    guarded([&]() -> nf4_status {
        std::vector<Gradient> g;
        if (nf4_status st = gradients_of(grads, count, "grads", g)) return st;
        bytes = nf4::grad_norm_ws_bytes(g.data(), count) + 256;
        return NF4_OK;
    });
    return bytes;
}

nf4_status qlora_grad_clip(const qlora_tensor* grads, const qlora_tensor* out, int64_t count, double max_norm, float* norm,
                           void* workspace, size_t workspace_bytes, void* stream) {
    return guarded([&]() -> nf4_status {
        std::vector<Gradient> g, o;
        if (nf4_status st = gradients_of(grads, count, "grads", g)) return st;
        if (nf4_status st = gradients_of(out, count, "out", o)) return st;
        if (!norm || !aligned(norm, 4)) return fail(NF4_ERR_ARG, "norm is NULL or misaligned");
        if (!(max_norm >= 0.0)) return fail(NF4_ERR_ARG, "max_norm must not be negative");
        for (int64_t i = 0; i < count; ++i)
            if (g[(size_t)i].n != o[(size_t)i].n || g[(size_t)i].bf16 != o[(size_t)i].bf16)
                return fail(NF4_ERR_ARG, "grads and out have different sizes or types");
        if (written_overlap(g, o)) return fail(NF4_ERR_ARG, "a tensor that is written overlaps another (or is given twice)");
        const size_t sums = nf4::grad_norm_ws_bytes(g.data(), count);
        if (!workspace || workspace_bytes < sums + 256) return fail(NF4_ERR_WORKSPACE, "workspace missing or too small");
        if (!aligned(workspace, 256)) return fail(NF4_ERR_ARG, "workspace must be 256-byte aligned");
        return hip_status(nf4::launch_grad_clip(g.data(), o.data(), count, max_norm, norm, (float*)((uint8_t*)workspace + sums), workspace,
                                                (hipStream_t)stream), "qlora_grad_clip");
    });
}

nf4_status qlora_logits_shape(const qlora_logit_rules* rules, int64_t rows, int64_t V, nf4_dtype dtype,
                              const qlora_rows* logits, const qlora_rows* out, void* stream) {
    return guarded([&]() -> nf4_status {
        if (!rules) return fail(NF4_ERR_ARG, "rules is NULL");
        if (!known(dtype)) return fail(NF4_ERR_ARG, "dtype must be NF4_F32 or NF4_BF16");
        if (rows < 0 || rows >= ((int64_t)1 << 24)) return fail(NF4_ERR_UNSUPPORTED, "rows must be 0 .. 2^24 - 1");
        if (V < 1 || V >= ((int64_t)1 << 28)) return fail(NF4_ERR_UNSUPPORTED, "V must be 1 .. 2^28 - 1");
        const qlora_logit_rules& q = *rules;
        for (int64_t n : {q.history_width, q.biases})
            if (n < 0 || n > (int64_t)0x7FFFFFFE) return fail(NF4_ERR_ARG, "history_width and biases must be 0 .. 2^31 - 2");
        if ((q.history && q.history_stride != 0 && q.history_stride < q.history_width) || (q.bias_ids && q.bias_ids_stride != 0 && q.bias_ids_stride < q.biases) ||
            (q.bias_ids && q.bias_stride != 0 && q.bias_stride < q.biases) || (q.allowed && q.allowed_stride != 0 && q.allowed_stride < (V + 31) / 32))
            return fail(NF4_ERR_ARG, "a row of the history, the biases or the mask is longer than its stride");
        if ((q.bias_ids != nullptr) != (q.bias != nullptr)) return fail(NF4_ERR_ARG, "bias_ids and bias go together");
        if (!q.history && (q.lengths || q.prompts)) return fail(NF4_ERR_ARG, "lengths and prompts need the history");
        for (const void* p : {(const void*)q.history, (const void*)q.lengths, (const void*)q.prompts, (const void*)q.repetitions, (const void*)q.presences,
                              (const void*)q.frequencies, (const void*)q.bias_ids, (const void*)q.bias, (const void*)q.allowed})
            if (!aligned(p, 4)) return fail(NF4_ERR_ARG, "a field of the rules is misaligned");
        if (q.history) {
            if (!q.repetitions && (!(q.repetition > 0.0f) || !isfinite(q.repetition))) return fail(NF4_ERR_ARG, "repetition must be positive and finite");
            if ((!q.presences && !isfinite(q.presence)) || (!q.frequencies && !isfinite(q.frequency)))
                return fail(NF4_ERR_ARG, "presence and frequency must be finite");
        }
        if (rows == 0) return NF4_OK;
        RowsView in, to;
        if (nf4_status st = check_rows(logits, "logits", true, false, rows, V, size_of(dtype), in)) return st;
        if (nf4_status st = check_rows(out, "out", true, true, rows, V, size_of(dtype), to)) return st;
        if (in.data == to.data && !same_rows(in, to, rows)) return fail(NF4_ERR_ARG, "in place needs the same stride");
        const Memory om = memory_of(to, rows, V, size_of(dtype));
        if (nf4_status st = check_apart(om, "out", {in.data == to.data ? Memory() : memory_of(in, rows, V, size_of(dtype)),
                                                    Memory(q.history, rows, q.history_stride, q.history_width, 4), Memory(q.lengths, rows, 1, 1, 4),
                                                    Memory(q.prompts, rows, 1, 1, 4), Memory(q.repetitions, rows, 1, 1, 4), Memory(q.presences, rows, 1, 1, 4),
                                                    Memory(q.frequencies, rows, 1, 1, 4), Memory(q.bias_ids, rows, q.bias_ids_stride, q.biases, 4),
                                                    Memory(q.bias, rows, q.bias_stride, q.biases, 4), Memory(q.allowed, rows, q.allowed_stride, (V + 31) / 32, 4)}))
            return st;
        const nf4::LogitRules r{rows, q.history, q.lengths, q.prompts, q.history_stride, (int)q.history_width, q.repetition, q.presence, q.frequency,
                                q.repetitions, q.presences, q.frequencies, q.bias_ids, q.bias, q.bias_ids_stride, q.bias_stride, (int)q.biases,
                                q.allowed, q.allowed_stride};
        return hip_status(nf4::launch_shape_logits(r, dtype == NF4_BF16, in.data, in.stride, to.data, to.stride, V, (hipStream_t)stream),
                          "qlora_logits_shape");
    });
}

}  // extern "C"
