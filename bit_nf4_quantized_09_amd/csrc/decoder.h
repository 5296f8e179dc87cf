// decoder.h -- host-side launchers of the operators around the linears (internal).
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "rotary.h"

namespace nf4 {

// ---- rotary positions ------------------------------------------------------
// `count` (1 or 2) tensors of M tokens, each in[i] -> out[i].
hipError_t launch_rope(const RopeView& rope, const int32_t* positions, int64_t M, int head_dim, bool bf16,
                       const HeadsView* in, const HeadsView* out, int count, hipStream_t s);

// ---- the paged cache -------------------------------------------------------
struct CacheView {
    uint8_t* codes;           // [pages][2][heads][page][dim]
    float* scales;            // [pages][2][heads]
    int64_t pages;
    int heads;                // key/value heads
    int page_log2;            // log2 of the tokens of a page
    int dim;
};
struct BatchView {
    const int32_t* starts;    // [seqs + 1]
    const int32_t* lengths;   // [seqs]
    const int32_t* table;     // [seqs][table_stride]
    int64_t table_stride;
    int tokens, seqs, table_width;
};
constexpr int KV_EXP_MIN = -50, KV_EXP_MAX = 50;   // exponents of a page's scale
hipError_t launch_kv_append(const CacheView& c, const BatchView& b, const HeadsView& k, const HeadsView& v,
                            const RopeView& rope, const HeadsView* q_in, const HeadsView* q_out, hipStream_t s);

size_t kv_attention_ws_bytes(const CacheView& c, const BatchView& b, int heads, int64_t max_new, int64_t max_length);
hipError_t launch_kv_attention(const CacheView& c, const BatchView& b, const HeadsView& q, const HeadsView& out,
                               float scale, int64_t max_new, int64_t max_length, void* ws, hipStream_t s);

// ---- the vocabulary head's loss --------------------------------------------
size_t head_loss_ws_bytes(int64_t M, int64_t K, int64_t V, bool dx, bool dw);
hipError_t launch_head_loss(const uint16_t* X, int64_t M, int64_t K, const uint16_t* W, int64_t V,
                            const int64_t* targets, int64_t ignore, const float* dloss, float* loss, uint16_t* dX,
                            uint16_t* dW, void* ws, hipStream_t s);
hipError_t launch_head_zero(uint16_t* p, int64_t n, hipStream_t s);   // n a multiple of 8, p 16-byte aligned

}  // namespace nf4
