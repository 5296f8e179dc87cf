// step.h -- host-side launchers of the operators of include/qlora_step.h (internal).
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace nf4 {

// ---- norms around a block --------------------------------------------------
constexpr int64_t NORM_MAX_WIDTH = 32768;
struct RowsView {
    void* data;
    int64_t stride;           // in values
};
// What lies between a block's output and the next block's input.  A null weight is one everywhere.
struct BlockNorm {
    const void *pre, *post, *gate;
    int64_t gate_rows;        // rows of the gate, each for tokens / gate_rows neighbouring tokens
    bool norm_pre, norm_post, weights_bf16, stream_bf16;
    float scale, eps;
};
hipError_t launch_block_norm_fwd(const BlockNorm& n, int64_t M, int64_t K, const RowsView& h, const RowsView& x,
                                 const RowsView& h_out, const RowsView& y, hipStream_t s);
size_t block_norm_ws_bytes(int64_t M, int64_t K, int64_t gate_rows, bool dpre, bool dpost, bool dgate);
hipError_t launch_block_norm_bwd(const BlockNorm& n, int64_t M, int64_t K, const RowsView& h, const RowsView& x,
                                 const RowsView& dy, const RowsView& dh, const RowsView& dh_out, const RowsView& dx,
                                 float* dpre, float* dpost, float* dgate, void* ws, hipStream_t s);

// ---- the gradients' norm and clipping --------------------------------------
struct Gradient {
    void* data;
    int64_t n;
    bool bf16;
};
size_t grad_norm_ws_bytes(const Gradient* g, int64_t count);
hipError_t launch_grad_norm(const Gradient* g, int64_t count, double max_norm, float* norm, float* factor, void* ws, hipStream_t s);
// norm and factor as above (factor is not always written); ws: of the norm.
hipError_t launch_grad_clip(const Gradient* g, const Gradient* out, int64_t count, double max_norm, float* norm, float* factor,
                            void* ws, hipStream_t s);

// ---- logits before the choice of a token -----------------------------------
struct LogitRules {
    int64_t rows;
    const int32_t *history, *lengths, *prompts;       // history null: no penalties
    int64_t history_stride;
    int history_width;
    float repetition, presence, frequency;            // of all rows, or
    const float *repetitions, *presences, *frequencies;     // of each (null: not)
    const int32_t* bias_ids;                          // null: no biases
    const float* bias;
    int64_t bias_ids_stride, bias_stride;
    int biases;
    const int32_t* allowed;                           // null: all
    int64_t allowed_stride;
};
hipError_t launch_shape_logits(const LogitRules& r, bool bf16, const void* in, int64_t in_stride, void* out, int64_t out_stride,
                               int64_t V, hipStream_t s);

}  // namespace nf4
