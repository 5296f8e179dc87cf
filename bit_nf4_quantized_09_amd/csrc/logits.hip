// logits.hip -- what lies between the vocabulary head's logits and the choice of a token: penalties for
// tokens that were there before, biases and a grammar's mask (gfx950).
//
// Mathematics.  Of row r and token v, with seen = v is among the row's tokens so far and count = how many times
// it is among those after the prompt:
//   z <- z / repetition if z > 0, else z repetition             (where seen)
//   z <- z - (frequency count + presence [count > 0])
//   z <- z + bias of the row's last entry with this token       (where there is one)
//   z <- -inf                                                   (where the mask's bit is 0)
// in fp32 with one rounding at the end.
//
// Shape.  Bound by HBM, or by a launch for a few rows: each logit is read once and written once.  A
// workgroup takes 8 neighbouring logits a thread of one row, and finds its tokens' counts by walking
// along the row's history with a counter for each of its own tokens in LDS: additions of whole numbers,
// whose order does not matter.  The logits are on their way while it counts.
#include "rows.h"
#include "step.h"

namespace nf4 {

struct LogitArgs {
    LogitRules r;
    const void* in;
    void* out;
    int64_t in_stride, out_stride;
    int V;
};

constexpr uint32_t SEEN = 0x80000000u;            // a counter's bit for tokens of the prompt and after

template <typename T, int THREADS, bool HISTORY, bool BIAS>
__global__ __launch_bounds__(THREADS)
void k_shape_logits(LogitArgs a) {
    constexpr int SLICE = 8 * THREADS;
    __shared__ uint32_t counts[HISTORY ? SLICE : 1], entries[BIAS ? SLICE : 1];
    const int64_t row = blockIdx.y + (int64_t)blockIdx.z * gridDim.y;
    if (row >= a.r.rows) return;
    const int first = blockIdx.x * SLICE, c = first + threadIdx.x * 8, left = a.V - c;
    const Eight<T> raw = load_eight((const T*)a.in + row * a.in_stride, c, a.V);
    uint32_t may = 0xFFu;
    if (a.r.allowed && left > 0) may = reinterpret_cast<const uint8_t*>(a.r.allowed + row * a.r.allowed_stride)[c >> 3];
    float rep = 1.0f, presence = 0.0f, frequency = 0.0f;
    if constexpr (HISTORY) {
        rep = a.r.repetitions ? a.r.repetitions[row] : a.r.repetition;
        presence = a.r.presences ? a.r.presences[row] : a.r.presence;
        frequency = a.r.frequencies ? a.r.frequencies[row] : a.r.frequency;
    }
    if constexpr (HISTORY || BIAS) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            if constexpr (HISTORY) reinterpret_cast<uint4*>(counts)[threadIdx.x + i * THREADS] = make_uint4(0, 0, 0, 0);
            if constexpr (BIAS) reinterpret_cast<uint4*>(entries)[threadIdx.x + i * THREADS] = make_uint4(0, 0, 0, 0);
        }
        __syncthreads();
        if constexpr (HISTORY) {
            const int32_t* tokens = a.r.history + row * a.r.history_stride;
            const int held = a.r.lengths ? a.r.lengths[row] : a.r.history_width;
            const int n = held < a.r.history_width ? held : a.r.history_width;
            const int prompt = a.r.prompts ? a.r.prompts[row] : 0;
            for (int i = threadIdx.x; i < n; i += THREADS) {
                const uint32_t v = (uint32_t)tokens[i] - (uint32_t)first;
                if (v >= (uint32_t)SLICE) continue;
                if (i >= prompt) atomicAdd(&counts[v], 1u);
                atomicOr(&counts[v], SEEN);
            }
        }
        if constexpr (BIAS) {
            const int32_t* ids = a.r.bias_ids + row * a.r.bias_ids_stride;
            for (int i = threadIdx.x; i < a.r.biases; i += THREADS) {
                const uint32_t v = (uint32_t)ids[i] - (uint32_t)first;
                if (v < (uint32_t)SLICE) atomicMax(&entries[v], (uint32_t)i + 1);
            }
        }
        __syncthreads();
    }
    if (left <= 0) return;
    float z[8];
    unpack_eight<T>(raw, z);
    if constexpr (HISTORY) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const uint32_t k = counts[threadIdx.x * 8 + j];
            if (k != 0) {
                z[j] = z[j] > 0.0f ? __fdiv_rn(z[j], rep) : z[j] * rep;
                const uint32_t n = k & ~SEEN;
                if (n != 0) z[j] -= frequency * (float)n + presence;
            }
        }
    }
    if constexpr (BIAS) {
        const float* bias = a.r.bias + row * a.r.bias_stride;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const uint32_t e = entries[threadIdx.x * 8 + j];
            if (e != 0) z[j] += bias[e - 1];
        }
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) z[j] = may >> j & 1u ? z[j] : -INFINITY;
    store_eight((T*)a.out + row * a.out_stride, c, a.V, pack_eight<T>(z));
}

hipError_t launch_shape_logits(const LogitRules& r, bool bf16, const void* in, int64_t in_stride, void* out, int64_t out_stride,
                               int64_t V, hipStream_t s) {
    LogitArgs a{r, in, out, in_stride, out_stride, (int)V};
    const bool history = r.history && r.history_width > 0, bias = r.bias_ids && r.biases > 0;
    // wide workgroups walk along a history less often, narrow ones spread few rows over more compute units
    const bool wide = history && r.rows * V > (int64_t)256 * 8 * 1024;
    const int slice = 8 * (wide ? 1024 : 256);
    const uint32_t y = (uint32_t)(r.rows < 65535 ? r.rows : 65535), z = (uint32_t)((r.rows + y - 1) / y);
    const dim3 grid((uint32_t)((V + slice - 1) / slice), y, z);
    auto run = [&](auto type, auto h, auto b) {
        constexpr bool H = decltype(h)::value, B = decltype(b)::value;
        using T = decltype(type);
        if (wide) hipLaunchKernelGGL((k_shape_logits<T, 1024, H, B>), grid, dim3(1024), 0, s, a);
        else hipLaunchKernelGGL((k_shape_logits<T, 256, H, B>), grid, dim3(256), 0, s, a);
    };
    auto with = [&](auto type) {
        if (history) bias ? run(type, std::true_type{}, std::true_type{}) : run(type, std::true_type{}, std::false_type{});
        else bias ? run(type, std::false_type{}, std::true_type{}) : run(type, std::false_type{}, std::false_type{});
    };
    if (bf16) with(uint16_t{});
    else with(float{});
    return hipGetLastError();
}

}  // namespace nf4
