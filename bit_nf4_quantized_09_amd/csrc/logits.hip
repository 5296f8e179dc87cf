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
// whose order does not matter.  The logits, the first 4 tokens a thread and the biases' ids are all on their way
// before it clears the counters.  256 rows of 128256 in fp32 (272 MB): 43 us without a history or biases (6.3 TB/s), 62
// with histories of up to 8000 tokens, which every workgroup of a row walks along, and 100 biases each; one row of
// 32000 in bf16 3.5 us.
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

// A row's int32 values, four a thread and load: the first ones are on their way from `start` on, and each time the next ones
// while the last are taken.
template <int THREADS>
struct Tokens {
    typedef int32_t i4 __attribute__((ext_vector_type(4), aligned(4)));
    const NF4_GLOBAL int32_t* p;
    int width;
    i4 now;
    __device__ __forceinline__ i4 load(int64_t i) const {
        i4 v = {-1, -1, -1, -1};
        if (i + 4 <= width) {
            v = *(const NF4_GLOBAL i4*)(p + i);
        } else {
#pragma unroll
            for (int j = 0; j < 3; ++j)
                if (i + j < width) v[j] = p[i + j];
        }
        return v;
    }
    __device__ __forceinline__ void start(const int32_t* row, int values) {
        p = (const NF4_GLOBAL int32_t*)(uintptr_t)row;
        width = values;
        now = load(threadIdx.x * 4);
    }
    // f(value, place) for those below n
    template <typename F>
    __device__ __forceinline__ void each(int n, F&& f) {
        for (int64_t i = threadIdx.x * 4; i < n; i += THREADS * 4) {
            const i4 next = load(i + THREADS * 4);
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (i + j < n) f(now[j], (int)(i + j));
            now = next;
        }
    }
};

// CHUNKS: vectors of 8 logits a thread.  PACKED: a token's entry of the biases (16 bits), whether the prompt has it and
// how often the answer does (15 bits) share one counter, else a counter of 31 bits and an entry are apart.
template <typename T, int THREADS, int CHUNKS, bool HISTORY, bool BIAS, bool PACKED>
__global__ __launch_bounds__(THREADS)
void k_shape_logits(LogitArgs a) {
    constexpr int SLICE = 8 * CHUNKS * THREADS;
    constexpr bool COUNTS = HISTORY || (BIAS && PACKED), ENTRIES = BIAS && !PACKED;
    constexpr uint32_t SEEN = PACKED ? 0x10000u : 0x80000000u, ONE = PACKED ? 0x20000u : 1u;
    __shared__ uint32_t counts[COUNTS ? SLICE : 4], entries[ENTRIES ? SLICE : 4];
    const int64_t row = blockIdx.y + (int64_t)blockIdx.z * gridDim.y;
    if (row >= a.r.rows) return;
    const int first = blockIdx.x * SLICE;
    // all that is read is on its way before the first barrier
    Tokens<THREADS> tokens, ids;
    if constexpr (HISTORY) tokens.start(a.r.history + row * a.r.history_stride, a.r.history_width);
    if constexpr (BIAS) ids.start(a.r.bias_ids + row * a.r.bias_ids_stride, a.r.biases);
    Eight<T> raw[CHUNKS];
    uint32_t may[CHUNKS];
#pragma unroll
    for (int u = 0; u < CHUNKS; ++u) {
        const int c = first + 8 * (threadIdx.x + u * THREADS);
        raw[u] = load_eight((const T*)a.in + row * a.in_stride, c, a.V);
        may[u] = 0xFFu;
        if (a.r.allowed && c < a.V) may[u] = reinterpret_cast<const uint8_t*>(a.r.allowed + row * a.r.allowed_stride)[c >> 3];
    }
    float rep = 1.0f, presence = 0.0f, frequency = 0.0f;
    int n = 0, prompt = 0;
    if constexpr (HISTORY) {
        rep = a.r.repetitions ? a.r.repetitions[row] : a.r.repetition;
        presence = a.r.presences ? a.r.presences[row] : a.r.presence;
        frequency = a.r.frequencies ? a.r.frequencies[row] : a.r.frequency;
        n = a.r.lengths ? a.r.lengths[row] : a.r.history_width;
        n = n < a.r.history_width ? n : a.r.history_width;
        prompt = a.r.prompts ? a.r.prompts[row] : 0;
    }
    if constexpr (HISTORY || BIAS) {
#pragma unroll
        for (int i = 0; i < 2 * CHUNKS; ++i) {
            if constexpr (COUNTS) reinterpret_cast<uint4*>(counts)[threadIdx.x + i * THREADS] = make_uint4(0, 0, 0, 0);
            if constexpr (ENTRIES) reinterpret_cast<uint4*>(entries)[threadIdx.x + i * THREADS] = make_uint4(0, 0, 0, 0);
        }
        __syncthreads();
        if constexpr (BIAS) {
            uint32_t* to = PACKED ? counts : entries;
            ids.each(a.r.biases, [&](int32_t id, int i) {
                const uint32_t v = (uint32_t)id - (uint32_t)first;
                if (v < (uint32_t)SLICE) atomicMax(&to[v], (uint32_t)i + 1);
            });
            if constexpr (PACKED && HISTORY) __syncthreads();         // the largest entry is of a counter without counts
        }
        if constexpr (HISTORY)
            tokens.each(n, [&](int32_t token, int i) {
                const uint32_t v = (uint32_t)token - (uint32_t)first;
                if (v >= (uint32_t)SLICE) return;
                if (i >= prompt) atomicAdd(&counts[v], ONE);
                else atomicOr(&counts[v], SEEN);
            });
        __syncthreads();
    }
#pragma unroll
    for (int u = 0; u < CHUNKS; ++u) {
        const int place = threadIdx.x + u * THREADS, c = first + 8 * place;
        if (c >= a.V) continue;
        float z[8];
        unpack_eight<T>(raw[u], z);
        if constexpr (HISTORY || BIAS) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                uint4 k4 = make_uint4(0, 0, 0, 0), e4 = k4;
                if constexpr (COUNTS) k4 = reinterpret_cast<const uint4*>(counts)[place * 2 + h];
                if constexpr (ENTRIES) e4 = reinterpret_cast<const uint4*>(entries)[place * 2 + h];
                if ((k4.x | k4.y | k4.z | k4.w | e4.x | e4.y | e4.z | e4.w) == 0) continue;
                const uint32_t k[4] = {k4.x, k4.y, k4.z, k4.w}, e[4] = {e4.x, e4.y, e4.z, e4.w};
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    float& x = z[4 * h + j];
                    if constexpr (HISTORY) {
                        const uint32_t seen = PACKED ? k[j] >> 16 : k[j], m = PACKED ? k[j] >> 17 : k[j] & ~SEEN;
                        if (seen != 0) {
                            x = x > 0.0f ? __fdiv_rn(x, rep) : x * rep;
                            if (m != 0) x -= frequency * (float)m + presence;
                        }
                    }
                    if constexpr (BIAS) {
                        const uint32_t entry = PACKED ? k[j] & 0xFFFFu : e[j];
                        if (entry != 0) x += (a.r.bias + row * a.r.bias_stride)[entry - 1];
                    }
                }
            }
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) z[j] = may[u] >> j & 1u ? z[j] : -INFINITY;
        store_eight((T*)a.out + row * a.out_stride, c, a.V, pack_eight<T>(z));
    }
}

hipError_t launch_shape_logits(const LogitRules& r, bool bf16, const void* in, int64_t in_stride, void* out, int64_t out_stride,
                               int64_t V, hipStream_t s) {
    LogitArgs a{r, in, out, in_stride, out_stride, (int)V};
    const bool history = r.history && r.history_width > 0, bias = r.bias_ids && r.biases > 0;
    const bool packed = r.history_width < 32768 && r.biases < 65536;
    // Wide workgroups walk along a history less often, narrow ones do not wait for so many others: 256 rows of 128256 with
    // up to 8000 tokens 62 us with slices of 16384 logits, 65 with 8192, 67 with 4096, 75 with 2048 (bf16: 41 and 47 for the
    // first two); with up to 500 53 with 8192, 47 and 47.  The widest where they leave a workgroup for each compute unit
    // (16 rows of 32000, up to 4000 tokens: 8.1 us with 16384, 5.9 with 8192, 6.6 with 2048).
    const bool wide = history && r.history_width > 1024, widest = wide && packed && r.rows * ((V + 16383) / 16384) >= 256;
    const int slice = widest ? 16384 : wide ? 8192 : 2048;
    const uint32_t y = (uint32_t)(r.rows < 65535 ? r.rows : 65535), z = (uint32_t)((r.rows + y - 1) / y);
    const dim3 grid((uint32_t)((V + slice - 1) / slice), y, z);
    auto run = [&](auto type, auto h, auto b) {
        constexpr bool H = decltype(h)::value, B = decltype(b)::value;
        using T = decltype(type);
        if constexpr (H) {
            if (widest) hipLaunchKernelGGL((k_shape_logits<T, 1024, 2, H, B, true>), grid, dim3(1024), 0, s, a);
            else if (wide && packed) hipLaunchKernelGGL((k_shape_logits<T, 1024, 1, H, B, true>), grid, dim3(1024), 0, s, a);
            else if (wide) hipLaunchKernelGGL((k_shape_logits<T, 1024, 1, H, B, false>), grid, dim3(1024), 0, s, a);
            else if (packed) hipLaunchKernelGGL((k_shape_logits<T, 256, 1, H, B, true>), grid, dim3(256), 0, s, a);
            else hipLaunchKernelGGL((k_shape_logits<T, 256, 1, H, B, false>), grid, dim3(256), 0, s, a);
        } else {
            hipLaunchKernelGGL((k_shape_logits<T, 256, 1, H, B, false>), grid, dim3(256), 0, s, a);
        }
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
