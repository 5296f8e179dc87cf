// gradients.hip -- the global norm of many gradients, and their clipping (gfx950).
//
// Mathematics.  norm = sqrt(sum over all tensors of g^2), factor = min(1, max_norm / norm), out = factor g.
// Every square is added in 64 bits: no gradient of fp32 overflows or vanishes there, and a sum over 10^9
// values keeps its digits; a lane's additions (one conversion and one fused multiply-add a value) stay below
// the time of its loads.  The factor is formed in 64 bits and rounded to fp32 once, the product to the
// tensor's type.  A norm of infinity makes the factor zero and one of NaN makes it NaN, as the formula says.
//
// Shape.  Bound by HBM: the norm reads each value once, the clipping reads and writes it once more.  The
// tensors' addresses and sizes travel in the kernels' arguments (240 or 160 of them in a launch), so that
// nothing is copied to the device and a captured graph holds them itself.  A launch's values are cut into
// spans, none across two tensors; workgroups take the spans in turn and leave one sum each, which one
// workgroup adds up in a fixed order: no atomics, the same call gives the same bits.
#include "rows.h"
#include "step.h"

namespace nf4 {

constexpr int NORM_TENSORS = 240, SCALE_TENSORS = 160;      // of a launch: 16 and 24 bytes each of 4 KiB of arguments
constexpr uint32_t IS_BF16 = 0x80000000u;

// Tensors of a launch.  size: values, below 2^31, and the type; span0: spans of the tensors before.
template <int MOST>
struct TensorTable {
    const void* in[MOST];
    uint32_t size[MOST];
    uint32_t span0[MOST];
    uint32_t spans;           // of all
    int count, span_log2;     // values of a span
};
struct ScaleTable : TensorTable<SCALE_TENSORS> {
    void* out[SCALE_TENSORS];
};

// The tensor of a span: the last one with span0 <= span.
template <int MOST>
__device__ __forceinline__ int tensor_of(const TensorTable<MOST>& t, uint32_t span) {
    int lo = 0, hi = t.count;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (t.span0[mid] <= span) lo = mid;
        else hi = mid;
    }
    return lo;
}

template <typename T>
__device__ __forceinline__ double squares_of(const T* p, uint32_t n) {
    double s[2] = {0.0, 0.0};
    constexpr int U = 4;                  // vectors in flight
    for (uint32_t i = threadIdx.x * 8; i < n; i += 256 * 8 * U) {
        Eight<T> e[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            e[u] = load_eight(p, i + 256 * 8 * u, n);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            float f[8];
            unpack_eight<T>(e[u], f);
#pragma unroll
            for (int j = 0; j < 8; ++j) s[j & 1] = fma((double)f[j], (double)f[j], s[j & 1]);
        }
    }
    return s[0] + s[1];
}

// Sum over a workgroup's threads, in thread 0.
template <int THREADS>
__device__ __forceinline__ double workgroup_sum(double v) {
    __shared__ double sums[THREADS / 64];
#pragma unroll
    for (int x = 1; x < 64; x <<= 1) v += __shfl_xor(v, x);
    if ((threadIdx.x & 63) == 0) sums[threadIdx.x >> 6] = v;
    __syncthreads();
    double s = 0.0;
    if (threadIdx.x == 0)
#pragma unroll
        for (int w = 0; w < THREADS / 64; ++w) s += sums[w];
    return s;
}

__global__ __launch_bounds__(256)
void k_grad_squares(TensorTable<NORM_TENSORS> t, double* part) {
    double s = 0.0;
    for (uint32_t span = blockIdx.x; span < t.spans; span += gridDim.x) {
        const int i = tensor_of(t, span);
        const uint32_t size = t.size[i] & ~IS_BF16, at = (span - t.span0[i]) << t.span_log2, most = 1u << t.span_log2;
        const uint32_t n = size - at < most ? size - at : most;
        if (t.size[i] & IS_BF16) s += squares_of((const uint16_t*)t.in[i] + at, n);
        else s += squares_of((const float*)t.in[i] + at, n);
    }
    s = workgroup_sum<256>(s);
    if (threadIdx.x == 0) part[blockIdx.x] = s;
}

__global__ __launch_bounds__(1024)
void k_grad_norm(const double* part, int parts, double max_norm, float* norm, float* factor) {
    double s = 0.0;
    for (int i = threadIdx.x; i < parts; i += 1024) s += part[i];
    s = workgroup_sum<1024>(s);
    if (threadIdx.x == 0) {
        const double n = sqrt(s);
        *norm = (float)n;
        if (factor) *factor = n > max_norm ? (float)(max_norm / n) : n == n ? 1.0f : (float)n;
    }
}

template <typename T>
__device__ __forceinline__ void scale_span(const T* in, T* out, uint32_t n, float f) {
    constexpr int U = 4;
    for (uint32_t i = threadIdx.x * 8; i < n; i += 256 * 8 * U) {
        Eight<T> e[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            e[u] = load_eight(in, i + 256 * 8 * u, n);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            float v[8];
            unpack_eight<T>(e[u], v);
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] *= f;
            store_eight(out, i + 256 * 8 * u, n, pack_eight<T>(v));
        }
    }
}

__global__ __launch_bounds__(256)
void k_grad_scale(ScaleTable t, const float* factor) {
    const float f = *factor;
    for (uint32_t span = blockIdx.x; span < t.spans; span += gridDim.x) {
        const int i = tensor_of<SCALE_TENSORS>(t, span);
        if (f == 1.0f && t.in[i] == t.out[i]) continue;         // in place, and nothing to clip
        const uint32_t size = t.size[i] & ~IS_BF16, at = (span - t.span0[i]) << t.span_log2, most = 1u << t.span_log2;
        const uint32_t n = size - at < most ? size - at : most;
        if (t.size[i] & IS_BF16) scale_span((const uint16_t*)t.in[i] + at, (uint16_t*)t.out[i] + at, n, f);
        else scale_span((const float*)t.in[i] + at, (float*)t.out[i] + at, n, f);
    }
}

// Spans of 2^log2 values: as long as some thousands of them are left, 2^16 at most.
static int span_log2_of(const Gradient* g, int64_t count) {
    int64_t total = 0;
    for (int64_t i = 0; i < count; ++i) total += g[i].n;
    int log2 = 11;
    while (log2 < 16 && (total >> (log2 + 1)) >= 4096) ++log2;
    return log2;
}
constexpr int64_t PIECE = (int64_t)1 << 30;       // longer tensors are several entries of the table
constexpr uint32_t GRAD_GRID = 2048;              // workgroups of a launch at most: those that run at once

// Calls launch(table) for tables of up to MOST pieces; add(table, entry, tensor, first value) fills in what else one holds.
template <int MOST, typename TABLE, typename A, typename F>
static hipError_t with_tables(const Gradient* g, int64_t count, int log2, A&& add, F&& launch) {
    TABLE t{};
    t.span_log2 = log2;
    auto flush = [&]() -> hipError_t {
        if (t.count == 0) return hipSuccess;
        const hipError_t e = launch(t);
        t.count = 0;
        t.spans = 0;
        return e;
    };
    for (int64_t i = 0; i < count; ++i)
        for (int64_t at = 0; at < g[i].n; at += PIECE) {
            const int64_t n = g[i].n - at < PIECE ? g[i].n - at : PIECE;
            const uint32_t spans = (uint32_t)((n + ((int64_t)1 << log2) - 1) >> log2);
            if (t.count == MOST || (uint64_t)t.spans + spans > 0x7FFFFFFFu)
                if (const hipError_t e = flush()) return e;
            t.in[t.count] = (const uint8_t*)g[i].data + at * (g[i].bf16 ? 2 : 4);
            t.size[t.count] = (uint32_t)n | (g[i].bf16 ? IS_BF16 : 0u);
            t.span0[t.count] = t.spans;
            add(t, t.count, i, at);
            t.spans += spans;
            ++t.count;
        }
    return flush();
}

// Launches, and so sums, of a norm over these tensors.
static int64_t norm_launches(const Gradient* g, int64_t count) {
    int64_t pieces = 0;
    for (int64_t i = 0; i < count; ++i) pieces += (g[i].n + PIECE - 1) / PIECE;
    return (pieces + NORM_TENSORS - 1) / NORM_TENSORS;
}
size_t grad_norm_ws_bytes(const Gradient* g, int64_t count) {
    return ((size_t)norm_launches(g, count) * GRAD_GRID * sizeof(double) + 255) & ~(size_t)255;
}

hipError_t launch_grad_norm(const Gradient* g, int64_t count, double max_norm, float* norm, float* factor, void* ws, hipStream_t s) {
    int64_t parts = 0;
    auto nothing = [](auto&, int, int64_t, int64_t) {};
    const hipError_t e = with_tables<NORM_TENSORS, TensorTable<NORM_TENSORS>>(g, count, span_log2_of(g, count), nothing, [&](const auto& t) {
        const uint32_t grid = t.spans < GRAD_GRID ? t.spans : GRAD_GRID;
        hipLaunchKernelGGL(k_grad_squares, dim3(grid), dim3(256), 0, s, t, (double*)ws + parts);
        parts += grid;
        return hipGetLastError();
    });
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(k_grad_norm, dim3(1), dim3(1024), 0, s, (const double*)ws, (int)parts, max_norm, norm, factor);
    return hipGetLastError();
}

hipError_t launch_grad_scale(const Gradient* g, const Gradient* out, int64_t count, const float* factor, hipStream_t s) {
    auto to = [&](ScaleTable& t, int entry, int64_t i, int64_t at) { t.out[entry] = (uint8_t*)out[i].data + at * (out[i].bf16 ? 2 : 4); };
    return with_tables<SCALE_TENSORS, ScaleTable>(g, count, span_log2_of(g, count), to, [&](const ScaleTable& t) {
        hipLaunchKernelGGL(k_grad_scale, dim3(t.spans < GRAD_GRID ? t.spans : GRAD_GRID), dim3(256), 0, s, t, factor);
        return hipGetLastError();
    });
}

}  // namespace nf4
