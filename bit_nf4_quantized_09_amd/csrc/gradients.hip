// gradients.hip -- the global norm of many gradients, and their clipping (gfx950).
//
// Mathematics.  norm = sqrt(sum over all tensors of g^2), factor = min(1, max_norm / norm), out = factor g.
// Every square is added in 64 bits: no gradient of fp32 overflows or vanishes there, and a sum over 10^9
// values keeps its digits; a lane's additions (one conversion and one fused multiply-add a value) stay below
// the time of its loads.  The factor is formed in 64 bits and rounded to fp32 once, the product to the
// tensor's type.  A norm of infinity makes the factor zero and one of NaN makes it NaN, as the formula says.
//
// Shape.  Bound by HBM: the norm reads each value once, the clipping reads and writes it once more.  The
// tensors' addresses and sizes travel in the kernels' arguments (240 of them in a launch, 160 with outputs apart), so that
// nothing is copied to the device and a captured graph holds them itself.  A launch's values are cut into
// spans of 8192, none across two tensors, and each workgroup walks along equally many neighbouring ones.  It leaves one
// sum; they are added up in a fixed order: no atomics, the same call gives the same bits.  1120 tensors of 3.2 GB in
// fp32: 1.84 ms, the norm's launches at 6.6 TB/s (nontemporal reads) and the scaling's at 5.1, a large copy's rate.
#include <vector>

#include "rows.h"
#include "step.h"

namespace nf4 {

// Tensors of a launch: 16 or (with outputs apart) 24 bytes each of 4 KiB of arguments; a list of up to 32 takes less (the arguments' way to
// the GPU is part of a call: 28 tensors clipped into others in 10.8 us, 12.2 with 4 KiB).
constexpr int NORM_TENSORS = 240, SCALE_TENSORS = 160, FEW_TENSORS = 32;
constexpr uint32_t IS_BF16 = 0x80000000u;
constexpr int SPAN_LOG2 = 13;                     // values of a span
constexpr int VECTORS = 8;                        // 16-byte vectors in flight a thread

// Tensors of a launch.  size: values, below 2^31, and the type; span0: spans of the tensors before.
template <int MOST>
struct TensorTable {
    const void* in[MOST];
    uint32_t size[MOST];
    uint32_t span0[MOST];
    uint32_t spans;           // of all
    int count;
    bool stream;              // more than the last-level cache keeps until it is read again
};
template <int MOST, bool APART>
struct ScaleTable : TensorTable<MOST> {
    void* out[MOST];
    __host__ __device__ void put(int i, void* p) { out[i] = p; }
    __device__ void* to(int i) const { return out[i]; }
};
// (all in place: an address each is enough, and fewer launches: 448 tensors 33 us, 38 with 160 a launch; 196 tensors 17 and 22)
template <int MOST>
struct ScaleTable<MOST, false> : TensorTable<MOST> {
    __host__ __device__ void put(int, void*) {}
    __device__ void* to(int i) const { return const_cast<void*>(this->in[i]); }
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

// Calls run(tensor, first value, values) for the workgroup's part of the launch's spans, tensor by tensor.
template <int MOST, typename F>
__device__ __forceinline__ void for_values(const TensorTable<MOST>& t, F&& run) {
    uint32_t span = (uint32_t)((uint64_t)t.spans * blockIdx.x / gridDim.x);
    const uint32_t end = (uint32_t)((uint64_t)t.spans * (blockIdx.x + 1) / gridDim.x);
    for (int i = span < end ? tensor_of(t, span) : 0; span < end; ++i) {
        const uint32_t next = i + 1 < t.count ? t.span0[i + 1] : t.spans, to = next < end ? next : end;
        const uint32_t size = t.size[i] & ~IS_BF16, first = (span - t.span0[i]) << SPAN_LOG2;
        const uint32_t last = to == next ? size : (to - t.span0[i]) << SPAN_LOG2;
        run(i, first, last - first);
        span = to;
    }
}

// Calls each(vector) for the whole 16-byte vectors of n values that the thread takes, VECTORS at a time: load(v) starts
// vector v's load, and take(v, it) has it; then one(value) for the last values.
template <typename T, typename L, typename K, typename O>
__device__ __forceinline__ void for_vectors(uint32_t n, L&& load, K&& take, O&& one) {
    constexpr uint32_t N = 16 / sizeof(T);
    const uint32_t vectors = n / N;
    uint32_t v = threadIdx.x;
    for (; v + 256 * (VECTORS - 1) < vectors; v += 256 * VECTORS) {
        uint4 w[VECTORS];
#pragma unroll
        for (int u = 0; u < VECTORS; ++u) w[u] = load(v + 256 * u);
#pragma unroll
        for (int u = 0; u < VECTORS; ++u) take(v + 256 * u, w[u]);
    }
    for (; v < vectors; v += 256) take(v, load(v));
    if (threadIdx.x < n % N) one(vectors * N + threadIdx.x);
}
template <typename T>
__device__ __forceinline__ uint4 vector_at(const T* p, uint32_t v, bool stream) {
    const NF4_GLOBAL typename Loose<T>::type* at = (const NF4_GLOBAL typename Loose<T>::type*)(uintptr_t)p + v;
    return __builtin_bit_cast(uint4, stream ? __builtin_nontemporal_load(at) : *at);
}

template <typename T>
__device__ __forceinline__ void add_squares(const T* p, uint32_t n, bool stream, double (&s)[2]) {
    constexpr int N = 16 / sizeof(T);
    for_vectors<T>(n, [&](uint32_t v) { return vector_at(p, v, stream); },
        [&](uint32_t, uint4 w) {
            float f[N];
            Vec16<T>::unpack(w, f);
#pragma unroll
            for (int j = 0; j < N; ++j) s[j & 1] = fma((double)f[j], (double)f[j], s[j & 1]);
        },
        [&](uint32_t i) {
            const double f = Vec16<T>::to_f32(p[i]);
            s[0] = fma(f, f, s[0]);
        });
}

// Sum over a workgroup's threads, the same in all of them.
template <int THREADS>
__device__ __forceinline__ double workgroup_sum(double v) {
    __shared__ double sums[THREADS / 64];
#pragma unroll
    for (int x = 1; x < 64; x <<= 1) v += __shfl_xor(v, x);
    if ((threadIdx.x & 63) == 0) sums[threadIdx.x >> 6] = v;
    __syncthreads();
    double s = 0.0;
#pragma unroll
    for (int w = 0; w < THREADS / 64; ++w) s += sums[w];
    return s;
}

template <int MOST>
__global__ __launch_bounds__(256)
void k_grad_squares(TensorTable<MOST> t, double* part) {
    double s[2] = {0.0, 0.0};
    for_values(t, [&](int i, uint32_t first, uint32_t n) {
        if (t.size[i] & IS_BF16) add_squares((const uint16_t*)t.in[i] + first, n, t.stream, s);
        else add_squares((const float*)t.in[i] + first, n, t.stream, s);
    });
    const double sum = workgroup_sum<256>(s[0] + s[1]);
    if (threadIdx.x == 0) part[blockIdx.x] = sum;
}

__device__ __forceinline__ float factor_of(double norm, double max_norm) {
    return norm > max_norm ? (float)(max_norm / norm) : norm == norm ? 1.0f : (float)norm;
}

__global__ __launch_bounds__(1024)
void k_grad_norm(const double* part, int parts, double max_norm, float* norm, float* factor) {
    double s = 0.0;
    for (int i = threadIdx.x; i < parts; i += 1024) s += part[i];
    s = workgroup_sum<1024>(s);
    if (threadIdx.x == 0) {
        const double n = sqrt(s);
        *norm = (float)n;
        if (factor) *factor = factor_of(n, max_norm);
    }
}

template <typename T>
__device__ __forceinline__ void scale_values(const T* in, T* out, uint32_t n, bool stream, float f) {
    constexpr int N = 16 / sizeof(T);
    for_vectors<T>(n, [&](uint32_t v) { return vector_at(in, v, stream); },
        [&](uint32_t v, uint4 w) {
            float x[N];
            Vec16<T>::unpack(w, x);
#pragma unroll
            for (int j = 0; j < N; ++j) x[j] *= f;
            *((NF4_GLOBAL typename Loose<T>::type*)(uintptr_t)out + v) = __builtin_bit_cast(typename Loose<T>::type, Vec16<T>::pack(x));
        },
        [&](uint32_t i) { out[i] = Vec16<T>::from_f32(Vec16<T>::to_f32(in[i]) * f); });
}

// JOIN: the norm's sums are so few that every workgroup adds them up for itself, and one of each launch says what they give.
template <int MOST, bool APART, bool JOIN>
__global__ __launch_bounds__(256)
void k_grad_scale(ScaleTable<MOST, APART> t, const double* part, int parts, double max_norm, float* norm, const float* factor) {
    float f;
    if constexpr (JOIN) {
        double s = 0.0;
        for (int i = threadIdx.x; i < parts; i += 256) s += part[i];
        const double n = sqrt(workgroup_sum<256>(s));
        f = factor_of(n, max_norm);
        if (blockIdx.x == 0 && threadIdx.x == 0) *norm = (float)n;
    } else {
        f = *factor;
    }
    for_values<MOST>(t, [&](int i, uint32_t first, uint32_t n) {
        if (f == 1.0f && t.in[i] == t.to(i)) return;            // in place, and nothing to clip
        if (t.size[i] & IS_BF16) scale_values((const uint16_t*)t.in[i] + first, (uint16_t*)t.to(i) + first, n, t.stream, f);
        else scale_values((const float*)t.in[i] + first, (float*)t.to(i) + first, n, t.stream, f);
    });
}

constexpr int64_t PIECE = (int64_t)1 << 30;       // longer tensors are several entries of the table
constexpr uint32_t GRAD_GRID = 2048;              // workgroups of a launch at most: those that run at once
constexpr int64_t KEPT = (int64_t)128 << 20;      // bytes that the last-level cache (256 MB) keeps while they are clipped

// Fills tables of up to MOST pieces each.  add(table, entry, tensor, first value) fills in what else an entry holds.
template <int MOST, typename TABLE, typename A>
static std::vector<TABLE> tables_of(const Gradient* g, int64_t count, A&& add) {
    std::vector<TABLE> all;
    int64_t left = 0;
    for (int64_t i = 0; i < count; ++i) left += g[i].n * (g[i].bf16 ? 2 : 4);
    for (int64_t i = 0; i < count; ++i)
        for (int64_t at = 0; at < g[i].n; at += PIECE) {
            const int64_t n = g[i].n - at < PIECE ? g[i].n - at : PIECE;
            if (all.empty() || all.back().count == MOST) {
                all.emplace_back();
                all.back().stream = left > KEPT;
            }
            TABLE& t = all.back();
            t.in[t.count] = (const uint8_t*)g[i].data + at * (g[i].bf16 ? 2 : 4);
            t.size[t.count] = (uint32_t)n | (g[i].bf16 ? IS_BF16 : 0u);
            t.span0[t.count] = t.spans;
            add(t, t.count, i, at);
            t.spans += (uint32_t)((n + ((int64_t)1 << SPAN_LOG2) - 1) >> SPAN_LOG2);
            ++t.count;
            left -= n * (g[i].bf16 ? 2 : 4);
        }
    return all;
}
template <typename TABLE>
static uint32_t grid_of(const TABLE& t) { return t.spans < GRAD_GRID ? t.spans : GRAD_GRID; }

static int64_t pieces_of(const Gradient* g, int64_t count) {
    int64_t pieces = 0;
    for (int64_t i = 0; i < count; ++i) pieces += (g[i].n + PIECE - 1) / PIECE;
    return pieces;
}
size_t grad_norm_ws_bytes(const Gradient* g, int64_t count) {
    const int64_t launches = (pieces_of(g, count) + NORM_TENSORS - 1) / NORM_TENSORS;
    return ((size_t)launches * GRAD_GRID * sizeof(double) + 255) & ~(size_t)255;
}

// The sums of all tensors' squares into ws; how many.
template <int MOST>
static int launch_squares_of(const Gradient* g, int64_t count, void* ws, hipStream_t s) {
    int parts = 0;
    for (const auto& t : tables_of<MOST, TensorTable<MOST>>(g, count, [](auto&, int, int64_t, int64_t) {})) {
        hipLaunchKernelGGL(k_grad_squares<MOST>, dim3(grid_of(t)), dim3(256), 0, s, t, (double*)ws + parts);
        parts += (int)grid_of(t);
    }
    return parts;
}
static int launch_squares(const Gradient* g, int64_t count, void* ws, hipStream_t s) {
    return pieces_of(g, count) <= FEW_TENSORS ? launch_squares_of<FEW_TENSORS>(g, count, ws, s) : launch_squares_of<NORM_TENSORS>(g, count, ws, s);
}

hipError_t launch_grad_norm(const Gradient* g, int64_t count, double max_norm, float* norm, float* factor, void* ws, hipStream_t s) {
    const int parts = launch_squares(g, count, ws, s);
    hipLaunchKernelGGL(k_grad_norm, dim3(1), dim3(1024), 0, s, (const double*)ws, parts, max_norm, norm, factor);
    return hipGetLastError();
}

// The tensors read last are clipped first: the last-level cache still has them.
template <int MOST, bool APART>
static void launch_scale(const Gradient* g, const Gradient* out, int64_t count, int parts, double max_norm, float* norm, float* factor, void* ws,
                         hipStream_t s) {
    const auto tables = tables_of<MOST, ScaleTable<MOST, APART>>(g, count, [&](ScaleTable<MOST, APART>& t, int entry, int64_t i, int64_t at) {
        t.put(entry, (uint8_t*)out[i].data + at * (out[i].bf16 ? 2 : 4));
    });
    // up to 1024 sums are added up by each workgroup (28 tensors of 0.3 million values in all: 10.8 us, 14.2 with a launch more)
    const bool join = !tables.empty() && parts <= 1024;
    if (!join) hipLaunchKernelGGL(k_grad_norm, dim3(1), dim3(1024), 0, s, (const double*)ws, parts, max_norm, norm, factor);
    for (auto t = tables.rbegin(); t != tables.rend(); ++t) {
        if (join) hipLaunchKernelGGL((k_grad_scale<MOST, APART, true>), dim3(grid_of(*t)), dim3(256), 0, s, *t, (const double*)ws, parts, max_norm, norm, (const float*)nullptr);
        else hipLaunchKernelGGL((k_grad_scale<MOST, APART, false>), dim3(grid_of(*t)), dim3(256), 0, s, *t, (const double*)nullptr, 0, 0.0, (float*)nullptr, (const float*)factor);
    }
}
hipError_t launch_grad_clip(const Gradient* g, const Gradient* out, int64_t count, double max_norm, float* norm, float* factor,
                            void* ws, hipStream_t s) {
    const int parts = launch_squares(g, count, ws, s);
    bool apart = false;
    for (int64_t i = 0; i < count; ++i) apart = apart || g[i].data != out[i].data;
    if (pieces_of(g, count) <= FEW_TENSORS) launch_scale<FEW_TENSORS, true>(g, out, count, parts, max_norm, norm, factor, ws, s);
    else if (apart) launch_scale<SCALE_TENSORS, true>(g, out, count, parts, max_norm, norm, factor, ws, s);
    else launch_scale<NORM_TENSORS, false>(g, out, count, parts, max_norm, norm, factor, ws, s);
    return hipGetLastError();
}

}  // namespace nf4
