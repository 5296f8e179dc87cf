// block_norm.hip -- the norms before and after a block with its gate, residual scale and residual
// addition, forward and backward (gfx950).
//
// Mathematics.  n(a) = a s(a), s(a) = 1 / sqrt(mean(a^2) + eps).  Forward, for each token's row:
//   p  = n(x) post            (or x, without a norm after the block)
//   h' = h + scale gate p     rounded to the stream's type
//   y  = n(h') pre            of the h' that was rounded, which is what the backward pass has
// Backward, with a = n(h'), b = n(x), t = dy pre, q = scale gate dh':
//   dh' = dh + s(h') (t - a mean(t a)),   dpre = sum over tokens of dy a
//   u = q post,  dx = s(x) (u - b mean(u b)),   dpost = sum of q b,   dgate = sum of scale p dh'
// and the stream's gradient is dh'.  Both factors s are computed again from h' and x, which have to be read
// anyway: nothing but the operands is kept between the passes.  Sums and products are fp32, each output is
// rounded once.  Squares that leave fp32 (values past 1.8e19) are summed again times 2^-160.
//
// Shape.  Bound by HBM: each operand is read once and each output written once, so a row stays in the
// registers of the threads that share it (8 values of 16 bytes a thread and operand), one wave up to a width
// of 1024, else a workgroup.  Workers (a wave or a workgroup) walk along a stretch of rows: the next row's
// operands are loaded while one is computed, the weights stay in registers, and the sums over tokens of dpre,
// dpost and dgate are kept there; the workers' sums are added up in a second launch, in a fixed order.
#include "rows.h"
#include "step.h"

namespace nf4 {

struct NormArgs {
    RowsView h, x, dy, dh;    // read; data of null: not there
    RowsView h_out, y;        // written: the stream (or its gradient) and the norm's output (or the block's gradient)
    const void *pre, *post, *gate;
    float *dpre, *dpost, *dgate;      // out, or
    float *part_pre, *part_post, *part_gate;      // the workers' sums: [worker][K], of gates [worker][2][K]
    int64_t M, gate_span;     // tokens; tokens of a gate's row
    int64_t rows;             // of a worker
    int K;
    bool norm_pre, norm_post;
    float scale, eps, per;    // per: 1 / K
};

constexpr float NORM_LARGE = 3e38f;
constexpr float NORM_SHRINK = 0x1p-80f;

// What turns a row into its norm: value * shrink * factor.
struct Factor {
    float shrink, factor;
};

// One row's operands in a thread.
template <typename S, typename W, int NC, bool BACK>
struct RowOperands {
    Eight<S> h[NC];
    Eight<S> dh[BACK ? NC : 1];
    Eight<uint16_t> x[NC];
    Eight<uint16_t> dy[BACK ? NC : 1];
    Eight<W> gate[NC];
};

template <typename S, typename W, int WAVES, int NC, bool BACK>
struct RowOf {
    static constexpr int THREADS = 64 * WAVES;
    const NormArgs& a;
    int t;                    // thread among those of the row
    __device__ __forceinline__ int column(int i) const { return 8 * (t + i * THREADS); }
    __device__ __forceinline__ void load(RowOperands<S, W, NC, BACK>& r, int64_t row) const {
#pragma unroll
        for (int i = 0; i < NC; ++i) {
            const int c = column(i), left = a.K - c;
            if (!BACK || a.norm_pre) r.h[i] = load_eight((const S*)a.h.data + row * a.h.stride + c, left);
            if (a.x.data) r.x[i] = load_eight((const uint16_t*)a.x.data + row * a.x.stride + c, left);
            if (a.gate) r.gate[i] = load_eight((const W*)a.gate + row / a.gate_span * a.K + c, left);
            if constexpr (BACK) {
                if (a.norm_pre) r.dy[i] = load_eight((const uint16_t*)a.dy.data + row * a.dy.stride + c, left);
                if (a.dh.data) r.dh[i] = load_eight((const S*)a.dh.data + row * a.dh.stride + c, left);
            }
        }
    }
    // weights of the thread's columns; ones where there are none
    __device__ __forceinline__ void weights(Eight<W> (&w)[NC], const void* p) const {
        const float one[8] = {1.0f, 1.0f, 1.0f, 1.0f, 1.0f, 1.0f, 1.0f, 1.0f};
#pragma unroll
        for (int i = 0; i < NC; ++i) w[i] = p ? load_eight((const W*)p + column(i), a.K - column(i)) : pack_eight<W>(one);
    }
};

// The factor of a row's norm from the sum of its squares; `again` sums its squares shrunk.
template <typename F>
__device__ __forceinline__ Factor factor_of(float squares, const NormArgs& a, F&& again) {
    if (__builtin_expect(squares < NORM_LARGE, 1)) return Factor{1.0f, __frsqrt_rn(squares * a.per + a.eps)};
    return Factor{NORM_SHRINK, __frsqrt_rn(again() * a.per)};       // (infinities and NaN come here too: eps 2^-160 is nothing)
}

template <int WAVES>
__device__ __forceinline__ int64_t worker_of() {
    return WAVES == 1 ? (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6) : (int64_t)blockIdx.x;
}

template <typename S, typename W, int WAVES, int NC>
__global__ __launch_bounds__(WAVES == 1 ? 256 : 64 * WAVES)
void k_block_norm_fwd(NormArgs a) {
    __shared__ float shared[2 * WAVES];
    int turn = 0;
    const RowOf<S, W, WAVES, NC, false> of{a, WAVES == 1 ? (int)(threadIdx.x & 63) : (int)threadIdx.x};
    const int64_t first = worker_of<WAVES>() * a.rows, end = first + a.rows < a.M ? first + a.rows : a.M;
    if (first >= end) return;             // (all threads of a barrier's workgroup together)
    Eight<W> pre[NC], post[NC];
    RowOperands<S, W, NC, false> next, now;
    of.load(next, first);
    of.weights(pre, a.pre);
    of.weights(post, a.post);
    for (int64_t row = first; row < end; ++row) {
        now = next;
        if (row + 1 < end) of.load(next, row + 1);
        float h[NC][8];
#pragma unroll
        for (int i = 0; i < NC; ++i) unpack_eight<S>(now.h[i], h[i]);
        if (a.x.data) {
            float p[NC][8];
#pragma unroll
            for (int i = 0; i < NC; ++i) unpack_eight<uint16_t>(now.x[i], p[i]);
            if (a.norm_post) {
                auto squares = [&](float shrink) {
                    float q[1] = {0.0f};
#pragma unroll
                    for (int i = 0; i < NC; ++i)
#pragma unroll
                        for (int j = 0; j < 8; ++j) q[0] = __fmaf_rn(p[i][j] * shrink, p[i][j] * shrink, q[0]);
                    row_sums<WAVES>(q, shared, turn);
                    return q[0];
                };
                const Factor f = factor_of(squares(1.0f), a, [&] { return squares(NORM_SHRINK); });
#pragma unroll
                for (int i = 0; i < NC; ++i) {
                    float w[8];
                    unpack_eight<W>(post[i], w);
#pragma unroll
                    for (int j = 0; j < 8; ++j) p[i][j] = p[i][j] * f.shrink * f.factor * w[j];
                }
            }
#pragma unroll
            for (int i = 0; i < NC; ++i) {
                float g[8] = {1.0f, 1.0f, 1.0f, 1.0f, 1.0f, 1.0f, 1.0f, 1.0f};
                if (a.gate) unpack_eight<W>(now.gate[i], g);
#pragma unroll
                for (int j = 0; j < 8; ++j) h[i][j] += a.scale * g[j] * p[i][j];
                const Eight<S> e = pack_eight<S>(h[i]);
                unpack_eight<S>(e, h[i]);
                const int c = of.column(i);
                store_eight((S*)a.h_out.data + row * a.h_out.stride + c, a.K - c, e);
            }
        }
        if (a.norm_pre) {
            auto squares = [&](float shrink) {
                float q[1] = {0.0f};
#pragma unroll
                for (int i = 0; i < NC; ++i)
#pragma unroll
                    for (int j = 0; j < 8; ++j) q[0] = __fmaf_rn(h[i][j] * shrink, h[i][j] * shrink, q[0]);
                row_sums<WAVES>(q, shared, turn);
                return q[0];
            };
            const Factor f = factor_of(squares(1.0f), a, [&] { return squares(NORM_SHRINK); });
#pragma unroll
            for (int i = 0; i < NC; ++i) {
                float w[8];
                unpack_eight<W>(pre[i], w);
#pragma unroll
                for (int j = 0; j < 8; ++j) w[j] = h[i][j] * f.shrink * f.factor * w[j];
                const int c = of.column(i);
                store_eight((uint16_t*)a.y.data + row * a.y.stride + c, a.K - c, pack_eight<uint16_t>(w));
            }
        }
    }
}

// LEARN: the sums over tokens are wanted.
template <typename S, typename W, int WAVES, int NC, bool LEARN>
__global__ __launch_bounds__(WAVES == 1 ? 256 : 64 * WAVES)
void k_block_norm_bwd(NormArgs a) {
    __shared__ float shared[2 * 3 * WAVES];
    int turn = 0;
    const RowOf<S, W, WAVES, NC, true> of{a, WAVES == 1 ? (int)(threadIdx.x & 63) : (int)threadIdx.x};
    const int64_t worker = worker_of<WAVES>(), first = worker * a.rows, end = first + a.rows < a.M ? first + a.rows : a.M;
    if (first >= end) return;
    Eight<W> pre[NC], post[NC];
    RowOperands<S, W, NC, true> next, now;
    of.load(next, first);
    of.weights(pre, a.pre);
    of.weights(post, a.post);
    float spre[NC][8] = {}, spost[NC][8] = {}, sgate[NC][8] = {};
    auto put = [&](float* to, const float (&v)[NC][8]) {
#pragma unroll
        for (int i = 0; i < NC; ++i) {
            const int c = of.column(i);
            store_eight(to + c, a.K - c, pack_eight<float>(v[i]));
        }
    };
    // one of the row sums in turn (the shared numbers are laid out for three)
    auto sum = [&](float v) {
        float q[3] = {v, 0.0f, 0.0f};
        row_sums<WAVES>(q, shared, turn);
        return q[0];
    };
    for (int64_t row = first; row < end; ++row) {
        now = next;
        if (row + 1 < end) of.load(next, row + 1);
        float d[NC][8], x[NC][8];
        // ---- through the norm before the next block ----
        float q[3] = {0.0f, 0.0f, 0.0f};          // squares of h', t h', squares of x
        if (a.norm_pre) {
#pragma unroll
            for (int i = 0; i < NC; ++i) {
                float h[8], t[8], w[8];
                unpack_eight<S>(now.h[i], h);
                unpack_eight<uint16_t>(now.dy[i], t);
                unpack_eight<W>(pre[i], w);
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    q[0] = __fmaf_rn(h[j], h[j], q[0]);
                    q[1] = __fmaf_rn(t[j] * w[j], h[j], q[1]);
                }
            }
        }
        if (a.x.data) {
#pragma unroll
            for (int i = 0; i < NC; ++i) {
                unpack_eight<uint16_t>(now.x[i], x[i]);
                if (a.norm_post)
#pragma unroll
                    for (int j = 0; j < 8; ++j) q[2] = __fmaf_rn(x[i][j], x[i][j], q[2]);
            }
        }
        row_sums<WAVES>(q, shared, turn);
        Factor f{1.0f, 0.0f}, g{1.0f, 1.0f};
        float mean = 0.0f;                        // of t a
        if (a.norm_pre) {
            f = factor_of(q[0], a, [&] {
                float v = 0.0f;
#pragma unroll
                for (int i = 0; i < NC; ++i) {
                    float h[8];
                    unpack_eight<S>(now.h[i], h);
#pragma unroll
                    for (int j = 0; j < 8; ++j) v = __fmaf_rn(h[j] * NORM_SHRINK, h[j] * NORM_SHRINK, v);
                }
                return sum(v);
            });
            mean = q[1] * f.factor * a.per;
            if (__builtin_expect(!(q[0] < NORM_LARGE && fabsf(q[1]) < NORM_LARGE), 0)) {      // t h' left fp32: the sum of t a itself
                float v = 0.0f;
#pragma unroll
                for (int i = 0; i < NC; ++i) {
                    float h[8], t[8], w[8];
                    unpack_eight<S>(now.h[i], h);
                    unpack_eight<uint16_t>(now.dy[i], t);
                    unpack_eight<W>(pre[i], w);
#pragma unroll
                    for (int j = 0; j < 8; ++j) v = __fmaf_rn(t[j] * w[j], h[j] * f.shrink * f.factor, v);
                }
                mean = sum(v) * a.per;
            }
        }
#pragma unroll
        for (int i = 0; i < NC; ++i) {
            float h[8], t[8], w[8];
            if (a.dh.data) unpack_eight<S>(now.dh[i], d[i]);
            else
#pragma unroll
                for (int j = 0; j < 8; ++j) d[i][j] = 0.0f;
            if (a.norm_pre) {
                unpack_eight<S>(now.h[i], h);
                unpack_eight<uint16_t>(now.dy[i], t);
                unpack_eight<W>(pre[i], w);
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const float n = h[j] * f.shrink * f.factor;
                    if (LEARN) spre[i][j] = __fmaf_rn(t[j], n, spre[i][j]);
                    d[i][j] += (t[j] * w[j] - n * mean) * f.factor * f.shrink;
                }
            }
            const int c = of.column(i);
            store_eight((S*)a.h_out.data + row * a.h_out.stride + c, a.K - c, pack_eight<S>(d[i]));
        }
        // ---- through the gate and the norm after the block ----
        if (a.y.data) {
            if (a.norm_post) {
                g = factor_of(q[2], a, [&] {
                    float v = 0.0f;
#pragma unroll
                    for (int i = 0; i < NC; ++i)
#pragma unroll
                        for (int j = 0; j < 8; ++j) v = __fmaf_rn(x[i][j] * NORM_SHRINK, x[i][j] * NORM_SHRINK, v);
                    return sum(v);
                });
            }
            float over = 0.0f;                    // the sum of u b
#pragma unroll
            for (int i = 0; i < NC; ++i) {
                float w[8], e[8] = {1.0f, 1.0f, 1.0f, 1.0f, 1.0f, 1.0f, 1.0f, 1.0f};
                if (a.gate) unpack_eight<W>(now.gate[i], e);
                unpack_eight<W>(post[i], w);
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const float b = x[i][j] * g.shrink * g.factor;
                    const float u = a.scale * e[j] * d[i][j];
                    if (LEARN) {
                        spost[i][j] = __fmaf_rn(u, b, spost[i][j]);
                        sgate[i][j] = __fmaf_rn(a.scale * d[i][j], b * w[j], sgate[i][j]);
                    }
                    d[i][j] = u * w[j];
                    over = __fmaf_rn(d[i][j], b, over);
                    x[i][j] = b;
                }
            }
            if (a.norm_post) {
                over = sum(over) * a.per;
#pragma unroll
                for (int i = 0; i < NC; ++i)
#pragma unroll
                    for (int j = 0; j < 8; ++j) d[i][j] = (d[i][j] - x[i][j] * over) * g.factor * g.shrink;
            }
#pragma unroll
            for (int i = 0; i < NC; ++i) {
                const int c = of.column(i);
                store_eight((uint16_t*)a.y.data + row * a.y.stride + c, a.K - c, pack_eight<uint16_t>(d[i]));
            }
            if (LEARN && a.dgate) {               // a gate's last token here: its sum leaves the registers
                const int64_t gate = row / a.gate_span, start = gate * a.gate_span;
                if (row + 1 == end || row + 1 == start + a.gate_span) {
                    const bool whole = start >= first && start + a.gate_span <= end;
                    put(whole ? a.dgate + gate * a.K : a.part_gate + (2 * worker + (first / a.gate_span == gate ? 0 : 1)) * a.K, sgate);
#pragma unroll
                    for (int i = 0; i < NC; ++i)
#pragma unroll
                        for (int j = 0; j < 8; ++j) sgate[i][j] = 0.0f;
                }
            }
        }
    }
    if constexpr (LEARN) {
        if (a.dpre) put(a.part_pre ? a.part_pre + worker * a.K : a.dpre, spre);
        if (a.dpost) put(a.part_post ? a.part_post + worker * a.K : a.dpost, spost);
    }
}

// The workers' sums, added up.  blockIdx.y: 0 of pre, 1 of post, then the gates that more than one worker has a part of.
// 16 threads hold 4 columns each, 16 others take every 16th worker; their sums are added in order.
struct JoinArgs {
    float *dpre, *dpost, *dgate;
    const float *part_pre, *part_post, *part_gate;
    int64_t gates, gate_span, rows, workers;
    int K;
};
__global__ __launch_bounds__(256)
void k_block_norm_join(JoinArgs a) {
    __shared__ float4 sums[16][16];
    const int lane = threadIdx.x & 15, slice = threadIdx.x >> 4;
    const int c = blockIdx.x * 64 + lane * 4;
    auto join = [&](int64_t from, int64_t to, float* out, auto&& row_of) {
        float4 s = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 4
        for (int64_t w = from + slice; w < to; w += 16) {
            const float* p = row_of(w) + c;
            if (c + 4 <= a.K) {
                typedef float f4 __attribute__((ext_vector_type(4), aligned(4)));
                const f4 v = *reinterpret_cast<const f4*>(p);
                s = make_float4(s.x + v.x, s.y + v.y, s.z + v.z, s.w + v.w);
            } else {
                if (c < a.K) s.x += p[0];
                if (c + 1 < a.K) s.y += p[1];
                if (c + 2 < a.K) s.z += p[2];
            }
        }
        sums[slice][lane] = s;
        __syncthreads();
        if (slice == 0) {
#pragma unroll
            for (int i = 1; i < 16; ++i) {
                const float4 v = sums[i][lane];
                s = make_float4(s.x + v.x, s.y + v.y, s.z + v.z, s.w + v.w);
            }
            const float v[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (c + i < a.K) out[c + i] = v[i];
        }
        __syncthreads();
    };
    if (blockIdx.y == 0) {
        if (a.dpre) join(0, a.workers, a.dpre, [&](int64_t w) { return a.part_pre + w * a.K; });
    } else if (blockIdx.y == 1) {
        if (a.dpost) join(0, a.workers, a.dpost, [&](int64_t w) { return a.part_post + w * a.K; });
    } else if (a.dgate) {
        for (int64_t g = blockIdx.y - 2; g < a.gates; g += gridDim.y - 2) {
            const int64_t start = g * a.gate_span, w0 = start / a.rows, w1 = a.workers > 0 ? (start + a.gate_span - 1) / a.rows : -1;
            if (w0 == w1) continue;       // (that worker has written it)
            join(w0, w1 + 1, a.dgate + g * a.K, [&](int64_t w) { return a.part_gate + (2 * w + (w * a.rows / a.gate_span == g ? 0 : 1)) * a.K; });
        }
    }
}

// Threads that share a row, and the rows that a worker walks along.
struct NormShape {
    int waves, chunks;        // waves of a row; times 8 values a thread
    int64_t rows, workers;
};
static NormShape norm_shape(int64_t M, int64_t K, bool learn) {
    NormShape p{};
    p.waves = K <= 1024 ? 1 : K <= 2048 ? 4 : K <= 4096 ? 8 : 16;
    p.chunks = K <= 512 ? 1 : K <= 1024 ? 2 : K <= 8192 ? 1 : K <= 16384 ? 2 : 4;
    // workers: those that run at once on 256 compute units
    const int64_t most = p.waves == 1 ? 4096 : p.waves == 4 ? 1024 : 512;
    p.rows = (M + most - 1) / most;
    p.rows = p.rows < 1 ? 1 : p.rows;
    p.workers = (M + p.rows - 1) / p.rows;
    (void)learn;
    return p;
}

template <typename F>
static void with_shape(const NormShape& p, F&& f) {
#define NF4_SHAPE(w, c) \
    if (p.waves == w && p.chunks == c) f(std::integral_constant<int, w>{}, std::integral_constant<int, c>{})
    NF4_SHAPE(1, 1);
    NF4_SHAPE(1, 2);
    NF4_SHAPE(4, 1);
    NF4_SHAPE(8, 1);
    NF4_SHAPE(16, 1);
    NF4_SHAPE(16, 2);
    NF4_SHAPE(16, 4);
#undef NF4_SHAPE
}
template <typename F>
static void with_types(const BlockNorm& n, F&& f) {
    if (n.stream_bf16) n.weights_bf16 ? f(uint16_t{}, uint16_t{}) : f(uint16_t{}, float{});
    else n.weights_bf16 ? f(float{}, uint16_t{}) : f(float{}, float{});
}

static NormArgs norm_args(const BlockNorm& n, int64_t M, int64_t K, const NormShape& p) {
    NormArgs a{};
    a.pre = n.pre;
    a.post = n.post;
    a.gate = n.gate;
    a.M = M;
    a.K = (int)K;
    a.gate_span = n.gate ? M / n.gate_rows : M;
    a.rows = p.rows;
    a.norm_pre = n.norm_pre;
    a.norm_post = n.norm_post;
    a.scale = n.scale;
    a.eps = n.eps;
    a.per = (float)(1.0 / (double)K);
    return a;
}

hipError_t launch_block_norm_fwd(const BlockNorm& n, int64_t M, int64_t K, const RowsView& h, const RowsView& x,
                                 const RowsView& h_out, const RowsView& y, hipStream_t s) {
    const NormShape p = norm_shape(M, K, false);
    NormArgs a = norm_args(n, M, K, p);
    a.h = h;
    a.x = x;
    a.h_out = h_out;
    a.y = y;
    with_types(n, [&](auto st, auto wt) {
        with_shape(p, [&](auto waves, auto chunks) {
            constexpr int W = decltype(waves)::value;
            const dim3 grid((uint32_t)(W == 1 ? (p.workers + 3) / 4 : p.workers)), block(W == 1 ? 256 : 64 * W);
            hipLaunchKernelGGL((k_block_norm_fwd<decltype(st), decltype(wt), W, decltype(chunks)::value>), grid, block, 0, s, a);
        });
    });
    return hipGetLastError();
}

// The workers' sums in the workspace: of pre, of post, of gates (two for each worker, where a worker's stretch can end
// inside a gate's tokens).
struct NormParts {
    size_t pre, post, gate, bytes;
};
static NormParts norm_parts(const NormShape& p, int64_t M, int64_t K, int64_t gate_rows, bool dpre, bool dpost, bool dgate) {
    NormParts q{};
    const size_t one = (size_t)p.workers * K * sizeof(float);
    if (p.workers == 1) return q;
    q.pre = 0;
    q.post = q.pre + (dpre ? one : 0);
    q.gate = q.post + (dpost ? one : 0);
    q.bytes = q.gate + (dgate && M > gate_rows ? 2 * one : 0);
    q.bytes = (q.bytes + 255) & ~(size_t)255;
    return q;
}
size_t block_norm_ws_bytes(int64_t M, int64_t K, int64_t gate_rows, bool dpre, bool dpost, bool dgate) {
    const NormShape p = norm_shape(M, K, dpre || dpost || dgate);
    return norm_parts(p, M, K, gate_rows, dpre, dpost, dgate).bytes;
}

hipError_t launch_block_norm_bwd(const BlockNorm& n, int64_t M, int64_t K, const RowsView& h, const RowsView& x,
                                 const RowsView& dy, const RowsView& dh, const RowsView& dh_out, const RowsView& dx,
                                 float* dpre, float* dpost, float* dgate, void* ws, hipStream_t s) {
    const bool learn = dpre || dpost || dgate;
    const NormShape p = norm_shape(M, K, learn);
    NormArgs a = norm_args(n, M, K, p);
    a.h = h;
    a.x = x;
    if (!n.norm_post && !learn) a.x = RowsView{};       // (the block's output itself is in none of what is wanted)
    a.dy = dy;
    a.dh = dh;
    a.h_out = dh_out;
    a.y = dx;
    a.dpre = dpre;
    a.dpost = dpost;
    a.dgate = dgate;
    const NormParts q = norm_parts(p, M, K, n.gate_rows, dpre, dpost, dgate);
    if (q.bytes > 0) {
        a.part_pre = (float*)((uint8_t*)ws + q.pre);
        a.part_post = (float*)((uint8_t*)ws + q.post);
        a.part_gate = (float*)((uint8_t*)ws + q.gate);
    }
    if (M > 0)
        with_types(n, [&](auto st, auto wt) {
            with_shape(p, [&](auto waves, auto chunks) {
                constexpr int W = decltype(waves)::value, C = decltype(chunks)::value;
                const dim3 grid((uint32_t)(W == 1 ? (p.workers + 3) / 4 : p.workers)), block(W == 1 ? 256 : 64 * W);
                if (learn) hipLaunchKernelGGL((k_block_norm_bwd<decltype(st), decltype(wt), W, C, true>), grid, block, 0, s, a);
                else hipLaunchKernelGGL((k_block_norm_bwd<decltype(st), decltype(wt), W, C, false>), grid, block, 0, s, a);
            });
        });
    if (q.bytes > 0 || (M == 0 && learn)) {
        const int64_t gates = dgate && M != n.gate_rows ? n.gate_rows : 0;      // (a token's own gate is never shared)
        const JoinArgs j{dpre, dpost, dgate, a.part_pre, a.part_post, a.part_gate, gates, a.gate_span, p.rows, p.workers, (int)K};
        const dim3 grid((uint32_t)((K + 63) / 64), (uint32_t)(2 + (gates < 4096 ? gates : 4096)));
        hipLaunchKernelGGL(k_block_norm_join, grid, dim3(256), 0, s, j);
    }
    return hipGetLastError();
}

}  // namespace nf4
