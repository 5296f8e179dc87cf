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
// rounded once.  Squares that leave fp32 (values past 1.8e19), or an eps next to its end, are summed again times 2^-160.
//
// Shape.  Bound by HBM: each operand is read once and each output written once, so a row stays in the
// registers of the threads that share it (8 values of 16 bytes a thread and operand), one wave up to a width
// of 512, else a workgroup of as many waves as it takes.  Workers (a wave or a workgroup) walk along a stretch of
// rows: the next row's operands are loaded while one is computed, the weights stay in registers, and the sums over
// tokens of dpre, dpost and dgate are kept there; the workers' sums are added up in a second launch, in a fixed
// order.  (Gradients with sums past a width of 4096 spill 4 to 17 registers where the stream or the weights are fp32.  Past a
// width of 8192 the sums lie in LDS, and the rows on their way and the weights do not stay.)  4096 tokens of
// width 8192, all bf16: forward 44 us (268 MB, 6.1 TB/s), backward with all sums 77 us
// (403 MB, 5.2 TB/s) and 5 for the join; 16 tokens of width 4096 3.5 us.
#include "rows.h"
#include "step.h"

namespace nf4 {

struct NormArgs {
    RowsView h, x, dy, dh;    // read; data of null: not there
    RowsView h_out, y;        // written: the stream (or its gradient) and the norm's output (or the block's gradient)
    const void *pre, *post, *gate;
    float *dpre, *dpost, *dgate;      // out, or
    float *part_pre, *part_post, *part_gate;      // the workgroups' sums: [workgroup][K], of gates [worker][2][K]
    uint32_t M, gate_span;    // tokens; tokens of a gate's row
    uint32_t rows;            // of a worker
    uint32_t K;
    bool norm_pre, norm_post;
    float scale, eps, per;    // per: 1 / K
    float large, eps_shrunk;  // sums of squares from which eps and they leave fp32; eps times 2^-160
};

constexpr float NORM_LARGE = 3e38f;
constexpr float NORM_SHRINK = 0x1p-80f;
// t h' is summed times 2^80, for gradients and rows whose products lie below fp32's normal numbers although s(h') brings them
// back; the sums that this takes past its end, like those that leave it by themselves, are summed again as t a.
constexpr float NORM_RAISE = 0x1p80f;     // (1 / NORM_SHRINK)
// 1 / the root of the mean square plus eps, from a row's sum of squares: whether that fits fp32, and from the squares times
// 2^-160 where it does not (there eps counts too, where it is large itself).
__device__ __forceinline__ bool fits(float squares, const NormArgs& a) { return squares < a.large; }
__device__ __forceinline__ float inverse_root(float squares, const NormArgs& a) { return __frsqrt_rn(squares * a.per + a.eps); }
__device__ __forceinline__ float inverse_root_shrunk(float squares, const NormArgs& a) {
    return __frsqrt_rn(squares * a.per + a.eps_shrunk) * NORM_SHRINK;
}

// One row's operands in a thread.
template <typename S, typename W, int NC, bool BACK>
struct RowOperands {
    Eight<S> h[NC];
    Eight<S> dh[BACK ? NC : 1];
    Eight<uint16_t> x[NC];
    Eight<uint16_t> dy[BACK ? NC : 1];
    Eight<W> gate[BACK && NC > 1 ? 1 : NC];       // (else read where it is needed)
};

// The rows of a worker, and the thread's columns of them.
template <typename S, typename W, bool GROUP, int NC, bool STREAM, bool BACK>
struct RowOf {
    typedef RowOperands<S, W, NC, BACK> Operands;
    static constexpr bool GATE = !BACK || NC == 1;        // the gate is among a row's operands
    const NormArgs& a;
    uint32_t t, threads;                  // thread among those of a row
    uint32_t worker, first, end;          // rows first .. end - 1
    bool tail;                            // some of the wave's columns are past the row's end
    uint32_t gate, gate_left;             // of the row loaded next: its gate, and the gate's tokens from it on
    __device__ __forceinline__ explicit RowOf(const NormArgs& args) : a(args) {
        const uint32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
        t = GROUP ? threadIdx.x : threadIdx.x & 63;
        threads = GROUP ? blockDim.x : 64;
        worker = GROUP ? blockIdx.x : blockIdx.x * 4 + wave;
        tail = 8 * ((GROUP ? 64 * wave : 0) + (NC - 1) * threads + 64) > a.K;
        const uint64_t from = (uint64_t)worker * a.rows;
        first = from < a.M ? (uint32_t)from : a.M;
        end = a.M - first > a.rows ? first + a.rows : a.M;
        gate = first / a.gate_span;
        gate_left = a.gate_span - first % a.gate_span;
    }
    __device__ __forceinline__ uint32_t column(int i) const { return 8 * (t + i * threads); }
    // (a row shared by waves is longer than 512 values, one wave's may be shorter than eight)
    template <bool ONCE = false, typename T>
    __device__ __forceinline__ Eight<T> start(const T* p, uint32_t c) const {
        if (!GROUP && a.K < 8) return load_eight(p, c, a.K);
        return load_late<T, ONCE>(p, c, a.K);
    }
    template <typename T>
    __device__ __forceinline__ void finish(Eight<T>& e, uint32_t c) const {
        if (GROUP || a.K >= 8) settle(e, c, a.K);
    }
    __device__ __forceinline__ void load(Operands& r, uint32_t row) {
#pragma unroll
        for (int i = 0; i < NC; ++i) {
            const uint32_t c = column(i);
            if (!BACK || a.norm_pre) r.h[i] = start<STREAM>((const S*)a.h.data + row * a.h.stride, c);
            if (a.x.data) r.x[i] = start<STREAM>((const uint16_t*)a.x.data + row * a.x.stride, c);
            if constexpr (GATE) {
                if (a.gate) r.gate[i] = start((const W*)a.gate + (uint64_t)gate * a.K, c);
            }
            if constexpr (BACK) {
                if (a.norm_pre) r.dy[i] = start<STREAM>((const uint16_t*)a.dy.data + row * a.dy.stride, c);
                if (a.dh.data) r.dh[i] = start<STREAM>((const S*)a.dh.data + row * a.dh.stride, c);
            }
        }
        if (--gate_left == 0) {
            ++gate;
            gate_left = a.gate_span;
        }
    }
    // Operands that are not there: zeros, and gates of one.
    __device__ __forceinline__ void neutral(Operands& r) const {
        const float one[8] = {1.0f, 1.0f, 1.0f, 1.0f, 1.0f, 1.0f, 1.0f, 1.0f};
#pragma unroll
        for (int i = 0; i < NC; ++i) {
            r.h[i] = {};
            r.x[i] = {};
            if constexpr (GATE) r.gate[i] = pack_eight<W>(one);
            if constexpr (BACK) {
                r.dy[i] = {};
                r.dh[i] = {};
            }
        }
    }
    __device__ __forceinline__ void settle_all(Operands& r) const {
        if (!tail) return;
#pragma unroll
        for (int i = 0; i < NC; ++i) {
            const uint32_t c = column(i);
            if (!BACK || a.norm_pre) finish(r.h[i], c);
            if (a.x.data) finish(r.x[i], c);
            if constexpr (GATE) {
                if (a.gate) finish(r.gate[i], c);
            }
            if constexpr (BACK) {
                if (a.norm_pre) finish(r.dy[i], c);
                if (a.dh.data) finish(r.dh[i], c);
            }
        }
    }
    // a weight's values in the thread's columns; ones where there are none
    __device__ __forceinline__ Eight<W> weight(const void* p, int i) const {
        const float one[8] = {1.0f, 1.0f, 1.0f, 1.0f, 1.0f, 1.0f, 1.0f, 1.0f};
        if (!p) return pack_eight<W>(one);
        Eight<W> e = start((const W*)p, column(i));
        if (tail) finish(e, column(i));
        return e;
    }
};

// Weights of the thread's columns: held in registers for all rows, or, where a thread has several vectors of a row and no
// registers to spare, read again for each (from the caches).
template <typename OF, typename W, int NC>
struct Weights {
    static constexpr bool HELD = NC == 1;
    const OF& of;
    const void* p;
    Eight<W> w[HELD ? NC : 1];
    __device__ __forceinline__ Weights(const OF& o, const void* weight) : of(o), p(weight) {
        if constexpr (HELD)
#pragma unroll
            for (int i = 0; i < NC; ++i) w[i] = of.weight(p, i);
    }
    __device__ __forceinline__ void get(int i, float (&v)[8]) const {
        if constexpr (HELD) unpack_eight<W>(w[i], v);
        else unpack_eight<W>(of.weight(p, i), v);
    }
};

// Sums over tokens of the thread's columns: in registers, or, of several vectors, in LDS (16 bytes a thread side by side; each
// thread reads and writes its own places, so that no barrier is needed).  128 KB are both sums of two vectors a thread
// (gradients of 2048 x 16384, bf16: 114 us, 322 with sums and rows on their way spilled), or one of four (1024 x 32768: 262
// and 757; the other is spilled).
template <int NC, bool LDS>
struct TokenSums {
    float v[NC][8] = {};
    __device__ __forceinline__ explicit TokenSums(float4*) {}
    template <typename F>
    __device__ __forceinline__ void each(int i, F&& f) {
        f(v[i]);
    }
};
template <int NC>
struct TokenSums<NC, true> {
    float4* own;
    __device__ __forceinline__ explicit TokenSums(float4* places) : own(places + threadIdx.x) {
#pragma unroll
        for (int i = 0; i < 2 * NC; ++i) own[i * 1024] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    }
    template <typename F>
    __device__ __forceinline__ void each(int i, F&& f) {
        const float4 a = own[2 * i * 1024], b = own[(2 * i + 1) * 1024];
        float v[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
        f(v);
        own[2 * i * 1024] = make_float4(v[0], v[1], v[2], v[3]);
        own[(2 * i + 1) * 1024] = make_float4(v[4], v[5], v[6], v[7]);
    }
};

// GROUP: a row is shared by the waves of a workgroup, else each of four waves has rows of its own.  STREAM: nontemporal
// loads of what is read once.
template <typename S, typename W, bool GROUP, int NC, bool STREAM>
__global__ __launch_bounds__(GROUP ? 1024 : 256)
void k_block_norm_fwd(NormArgs a) {
    __shared__ float4 shared[2 * 4];
    int turn = 0;
    const int waves = blockDim.x >> 6;
    if constexpr (GROUP) {
        if (threadIdx.x < 8) shared[threadIdx.x] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        __syncthreads();
    }
    typedef RowOf<S, W, GROUP, NC, STREAM, false> Of;
    Of of(a);
    if (of.first >= of.end) return;       // (all threads of a barrier's workgroup together)
    constexpr bool UNIFORM = NC <= 2;
    // (the next row on its way: up to two vectors a thread there are registers for it, but for 13 that an fp32 stream with fp32
    // weights spills; 1024 x 32768 with four: 74 us, 122 with)
    constexpr bool AHEAD = NC <= 2;
    typename Of::Operands next, now;
    if constexpr (AHEAD) {
        of.neutral(next);
        of.load(next, of.first);
    }
    const Weights<Of, W, NC> pre(of, a.pre), post(of, a.post);
    // 1 / the root of the mean square of a row
    auto factor = [&](const float (&v)[NC][8]) {
        auto squares = [&](float shrink) {
            float q[1] = {0.0f};
#pragma unroll
            for (int i = 0; i < NC; ++i)
#pragma unroll
                for (int j = 0; j < 8; ++j) q[0] = __fmaf_rn(v[i][j] * shrink, v[i][j] * shrink, q[0]);
            row_sums<GROUP, UNIFORM>(q, shared, turn, waves);
            return q[0];
        };
        const float q = squares(1.0f);
        if (__builtin_expect(fits(q, a), 1)) return inverse_root(q, a);
        return inverse_root_shrunk(squares(NORM_SHRINK), a);         // (infinities and NaN come here too)
    };
    for (uint32_t row = of.first; row < of.end; ++row) {
        if constexpr (AHEAD) {
            now = next;
            if (row + 1 < of.end) of.load(next, row + 1);
        } else {
            of.neutral(now);
            of.load(now, row);
        }
        of.settle_all(now);
        float h[NC][8];
#pragma unroll
        for (int i = 0; i < NC; ++i) unpack_eight<S>(now.h[i], h[i]);
        if (a.x.data) {
            float p[NC][8];
#pragma unroll
            for (int i = 0; i < NC; ++i) unpack_eight<uint16_t>(now.x[i], p[i]);
            if (a.norm_post) {
                const float f = factor(p);
#pragma unroll
                for (int i = 0; i < NC; ++i) {
                    float w[8];
                    post.get(i, w);
#pragma unroll
                    for (int j = 0; j < 8; ++j) p[i][j] = p[i][j] * f * w[j];
                }
            }
#pragma unroll
            for (int i = 0; i < NC; ++i) {
                float g[8];
                unpack_eight<W>(now.gate[i], g);
#pragma unroll
                for (int j = 0; j < 8; ++j) h[i][j] += a.scale * g[j] * p[i][j];
                const Eight<S> e = pack_eight<S>(h[i]);
                unpack_eight<S>(e, h[i]);
                store_eight((S*)a.h_out.data + row * a.h_out.stride, of.column(i), a.K, e);
            }
        }
        if (a.norm_pre) {
            const float f = factor(h);
#pragma unroll
            for (int i = 0; i < NC; ++i) {
                float w[8];
                pre.get(i, w);
#pragma unroll
                for (int j = 0; j < 8; ++j) w[j] = h[i][j] * f * w[j];
                store_eight((uint16_t*)a.y.data + row * a.y.stride, of.column(i), a.K, pack_eight<uint16_t>(w));
            }
        }
    }
}

// LEARN: the sums over tokens are wanted.  dpost and dgate are both sums of scale d b (b = n(x)): of each gate's tokens
// that sum is kept, and leaves for both where a gate's tokens end.  One gate for all has one sum, which the join
// multiplies out; a gate of one token's own has no sum to keep, and dpost's takes the registers.
// THREADS: of a workgroup at most.  LEARN: 0, 1, or 2 where the gates are the tokens' own.
template <typename S, typename W, int THREADS, bool GROUP, int NC, bool STREAM, int LEARN>
__global__ __launch_bounds__(THREADS)
void k_block_norm_bwd(NormArgs a) {
    __shared__ float4 shared[2 * 3 * 4];
    __shared__ float4 places[LEARN && NC > 1 ? 8 * 1024 : 1];
    int turn = 0;
    const int waves = blockDim.x >> 6;
    if constexpr (GROUP) {
        if (threadIdx.x < 24) shared[threadIdx.x] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        __syncthreads();
    }
    typedef RowOf<S, W, GROUP, NC, STREAM, true> Of;
    Of of(a);
    // The next row's operands are loaded while one is computed, but for several vectors a thread, whose registers the rows on
    // their way would spill (gradient of 2048 x 16384, bf16: 91 us, 105 with them; fp32 129 and 178).
    constexpr bool AHEAD = NC == 1, UNIFORM = NC <= 2;
    typename Of::Operands next, now;
    if (of.first >= of.end) return;       // (all threads of a barrier's workgroup together)
    if constexpr (AHEAD) {
        of.neutral(next);
        of.load(next, of.first);
    }
    const Weights<Of, W, NC> pre(of, a.pre), post(of, a.post);
    TokenSums<LEARN ? NC : 1, LEARN && NC != 1> spre(places);
    TokenSums<LEARN ? NC : 1, LEARN && NC == 2> sover(places + (LEARN && NC == 2 ? 4 * 1024 : 0));
    constexpr bool OWN = LEARN == 2;
    const bool one_gate = a.gate && a.gate_span == a.M;
    bool posted = false;                          // the worker's sum of dpost is partly in memory
    auto put = [&](float* to, auto& sums) {
#pragma unroll
        for (int i = 0; i < NC; ++i) sums.each(i, [&](float (&v)[8]) { store_eight(to, of.column(i), a.K, pack_eight<float>(v)); });
    };
    // one of the row sums in turn (the shared numbers are laid out for three)
    auto sum = [&](float v) {
        float q[3] = {v, 0.0f, 0.0f};
        row_sums<GROUP, UNIFORM>(q, shared, turn, waves);
        return q[0];
    };
    uint32_t gate = of.first / a.gate_span, gate_first = gate * a.gate_span;        // of the row computed
    auto gate_of = [&](int i, float (&v)[8]) {
        if constexpr (Of::GATE) unpack_eight<W>(now.gate[i], v);
        else unpack_eight<W>(of.weight(a.gate ? (const W*)a.gate + (uint64_t)gate * a.K : nullptr, i), v);
    };
    // (the block's output stays as it was read where a thread has several vectors of it)
    constexpr bool KEPT = NC == 1;
    float kept[KEPT ? NC : 1][8];
    auto block = [&](int i, float factor, float (&v)[8]) {
        if constexpr (KEPT) {
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] = kept[i][j] * factor;
        } else {
            unpack_eight<uint16_t>(now.x[i], v);
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] *= factor;
        }
    };
    for (uint32_t row = of.first; row < of.end; ++row) {
        if constexpr (AHEAD) {
            now = next;
            if (row + 1 < of.end) of.load(next, row + 1);
        } else {
            of.neutral(now);
            of.load(now, row);
        }
        of.settle_all(now);
        float d[NC][8];
        // ---- through the norm before the next block (without one, h' and dy are zero) ----
        float q[3] = {0.0f, 0.0f, 0.0f};          // squares of h', t h' 2^80, squares of x
#pragma unroll
        for (int i = 0; i < NC; ++i) {
            float h[8], t[8], w[8], x[8];
            unpack_eight<S>(now.h[i], h);
            unpack_eight<uint16_t>(now.dy[i], t);
            pre.get(i, w);
            unpack_eight<uint16_t>(now.x[i], x);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                q[0] = __fmaf_rn(h[j], h[j], q[0]);
                q[1] = __fmaf_rn(t[j] * w[j], h[j] * NORM_RAISE, q[1]);
                q[2] = __fmaf_rn(x[j], x[j], q[2]);
                if constexpr (KEPT) kept[i][j] = x[j];
            }
        }
        row_sums<GROUP, UNIFORM>(q, shared, turn, waves);
        float f, mean;                            // s(h'); the mean of t a
        if (__builtin_expect(fits(q[0], a), 1)) {
            f = inverse_root(q[0], a);
        } else {
            float v = 0.0f;
#pragma unroll
            for (int i = 0; i < NC; ++i) {
                float h[8];
                unpack_eight<S>(now.h[i], h);
#pragma unroll
                for (int j = 0; j < 8; ++j) v = __fmaf_rn(h[j] * NORM_SHRINK, h[j] * NORM_SHRINK, v);
            }
            f = inverse_root_shrunk(sum(v), a);
        }
        mean = (f > 1.0f ? q[1] * (f * NORM_SHRINK) : q[1] * NORM_SHRINK * f) * a.per;
        if (__builtin_expect(!(fabsf(q[1]) < NORM_LARGE), 0)) {           // the sum of t a itself
            float v = 0.0f;
#pragma unroll
            for (int i = 0; i < NC; ++i) {
                float h[8], t[8], w[8];
                unpack_eight<S>(now.h[i], h);
                unpack_eight<uint16_t>(now.dy[i], t);
                pre.get(i, w);
#pragma unroll
                for (int j = 0; j < 8; ++j) v = __fmaf_rn(t[j] * w[j], h[j] * f, v);
            }
            mean = sum(v) * a.per;
        }
#pragma unroll
        for (int i = 0; i < NC; ++i) {
            float h[8], t[8], w[8];
            unpack_eight<S>(now.dh[i], d[i]);
            unpack_eight<S>(now.h[i], h);
            unpack_eight<uint16_t>(now.dy[i], t);
            pre.get(i, w);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                h[j] *= f;
                d[i][j] = __fmaf_rn(__fmaf_rn(t[j], w[j], -h[j] * mean), f, d[i][j]);
            }
            if constexpr (LEARN != 0)
                spre.each(i, [&](float (&s)[8]) {
#pragma unroll
                    for (int j = 0; j < 8; ++j) s[j] = __fmaf_rn(t[j], h[j], s[j]);
                });
            store_eight((S*)a.h_out.data + row * a.h_out.stride, of.column(i), a.K, pack_eight<S>(d[i]));
        }
        // ---- through the gate and the norm after the block ----
        if (a.y.data) {
            float g = 1.0f;                       // s(x)
            if (a.norm_post) {
                if (__builtin_expect(fits(q[2], a), 1)) {
                    g = inverse_root(q[2], a);
                } else {
                    float v = 0.0f;
#pragma unroll
                    for (int i = 0; i < NC; ++i) {
                        float x[8];
                        block(i, NORM_SHRINK, x);
#pragma unroll
                        for (int j = 0; j < 8; ++j) v = __fmaf_rn(x[j], x[j], v);
                    }
                    g = inverse_root_shrunk(sum(v), a);
                }
            }
            if constexpr (OWN) {
#pragma unroll
                for (int i = 0; i < NC; ++i) {
                    float w[8], e[8], x[8];
                    gate_of(i, e);
                    post.get(i, w);
                    block(i, g, x);
                    sover.each(i, [&](float (&s)[8]) {
#pragma unroll
                        for (int j = 0; j < 8; ++j) {
                            const float v = a.scale * d[i][j] * x[j];
                            s[j] = __fmaf_rn(v, e[j], s[j]);
                            w[j] *= v;
                        }
                    });
                    if (a.dgate) store_eight(a.dgate + (uint64_t)row * a.K, of.column(i), a.K, pack_eight<float>(w));
                }
            }
            float over = 0.0f;                    // the sum of u b
#pragma unroll
            for (int i = 0; i < NC; ++i) {
                float w[8], e[8], x[8];
                gate_of(i, e);
                post.get(i, w);
                block(i, g, x);
#pragma unroll
                for (int j = 0; j < 8; ++j) d[i][j] *= a.scale;
                if constexpr (LEARN != 0 && !OWN)
                    sover.each(i, [&](float (&s)[8]) {
#pragma unroll
                        for (int j = 0; j < 8; ++j) s[j] = __fmaf_rn(d[i][j], x[j], s[j]);
                    });
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    d[i][j] = d[i][j] * e[j] * w[j];
                    over = __fmaf_rn(d[i][j], x[j], over);
                    if constexpr (KEPT) kept[i][j] = x[j];
                }
            }
            if (a.norm_post) {
                over = sum(over) * a.per;
#pragma unroll
                for (int i = 0; i < NC; ++i) {
                    float x[8];
                    block(i, KEPT ? 1.0f : g, x);
#pragma unroll
                    for (int j = 0; j < 8; ++j) d[i][j] = __fmaf_rn(-x[j], over, d[i][j]) * g;
                }
            }
#pragma unroll
            for (int i = 0; i < NC; ++i) store_eight((uint16_t*)a.y.data + row * a.y.stride, of.column(i), a.K, pack_eight<uint16_t>(d[i]));
            if (LEARN && !OWN && a.gate && !one_gate && (row + 1 == of.end || row + 1 == gate_first + a.gate_span)) {
                // a gate's last token here: its sums leave the registers
                const bool whole = gate_first >= of.first && gate_first + a.gate_span <= of.end;
                float* to = whole ? a.dgate + (uint64_t)gate * a.K
                                  : a.part_gate + (2 * (uint64_t)of.worker + (gate_first <= of.first ? 0 : 1)) * a.K;
#pragma unroll
                for (int i = 0; i < NC; ++i) {
                    float w[8], e[8], s[8], was[8] = {};
                    float over[8];
                    post.get(i, w);
                    gate_of(i, e);
                    sover.each(i, [&](float (&v)[8]) {
#pragma unroll
                        for (int j = 0; j < 8; ++j) {
                            over[j] = v[j];
                            v[j] = 0.0f;
                        }
                    });
#pragma unroll
                    for (int j = 0; j < 8; ++j) s[j] = over[j] * w[j];
                    if (a.dgate) store_eight(to, of.column(i), a.K, pack_eight<float>(s));
                    if (a.dpost) {
                        float* post_to = (a.part_post ? a.part_post + (uint64_t)of.worker * a.K : a.dpost);
                        if (posted) unpack_eight<float>(load_eight((const float*)post_to, of.column(i), a.K), was);
#pragma unroll
                        for (int j = 0; j < 8; ++j) was[j] = __fmaf_rn(over[j], e[j], was[j]);
                        store_eight(post_to, of.column(i), a.K, pack_eight<float>(was));
                    }
                }
                posted = true;
            }
        }
        if (row + 1 == gate_first + a.gate_span) {
            ++gate;
            gate_first += a.gate_span;
        }
    }
    if constexpr (LEARN) {
        if (a.dpre) put(a.part_pre ? a.part_pre + (uint64_t)of.worker * a.K : a.dpre, spre);
        if (!OWN && one_gate && !a.part_post) {   // one worker
#pragma unroll
            for (int i = 0; i < NC; ++i) {
                float w[8], e[8], over[8];
                sover.each(i, [&](float (&v)[8]) { __builtin_memcpy(over, v, sizeof(v)); });
                post.get(i, w);
                unpack_eight<W>(of.weight(a.gate, i), e);
#pragma unroll
                for (int j = 0; j < 8; ++j) w[j] *= over[j], e[j] *= over[j];
                if (a.dgate) store_eight(a.dgate, of.column(i), a.K, pack_eight<float>(w));
                if (a.dpost) store_eight(a.dpost, of.column(i), a.K, pack_eight<float>(e));
            }
        } else if ((a.dpost || (a.dgate && one_gate)) && !posted) {
            put(a.part_post ? a.part_post + (uint64_t)of.worker * a.K : a.dpost, sover);
        }
    }
}

// The workers' sums, added up.  blockIdx.y: 0 of pre, 1 of post (and of the one gate for all), then the gates that more than
// one worker has a part of.  8 threads hold 4 columns each; 128 such groups take the workers in turn, and
// their sums are added in a fixed order.
struct JoinArgs {
    float *dpre, *dpost, *dgate;
    const float *part_pre, *part_post, *part_gate;
    const void *post, *gate;  // one gate for all: the factors of its sum (null: ones), else null
    int64_t gates, gate_span, rows, workers;
    int K;
    bool one_gate, weights_bf16;
};
constexpr int JOIN_COLUMNS = 32;
__global__ __launch_bounds__(1024)
void k_block_norm_join(JoinArgs a) {
    constexpr int SLICES = 128;
    __shared__ float4 sums[SLICES][8];
    const int lane = threadIdx.x & 7, slice = threadIdx.x >> 3;
    const int c = blockIdx.x * JOIN_COLUMNS + lane * 4;
    auto join = [&](int64_t from, int64_t to, auto&& row_of, auto&& put) {
        float4 s = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 4
        for (int64_t w = from + slice; w < to; w += SLICES) {
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
        float* column = reinterpret_cast<float*>(&sums[0][0]) + threadIdx.x % JOIN_COLUMNS;
        const int part = threadIdx.x / JOIN_COLUMNS, k = blockIdx.x * JOIN_COLUMNS + threadIdx.x % JOIN_COLUMNS;
        if (part < 8) {
            float v = 0.0f;
#pragma unroll
            for (int i = 0; i < SLICES / 8; ++i) v += column[(part * (SLICES / 8) + i) * JOIN_COLUMNS];
            column[part * (SLICES / 8) * JOIN_COLUMNS] = v;
        }
        __syncthreads();
        if (part == 0 && k < a.K) {
            float v = 0.0f;
#pragma unroll
            for (int i = 0; i < 8; ++i) v += column[i * (SLICES / 8) * JOIN_COLUMNS];
            put(k, v);
        }
        __syncthreads();
    };
    auto weight = [&](const void* p, int k) { return !p ? 1.0f : a.weights_bf16 ? bf16_to_f32(((const uint16_t*)p)[k]) : ((const float*)p)[k]; };
    if (blockIdx.y == 0) {
        if (a.dpre) join(0, a.workers, [&](int64_t w) { return a.part_pre + w * a.K; }, [&](int k, float v) { a.dpre[k] = v; });
    } else if (blockIdx.y == 1) {
        if (a.dpost || (a.dgate && a.one_gate))
            join(0, a.workers, [&](int64_t w) { return a.part_post + w * a.K; }, [&](int k, float v) {
                if (a.dpost) a.dpost[k] = v * weight(a.gate, k);
                if (a.dgate && a.one_gate) a.dgate[k] = v * weight(a.post, k);
            });
    } else {
        for (int64_t g = blockIdx.y - 2; g < a.gates; g += gridDim.y - 2) {
            const int64_t start = g * a.gate_span, w0 = start / a.rows, w1 = a.workers > 0 ? (start + a.gate_span - 1) / a.rows : -1;
            if (w0 == w1) continue;       // (that worker has written it)
            join(w0, w1 + 1, [&](int64_t w) { return a.part_gate + (2 * w + (w * a.rows >= start ? 0 : 1)) * a.K; },
                 [&](int k, float v) { a.dgate[g * a.K + k] = v; });
        }
    }
}

// Threads that share a row, and the rows that a worker walks along.  One vector a thread as far as a workgroup reaches: with
// two, 512 threads have the registers for the backward pass without spilling, but two waves a SIMD do not cover the sums'
// waits (gradient of 4096 x 8192: 105.7 us with two, 90.3 with one; of 4000 x 4099, where five waves of two vectors leave
// SIMDs idle, 95 and 68).
struct NormShape {
    int waves, chunks;        // waves of a row; times 8 values a thread
    int64_t rows, workers;
    bool group() const { return waves > 1; }
    dim3 grid() const { return dim3((uint32_t)(group() ? workers : (workers + 3) / 4)); }
    dim3 block() const { return dim3(group() ? 64 * waves : 256); }
};
// Workers: those that run at once.  `at_once` waves a compute unit, but one workgroup of more than 8 waves (forward 4096 x
// 8192: 46 us with one a compute unit, 47 with two, 53 with four).  Forward 32 (6000 x 256: 7.5 us, 13 with a quarter of them);
// backward, which has fewer waves at once, 16 (1001 x 2501: 12.6 us with 2 or 3 workgroups, 15.8 with 6); with sums over tokens
// 8, for each worker leaves sums to be joined (gradients of 6000 x 1000: 25 us with 4 workers of two waves a compute unit,
// 29 with 8; of 4096 x 4096: 45 us with one of eight, 48 with two, 73 with eight).
constexpr int FORWARD = 32, BACKWARD = 16, WITH_SUMS = 8;
static NormShape norm_shape(int64_t M, int64_t K, int at_once) {
    NormShape p{};
    p.chunks = K > 16384 ? 4 : K > 8192 ? 2 : 1;
    p.waves = (int)((K + 512 * p.chunks - 1) / (512 * p.chunks));
    const int per_unit = p.waves > 8 ? 1 : at_once / p.waves;
    const int64_t most = 256 * (int64_t)per_unit;
    p.rows = (M + most - 1) / most;
    p.rows = p.rows < 1 ? 1 : p.rows;
    p.workers = (M + p.rows - 1) / p.rows;
    return p;
}

template <typename F>
static void with_types(const BlockNorm& n, F&& f) {
    if (n.stream_bf16) n.weights_bf16 ? f(uint16_t{}, uint16_t{}) : f(uint16_t{}, float{});
    else n.weights_bf16 ? f(float{}, uint16_t{}) : f(float{}, float{});
}

// 32 MB of a bf16 operand and more, in whole lines of 128 bytes: nontemporal loads (4096 x 8192: 47 us forward and 82 backward,
// 55 and 92 without; rows that begin inside a line, which two workgroups read: 28.0 us backward of 1001 x 2501, 24.6 without).
// Past a width of 8192 from 64 MB on (backward with sums 2048 x 16384: 114 us, 121 without; forward 2048 x 8704 in fp32, 53
// and 46).
static bool streams(int64_t M, int64_t K, const NormShape& p) { return p.group() && M * K >= (int64_t)1 << (p.chunks == 1 ? 24 : 25) && K % 64 == 0; }

static NormArgs norm_args(const BlockNorm& n, int64_t M, int64_t K, const NormShape& p) {
    NormArgs a{};
    a.pre = n.pre;
    a.post = n.post;
    a.gate = n.gate;
    a.M = (uint32_t)M;
    a.K = (uint32_t)K;
    a.gate_span = (uint32_t)(n.gate ? M / n.gate_rows : M);
    a.rows = (uint32_t)p.rows;
    a.norm_pre = n.norm_pre;
    a.norm_post = n.norm_post;
    a.scale = n.scale;
    a.eps = n.eps;
    a.large = NORM_LARGE - n.eps;
    a.eps_shrunk = n.eps * NORM_SHRINK * NORM_SHRINK;
    a.per = (float)(1.0 / (double)K);
    return a;
}

hipError_t launch_block_norm_fwd(const BlockNorm& n, int64_t M, int64_t K, const RowsView& h, const RowsView& x,
                                 const RowsView& h_out, const RowsView& y, hipStream_t s) {
    const NormShape p = norm_shape(M, K, FORWARD);
    NormArgs a = norm_args(n, M, K, p);
    a.h = h;
    a.x = x;
    a.h_out = h_out;
    a.y = y;
    with_types(n, [&](auto st, auto wt) {
        auto run = [&](auto group, auto chunks, auto stream) {
            hipLaunchKernelGGL((k_block_norm_fwd<decltype(st), decltype(wt), decltype(group)::value, decltype(chunks)::value, decltype(stream)::value>),
                               p.grid(), p.block(), 0, s, a);
        };
        auto group = [&](auto chunks) {
            if (streams(M, K, p)) run(std::true_type{}, chunks, std::true_type{});
            else run(std::true_type{}, chunks, std::false_type{});
        };
        if (!p.group()) run(std::false_type{}, std::integral_constant<int, 1>{}, std::false_type{});
        else if (p.chunks == 1) group(std::integral_constant<int, 1>{});
        else if (p.chunks == 2) group(std::integral_constant<int, 2>{});
        else group(std::integral_constant<int, 4>{});
    });
    return hipGetLastError();
}

// The workers' sums in the workspace: of pre, of post (or of the one gate), of gates (two for each worker, whose stretch can
// begin and end inside a gate's tokens).
struct NormParts {
    size_t pre, post, gate, bytes;
};
static NormParts norm_parts(const NormShape& p, int64_t M, int64_t K, int64_t gate_rows, bool dpre, bool dpost, bool dgate) {
    NormParts q{};
    const size_t one = (size_t)p.workers * K * sizeof(float);
    if (p.workers <= 1) return q;
    q.pre = 0;
    q.post = q.pre + (dpre ? one : 0);
    q.gate = q.post + (dpost || (dgate && gate_rows == 1) ? one : 0);
    q.bytes = q.gate + (dgate && gate_rows > 1 && gate_rows < M ? 2 * one : 0);
    q.bytes = (q.bytes + 255) & ~(size_t)255;
    return q;
}
size_t block_norm_ws_bytes(int64_t M, int64_t K, int64_t gate_rows, bool dpre, bool dpost, bool dgate) {
    return norm_parts(norm_shape(M, K, WITH_SUMS), M, K, gate_rows, dpre, dpost, dgate).bytes;
}

hipError_t launch_block_norm_bwd(const BlockNorm& n, int64_t M, int64_t K, const RowsView& h, const RowsView& x,
                                 const RowsView& dy, const RowsView& dh, const RowsView& dh_out, const RowsView& dx,
                                 float* dpre, float* dpost, float* dgate, void* ws, hipStream_t s) {
    const bool learn = dpre || dpost || dgate;
    const NormShape p = norm_shape(M, K, learn ? WITH_SUMS : BACKWARD);
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
            auto run = [&](auto threads, auto group, auto chunks, auto stream) {
                constexpr int T = decltype(threads)::value, C = decltype(chunks)::value;
                constexpr bool G = decltype(group)::value, N = decltype(stream)::value;
                auto with = [&](auto kernel) { hipLaunchKernelGGL(kernel, p.grid(), p.block(), 0, s, a); };
                if (learn && n.gate && n.gate_rows == M && M > 1) with(k_block_norm_bwd<decltype(st), decltype(wt), T, G, C, N, 2>);
                else if (learn) with(k_block_norm_bwd<decltype(st), decltype(wt), T, G, C, N, 1>);
                else with(k_block_norm_bwd<decltype(st), decltype(wt), T, G, C, N, 0>);
            };
            auto group = [&](auto threads, auto chunks) {
                if (streams(M, K, p)) run(threads, std::true_type{}, chunks, std::true_type{});
                else run(threads, std::true_type{}, chunks, std::false_type{});
            };
            // (a workgroup of 1024 threads has 128 registers a thread: of a row of one or two vectors a thread none is spilled in
            // bf16 and up to 17 with fp32, of one of four 70 to 115 without sums and 186 to 270 with them)
            if (!p.group()) run(std::integral_constant<int, 256>{}, std::false_type{}, std::integral_constant<int, 1>{}, std::false_type{});
            else if (p.chunks == 1 && p.waves <= 8) group(std::integral_constant<int, 512>{}, std::integral_constant<int, 1>{});
            else if (p.chunks == 1) group(std::integral_constant<int, 1024>{}, std::integral_constant<int, 1>{});
            else if (p.chunks == 2) group(std::integral_constant<int, 1024>{}, std::integral_constant<int, 2>{});
            else group(std::integral_constant<int, 1024>{}, std::integral_constant<int, 4>{});
        });
    if (q.bytes > 0 || (M == 0 && learn)) {
        // (a token's own gate is never shared)
        const bool one = n.gate && n.gate_rows == 1;
        const int64_t gates = dgate && !one && M != n.gate_rows ? n.gate_rows : 0;
        const JoinArgs j{dpre, dpost, dgate, a.part_pre, a.part_post, a.part_gate, one ? n.post : nullptr, one ? n.gate : nullptr,
                         gates, a.gate_span, p.rows, p.workers, (int)K, one, n.weights_bf16};
        const dim3 grid((uint32_t)((K + JOIN_COLUMNS - 1) / JOIN_COLUMNS), (uint32_t)(2 + (gates < 4096 ? gates : 4096)));
        hipLaunchKernelGGL(k_block_norm_join, grid, dim3(1024), 0, s, j);
    }
    return hipGetLastError();
}

}  // namespace nf4
