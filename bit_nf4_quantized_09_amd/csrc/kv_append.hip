// kv_append.hip -- keys and values into the paged 8-bit cache, rotated on the way (gfx950).
//
// A page's scale is one power of two per head and kind: the smallest 2^e with every value
// there within +-448 2^e.  E4M3 keeps the same relative precision at every magnitude above
// 2^-6 of its unit, so a power of two loses nothing against a free scale, and a page's
// earlier codes move to a larger scale by an exact change of exponent (but for those that
// become subnormal).  Rotation keeps a pair's norm, so the scale is taken from pair norms,
// before the rotation: it needs no cos or sin and no second rotation.
//
// One wave owns one (page, kv head) of one sequence, so nothing races on a scale: it reads
// the page's new keys and values twice (from memory, then from cache), once for the scale
// and once to rotate, round and store them.  The page's wave is the one whose span of
// `span` packed tokens holds the page's first new token.  Bound by HBM for prompts (4 bytes
// read and 2 written per key/value pair, 4 per query value) and by the chain of dependent
// loads (starts, length, table, values) for single tokens.
#include "paged.h"

namespace nf4 {

struct AppendArgs {
    CacheView c;
    BatchView b;
    RopeView rope;
    HeadsView k, v, q, qo;
    int span;                 // packed tokens per workgroup column
    int spans;
    int kv_blocks;            // workgroups that append; the rest rotate queries
    int q_parts;              // workgroups per token for its queries
};

// Smallest e of KV_EXP_MIN .. KV_EXP_MAX with squares <= (448 2^e)^2, decided exactly:
// 448^2 = 0.765625 * 2^18.
__device__ __forceinline__ int scale_exponent(float squares) {
    if (!(squares > 0.0f)) return KV_EXP_MIN;
    if (squares > 0x1p127f) return KV_EXP_MAX;
    int x;
    const float f = frexpf(squares, &x);
    const int c = f > 0.765625f ? x - 17 : x - 18;
    const int e = (c + 1) >> 1;
    return e < KV_EXP_MIN ? KV_EXP_MIN : (e > KV_EXP_MAX ? KV_EXP_MAX : e);
}

__device__ __forceinline__ float pow2(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }

// Four values to four E4M3 codes, clamped to +-448, round to nearest even.
__device__ __forceinline__ uint32_t encode4(float a, float b, float c, float d) {
    auto cl = [](float x) { return fminf(fmaxf(x, -448.0f), 448.0f); };
    int w = __builtin_amdgcn_cvt_pk_fp8_f32(cl(a), cl(b), 0, false);
    w = __builtin_amdgcn_cvt_pk_fp8_f32(cl(c), cl(d), w, true);
    return (uint32_t)w;
}

// Four codes times 2^d (d <= 0), rounded again; a NaN code stays one.
__device__ __forceinline__ uint32_t recode4(uint32_t w, float factor) {
    uint32_t out = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t code = (w >> (8 * i)) & 0xFFu;
        const float x = e4m3_to_f32(code) * factor;
        const uint32_t y = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(x, 0.0f, 0, false) & 0xFFu;
        out |= ((code & 0x7Fu) == 0x7Fu ? code : y) << (8 * i);
    }
    return out;
}

template <int D, bool INTER>
__device__ __forceinline__ void append_page(const AppendArgs& a, int seq, int t0, int n, int page, int slot0, int head,
                                            int position, int lane) {
    constexpr int LPT = D / 8;            // lanes per token, 8 values each
    constexpr int TPP = 64 / LPT;         // tokens per pass of the wave
    const int d0 = (lane % LPT) * 8;
    const int64_t P = (int64_t)1 << a.c.page_log2;
    const uint16_t* kp = (const uint16_t*)a.k.data + head * a.k.head_stride;
    const uint16_t* vp = (const uint16_t*)a.v.data + head * a.v.head_stride;
    const int rd = a.rope.rotary, half = rd >> 1;
    const float mag = a.rope.magnitude;
    // partner of value d in its pair, or d itself past the rotated part
    auto partner = [&](int d) { return d >= rd ? d : INTER ? d ^ 1 : (d < half ? d + half : d - half); };
    // half layout: a lane's 8 partners are one aligned vector when the pairs come in whole eights
    const bool whole = INTER ? rd % 2 == 0 : half % 8 == 0;
    struct Values {
        float k[8], p[8], v[8];           // keys, their partners (the magnitude multiplied into both), values
        bool bad;                         // the token has a non-finite entry
    };
    auto read = [&](int t) {
        Values x;
        const uint16_t* kt = kp + (int64_t)t * a.k.token_stride;
        Vec16<uint16_t>::unpack(*reinterpret_cast<const uint4*>(kt + d0), x.k);
        Vec16<uint16_t>::unpack(*reinterpret_cast<const uint4*>(vp + (int64_t)t * a.v.token_stride + d0), x.v);
        if constexpr (INTER) {
#pragma unroll
            for (int i = 0; i < 8; ++i) x.p[i] = x.k[i ^ 1];
        } else if (whole) {
            Vec16<uint16_t>::unpack(*reinterpret_cast<const uint4*>(kt + partner(d0)), x.p);
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) x.p[i] = bf16_to_f32(kt[partner(d0 + i)]);
        }
        bool bad = false;
#pragma unroll
        for (int i = 0; i < 8; ++i) bad = bad || !(fabsf(x.k[i]) < INFINITY) || !(fabsf(x.v[i]) < INFINITY);
        const uint64_t lanes = __ballot(bad);
        const uint64_t group = LPT == 64 ? ~0ull : ((1ull << (LPT & 63)) - 1) << (lane / LPT * LPT);
        x.bad = (lanes & group) != 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            if (d0 + i < rd) {
                x.k[i] *= mag;
                x.p[i] *= mag;
            }
        }
        return x;
    };
    // ---- the scale ----
    float k2 = 0.0f, v2 = 0.0f;
    for (int i = 0; i < n; i += TPP) {
        const int j = i + lane / LPT;
        const Values x = read(t0 + (j < n ? j : n - 1));
        if (x.bad) continue;
#pragma unroll
        for (int u = 0; u < 8; ++u) {
            k2 = fmaxf(k2, d0 + u < rd ? x.k[u] * x.k[u] + x.p[u] * x.p[u] : x.k[u] * x.k[u]);
            v2 = fmaxf(v2, x.v[u] * x.v[u]);
        }
    }
#pragma unroll
    for (int m = 1; m < 64; m <<= 1) {
        k2 = fmaxf(k2, __shfl_xor(k2, m));
        v2 = fmaxf(v2, __shfl_xor(v2, m));
    }
    int e[2] = {scale_exponent(k2), scale_exponent(v2)};
#pragma unroll
    for (int kind = 0; kind < 2; ++kind) {
        const int64_t block = ((int64_t)page * 2 + kind) * a.c.heads + head;
        float* sp = a.c.scales + block;
        if (slot0 > 0) {                  // earlier tokens stay: their scale may only grow
            int old;
            frexpf(*sp, &old);
            old = old - 1 < KV_EXP_MIN ? KV_EXP_MIN : (old - 1 > KV_EXP_MAX ? KV_EXP_MAX : old - 1);
            if (e[kind] <= old) {
                e[kind] = old;
            } else {
                const float factor = pow2(old - e[kind]);
                uint2* row = reinterpret_cast<uint2*>(a.c.codes + block * P * D);
                for (int i = lane; i < slot0 * LPT; i += 64) {
                    const uint2 w = row[i];
                    row[i] = make_uint2(recode4(w.x, factor), recode4(w.y, factor));
                }
            }
        }
        if (lane == 0) *sp = pow2(e[kind]);
    }
    // ---- rotate, round, store ----
    const float ik = pow2(-e[0]), iv = pow2(-e[1]);
    uint8_t* kc = a.c.codes + (((int64_t)page * 2) * a.c.heads + head) * P * D;
    uint8_t* vc = kc + (int64_t)a.c.heads * P * D;
    for (int i = 0; i < n; i += TPP) {
        const int j = i + lane / LPT;
        const Values x = read(t0 + (j < n ? j : n - 1));
        float y[8];
#pragma unroll
        for (int u = 0; u < 8; ++u) {
            const int d = d0 + u;
            y[u] = x.k[u];
            if (d < rd) {
                const bool second = INTER ? (u & 1) != 0 : d >= half;
                const int pair = INTER ? d >> 1 : (second ? d - half : d);
                const float2 cs = rope_cos_sin(a.rope.freq[pair], position + j);
                const float2 r = second ? rope_turn(x.p[u], x.k[u], cs) : rope_turn(x.k[u], x.p[u], cs);
                y[u] = second ? r.y : r.x;
            }
            y[u] *= ik;
        }
        if (j < n) {
            const int64_t at = (int64_t)(slot0 + j) * D + d0;
            const uint32_t nan4 = 0x7F7F7F7Fu;
            uint2 kw = make_uint2(encode4(y[0], y[1], y[2], y[3]), encode4(y[4], y[5], y[6], y[7]));
            uint2 vw = make_uint2(encode4(x.v[0] * iv, x.v[1] * iv, x.v[2] * iv, x.v[3] * iv),
                                  encode4(x.v[4] * iv, x.v[5] * iv, x.v[6] * iv, x.v[7] * iv));
            if (x.bad) {
                kw = make_uint2(nan4, nan4);
                vw = make_uint2(0u, 0u);
            }
            *reinterpret_cast<uint2*>(kc + at) = kw;
            *reinterpret_cast<uint2*>(vc + at) = vw;
        }
    }
}

template <int D, bool INTER, bool VECQ>
__global__ __launch_bounds__(256)
void k_append(AppendArgs a) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    if ((int)blockIdx.x >= a.kv_blocks) {          // queries: one token (or part of its heads) per workgroup
        __shared__ float2 cs[D / 2];
        const int id = (int)blockIdx.x - a.kv_blocks;
        const int t = id / a.q_parts, part = id - t * a.q_parts;
        const int seq = sequence_of(a.b.starts, a.b.seqs, t, lane);
        const int position = a.b.lengths[seq] + t - a.b.starts[seq];
        rope_fill(a.rope, position, cs, threadIdx.x, 256);
        __syncthreads();
        const int per = rope_items<uint16_t, VECQ>(a.rope.rotary, D);
        for (int i = part * 256 + threadIdx.x; i < per * a.q.heads; i += 256 * a.q_parts) {
            const int h = i / per, c = i - h * per;
            rope_item<uint16_t, INTER, VECQ>(
                (const uint16_t*)a.q.data + (int64_t)t * a.q.token_stride + h * a.q.head_stride,
                (uint16_t*)a.qo.data + (int64_t)t * a.qo.token_stride + h * a.qo.head_stride, c, a.rope, cs);
        }
        return;
    }
    const int span = (int)blockIdx.x % a.spans;
    const int head = ((int)blockIdx.x / a.spans) * 4 + wave;
    if (head >= a.c.heads) return;
    const int P = 1 << a.c.page_log2;
    const int first = span * a.span;
    const int last = first + a.span < a.b.tokens ? first + a.span : a.b.tokens;
    int t = first;
    int seq = sequence_of(a.b.starts, a.b.seqs, first, lane);
    while (t < last) {
        int begin = a.b.starts[seq], end = a.b.starts[seq + 1];
        while (t >= end && seq + 1 < a.b.seqs) {      // the next sequence that has tokens
            ++seq;
            begin = end;
            end = a.b.starts[seq + 1];
        }
        if (t >= end || t < begin) return;
        const int position = a.b.lengths[seq] + t - begin;
        if (position < 0) {
            ++t;
            continue;
        }
        const int slot = position & (P - 1);
        int n = P - slot < end - t ? P - slot : end - t;      // the page's tokens from t on
        n = n < a.b.tokens - t ? n : a.b.tokens - t;
        // another wave has the page if an earlier new token lies on it
        const bool mine = slot == 0 || t == begin || position - 1 < 0 || a.b.lengths[seq] + t - 1 - begin < 0;
        if (mine) {
            const int page = page_of(a.c, a.b, seq, position >> a.c.page_log2);
            if (page >= 0) append_page<D, INTER>(a, seq, t, n, page, slot, head, position, lane);
        }
        t += n;
    }
}

hipError_t launch_kv_append(const CacheView& c, const BatchView& b, const HeadsView& k, const HeadsView& v,
                            const RopeView& rope, const HeadsView* q_in, const HeadsView* q_out, hipStream_t s) {
    AppendArgs a{};
    a.c = c;
    a.b = b;
    a.rope = rope;
    a.k = k;
    a.v = v;
    // a span of about as many tokens as a sequence brings, a page's at most: single tokens of
    // many sequences go to a wave each, a prompt's pages too
    const int page = 1 << c.page_log2;
    const int mean = b.tokens / b.seqs;
    a.span = mean < 1 ? 1 : (mean < page ? mean : page);
    a.spans = (b.tokens + a.span - 1) / a.span;
    a.kv_blocks = a.spans * ((c.heads + 3) / 4);
    int q_blocks = 0;
    bool vec = true;
    if (q_in) {
        a.q = *q_in;
        a.qo = *q_out;
        vec = rope.rotary % 16 == 0;
        const int items = (rope.rotary / (vec ? 16 : 2) + (c.dim - rope.rotary) / (vec ? 8 : 1)) * a.q.heads;
        const int rounds = (items + 255) / 256;
        a.q_parts = b.tokens >= 1024 ? 1 : (1024 + b.tokens - 1) / b.tokens;
        a.q_parts = a.q_parts < rounds ? a.q_parts : rounds;
        q_blocks = b.tokens * a.q_parts;
    }
    const dim3 grid((uint32_t)(a.kv_blocks + q_blocks));
    auto run = [&](auto kernel) { hipLaunchKernelGGL(kernel, grid, dim3(256), 0, s, a); };
    auto with = [&](auto dim) {
        constexpr int D = decltype(dim)::value;
        if (rope.interleaved) vec ? run(k_append<D, true, true>) : run(k_append<D, true, false>);
        else vec ? run(k_append<D, false, true>) : run(k_append<D, false, false>);
    };
    if (c.dim == 64) with(std::integral_constant<int, 64>{});
    else if (c.dim == 128) with(std::integral_constant<int, 128>{});
    else with(std::integral_constant<int, 256>{});
    return hipGetLastError();
}

}  // namespace nf4
