// kv_append.hip -- keys and values into the paged 8-bit cache, rotated on the way (gfx950).
//
// A page's scale is one power of two per head and kind: the smallest 2^e with every value
// there within +-448 2^e.  E4M3 keeps the same relative precision at every magnitude above
// 2^-6 of its unit, so a power of two loses nothing against a free scale, and a page's
// earlier codes move to a larger scale by an exact change of exponent (but for those that
// become subnormal).  Rotation keeps a pair's norm, so the scale is taken from pair norms,
// before the rotation: it needs no cos or sin and no second rotation.
//
// A page's new tokens of one kv head belong to one wave, or, where a page is longer than one wave's
// registers hold, to the four waves of a workgroup that join their maxima through LDS: nothing races on
// a scale.  Keys and values are read once (long pages: what four rounds do not hold is read again), the
// cos and sin of 8 KB worth of (token, pair) at a time are computed once per workgroup into LDS.  The
// workgroup of a page is the one whose span of `span` packed tokens holds the page's first new token.
// Queries are rotated by further workgroups of the same launch, a wave per token and part of its heads.
// Bound by HBM for prompts (4 bytes read and 2 written per key/value pair, 4 per query value) and by the
// chain of dependent loads (starts, length, table, values) for single tokens.  9 prompts of up to 1023 tokens, 32
// heads of 128, pages of 16 (272 MB): 70 us, 3.9 TB/s; one token of 16 sequences, 64 heads: 7.2 us.
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
    int q_parts;              // waves per token for its queries
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

// One page's new tokens t0 .. t0 + n - 1, positions `position` .., slots slot0 ...  Lane l has values
// 8 (l % (D/8)) .. of token l / (D/8) of its round; a round is TPP tokens of a wave.  SPLIT: the four
// waves share one head and take the rounds in turn; otherwise each wave has a head of its own.  Every wave
// of the workgroup makes the same calls (`on`: whether its head exists).
template <int D, bool INTER, bool SPLIT>
__device__ __forceinline__ void append_page(const AppendArgs& a, int t0, int n, int page, int slot0, int head, bool on, int position,
                                            int wave, int lane, float2* table, float* join) {
    constexpr int LPT = D / 8, TPP = 64 / LPT;
    constexpr int CHUNK = 4 * TPP;        // tokens of the table: four rounds of a wave, or one of four waves
    const int d0 = (lane % LPT) * 8, sub = lane / LPT;
    const int64_t P = (int64_t)1 << a.c.page_log2;
    const uint16_t* kp = (const uint16_t*)a.k.data + head * a.k.head_stride;
    const uint16_t* vp = (const uint16_t*)a.v.data + head * a.v.head_stride;
    const int rd = a.rope.rotary, half = rd >> 1;
    const float mag = a.rope.magnitude;
    const int rounds = SPLIT ? (n + CHUNK - 1) / CHUNK : (n + TPP - 1) / TPP;
    auto token_of = [&](int round) { return (SPLIT ? round * CHUNK + wave * TPP : round * TPP) + sub; };
    // partner of value d in its pair, or d itself past the rotated part
    auto partner = [&](int d) { return d >= rd ? d : INTER ? d ^ 1 : (d < half ? d + half : d - half); };
    // half layout: a lane's 8 partners are one aligned vector when the pairs come in whole eights
    const bool whole = half % 8 == 0;
    struct Raw {
        uint4 k, v;                       // keys and values
        bool bad;                         // the token has a non-finite entry
    };
    auto read = [&](Raw& x, int round) {
        const int j = token_of(round);
        const int64_t t = t0 + (j < n ? j : n - 1);
        x.k = *reinterpret_cast<const uint4*>(kp + t * a.k.token_stride + d0);
        x.v = *reinterpret_cast<const uint4*>(vp + t * a.v.token_stride + d0);
    };
    auto judge = [&](Raw& x) {            // an exponent of all ones: infinity or NaN
        auto any = [](uint32_t w) { return (w & 0x7F80u) == 0x7F80u || (w & 0x7F800000u) == 0x7F800000u; };
        const bool bad = any(x.k.x) || any(x.k.y) || any(x.k.z) || any(x.k.w) || any(x.v.x) || any(x.v.y) || any(x.v.z) || any(x.v.w);
        x.bad = (__ballot(bad) & ((1ull << LPT) - 1) << (sub * LPT)) != 0;
    };
    const int partner_lane = sub * LPT + partner(d0) / 8;
    // keys and their partners, the magnitude multiplied into rotated ones
    auto widen = [&](const Raw& x, int round, float* k, float* p) {
        Vec16<uint16_t>::unpack(x.k, k);
        if constexpr (INTER) {
#pragma unroll
            for (int i = 0; i < 8; ++i) p[i] = k[i ^ 1];
        } else if (whole) {
            const uint4 w = make_uint4(__shfl(x.k.x, partner_lane), __shfl(x.k.y, partner_lane), __shfl(x.k.z, partner_lane),
                                       __shfl(x.k.w, partner_lane));
            Vec16<uint16_t>::unpack(w, p);
        } else {
            const int j = token_of(round);
            const uint16_t* kt = kp + (int64_t)(t0 + (j < n ? j : n - 1)) * a.k.token_stride;
#pragma unroll
            for (int i = 0; i < 8; ++i) p[i] = bf16_to_f32(kt[partner(d0 + i)]);
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            if (d0 + i < rd) {
                k[i] *= mag;
                p[i] *= mag;
            }
        }
    };
    // ---- the scale ----
    float k2 = 0.0f, v2 = 0.0f;
    auto reach = [&](const Raw& x, int round) {
        float k[8], p[8], v[8];
        widen(x, round, k, p);
        Vec16<uint16_t>::unpack(x.v, v);
#pragma unroll
        for (int u = 0; u < 8; ++u) {
            const float y = d0 + u < rd ? k[u] * k[u] + p[u] * p[u] : k[u] * k[u];
            k2 = fmaxf(k2, x.bad ? 0.0f : y);
            v2 = fmaxf(v2, x.bad ? 0.0f : v[u] * v[u]);
        }
    };
    // four rounds at a time in registers (the fences keep one round's temporaries from another's)
    const int groups = (rounds + 3) / 4;
    Raw held[4];
    auto read4 = [&](int g) {
#pragma unroll
        for (int i = 0; i < 4; ++i) read(held[i], 4 * g + i < rounds ? 4 * g + i : rounds - 1);
#pragma unroll
        for (int i = 0; i < 4; ++i) judge(held[i]);
    };
    for (int g = 0; g < groups; ++g) {
        read4(g);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            __builtin_amdgcn_sched_barrier(0);
            if (4 * g + i < rounds) reach(held[i], 4 * g + i);
        }
    }
#pragma unroll
    for (int m = 1; m < 64; m <<= 1) {
        k2 = fmaxf(k2, __shfl_xor(k2, m));
        v2 = fmaxf(v2, __shfl_xor(v2, m));
    }
    if constexpr (SPLIT) {
        if (lane == 0) {
            join[wave] = k2;
            join[4 + wave] = v2;
        }
        __syncthreads();
        k2 = fmaxf(fmaxf(join[0], join[1]), fmaxf(join[2], join[3]));
        v2 = fmaxf(fmaxf(join[4], join[5]), fmaxf(join[6], join[7]));
    }
    int e[2] = {scale_exponent(k2), scale_exponent(v2)};
    int old[2] = {0, 0};
    const int64_t block0 = ((int64_t)page * 2) * a.c.heads + head, block1 = block0 + a.c.heads;
    if (slot0 > 0) {                      // earlier tokens stay: their scale may only grow
#pragma unroll
        for (int kind = 0; kind < 2; ++kind) {
            int x;
            frexpf(a.c.scales[kind ? block1 : block0], &x);
            x -= 1;
            old[kind] = x < KV_EXP_MIN ? KV_EXP_MIN : (x > KV_EXP_MAX ? KV_EXP_MAX : x);
        }
    }
    if constexpr (SPLIT) __syncthreads();                    // every wave has read the old scale (and `join`)
#pragma unroll
    for (int kind = 0; kind < 2; ++kind) {
        const int64_t block = kind ? block1 : block0;
        if (slot0 > 0) {
            if (e[kind] <= old[kind]) {
                e[kind] = old[kind];
            } else if (on) {
                const float factor = pow2(old[kind] - e[kind]);
                uint2* row = reinterpret_cast<uint2*>(a.c.codes + block * P * D);
                for (int i = (SPLIT ? wave * 64 : 0) + lane; i < slot0 * LPT; i += SPLIT ? 256 : 64) {
                    const uint2 w = row[i];
                    row[i] = make_uint2(recode4(w.x, factor), recode4(w.y, factor));
                }
            }
        }
        if (on && lane == 0 && (!SPLIT || wave == 0)) a.c.scales[block] = pow2(e[kind]);
    }
    // ---- rotate, round, store ----
    const float ik = pow2(-e[0]), iv = pow2(-e[1]);
    uint8_t* kc = a.c.codes + block0 * P * D;
    uint8_t* vc = a.c.codes + block1 * P * D;
    auto store = [&](const Raw& x, int round) {
        const int j = token_of(round);
        float k[8], p[8], v[8], y[8];
        widen(x, round, k, p);
        Vec16<uint16_t>::unpack(x.v, v);
#pragma unroll
        for (int u = 0; u < 8; ++u) {
            const int d = d0 + u;
            y[u] = k[u];
            if (d < rd) {
                const bool second = INTER ? (u & 1) != 0 : d >= half;
                const int pair = INTER ? d >> 1 : (second ? d - half : d);
                const float2 cs = table[(j % CHUNK) * (D / 2) + pair];
                const float2 r = second ? rope_turn(p[u], k[u], cs) : rope_turn(k[u], p[u], cs);
                y[u] = second ? r.y : r.x;
            }
            y[u] *= ik;
        }
        if (on && j < n) {
            const int64_t at = (int64_t)(slot0 + j) * D + d0;
            const uint32_t nan4 = 0x7F7F7F7Fu;
            uint2 kw = make_uint2(encode4(y[0], y[1], y[2], y[3]), encode4(y[4], y[5], y[6], y[7]));
            uint2 vw = make_uint2(encode4(v[0] * iv, v[1] * iv, v[2] * iv, v[3] * iv),
                                  encode4(v[4] * iv, v[5] * iv, v[6] * iv, v[7] * iv));
            if (x.bad) {
                kw = make_uint2(nan4, nan4);
                vw = make_uint2(0u, 0u);
            }
            *reinterpret_cast<uint2*>(kc + at) = kw;
            *reinterpret_cast<uint2*>(vc + at) = vw;
        }
    };
    auto fill = [&](int chunk) {          // cos and sin of the chunk's tokens
        __syncthreads();
        const int left = n - chunk * CHUNK < CHUNK ? n - chunk * CHUNK : CHUNK;
        if (half > 0)
            for (int i = wave * 64 + lane; i < left * (D / 2); i += 256) {
                const int j = i / (D / 2), pair = i % (D / 2);
                if (pair < half) table[i] = rope_cos_sin(a.rope.freq[pair], position + chunk * CHUNK + j);
            }
        __syncthreads();
    };
    constexpr int PER = SPLIT ? 1 : 4;    // rounds of a chunk
    for (int g = 0; g < groups; ++g) {
        if (groups > 1) read4(g);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            __builtin_amdgcn_sched_barrier(0);
            if (4 * g + i < rounds) {
                if (i % PER == 0) fill((4 * g + i) / PER);
                store(held[i], 4 * g + i);
            }
        }
    }
    __syncthreads();                      // the table may be filled again, for another page
}

template <int D, bool INTER, bool VECQ, bool SPLIT>
__global__ __launch_bounds__(256)
void k_append(AppendArgs a) {
    __shared__ float2 table[1024];        // 4 rounds x 64 / (D/8) tokens x D/2 pairs: 8 KB at every head size
    __shared__ float join[8];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    if ((int)blockIdx.x >= a.kv_blocks) {          // queries: a wave per token and part of its heads
        const int id = ((int)blockIdx.x - a.kv_blocks) * 4 + wave;
        const int t = id / a.q_parts, part = id - t * a.q_parts;
        if (t >= a.b.tokens) return;
        const int seq = sequence_of(a.b.starts, a.b.seqs, t, lane);
        const int position = position_at(a.b.lengths[seq], t - a.b.starts[seq]);
        float2* cs = table + wave * (D / 2);       // of this wave alone
        rope_fill(a.rope, position, cs, lane, 64);
        __builtin_amdgcn_wave_barrier();
        __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
        const int per = rope_items<uint16_t, VECQ>(a.rope.rotary, D);
        for (int i = part * 64 + lane; i < per * a.q.heads; i += 64 * a.q_parts) {
            const int h = i / per, c = i - h * per;
            rope_item<uint16_t, INTER, VECQ>(
                (const uint16_t*)a.q.data + (int64_t)t * a.q.token_stride + h * a.q.head_stride,
                (uint16_t*)a.qo.data + (int64_t)t * a.qo.token_stride + h * a.qo.head_stride, c, a.rope, cs);
        }
        return;
    }
    const int span = (int)blockIdx.x % a.spans;
    const int head0 = (int)blockIdx.x / a.spans * (SPLIT ? 1 : 4) + (SPLIT ? 0 : wave);
    const bool on = head0 < a.c.heads;
    const int head = on ? head0 : a.c.heads - 1;
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
        const int position = position_at(a.b.lengths[seq], t - begin);
        if (position < 0) {
            ++t;
            continue;
        }
        const int slot = position & (P - 1);
        int n = P - slot < end - t ? P - slot : end - t;      // the page's tokens from t on
        n = n < a.b.tokens - t ? n : a.b.tokens - t;
        // another workgroup has the page if an earlier new token lies on it
        const bool mine = slot == 0 || t == begin || position_at(position, -1) < 0;
        if (mine) {
            const int page = page_of(a.c, a.b, seq, position >> a.c.page_log2);
            if (page >= 0) append_page<D, INTER, SPLIT>(a, t, n, page, slot, head, on, position, wave, lane, table, join);
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
    // many sequences go to a workgroup each, a prompt's pages too
    const int page = 1 << c.page_log2;
    const int mean = b.tokens / b.seqs;
    a.span = mean < 1 ? 1 : (mean < page ? mean : page);
    // four waves share a head's page where its tokens are more than the rounds one wave holds in registers (8 prompts of
    // up to 1000 tokens, 32 heads of 128: pages of 128 80 us, 117 unshared; 9 on pages of 16: 65 unshared, 128 shared)
    const bool split = a.span > 4 * 512 / c.dim;
    const int columns = split ? c.heads : (c.heads + 3) / 4;
    // a span in which two pages begin takes them one after the other: shorter spans, some of them without a page, while
    // the workgroups fit the compute units twice (3 sequences of up to 125 tokens, 16 heads, pages of 16: 16 us, 11
    // with spans of 4; but 9 of 1023: 65 and 79)
    while (a.span > 1 && (int64_t)((b.tokens + a.span / 2 - 1) / (a.span / 2)) * columns <= 512) a.span /= 2;
    a.spans = (b.tokens + a.span - 1) / a.span;
    a.kv_blocks = a.spans * columns;
    int q_blocks = 0;
    bool vec = true;
    if (q_in) {
        a.q = *q_in;
        a.qo = *q_out;
        vec = rope.rotary % 16 == 0;
        // a wave takes 8 items a lane, or, of few tokens, one (until about 4096 waves are there)
        const int items = (rope.rotary / (vec ? 16 : 2) + (c.dim - rope.rotary) / (vec ? 8 : 1)) * a.q.heads;
        const int most = (items + 63) / 64, least = (items + 511) / 512;
        const int want = (4096 + b.tokens - 1) / b.tokens;
        a.q_parts = want < least ? least : (want < most ? want : most);
        q_blocks = (int)(((int64_t)b.tokens * a.q_parts + 3) / 4);
    }
    const dim3 grid((uint32_t)(a.kv_blocks + q_blocks));
    auto run = [&](auto kernel) { hipLaunchKernelGGL(kernel, grid, dim3(256), 0, s, a); };
    auto with = [&](auto dim) {
        constexpr int D = decltype(dim)::value;
        if (rope.interleaved) {
            if (split) vec ? run(k_append<D, true, true, true>) : run(k_append<D, true, false, true>);
            else vec ? run(k_append<D, true, true, false>) : run(k_append<D, true, false, false>);
        } else {
            if (split) vec ? run(k_append<D, false, true, true>) : run(k_append<D, false, false, true>);
            else vec ? run(k_append<D, false, true, false>) : run(k_append<D, false, false, false>);
        }
    };
    if (c.dim == 64) with(std::integral_constant<int, 64>{});
    else if (c.dim == 128) with(std::integral_constant<int, 128>{});
    else with(std::integral_constant<int, 256>{});
    return hipGetLastError();
}

}  // namespace nf4
