// kv_attention.hip -- causal attention over the paged 8-bit cache (gfx950).
//
// Mathematics.  One pass over the keys with the running maximum and sum of a softmax.  With
// base-2 scores x_j = scale log2(e) q.k_j and page exponents f_j of the values (v = code 2^f),
// the kernel sums w_j = 2^(x_j + f_j - m) against the bare codes, m a running reference of
// x + f, and 2^(-f_j) w_j for the denominator: the value scales cost one addition per score.
// Rounding: keys are exact in bf16 (E4M3 has 4 significant bits, the scale is a power of
// two), scores, maxima, sums and outputs are fp32, and the weights go into the second
// product as fp16, scaled to at most 2^15: 11 significant bits down to 2^-29 of the largest,
// an eighth of bf16's error (the output itself is bf16).
//
// Shape.  A tile is up to 16 rows (query heads of one kv head, of one or more tokens) and a
// step 32 keys.  Both products are v_mfma_f32_16x16x32 with the keys or the value dimensions
// as rows and the queries as columns, so a column's maximum, sum and factors live in the lanes
// of that column, and the scores leave the first product in the very lanes and order in which
// the second takes its weights: no exchange between lanes.  Keys: lane (key l % 16, quarter
// l / 16) reads 16-byte pieces of its key's row.  Values: lane (l % 16, quarter) reads
// D / 16 bytes of each of 8 tokens, and byte permutes pair the tokens up for the conversion.
// A wave's loads of the next step are in flight while it computes one, so a workgroup of four
// waves keeps 4 steps of 32 keys x 2 D bytes outstanding.
//
// Work.  Workgroups of four waves own (sequence, kv head, row tile, chunk of keys); the waves
// take the chunk's steps in turn and join through LDS, and chunks of one row join in a second
// launch.  Bound by HBM: each key and value byte is read once per row tile.
#include "paged.h"

namespace nf4 {

typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));

constexpr int KV_STEP = 32;               // keys of a step
constexpr int KV_WAVES = 4;
constexpr float KV_FLOOR = -3e38f;        // reference before any key: finite, so that no inf - inf arises
constexpr float KV_BIAS = 10.0f;          // weights are at most 2^(KV_BIAS + KV_SLACK) = 2^15 (fp16 reaches 2^16)
constexpr float KV_SLACK = 5.0f;          // a reference is raised once a score passes it by more than this

struct AttendArgs {
    CacheView c;
    BatchView b;
    HeadsView q, out;
    int group;                // query heads per kv head
    int row_tiles;            // launched row tiles per (sequence, kv head)
    int chunk;                // keys per chunk, a multiple of 4 * KV_STEP
    int splits;               // launched chunks per row tile
    float scale2;             // scale * log2(e)
    float* part;              // [token][head][split]: D sums, reference, denominator (splits > 1)
};

__device__ __forceinline__ bf16x8 codes_to_bf16(uint2 w, float scale) {
    typedef __bf16 b2 __attribute__((ext_vector_type(2)));
    const b2 a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w.x, scale, false);
    const b2 b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w.x, scale, true);
    const b2 c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w.y, scale, false);
    const b2 d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w.y, scale, true);
    return bf16x8{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}

// One step's codes and scales of a wave: two tiles of 16 keys.
template <int D>
struct StepCodes {
    uint4 k[2][D / 64];                   // [tile][piece]: 16 bytes of the lane's key
    uint32_t v[2][4][D / 64];             // [tile][token 4 g + r]: D / 16 bytes of its values
    float ks[2], vf[2];                   // key scale; value exponent
    int end[2];                           // keys of the tile that count lie below
};

template <int D>
__global__ __launch_bounds__(256)
void k_attend_rows(AttendArgs a) {
    constexpr int PIECES = D / 64;        // 16-byte pieces of a key per lane; values dwords per token
    constexpr int KSTEPS = D / 32;        // products along the dimensions
    constexpr int TILES = D / 16;         // value dimension tiles of the output
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int col = lane & 15, quarter = lane >> 4;
    const int split = blockIdx.x;
    const int head = blockIdx.y % a.c.heads, tile0 = blockIdx.y / a.c.heads;
    const int seq = blockIdx.z;
    const int begin = a.b.starts[seq], fresh = a.b.starts[seq + 1] - begin;
    const int before = a.b.lengths[seq];
    const int rows = fresh * a.group;
    const int reach = a.b.table_width << a.c.page_log2;      // positions the table can hold
    const int P = 1 << a.c.page_log2;
    const int64_t page_bytes = (int64_t)P * D;
    __shared__ float sm[KV_WAVES][16], sl[KV_WAVES][16];
    __shared__ f32x4 so[2][TILES][64];

    for (int tile = tile0; tile * 16 < rows; tile += a.row_tiles) {
        const int row = tile * 16 + col;
        const bool live = row < rows;
        const int token = (live ? row : rows - 1) / a.group;
        const int qhead = head * a.group + (live ? row : rows - 1) % a.group;
        int position = before + token;
        if (position >= reach) position = -1;                 // left out: attends to nothing
        const int last_row = tile * 16 + 15 < rows ? tile * 16 + 15 : rows - 1;
        int keys = before + last_row / a.group + 1;           // keys the tile's last row sees
        keys = keys < reach ? keys : reach;
        // queries: the lane's dimensions of MFMA step s, in the order of the key pieces
        bf16x8 qf[KSTEPS];
        {
            const uint16_t* qp = (const uint16_t*)a.q.data + (int64_t)(begin + token) * a.q.token_stride +
                                 (int64_t)qhead * a.q.head_stride;
#pragma unroll
            for (int s = 0; s < KSTEPS; ++s)
                qf[s] = *reinterpret_cast<const bf16x8*>(qp + 64 * (s >> 1) + 16 * quarter + 8 * (s & 1));
        }
        f32x4 acc[TILES];
#pragma unroll
        for (int i = 0; i < TILES; ++i) acc[i] = f32x4{};
        float m = KV_FLOOR, l = 0.0f;     // m is shared by a column's four lanes, l is the lane's own part

        const int chunks = (keys + a.chunk - 1) / a.chunk;
        for (int ch = split; ch < chunks; ch += a.splits) {
            const int lo = ch * a.chunk;
            const int hi = lo + a.chunk < keys ? lo + a.chunk : keys;
            const int steps = (hi - lo + KV_STEP - 1) / KV_STEP;
            auto load = [&](StepCodes<D>& x, int step) {
#pragma unroll
                for (int t = 0; t < 2; ++t) {
                    int at = lo + step * KV_STEP + 16 * t;
                    at = at < keys ? at : (keys - 1) & ~15;   // a tile past the last key: any held one, masked later
                    const int page = page_of(a.c, a.b, seq, at >> a.c.page_log2);
                    const int64_t block = (int64_t)(page < 0 ? 0 : page) * 2 * a.c.heads + head;
                    const int slot = at & (P - 1);
                    const int have = keys - at < 16 ? keys - at : 16;
                    x.end[t] = page < 0 ? 0 : hi;         // a page outside the pool holds no keys
                    x.ks[t] = a.c.scales[block];
                    x.vf[t] = (float)((int)((__float_as_uint(a.c.scales[block + a.c.heads]) >> 23) & 0xFFu) - 127);
                    const uint8_t* kb = a.c.codes + block * page_bytes + (int64_t)slot * D;
                    const uint8_t* vb = kb + a.c.heads * page_bytes;
#pragma unroll
                    for (int p = 0; p < PIECES; ++p)
                        x.k[t][p] = *reinterpret_cast<const uint4*>(kb + col * D + 64 * p + 16 * quarter);
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        // slots past the last key may hold anything: their values come from the last key
                        int n = 4 * quarter + r;
                        n = n < have ? n : have - 1;
                        const uint8_t* vp = vb + n * D + col * (D / 16);
                        if constexpr (D == 64) x.v[t][r][0] = *reinterpret_cast<const uint32_t*>(vp);
                        if constexpr (D == 128) {
                            const uint2 w = *reinterpret_cast<const uint2*>(vp);
                            x.v[t][r][0] = w.x;
                            x.v[t][r][1] = w.y;
                        }
                        if constexpr (D == 256) {
                            const uint4 w = *reinterpret_cast<const uint4*>(vp);
                            x.v[t][r][0] = w.x;
                            x.v[t][r][1] = w.y;
                            x.v[t][r][2] = w.z;
                            x.v[t][r][3] = w.w;
                        }
                    }
                    if (page < 0) {
#pragma unroll
                        for (int r = 0; r < 4; ++r)
#pragma unroll
                            for (int d = 0; d < PIECES; ++d) x.v[t][r][d] = 0;
                    }
                }
            };
            auto compute = [&](const StepCodes<D>& x, int step) {
                float y[8];
#pragma unroll
                for (int t = 0; t < 2; ++t) {
                    f32x4 s = {};
#pragma unroll
                    for (int i = 0; i < KSTEPS; ++i) {
                        const uint4 w = x.k[t][i >> 1];
                        const bf16x8 kf = codes_to_bf16((i & 1) ? make_uint2(w.z, w.w) : make_uint2(w.x, w.y), 1.0f);
                        s = __builtin_amdgcn_mfma_f32_16x16x32_bf16(kf, qf[i], s, 0, 0, 0);
                    }
                    const int key = lo + step * KV_STEP + 16 * t + 4 * quarter;
                    const float f = x.ks[t] * a.scale2;
#pragma unroll
                    for (int r = 0; r < 4; ++r)
                        y[4 * t + r] = key + r <= position && key + r < x.end[t] ? s[r] * f + x.vf[t] : -INFINITY;
                }
                float top = fmaxf(fmaxf(fmaxf(y[0], y[1]), fmaxf(y[2], y[3])), fmaxf(fmaxf(y[4], y[5]), fmaxf(y[6], y[7])));
                if (__any(top > m + KV_SLACK)) {
                    top = fmaxf(top, __shfl_xor(top, 16));
                    top = fmaxf(top, __shfl_xor(top, 32));
                    const float now = fmaxf(m, top);
                    const float f = __builtin_amdgcn_exp2f(m - now);
                    m = now;
                    l *= f;
#pragma unroll
                    for (int i = 0; i < TILES; ++i) acc[i] *= f;
                }
                f16x8 w;
                const float ref = m - KV_BIAS;
#pragma unroll
                for (int t = 0; t < 2; ++t) {
                    float sum = 0.0f;
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        const float p = __builtin_amdgcn_exp2f(y[4 * t + r] - ref);
                        sum += p;
                        w[4 * t + r] = (_Float16)p;
                    }
                    l += sum * __builtin_amdgcn_exp2f(-x.vf[t]);
                }
#pragma unroll
                for (int d = 0; d < PIECES; ++d)
#pragma unroll
                    for (int h = 0; h < 2; ++h) {             // bytes 2 h and 2 h + 1 of dword d: two dimension tiles
                        f16x8 v0, v1;
#pragma unroll
                        for (int j = 0; j < 4; ++j) {         // token pairs
                            const uint32_t w0 = x.v[j >> 1][2 * (j & 1)][d], w1 = x.v[j >> 1][2 * (j & 1) + 1][d];
                            // bytes (tok0.b, tok1.b, tok0.b+1, tok1.b+1)
                            const uint32_t pk = __builtin_amdgcn_perm(w1, w0, h ? 0x07030602u : 0x05010400u);
                            const f16x2 lo2 = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(pk, 1.0f, false);
                            const f16x2 hi2 = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(pk, 1.0f, true);
                            v0[2 * j] = lo2[0];
                            v0[2 * j + 1] = lo2[1];
                            v1[2 * j] = hi2[0];
                            v1[2 * j + 1] = hi2[1];
                        }
                        acc[4 * d + 2 * h] = __builtin_amdgcn_mfma_f32_16x16x32_f16(v0, w, acc[4 * d + 2 * h], 0, 0, 0);
                        acc[4 * d + 2 * h + 1] = __builtin_amdgcn_mfma_f32_16x16x32_f16(v1, w, acc[4 * d + 2 * h + 1], 0, 0, 0);
                    }
            };
            if (wave < steps) {
                StepCodes<D> cur, nxt;
                load(cur, wave);
                for (int s = wave; s < steps; s += KV_WAVES) {
                    if (s + KV_WAVES < steps) load(nxt, s + KV_WAVES);
                    compute(cur, s);
                    cur = nxt;
                }
            }
        }
        // ---- the waves join: a common reference, then the sums ----
        l += __shfl_xor(l, 16);
        l += __shfl_xor(l, 32);
        if (quarter == 0) {
            sm[wave][col] = m;
            sl[wave][col] = l;
        }
        __syncthreads();
        float top = sm[0][col], total = 0.0f;
#pragma unroll
        for (int w = 1; w < KV_WAVES; ++w) top = fmaxf(top, sm[w][col]);
#pragma unroll
        for (int w = 0; w < KV_WAVES; ++w) total += sl[w][col] * __builtin_amdgcn_exp2f(sm[w][col] - top);
        const float f = __builtin_amdgcn_exp2f(m - top);
#pragma unroll
        for (int i = 0; i < TILES; ++i) acc[i] *= f;
        for (int half = 2; half >= 1; half >>= 1) {           // waves 2, 3 onto 0, 1, then 1 onto 0
            if (wave >= half && wave < 2 * half) {
#pragma unroll
                for (int i = 0; i < TILES; ++i) so[wave - half][i][lane] = acc[i];
            }
            __syncthreads();
            if (wave < half) {
#pragma unroll
                for (int i = 0; i < TILES; ++i) acc[i] += so[wave][i][lane];
            }
            __syncthreads();
        }
        if (wave == 0 && live) {
            // accumulator (tile i, register r): dimension (4 quarter + r) * TILES + i
            const int64_t t = begin + token;
            if (a.splits == 1) {
                const float inv = total > 0.0f || total != total ? 1.0f / total : 0.0f;
                uint16_t* o = (uint16_t*)a.out.data + t * a.out.token_stride + qhead * a.out.head_stride;
#pragma unroll
                for (int r = 0; r < 4; ++r)
#pragma unroll
                    for (int i = 0; i < TILES; i += 4) {
                        const uint2 w = make_uint2(pack_bf16x2(acc[i][r] * inv, acc[i + 1][r] * inv),
                                                   pack_bf16x2(acc[i + 2][r] * inv, acc[i + 3][r] * inv));
                        *reinterpret_cast<uint2*>(o + (4 * quarter + r) * TILES + i) = w;
                    }
            } else {
                float* p = a.part + ((t * (int64_t)(a.c.heads * a.group) + qhead) * a.splits + split) * (D + 2);
#pragma unroll
                for (int r = 0; r < 4; ++r)
#pragma unroll
                    for (int i = 0; i < TILES; i += 2)
                        *reinterpret_cast<float2*>(p + (4 * quarter + r) * TILES + i) = make_float2(acc[i][r], acc[i + 1][r]);
                if (quarter == 0) *reinterpret_cast<float2*>(p + D) = make_float2(top, total);
            }
        }
    }
}

// Joins the chunks of each row: one wave per (token, head).
template <int D>
__global__ __launch_bounds__(256)
void k_attend_join(AttendArgs a) {
    constexpr int N = D / 64;
    const int lane = threadIdx.x & 63;
    const int heads = a.c.heads * a.group;
    const int64_t row = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
    if (row >= (int64_t)a.b.tokens * heads) return;
    const float* p = a.part + row * a.splits * (D + 2);
    float top = KV_FLOOR;
    for (int s = lane; s < a.splits; s += 64) top = fmaxf(top, p[(int64_t)s * (D + 2) + D]);
#pragma unroll
    for (int x = 1; x < 64; x <<= 1) top = fmaxf(top, __shfl_xor(top, x));
    float total = 0.0f, o[N] = {};
    for (int s = 0; s < a.splits; ++s) {
        const float* ps = p + (int64_t)s * (D + 2);
        const float f = __builtin_amdgcn_exp2f(ps[D] - top);
        total += ps[D + 1] * f;
#pragma unroll
        for (int i = 0; i < N; ++i) o[i] += ps[lane + 64 * i] * f;
    }
    const float inv = total > 0.0f || total != total ? 1.0f / total : 0.0f;
    uint16_t* out = (uint16_t*)a.out.data + (row / heads) * a.out.token_stride + (row % heads) * a.out.head_stride;
#pragma unroll
    for (int i = 0; i < N; ++i) out[lane + 64 * i] = f32_to_bf16(o[i] * inv);
}

struct AttendPlan {
    int row_tiles, chunk, splits;
    size_t bytes;
};

// Chunks are sized for about 2048 workgroups (two rounds of four on each compute unit) at the
// stated lengths, and of at least 256 keys: a join costs a launch.
static AttendPlan attend_plan(const CacheView& c, int seqs, int64_t tokens, int heads, int64_t max_new,
                              int64_t max_length) {
    AttendPlan p{};
    const int group = heads / c.heads;
    int64_t tiles = (max_new * group + 15) / 16;
    const int64_t most = 32768 / c.heads < 512 ? 32768 / c.heads : 512;   // the launch's second dimension is 65535 at most
    tiles = tiles < 1 ? 1 : (tiles < most ? tiles : most);
    p.row_tiles = (int)tiles;
    const int64_t groups = (int64_t)seqs * c.heads * tiles;
    constexpr int64_t unit = KV_WAVES * KV_STEP;
    int64_t chunk = (max_length * groups / 2048 + unit - 1) / unit * unit;
    if (chunk < 256) chunk = 256;
    if (chunk > (1 << 20)) chunk = 1 << 20;
    p.chunk = (int)chunk;
    int64_t splits = (max_length + chunk - 1) / chunk;
    splits = splits < 1 ? 1 : (splits < 1024 ? splits : 1024);
    p.splits = (int)splits;
    p.bytes = splits > 1 ? (size_t)tokens * heads * splits * (c.dim + 2) * sizeof(float) : 0;
    return p;
}

size_t kv_attention_ws_bytes(const CacheView& c, int seqs, int64_t tokens, int heads, int64_t max_new,
                             int64_t max_length) {
    return attend_plan(c, seqs, tokens, heads, max_new, max_length).bytes;
}

hipError_t launch_kv_attention(const CacheView& c, const BatchView& b, const HeadsView& q, const HeadsView& out,
                               float scale, int64_t max_new, int64_t max_length, void* ws, hipStream_t s) {
    const AttendPlan p = attend_plan(c, b.seqs, b.tokens, q.heads, max_new, max_length);
    AttendArgs a{c, b, q, out, q.heads / c.heads, p.row_tiles, p.chunk, p.splits, scale * 1.4426950408889634f, (float*)ws};
    const dim3 grid((uint32_t)p.splits, (uint32_t)(c.heads * p.row_tiles), (uint32_t)b.seqs);
    const dim3 join((uint32_t)(((int64_t)b.tokens * q.heads + 3) / 4));
    auto with = [&](auto dim) {
        constexpr int D = decltype(dim)::value;
        hipLaunchKernelGGL(k_attend_rows<D>, grid, dim3(256), 0, s, a);
        if (p.splits > 1) hipLaunchKernelGGL(k_attend_join<D>, join, dim3(256), 0, s, a);
    };
    if (c.dim == 64) with(std::integral_constant<int, 64>{});
    else if (c.dim == 128) with(std::integral_constant<int, 128>{});
    else with(std::integral_constant<int, 256>{});
    return hipGetLastError();
}

}  // namespace nf4
