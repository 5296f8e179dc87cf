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
#include "bufio.h"
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
    float* part;              // [token][head][split][D] sums, and
    float2* sums;             // [token][head][split] reference and denominator (splits > 1)
};

__device__ __forceinline__ bf16x8 codes_to_bf16(uint2 w, float scale) {
    typedef __bf16 b2 __attribute__((ext_vector_type(2)));
    const b2 a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w.x, scale, false);
    const b2 b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w.x, scale, true);
    const b2 c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w.y, scale, false);
    const b2 d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w.y, scale, true);
    return bf16x8{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}

// Uniform values that no kernel here writes, through the scalar cache (a vector load among the
// prefetched codes would wait for all of them).
template <typename T>
__device__ __forceinline__ T scalar_load(const T* p) {
    return *(const __attribute__((address_space(4))) T*)(uintptr_t)p;
}

// page_of through scalar loads.
__device__ __forceinline__ int uniform_page_of(const CacheView& c, const BatchView& b, int seq, int page_index) {
    if (page_index < 0 || page_index >= b.table_width) return -1;
    const int page = scalar_load(b.table + seq * b.table_stride + page_index);
    return page >= 0 && page < c.pages ? page : -1;
}

// The codes of 16 keys of one kv head from `slot` of a page on, and their values': ranges that
// end with the last key that counts, so that whatever lies behind it reads as zero.
struct TileView {
    __amdgpu_buffer_rsrc_t k, v;
    float ks, vf;             // key scale; value exponent
};
template <int D>
__device__ __forceinline__ TileView tile_view(const CacheView& c, int page, int head, int slot, int have) {
    const int64_t block = (int64_t)(page < 0 ? 0 : page) * 2 * c.heads + head;
    const int64_t page_bytes = (int64_t)D << c.page_log2;
    const uint8_t* kb = c.codes + block * page_bytes + slot * D;
    const int bytes = page < 0 || have <= 0 ? 0 : (have < 16 ? have : 16) * D;
    TileView t;
    t.k = make_rsrc(kb, bytes);
    t.v = make_rsrc(kb + c.heads * page_bytes, bytes);
    t.ks = scalar_load(c.scales + block);
    t.vf = (float)((int)((__float_as_uint(scalar_load(c.scales + block + c.heads)) >> 23) & 0xFFu) - 127);
    return t;
}

// One step's codes of a wave: two tiles of 16 keys.
template <int D>
struct StepCodes {
    uint4 k[2][D / 64];                   // [tile][piece]: 16 bytes of the lane's key
    uint32_t v[2][4][D / 64];             // [tile][token 4 g + r]: D / 16 bytes of its values
    float ks[2], vf[2];
    int end[2];                           // keys of the tile that count lie below
};

// The state of a tile of 16 columns (query rows) in a wave.
template <int D>
struct RowsState {
    f32x4 acc[D / 16];                    // dimension tile i: dimensions (4 quarter + r) * D / 16 + i
    float m, l;                           // reference (the same in a column's four lanes), the lane's part of the sum
};

// The scores y of 32 keys (lane: column col, keys 4 quarter + r of tile t) join the state.
template <int D>
__device__ __forceinline__ void attend_step(RowsState<D>& st, float* y, const uint32_t (&v)[2][4][D / 64], const float* vf) {
    constexpr int TILES = D / 16, PIECES = D / 64;
    float top = fmaxf(fmaxf(fmaxf(y[0], y[1]), fmaxf(y[2], y[3])), fmaxf(fmaxf(y[4], y[5]), fmaxf(y[6], y[7])));
    if (__any(top > st.m + KV_SLACK)) {
        top = fmaxf(top, __shfl_xor(top, 16));
        top = fmaxf(top, __shfl_xor(top, 32));
        const float now = fmaxf(st.m, top);
        const float f = __builtin_amdgcn_exp2f(st.m - now);
        st.m = now;
        st.l *= f;
#pragma unroll
        for (int i = 0; i < TILES; ++i) st.acc[i] *= f;
    }
    f16x8 w;
    const float ref = st.m - KV_BIAS;
#pragma unroll
    for (int t = 0; t < 2; ++t) {
        float p[4];
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            p[r] = __builtin_amdgcn_exp2f(y[4 * t + r] - ref);
            w[4 * t + r] = (_Float16)p[r];
        }
        st.l = __fmaf_rn((p[0] + p[1]) + (p[2] + p[3]), __builtin_amdgcn_exp2f(-vf[t]), st.l);
    }
#pragma unroll
    for (int d = 0; d < PIECES; ++d)
#pragma unroll
        for (int h = 0; h < 2; ++h) {             // bytes 2 h and 2 h + 1 of dword d: two dimension tiles
            f16x8 v0, v1;
#pragma unroll
            for (int j = 0; j < 4; ++j) {         // token pairs
                const uint32_t w0 = v[j >> 1][2 * (j & 1)][d], w1 = v[j >> 1][2 * (j & 1) + 1][d];
                // bytes (tok0.b, tok1.b, tok0.b+1, tok1.b+1)
                const uint32_t pk = __builtin_amdgcn_perm(w1, w0, h ? 0x07030602u : 0x05010400u);
                const f16x2 lo2 = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(pk, 1.0f, false);
                const f16x2 hi2 = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(pk, 1.0f, true);
                v0[2 * j] = lo2[0];
                v0[2 * j + 1] = lo2[1];
                v1[2 * j] = hi2[0];
                v1[2 * j + 1] = hi2[1];
            }
            st.acc[4 * d + 2 * h] = __builtin_amdgcn_mfma_f32_16x16x32_f16(v0, w, st.acc[4 * d + 2 * h], 0, 0, 0);
            st.acc[4 * d + 2 * h + 1] = __builtin_amdgcn_mfma_f32_16x16x32_f16(v1, w, st.acc[4 * d + 2 * h + 1], 0, 0, 0);
        }
}

template <int D>
__global__ __launch_bounds__(256) __attribute__((amdgpu_waves_per_eu(D == 256 ? 2 : 3)))
void k_attend_rows(AttendArgs a) {
    constexpr int PIECES = D / 64;        // 16-byte pieces of a key per lane; values dwords per token
    constexpr int KSTEPS = D / 32;        // products along the dimensions
    constexpr int TILES = D / 16;         // value dimension tiles of the output
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int col = lane & 15, quarter = lane >> 4;
    const int split = blockIdx.x;
    const int head = blockIdx.y % a.c.heads, tile0 = blockIdx.y / a.c.heads;
    const int seq = blockIdx.z;
    const int begin = scalar_load(a.b.starts + seq), fresh = scalar_load(a.b.starts + seq + 1) - begin;
    const int before = scalar_load(a.b.lengths + seq);
    const int rows = fresh * a.group;
    const int reach = a.b.table_width << a.c.page_log2;      // positions the table can hold
    const int P = 1 << a.c.page_log2;
    __shared__ float sm[KV_WAVES][16], sl[KV_WAVES][16];
    __shared__ f32x4 so[2][TILES][64];
    const uint32_t koff = col * D + 16 * quarter, voff = 4 * quarter * D + col * (D / 16);

    for (int tile = tile0; tile * 16 < rows; tile += a.row_tiles) {
        const int row = tile * 16 + col;
        const bool live = row < rows;
        const int token = (live ? row : rows - 1) / a.group;
        const int qhead = head * a.group + (live ? row : rows - 1) % a.group;
        int position = before + token;
        if (position >= reach) position = -1;                 // left out: attends to nothing
        const int last_row = tile * 16 + 15 < rows ? tile * 16 + 15 : rows - 1;
        const int low = before + tile * 16 / a.group;         // the first row's position
        int keys = before + last_row / a.group + 1;           // keys the tile's last row sees
        const bool past = keys > reach;
        keys = past ? reach : keys;
        // queries: the lane's dimensions of MFMA step s, in the order of the key pieces
        bf16x8 qf[KSTEPS];
        {
            const uint16_t* qp = (const uint16_t*)a.q.data + (int64_t)(begin + token) * a.q.token_stride +
                                 (int64_t)qhead * a.q.head_stride;
#pragma unroll
            for (int s = 0; s < KSTEPS; ++s)
                qf[s] = *reinterpret_cast<const bf16x8*>(qp + 64 * (s >> 1) + 16 * quarter + 8 * (s & 1));
        }
        RowsState<D> st;
#pragma unroll
        for (int i = 0; i < TILES; ++i) st.acc[i] = f32x4{};
        st.m = KV_FLOOR;
        st.l = 0.0f;

        const int chunks = (keys + a.chunk - 1) / a.chunk;
        for (int ch = split; ch < chunks; ch += a.splits) {
            const int lo = ch * a.chunk;
            const int hi = lo + a.chunk < keys ? lo + a.chunk : keys;
            // this wave's steps: keys lo + 32 (wave + 4 i) ..
            const int all = (hi - lo + KV_STEP - 1) / KV_STEP;
            const int steps = (all - wave + KV_WAVES - 1) / KV_WAVES;
            auto first_key = [&](int i) { return lo + KV_STEP * (wave + KV_WAVES * i); };
            struct Pages {
                int p[2];
            };
            auto pages = [&](int i) {
                Pages g;
#pragma unroll
                for (int t = 0; t < 2; ++t) g.p[t] = uniform_page_of(a.c, a.b, seq, (first_key(i) + 16 * t) >> a.c.page_log2);
                return g;
            };
            auto load = [&](StepCodes<D>& x, int i, const Pages& g) {
#pragma unroll
                for (int t = 0; t < 2; ++t) {
                    const int at = first_key(i) + 16 * t;
                    const TileView v = tile_view<D>(a.c, g.p[t], head, at & (P - 1), hi - at);
                    x.ks[t] = v.ks;
                    x.vf[t] = v.vf;
                    x.end[t] = g.p[t] < 0 ? 0 : hi;           // a page outside the pool holds no keys
#pragma unroll
                    for (int p = 0; p < PIECES; ++p) x.k[t][p] = buf_load16(v.k, koff + 64 * p, 0);
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        if constexpr (D == 64) x.v[t][r][0] = buf_load4(v.v, voff + r * D, 0);
                        if constexpr (D == 128) {
                            const uint2 w = buf_load8(v.v, voff + r * D, 0);
                            x.v[t][r][0] = w.x;
                            x.v[t][r][1] = w.y;
                        }
                        if constexpr (D == 256) {
                            const uint4 w = buf_load16(v.v, voff + r * D, 0);
                            x.v[t][r][0] = w.x;
                            x.v[t][r][1] = w.y;
                            x.v[t][r][2] = w.z;
                            x.v[t][r][3] = w.w;
                        }
                    }
                }
            };
            auto compute = [&](const StepCodes<D>& x, int i) {
                float y[8];
#pragma unroll
                for (int t = 0; t < 2; ++t) {
                    f32x4 s = {};
#pragma unroll
                    for (int u = 0; u < KSTEPS; ++u) {
                        const uint4 w = x.k[t][u >> 1];
                        const bf16x8 kf = codes_to_bf16((u & 1) ? make_uint2(w.z, w.w) : make_uint2(w.x, w.y), 1.0f);
                        s = __builtin_amdgcn_mfma_f32_16x16x32_bf16(kf, qf[u], s, 0, 0, 0);
                    }
                    const int key = first_key(i) + 16 * t;
                    const float f = x.ks[t] * a.scale2;
#pragma unroll
                    for (int r = 0; r < 4; ++r) y[4 * t + r] = __fmaf_rn(s[r], f, x.vf[t]);
                    if (key + 15 > low || key + 16 > x.end[t] || past) {     // some column does not see some key
#pragma unroll
                        for (int r = 0; r < 4; ++r) {
                            const int k = key + 4 * quarter + r;
                            y[4 * t + r] = k <= position && k < x.end[t] ? y[4 * t + r] : -INFINITY;
                        }
                    }
                }
                attend_step<D>(st, y, x.v, x.vf);
            };
            if (steps > 0) {
                StepCodes<D> x0, x1;
                load(x0, 0, pages(0));
                Pages g1 = pages(steps > 1 ? 1 : 0);
                int i = 0;
                for (; i + 2 < steps; i += 2) {
                    const Pages g2 = pages(i + 2);
                    load(x1, i + 1, g1);
                    compute(x0, i);
                    g1 = pages(i + 3 < steps ? i + 3 : i + 2);
                    load(x0, i + 2, g2);
                    compute(x1, i + 1);
                }
                if (i + 1 < steps) {
                    load(x1, i + 1, g1);
                    compute(x0, i);
                    compute(x1, i + 1);
                } else {
                    compute(x0, i);
                }
            }
        }
        // ---- the waves join: a common reference, then the sums ----
        float l = st.l;
        l += __shfl_xor(l, 16);
        l += __shfl_xor(l, 32);
        if (quarter == 0) {
            sm[wave][col] = st.m;
            sl[wave][col] = l;
        }
        __syncthreads();
        float top = sm[0][col], total = 0.0f;
#pragma unroll
        for (int w = 1; w < KV_WAVES; ++w) top = fmaxf(top, sm[w][col]);
#pragma unroll
        for (int w = 0; w < KV_WAVES; ++w) total += sl[w][col] * __builtin_amdgcn_exp2f(sm[w][col] - top);
        const float f = __builtin_amdgcn_exp2f(st.m - top);
#pragma unroll
        for (int i = 0; i < TILES; ++i) st.acc[i] *= f;
        for (int half = 2; half >= 1; half >>= 1) {           // waves 2, 3 onto 0, 1, then 1 onto 0
            if (wave >= half && wave < 2 * half) {
#pragma unroll
                for (int i = 0; i < TILES; ++i) so[wave - half][i][lane] = st.acc[i];
            }
            __syncthreads();
            if (wave < half) {
#pragma unroll
                for (int i = 0; i < TILES; ++i) st.acc[i] += so[wave][i][lane];
            }
            __syncthreads();
        }
        if (wave == 0 && live) {
            const int64_t t = begin + token;
            if (a.splits == 1) {
                const float inv = total > 0.0f || total != total ? 1.0f / total : 0.0f;
                uint16_t* o = (uint16_t*)a.out.data + t * a.out.token_stride + qhead * a.out.head_stride;
#pragma unroll
                for (int r = 0; r < 4; ++r)
#pragma unroll
                    for (int i = 0; i < TILES; i += 4) {
                        const uint2 w = make_uint2(pack_bf16x2(st.acc[i][r] * inv, st.acc[i + 1][r] * inv),
                                                   pack_bf16x2(st.acc[i + 2][r] * inv, st.acc[i + 3][r] * inv));
                        *reinterpret_cast<uint2*>(o + (4 * quarter + r) * TILES + i) = w;
                    }
            } else {
                const int64_t at = (t * (int64_t)(a.c.heads * a.group) + qhead) * a.splits + split;
                float* p = a.part + at * D;
#pragma unroll
                for (int r = 0; r < 4; ++r)
#pragma unroll
                    for (int i = 0; i < TILES; i += 4)
                        *reinterpret_cast<f32x4*>(p + (4 * quarter + r) * TILES + i) =
                            f32x4{st.acc[i][r], st.acc[i + 1][r], st.acc[i + 2][r], st.acc[i + 3][r]};
                if (quarter == 0) a.sums[at] = make_float2(top, total);
            }
        }
    }
}

// Joins the chunks of each row: W waves per (token, head), D / 4 lanes per chunk.
template <int D, int W>
__global__ __launch_bounds__(256)
void k_attend_join(AttendArgs a) {
    constexpr int LANES = D / 4, GROUPS = W * 64 / LANES;     // chunks at a time
    const int in = threadIdx.x % (W * 64), lane = in & 63;
    const int heads = a.c.heads * a.group;
    const int64_t row = (int64_t)blockIdx.x * (4 / W) + threadIdx.x / (W * 64);
    const bool on = row < (int64_t)a.b.tokens * heads;
    const int64_t base = on ? row * a.splits : 0;
    const int splits = on ? a.splits : 0;
    const int group = in / LANES, c = in % LANES;
    // every wave finds the row's reference for itself
    float top = KV_FLOOR;
    for (int s = lane; s < splits; s += 64) top = fmaxf(top, a.sums[base + s].x);
#pragma unroll
    for (int x = 1; x < 64; x <<= 1) top = fmaxf(top, __shfl_xor(top, x));
    float total = 0.0f;
    f32x4 o = {};
#pragma unroll 4
    for (int s = group; s < splits; s += GROUPS) {
        const float2 ml = a.sums[base + s];
        const f32x4 p = *reinterpret_cast<const f32x4*>(a.part + (base + s) * D + 4 * c);
        const float f = __builtin_amdgcn_exp2f(ml.x - top);
        total += ml.y * f;
        o += p * f;
    }
#pragma unroll
    for (int x = LANES; x < 64; x <<= 1) {
        total += __shfl_xor(total, x);
#pragma unroll
        for (int i = 0; i < 4; ++i) o[i] += __shfl_xor(o[i], x);
    }
    if constexpr (W > 1) {
        __shared__ f32x4 so[W][LANES];
        __shared__ float st[W];
        const int wave = in >> 6;
        if (lane < LANES) so[wave][lane] = o;
        if (lane == 0) st[wave] = total;
        __syncthreads();
        if (wave != 0) return;
#pragma unroll
        for (int w = 1; w < W; ++w) {
            o += so[w][c];
            total += st[w];
        }
    }
    if (!on || lane >= LANES) return;
    const float inv = total > 0.0f || total != total ? 1.0f / total : 0.0f;
    uint16_t* out = (uint16_t*)a.out.data + (row / heads) * a.out.token_stride + (row % heads) * a.out.head_stride;
    *reinterpret_cast<uint2*>(out + 4 * c) = make_uint2(pack_bf16x2(o[0] * inv, o[1] * inv), pack_bf16x2(o[2] * inv, o[3] * inv));
}

struct AttendPlan {
    int row_tiles, chunk, splits;
    size_t bytes;
};

// Chunks are sized for about 4096 workgroups (some rounds of three or four on each compute unit) at the
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
    int64_t chunk = (max_length * groups / 4096 + unit - 1) / unit * unit;
    if (chunk < 256) chunk = 256;
    if (chunk > (1 << 20)) chunk = 1 << 20;
    p.chunk = (int)chunk;
    int64_t splits = (max_length + chunk - 1) / chunk;
    splits = splits < 1 ? 1 : (splits < 1024 ? splits : 1024);
    p.splits = (int)splits;
    p.bytes = splits > 1 ? (size_t)tokens * heads * splits * (c.dim + 2) * sizeof(float) : 0;   // sums, then references
    return p;
}

size_t kv_attention_ws_bytes(const CacheView& c, int seqs, int64_t tokens, int heads, int64_t max_new,
                             int64_t max_length) {
    return attend_plan(c, seqs, tokens, heads, max_new, max_length).bytes;
}

hipError_t launch_kv_attention(const CacheView& c, const BatchView& b, const HeadsView& q, const HeadsView& out,
                               float scale, int64_t max_new, int64_t max_length, void* ws, hipStream_t s) {
    const AttendPlan p = attend_plan(c, b.seqs, b.tokens, q.heads, max_new, max_length);
    AttendArgs a{c, b, q, out, q.heads / c.heads, p.row_tiles, p.chunk, p.splits, scale * 1.4426950408889634f, (float*)ws,
                 (float2*)((float*)ws + (size_t)b.tokens * q.heads * p.splits * c.dim)};
    const dim3 grid((uint32_t)p.splits, (uint32_t)(c.heads * p.row_tiles), (uint32_t)b.seqs);
    const int64_t rows = (int64_t)b.tokens * q.heads;
    const bool wide = p.splits > 16;      // four waves to a row: its chunks' loads take turns otherwise
    auto with = [&](auto dim) {
        constexpr int D = decltype(dim)::value;
        hipLaunchKernelGGL(k_attend_rows<D>, grid, dim3(256), 0, s, a);
        if (p.splits > 1 && wide) hipLaunchKernelGGL((k_attend_join<D, 4>), dim3((uint32_t)rows), dim3(256), 0, s, a);
        else if (p.splits > 1) hipLaunchKernelGGL((k_attend_join<D, 1>), dim3((uint32_t)((rows + 3) / 4)), dim3(256), 0, s, a);
    };
    if (c.dim == 64) with(std::integral_constant<int, 64>{});
    else if (c.dim == 128) with(std::integral_constant<int, 128>{});
    else with(std::integral_constant<int, 256>{});
    return hipGetLastError();
}

}  // namespace nf4
