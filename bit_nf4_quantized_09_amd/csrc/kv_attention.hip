// kv_attention.hip -- causal attention over the paged 8-bit cache (gfx950).
//
// Mathematics.  One pass over the keys with the running maximum and sum of a softmax.  With
// base-2 scores x_j = scale log2(e) q.k_j and page exponents f_j of the values (v = code 2^f),
// the kernel sums w_j = 2^(x_j + f_j - m) against the bare codes, m a running reference of
// x + f, and 2^(-f_j) w_j for the denominator: the value scales cost one addition per score.
// Rounding: keys are exact in bf16 (E4M3 has 4 significant bits, the scale is a power of
// two), scores, maxima, sums and outputs are fp32, and the weights go into the second
// product as fp16, the largest between 2^10 and 2^15: 11 significant bits down to 2^-24 of the
// largest, an eighth of bf16's error (the output itself is bf16).
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
// Work.  Up to 32 rows of a (sequence, kv head), k_attend_rows: workgroups of four waves own
// (sequence, kv head, row tile, chunk of keys); the waves take the chunk's steps in turn and join
// through LDS, and chunks of one row join in a second launch.  Bound by HBM, each key and value byte
// read once per row tile: 24 sequences of up to 4096 keys, 64 heads of 128 (716 MB): 126 us, 5.7 TB/s;
// two of 120001, 8 kv heads (343 MB): 76 us with the join.  A short sequence is bound by its chain
// of loads (length, page, codes): 6.3 us for one of 131 keys.
// More rows, k_attend_block: one, two or four waves own (sequence, kv head, 16 CT rows, chunk).  Bound by latency:
// a wave waits for its own loads, matrix and vector instructions in turn, registers leave room for two waves a
// SIMD, and blocks of unequal length leave one in the last third of the time.  3 prompts of up to 1500 tokens
// behind up to 1100 cached, 32 heads of 128 (74 GFLOP): 137 us alone, 127 a call among others, whose blocks fill
// that third (540 and 585 TFLOP/s); 1.5 of 2 waves resident, vector instructions issued 39% of the time, matrix
// cores busy 22%.
#include "bufio.h"
#include "paged.h"
#include "attend_plan.h"

namespace nf4 {

typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));

constexpr float KV_FLOOR = -3e38f;        // reference before any key: finite, so that no inf - inf arises
constexpr float KV_BIAS = 10.0f;          // weights are at most 2^(KV_BIAS + KV_SLACK) = 2^15 (fp16 reaches 2^16)
constexpr float KV_SLACK = 5.0f;          // a reference is raised once a score passes it by more than this

struct AttendArgs {
    CacheView c;
    BatchView b;
    HeadsView q, out;
    int group;                // query heads per kv head
    int row_tiles;            // k_attend_rows: launched row tiles per (sequence, kv head)
    int blocks;               // k_attend_block: launched blocks of CT row tiles per (sequence, kv head)
    int ordered;              // k_attend_block: blocks start in the order of their keys
    int chunk;                // keys per chunk, a multiple of 4 * KV_STEP
    int splits;               // launched chunks per row tile
    float scale2;             // |scale| * log2(e)
    uint32_t flip;            // sign bits of a bf16 pair if scale < 0
    int limit;                // rows of a (sequence, kv head) up to which k_attend_rows takes it (else k_attend_block)
    int few;                  // k_attend_rows: rows of each up to which they have slots for their chunks' parts
    float* part;              // [row slot][split][D] sums, and
    float2* sums;             // [row slot][split] reference and denominator (splits > 1)
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

// The table's entry for a page index of a sequence, through a scalar load that no branch and no check
// waits for: where the entry is looked at, page_or_none checks it.
__device__ __forceinline__ int page_entry(const BatchView& b, int seq, int page_index) {
    const int last = b.table_width - 1;
    return scalar_load(b.table + seq * b.table_stride + (page_index < last ? page_index : last));
}
__device__ __forceinline__ int page_or_none(const CacheView& c, int entry) { return entry >= 0 && entry < c.pages ? entry : -1; }

// Scales of a tile as bits.  They are looked at a step after their load was started.
struct TileScales {
    uint32_t k, v;
    int end;                              // keys of the tile that count lie below; 0: none, and the scales are anything
};
__device__ __forceinline__ float key_scale(const TileScales& t) { return t.end > 0 ? __uint_as_float(t.k) : 1.0f; }
// The factor from a product to its score is neither zero nor infinite: a hidden product is -inf and has to stay it, and
// a product of zero has to stay zero.
__device__ __forceinline__ float score_factor(float f) { return __builtin_amdgcn_fmed3f(f, 0x1p-126f, 0x1.fffffep127f); }
// A query's part of it, such that the product with any key scale (2^-50 .. 2^50) is so without a look at each step (1.5%
// of a prompt's time).  Products reach 2^25 where a query is scaled, so scores below the lower end are below 2^-23
// and those past the upper end are 2^5 apart at least: neither end changes a weight.
__device__ __forceinline__ float query_factor(float f) { return __builtin_amdgcn_fmed3f(f, 0x1p-98f, 0x1p77f); }
__device__ __forceinline__ float value_exponent(const TileScales& t) {
    return t.end > 0 ? (float)((int)((t.v >> 23) & 0xFFu) - 127) : 0.0f;
}

// One step's codes of a wave: two tiles of 16 keys.
template <int D>
struct StepCodes {
    uint4 k[2][D / 64];                   // [tile][piece]: 16 bytes of the lane's key
    uint32_t v[2][4][D / 64];             // [tile][token 4 g + r]: D / 16 bytes of its values
    TileScales scale[2];
    __amdgpu_buffer_rsrc_t values[2];
};

// The step's codes at key `first` of a sequence whose keys end at `hi`: ranges that end with the last key that
// counts, so that whatever lies behind it reads as zero; a page outside the pool holds no keys.  WIDE: both
// tiles are of one page.
template <int D, int AUX, bool WIDE>
__device__ __forceinline__ void load_values(StepCodes<D>& x, uint32_t voff) {
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const __amdgpu_buffer_rsrc_t rv = x.values[WIDE ? 0 : t];
            const uint32_t at = voff + (WIDE ? 16 * t * D : 0) + r * D;
            if constexpr (D == 64) x.v[t][r][0] = buf_load4_as<AUX>(rv, at);
            if constexpr (D == 128) {
                const uint2 w = buf_load8_as<AUX>(rv, at);
                x.v[t][r][0] = w.x;
                x.v[t][r][1] = w.y;
            }
            if constexpr (D == 256) {
                const uint4 w = buf_load16_as<AUX>(rv, at);
                x.v[t][r][0] = w.x;
                x.v[t][r][1] = w.y;
                x.v[t][r][2] = w.z;
                x.v[t][r][3] = w.w;
            }
        }
}
template <int D, int AUX, bool WIDE>
__device__ __forceinline__ void load_keys(StepCodes<D>& x, const CacheView& c, int head, int first, int hi, const int* entries,
                                          uint32_t koff) {
    constexpr int KEYS = WIDE ? 32 : 16;
    const int64_t page_bytes = (int64_t)D << c.page_log2;
    __amdgpu_buffer_rsrc_t rk;
#pragma unroll
    for (int t = 0; t < 2; ++t) {
        if (!WIDE || t == 0) {
            const int at = first + 16 * t, page = page_or_none(c, entries[t]);
            const int have = page < 0 || hi <= at ? 0 : (hi - at < KEYS ? hi - at : KEYS);
            const int64_t block = (int64_t)(page < 0 ? 0 : page) * 2 * c.heads + head;
            const uint8_t* kb = c.codes + block * page_bytes + (at & ((1 << c.page_log2) - 1)) * D;
            rk = make_rsrc(kb, have * D);
            x.values[t] = make_rsrc(kb + c.heads * page_bytes, have * D);
            x.scale[t] = TileScales{scalar_load((const uint32_t*)c.scales + block), scalar_load((const uint32_t*)c.scales + block + c.heads),
                                    have > 0 ? hi : 0};
        } else {
            x.scale[t] = x.scale[0];
        }
#pragma unroll
        for (int p = 0; p < D / 64; ++p) x.k[t][p] = buf_load16_as<AUX>(rk, koff + (WIDE ? 16 * t * D : 0) + 64 * p);
    }
}

// Values of 8 tokens in the order of the weights: bytes 2 h and 2 h + 1 of dword d.
template <int D>
__device__ __forceinline__ void values_of(const uint32_t (&v)[2][4][D / 64], int d, int h, f16x8& v0, f16x8& v1) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {             // token pairs
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
}

// The state of a tile of 16 columns (query rows) in a wave.
template <int D>
struct RowsState {
    f32x4 acc[D / 16];                    // dimension tile i: dimensions (4 quarter + r) * D / 16 + i
    float m, l;                           // reference (the same in a column's four lanes), the lane's part of the sum
};

// The scores of 32 keys (lane: column col, keys 4 quarter + r of tile t; s: products, f: scale) raise the
// state's reference where they must, and become weights.  vf: exponents of the values; ev: 2^-vf.
template <int D>
__device__ __forceinline__ f16x8 weights_of(RowsState<D>& st, const f32x4* s, const float* f, const float* vf, const float* ev) {
    float top = -INFINITY;
#pragma unroll
    for (int t = 0; t < 2; ++t)               // f > 0: the largest product has the largest score
        top = fmaxf(top, __fmaf_rn(fmaxf(fmaxf(s[t][0], s[t][1]), fmaxf(s[t][2], s[t][3])), f[t], vf[t]));
    if (__any(top > st.m + KV_SLACK)) {
        top = fmaxf(top, __shfl_xor(top, 16));
        top = fmaxf(top, __shfl_xor(top, 32));
        const float now = fmaxf(st.m, top);
        const float g = __builtin_amdgcn_exp2f(st.m - now);
        st.m = now;
        st.l *= g;
#pragma unroll
        for (int i = 0; i < D / 16; ++i) st.acc[i] *= g;
    }
    f16x8 w;
#pragma unroll
    for (int t = 0; t < 2; ++t) {
        const float shift = vf[t] - (st.m - KV_BIAS);
        float p[4];
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            p[r] = __builtin_amdgcn_exp2f(__fmaf_rn(s[t][r], f[t], shift));
            w[4 * t + r] = (_Float16)p[r];
        }
        st.l = __fmaf_rn((p[0] + p[1]) + (p[2] + p[3]), ev[t], st.l);
    }
    return w;
}

// A finished row, and a chunk's part of one, from the accumulators of a column's four lanes.
template <int D>
__device__ __forceinline__ void write_row(const f32x4* acc, float total, uint16_t* o, int quarter) {
    constexpr int TILES = D / 16;
    const float inv = total > 0.0f || total != total ? 1.0f / total : 0.0f;      // no key: zeros
#pragma unroll
    for (int r = 0; r < 4; ++r)
#pragma unroll
        for (int i = 0; i < TILES; i += 4)
            *reinterpret_cast<uint2*>(o + (4 * quarter + r) * TILES + i) =
                make_uint2(pack_bf16x2(acc[i][r] * inv, acc[i + 1][r] * inv), pack_bf16x2(acc[i + 2][r] * inv, acc[i + 3][r] * inv));
}
template <int D>
__device__ __forceinline__ void write_part(const f32x4* acc, float m, float total, float* p, float2* sums, int quarter) {
    constexpr int TILES = D / 16;
#pragma unroll
    for (int r = 0; r < 4; ++r)
#pragma unroll
        for (int i = 0; i < TILES; i += 4)
            *reinterpret_cast<f32x4*>(p + (4 * quarter + r) * TILES + i) = f32x4{acc[i][r], acc[i + 1][r], acc[i + 2][r], acc[i + 3][r]};
    if (quarter == 0) *sums = make_float2(m, total);
}

// Products of keys that a column does not see become -inf (a tile that every column sees passes).
__device__ __forceinline__ f32x4 hide(f32x4 s, int key, int quarter, int low, int position, int end, bool always) {
    if (key + 15 > low || key + 16 > end || always) {
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const int k = key + 4 * quarter + r;
            s[r] = k <= position && k < end ? s[r] : -INFINITY;
        }
    }
    return s;
}

// A query row as operands of the bf16 products: the lane's dimensions of product s, in the order of the key pieces.  A
// negative scale changes the queries' sign instead.  An infinity makes every score infinite or NaN, and a row
// of nothing but -inf would look like one without keys: it becomes a NaN at once.
template <int D>
__device__ __forceinline__ void load_query(const uint16_t* row, int quarter, uint32_t flip, bf16x8 (&q)[D / 32]) {
    typedef unsigned short u16x2 __attribute__((ext_vector_type(2)));
    u16x2 top = {0, 0};
#pragma unroll
    for (int s = 0; s < D / 32; ++s) {
        uint4 w = *reinterpret_cast<const uint4*>(row + 64 * (s >> 1) + 16 * quarter + 8 * (s & 1));
#pragma unroll
        for (uint32_t x : {w.x, w.y, w.z, w.w}) top = __builtin_elementwise_max(top, __builtin_bit_cast(u16x2, x & 0x7FFF7FFFu));
        w.x ^= flip;
        w.y ^= flip;
        w.z ^= flip;
        w.w ^= flip;
        q[s] = __builtin_bit_cast(bf16x8, w);
    }
    if (top[0] >= 0x7F80 || top[1] >= 0x7F80) q[0][0] = __builtin_bit_cast(__bf16, (unsigned short)0x7FC0);
}

// A query row for the 8-bit matrix instructions, in the order of the key pieces: times a power of two
// that brings its largest value to 128 .. 255, as the sum of two E4M3 numbers, the nearest one and 16 times
// what that leaves.  8 significant bits are two of 4 (the second has a sign), so this is exact down to
// 2^-14 of the largest value, and within 2^-23 of it below.  Returns what undoes the power of two.
typedef int i32x8 __attribute__((ext_vector_type(8)));
template <int D>
__device__ __forceinline__ float split_query(const uint16_t* row, int quarter, uint32_t flip, i32x8 (&q1)[D / 128], i32x8 (&q2)[D / 128]) {
    float x[D / 64][16], top = 0.0f;
#pragma unroll
    for (int p = 0; p < D / 64; ++p) {
        uint4 w[2];
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            w[u] = *reinterpret_cast<const uint4*>(row + 64 * p + 16 * quarter + 8 * u);
            w[u] = make_uint4(w[u].x ^ flip, w[u].y ^ flip, w[u].z ^ flip, w[u].w ^ flip);
            Vec16<uint16_t>::unpack(w[u], x[p] + 8 * u);
        }
#pragma unroll
        for (int i = 0; i < 16; ++i) top = fmaxf(top, fabsf(x[p][i]));
    }
    top = fmaxf(top, __shfl_xor(top, 16));
    top = fmaxf(top, __shfl_xor(top, 32));
    int e = 0;
    if (top > 0.0f && top < INFINITY) frexpf(top, &e);            // top = [0.5, 1) 2^e
    e = e < -110 ? -110 : e;                                      // (e <= 128: both powers are finite and normal)
    const float up = __uint_as_float((uint32_t)(127 + 8 - e) << 23);
#pragma unroll
    for (int p = 0; p < D / 64; ++p)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float y[4], r[4];
#pragma unroll
            for (int u = 0; u < 4; ++u) y[u] = x[p][4 * i + u] * up;
            int w = __builtin_amdgcn_cvt_pk_fp8_f32(y[0], y[1], 0, false);
            w = __builtin_amdgcn_cvt_pk_fp8_f32(y[2], y[3], w, true);
#pragma unroll
            for (int u = 0; u < 4; ++u) r[u] = (y[u] - e4m3_to_f32((uint32_t)w >> (8 * u) & 0xFFu)) * 16.0f;
            int v = __builtin_amdgcn_cvt_pk_fp8_f32(r[0], r[1], 0, false);
            v = __builtin_amdgcn_cvt_pk_fp8_f32(r[2], r[3], v, true);
            q1[p >> 1][4 * (p & 1) + i] = w;
            q2[p >> 1][4 * (p & 1) + i] = v;
        }
    return 1.0f / up;
}

// Calls f(first key, end) for chunks split, split + splits, .. of `keys` keys (none or fewer: no chunk; up to 2^31 - 1).
// In 32 bits without sign: splits * chunk is at most max_length + chunk, so nothing passes them, and no division is needed.
template <typename F>
__device__ __forceinline__ void for_chunks(int keys, int chunk, int split, int splits, F&& f) {
    const uint32_t end = keys > 0 ? keys : 0, jump = (uint32_t)splits * (uint32_t)chunk;
    uint32_t lo = (uint32_t)split * (uint32_t)chunk;
    while (lo < end) {
        f((int)lo, (int)(end - lo > (uint32_t)chunk ? lo + chunk : end));
        if (end - lo <= jump) break;
        lo += jump;
    }
}

template <int D, int AUX>
__global__ __launch_bounds__(256) __attribute__((amdgpu_waves_per_eu(D == 256 ? 1 : 3)))
void k_attend_rows(AttendArgs a) {
    constexpr int PIECES = D / 64;        // 16-byte pieces of a key per lane; values dwords per token
    constexpr int KSTEPS = D / 32;        // products along the dimensions
    constexpr int TILES = D / 16;         // value dimension tiles of the output
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int col = lane & 15, quarter = lane >> 4;
    const int split = blockIdx.x;
    const int head = blockIdx.y % a.c.heads, tile0 = blockIdx.y / a.c.heads;
    const int seq = blockIdx.z;
    const NewTokens fresh = new_tokens(a.b, scalar_load(a.b.starts + seq), scalar_load(a.b.starts + seq + 1));
    const int before = scalar_load(a.b.lengths + seq), begin = fresh.begin;
    const int rows = fresh.count * a.group;
    if (rows > a.limit) return;
    const int reach = a.b.table_width << a.c.page_log2;      // positions the table can hold
    __shared__ float sm[KV_WAVES][16], sl[KV_WAVES][16];
    __shared__ f32x4 so[2][TILES][64];
    const uint32_t koff = col * D + 16 * quarter, voff = 4 * quarter * D + col * (D / 16);

    for (int tile = tile0; tile * 16 < rows; tile += a.row_tiles) {
        // a sequence with more rows than were announced has no slots: one workgroup takes all of its chunks
        const bool whole = a.splits == 1 || rows > a.few;
        if (whole && split > 0) continue;
        const int stride = whole ? 1 : a.splits;
        const int row = tile * 16 + col;
        const bool live = row < rows;
        const int token = (live ? row : rows - 1) / a.group;
        const int qhead = head * a.group + (live ? row : rows - 1) % a.group;
        int position = position_at(before, token);
        if (position >= reach) position = -1;                 // left out: attends to nothing
        const int last_row = tile * 16 + 15 < rows ? tile * 16 + 15 : rows - 1;
        const int low = position_at(before, tile * 16 / a.group);         // the first row's position
        int keys = position_at(before, last_row / a.group + 1);           // keys the tile's last row sees
        const bool past = keys > reach;
        keys = past ? reach : keys;
        bf16x8 qf[KSTEPS];
        {
            const uint16_t* qp = (const uint16_t*)a.q.data + (int64_t)(begin + token) * a.q.token_stride +
                                 (int64_t)qhead * a.q.head_stride;
            load_query<D>(qp, quarter, a.flip, qf);
        }
        RowsState<D> st;
#pragma unroll
        for (int i = 0; i < TILES; ++i) st.acc[i] = f32x4{};
        st.m = KV_FLOOR;
        st.l = 0.0f;

        for_chunks(keys, a.chunk, split, stride, [&](int lo, int hi) {
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
                for (int t = 0; t < 2; ++t) g.p[t] = page_entry(a.b, seq, (first_key(i) + 16 * t) >> a.c.page_log2);
                return g;
            };
            auto load = [&](StepCodes<D>& x, int i, const Pages& g) {
                load_keys<D, AUX, false>(x, a.c, head, first_key(i), hi, g.p, koff);
                load_values<D, AUX, false>(x, voff);
            };
            auto compute = [&](const StepCodes<D>& x, int i) {
                f32x4 sc[2];
                float f[2], vf[2], ev[2];
#pragma unroll
                for (int t = 0; t < 2; ++t) {
                    f32x4 s = {};
#pragma unroll
                    for (int u = 0; u < KSTEPS; ++u) {
                        const uint4 w = x.k[t][u >> 1];
                        const bf16x8 kf = codes_to_bf16((u & 1) ? make_uint2(w.z, w.w) : make_uint2(w.x, w.y), 1.0f);
                        s = __builtin_amdgcn_mfma_f32_16x16x32_bf16(kf, qf[u], s, 0, 0, 0);
                    }
                    f[t] = score_factor(key_scale(x.scale[t]) * a.scale2);
                    vf[t] = value_exponent(x.scale[t]);
                    ev[t] = __builtin_amdgcn_exp2f(-vf[t]);
                    sc[t] = hide(s, first_key(i) + 16 * t, quarter, low, position, x.scale[t].end, past);
                }
                const f16x8 w = weights_of<D>(st, sc, f, vf, ev);
#pragma unroll
                for (int d = 0; d < PIECES; ++d)
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        f16x8 v0, v1;
                        values_of<D>(x.v, d, h, v0, v1);
                        st.acc[4 * d + 2 * h] = __builtin_amdgcn_mfma_f32_16x16x32_f16(v0, w, st.acc[4 * d + 2 * h], 0, 0, 0);
                        st.acc[4 * d + 2 * h + 1] = __builtin_amdgcn_mfma_f32_16x16x32_f16(v1, w, st.acc[4 * d + 2 * h + 1], 0, 0, 0);
                    }
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
        });
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
            if (whole) {
                write_row<D>(st.acc, total, (uint16_t*)a.out.data + t * a.out.token_stride + qhead * a.out.head_stride, quarter);
            } else {
                const int64_t at = (((int64_t)seq * a.c.heads + head) * a.few + row) * a.splits + split;
                write_part<D>(st.acc, top, total, a.part + at * D, a.sums + at, quarter);
            }
        }
    }
}

// The block of rank `rank` among those of an XCD's `here` <= 64 (sequence, kv head) pairs, the one with most keys
// first: the pair's index in x, its block in y (-1: there are not that many).  A lane has a pair; a block's
// keys are counted in blocks of rows, base + block, and the least count that `rank` blocks do not pass is
// searched for.
template <int BLOCK>
__device__ __forceinline__ int2 block_of_rank(const AttendArgs& a, int here, int rank, int lane) {
    const int pair = lane * XCDS + (int)(blockIdx.x % XCDS);
    int blocks = 0, base = 0;
    if (lane < here && pair < a.b.seqs * a.c.heads) {
        const int seq = pair / a.c.heads, rows = new_tokens(a.b, a.b.starts[seq], a.b.starts[seq + 1]).count * a.group;
        blocks = rows <= a.limit ? 0 : (rows + BLOCK - 1) / BLOCK;
        const int64_t rows_before = (int64_t)a.b.lengths[seq] * a.group / BLOCK;
        base = rows_before < 0 ? 0 : rows_before < (1 << 28) ? (int)rows_before : 1 << 28;
    }
    auto total = [&](int x) {
        for (int i = 1; i < here; i <<= 1) x += __shfl_xor(x, i);
        return __builtin_amdgcn_readfirstlane(x);
    };
    auto reaching = [&](int t) {              // this lane's blocks with t keys or more
        const int n = base + blocks - t;
        return n < 0 ? 0 : n < blocks ? n : blocks;
    };
    if (rank >= total(blocks)) return make_int2(0, -1);
    int low = 0, high = blocks > 0 ? base + blocks : 0;      // rank < count at `low`, not at `high`
    for (int i = 1; i < here; i <<= 1) high = max(high, __shfl_xor(high, i));
    high = __builtin_amdgcn_readfirstlane(high);
    while (high - low > 1) {
        const int mid = (low + high) >> 1;
        if (rank < total(reaching(mid))) low = mid;
        else high = mid;
    }
    // among the pairs that have a block of exactly `low`, the one that is as many places on
    int left = rank - total(reaching(low + 1));
    const uint64_t have = __ballot(reaching(low) > reaching(low + 1));
    uint64_t rest = have;
    for (; left > 0; --left) rest &= rest - 1;
    const int at = __ffsll((unsigned long long)rest) - 1;
    return make_int2(at, low - __builtin_amdgcn_readlane(base, at));
}

// Rows of a (sequence, kv head) beyond a few: a wave owns CT tiles of 16 rows and reads the codes itself,
// each decoded once for all of its tiles; no LDS, no barrier, but where W waves share the keys, at the end.  Scores
// by 8-bit products (D >= 128): the codes of the keys are the operand as they lie.  The workgroups of one (sequence, kv
// head) run on one XCD, whose L2 holds its keys; those that see most keys start first.
// (Heads of 64: three waves a SIMD, 74 us for 3 prompts of up to 1500 tokens behind up to 1100 cached, 32 heads; two 84.)
template <int D, int CT, bool WIDE, int W>
__global__ __launch_bounds__(64 * W) __attribute__((amdgpu_waves_per_eu(D == 64 && W == 1 ? 3 : 2)))
void k_attend_block(AttendArgs a) {
    constexpr int KSTEPS = D / 32, TILES = D / 16, PIECES = D / 64;
    constexpr bool F8 = D >= 128;
    const int lane = threadIdx.x & 63, wave = W > 1 ? __builtin_amdgcn_readfirstlane(threadIdx.x >> 6) : 0;
    const int col = lane & 15, quarter = lane >> 4;
    const int pairs = a.b.seqs * a.c.heads;
    const int local = (int)(blockIdx.x / XCDS), here = (pairs + XCDS - 1) / XCDS;      // of this XCD: workgroup, pairs
    const int split = blockIdx.y;
    const int reach = a.b.table_width << a.c.page_log2;
    const uint32_t koff = col * D + 16 * quarter, voff = 4 * quarter * D + col * (D / 16);
    constexpr int BLOCK = CT * 16;
    for (int rank = local;; rank += here * a.blocks) {
        int pair = rank % here * XCDS + (int)(blockIdx.x % XCDS), block = 0;
        if (a.ordered) {
            const int2 own = block_of_rank<BLOCK>(a, here, rank, lane);
            if (own.y < 0) return;
            pair = own.x * XCDS + (int)(blockIdx.x % XCDS);
            block = own.y;
        } else if (pair >= pairs) {
            return;
        }
        const int head = pair % a.c.heads, seq = pair / a.c.heads;
        const NewTokens fresh = new_tokens(a.b, scalar_load(a.b.starts + seq), scalar_load(a.b.starts + seq + 1));
        const int before = scalar_load(a.b.lengths + seq), begin = fresh.begin;
        const int rows = fresh.count * a.group;
        if (!a.ordered) {                     // a pair's last block first (every rank of this workgroup is of one pair)
            block = (rows + BLOCK - 1) / BLOCK - 1 - rank / here;
            if (block < 0 || rows <= a.limit) return;
        }
        const int row0 = block * BLOCK;
        const int last_row = row0 + BLOCK <= rows ? row0 + BLOCK - 1 : rows - 1;
        int keys = position_at(before, last_row / a.group + 1);
        const bool past = keys > reach;
        keys = past ? reach : keys;
        bf16x8 qf[F8 ? 1 : CT][KSTEPS];
        i32x8 q1[CT][F8 ? D / 128 : 1], q2[CT][F8 ? D / 128 : 1];
        float qs[CT];
        RowsState<D> st[CT];
        int position[CT], low[CT];                // of the lane's column; of the tile's first row
#pragma unroll
        for (int c = 0; c < CT; ++c) {
            const int row = row0 + 16 * c + col < rows ? row0 + 16 * c + col : rows - 1;
            const int token = row / a.group, qhead = head * a.group + row % a.group;
            position[c] = position_at(before, token);
            position[c] = position[c] < reach ? position[c] : -1;
            low[c] = position_at(before, (row0 + 16 * c) / a.group);
            const uint16_t* qp = (const uint16_t*)a.q.data + (int64_t)(begin + token) * a.q.token_stride +
                                 (int64_t)qhead * a.q.head_stride;
            if constexpr (!F8) {
                qs[c] = query_factor(a.scale2);
                load_query<D>(qp, quarter, a.flip, qf[c]);
            } else {
                qs[c] = query_factor(split_query<D>(qp, quarter, a.flip, q1[c], q2[c]) * a.scale2);
            }
#pragma unroll
            for (int i = 0; i < TILES; ++i) st[c].acc[i] = f32x4{};
            st[c].m = KV_FLOOR;
            st[c].l = 0.0f;
        }
        for_chunks(keys, a.chunk, split, a.splits, [&](int lo, int hi) {
            const int steps = ((hi - lo + KV_STEP - 1) / KV_STEP - wave + W - 1) / W;     // of this wave: every W-th
            auto first_key = [&](int i) { return lo + KV_STEP * (W * i + wave); };
            struct Pages {
                int p[2];
            };
            auto pages = [&](int i) {
                Pages g;
#pragma unroll
                for (int t = 0; t < (WIDE ? 1 : 2); ++t) g.p[t] = page_entry(a.b, seq, (first_key(i) + 16 * t) >> a.c.page_log2);
                return g;
            };
            auto load = [&](StepCodes<D>& x, int i, const Pages& g) {
                load_keys<D, 0, WIDE>(x, a.c, head, first_key(i), hi, g.p, koff);
            };
            // (a step's values are started as it begins, its keys a step before: 16 D / 64 registers fewer)
            auto values = [&](StepCodes<D>& x) { load_values<D, 0, WIDE>(x, voff); };
            auto compute = [&](const StepCodes<D>& x, int i) {
                const int first = first_key(i);
                f32x4 sc[CT][2];
                float ks[2], vf[2], ev[2];
#pragma unroll
                for (int t = 0; t < 2; ++t) {
                    ks[t] = key_scale(x.scale[t]);
                    vf[t] = value_exponent(x.scale[t]);
                    ev[t] = __builtin_amdgcn_exp2f(-vf[t]);
#pragma unroll
                    for (int c = 0; c < CT; ++c) sc[c][t] = f32x4{};
                    if constexpr (!F8) {
#pragma unroll
                        for (int u = 0; u < KSTEPS; ++u) {
                            const uint4 w = x.k[t][u >> 1];
                            const bf16x8 kf = codes_to_bf16((u & 1) ? make_uint2(w.z, w.w) : make_uint2(w.x, w.y), 1.0f);
#pragma unroll
                            for (int c = 0; c < CT; ++c) sc[c][t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(kf, qf[c][u], sc[c][t], 0, 0, 0);
                        }
                    } else {
#pragma unroll
                        for (int b = 0; b < D / 128; ++b) {
                            const uint4 w0 = x.k[t][2 * b], w1 = x.k[t][2 * b + 1];
                            const i32x8 kf = {(int)w0.x, (int)w0.y, (int)w0.z, (int)w0.w, (int)w1.x, (int)w1.y, (int)w1.z, (int)w1.w};
                            // (formats E4M3; scales 2^0, and 2^-4 for the second part of the queries)
#pragma unroll
                            for (int c = 0; c < CT; ++c) {
                                sc[c][t] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(kf, q1[c][b], sc[c][t], 0, 0, 0, 127, 0, 127);
                                sc[c][t] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(kf, q2[c][b], sc[c][t], 0, 0, 0, 127, 0, 123);
                            }
                        }
                    }
                }
                f16x8 w[CT];
#pragma unroll
                for (int c = 0; c < CT; ++c) {
#pragma unroll
                    for (int t = 0; t < 2; ++t)
                        sc[c][t] = hide(sc[c][t], first + 16 * t, quarter, low[c], position[c], x.scale[t].end, past);
                    const float f[2] = {ks[0] * qs[c], ks[1] * qs[c]};
                    w[c] = weights_of<D>(st[c], sc[c], f, vf, ev);
                }
#pragma unroll
                for (int d = 0; d < PIECES; ++d)
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        f16x8 v0, v1;
                        values_of<D>(x.v, d, h, v0, v1);
#pragma unroll
                        for (int c = 0; c < CT; ++c) {
                            f32x4 &o0 = st[c].acc[4 * d + 2 * h], &o1 = st[c].acc[4 * d + 2 * h + 1];
                            o0 = __builtin_amdgcn_mfma_f32_16x16x32_f16(v0, w[c], o0, 0, 0, 0);
                            o1 = __builtin_amdgcn_mfma_f32_16x16x32_f16(v1, w[c], o1, 0, 0, 0);
                        }
                    }
            };
            if (steps > 0) {
                StepCodes<D> x0, x1;
                load(x0, 0, pages(0));
                Pages g1 = pages(1);
                int i = 0;
                for (; i + 2 < steps; i += 2) {
                    const Pages g2 = pages(i + 2);
                    values(x0);
                    load(x1, i + 1, g1);
                    compute(x0, i);
                    g1 = pages(i + 3);
                    values(x1);
                    load(x0, i + 2, g2);
                    compute(x1, i + 1);
                }
                values(x0);
                if (i + 1 < steps) {
                    load(x1, i + 1, g1);
                    compute(x0, i);
                    values(x1);
                    compute(x1, i + 1);
                } else {
                    compute(x0, i);
                }
            }
        });
        if constexpr (W > 1) {                // the first wave adds the others' parts to its own
            __shared__ f32x4 parts[W - 1][CT][TILES][64];
            __shared__ float2 ends[W - 1][CT][64];
            if (wave > 0) {
#pragma unroll
                for (int c = 0; c < CT; ++c) {
                    ends[wave - 1][c][lane] = make_float2(st[c].m, st[c].l);
#pragma unroll
                    for (int i = 0; i < TILES; ++i) parts[wave - 1][c][i][lane] = st[c].acc[i];
                }
            }
            __syncthreads();
            if (wave == 0) {
#pragma unroll
                for (int c = 0; c < CT; ++c)
#pragma unroll
                    for (int w = 0; w < W - 1; ++w) {
                        const float2 other = ends[w][c][lane];
                        const float now = fmaxf(st[c].m, other.x);
                        const float mine = __builtin_amdgcn_exp2f(st[c].m - now), theirs = __builtin_amdgcn_exp2f(other.x - now);
                        st[c].m = now;
                        st[c].l = st[c].l * mine + other.y * theirs;
#pragma unroll
                        for (int i = 0; i < TILES; ++i) st[c].acc[i] = st[c].acc[i] * mine + parts[w][c][i][lane] * theirs;
                    }
            }
            __syncthreads();                  // the parts have been read before another block's are written
            if (wave > 0) continue;
        }
#pragma unroll
        for (int c = 0; c < CT; ++c) {
            float l = st[c].l;
            l += __shfl_xor(l, 16);
            l += __shfl_xor(l, 32);
            const int row = row0 + 16 * c + col;
            if (row >= rows) continue;
            const int64_t t = begin + row / a.group;
            const int qhead = head * a.group + row % a.group;
            if (a.splits == 1) {
                write_row<D>(st[c].acc, l, (uint16_t*)a.out.data + t * a.out.token_stride + qhead * a.out.head_stride, quarter);
            } else {
                const int64_t at = (t * (int64_t)(a.c.heads * a.group) + qhead) * a.splits + split;
                write_part<D>(st[c].acc, st[c].m, l, a.part + at * D, a.sums + at, quarter);
            }
        }
    }
}

// Joins the chunks of each row: W waves per row, D / 4 lanes per chunk.  FEW: the rows of
// k_attend_rows (slot: sequence, kv head, row), else those of k_attend_block (slot: token, head).
template <int D, int W, bool FEW>
__global__ __launch_bounds__(256)
void k_attend_join(AttendArgs a) {
    constexpr int LANES = D / 4, GROUPS = W * 64 / LANES;     // chunks at a time
    const int in = threadIdx.x % (W * 64), lane = in & 63;
    const int heads = a.c.heads * a.group;
    const int64_t slot = (int64_t)blockIdx.x * (4 / W) + threadIdx.x / (W * 64);
    int64_t token, qhead;
    bool on;
    if constexpr (FEW) {
        const int64_t pair = slot / a.few, row = slot % a.few;
        const int seq = (int)(pair / a.c.heads), head = (int)(pair % a.c.heads);
        on = seq < a.b.seqs;
        const NewTokens fresh = on ? new_tokens(a.b, a.b.starts[seq], a.b.starts[seq + 1]) : NewTokens{0, 0};
        const int begin = fresh.begin, rows = fresh.count * a.group;
        on = on && rows <= a.few && row < rows;
        token = begin + row / a.group;
        qhead = head * a.group + row % a.group;
    } else {
        token = slot / heads;
        qhead = slot % heads;
        on = token < a.b.tokens;
        if (on && a.limit > 0) {
            const int seq = sequence_of(a.b.starts, a.b.seqs, (int)token, lane);
            on = new_tokens(a.b, a.b.starts[seq], a.b.starts[seq + 1]).count * a.group > a.limit;
        }
    }
    const int64_t base = slot * a.splits;
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
    uint16_t* out = (uint16_t*)a.out.data + token * a.out.token_stride + qhead * a.out.head_stride;
    *reinterpret_cast<uint2*>(out + 4 * c) = make_uint2(pack_bf16x2(o[0] * inv, o[1] * inv), pack_bf16x2(o[2] * inv, o[3] * inv));
}

static AttendPlan plan_of(const CacheView& c, const BatchView& b, int heads, int64_t max_new, int64_t max_length) {
    return attend_plan(AttendShape{c.dim, c.heads, b.seqs, b.tokens, heads, max_new, max_length});
}

size_t kv_attention_ws_bytes(const CacheView& c, const BatchView& b, int heads, int64_t max_new, int64_t max_length) {
    const AttendPlan p = plan_of(c, b, heads, max_new, max_length);
    return p.rows.bytes + p.block.bytes;
}

hipError_t launch_kv_attention(const CacheView& c, const BatchView& b, const HeadsView& q, const HeadsView& out,
                               float scale, int64_t max_new, int64_t max_length, void* ws, hipStream_t s) {
    const AttendPlan p = plan_of(c, b, q.heads, max_new, max_length);
    AttendArgs a{};
    a.c = c;
    a.b = b;
    a.q = q;
    a.out = out;
    a.group = q.heads / c.heads;
    a.scale2 = fabsf(scale) * 1.4426950408889634f;
    a.flip = scale < 0.0f ? 0x80008000u : 0u;
    a.limit = !p.block.on ? 0x7FFFFFFF : p.rows.on ? KV_FEW : 0;
    auto part = [&](const AttendPart& q, void* at) {
        a.chunk = q.chunk;
        a.splits = q.splits;
        a.part = (float*)at;
        a.sums = (float2*)((float*)at + q.slots * q.splits * c.dim);
    };
    auto with = [&](auto dim) {
        constexpr int D = decltype(dim)::value;
        // W: four waves to a row of many chunks, whose loads would take turns otherwise
        if (p.block.on) {
            part(p.block, (uint8_t*)ws + p.rows.bytes);
            a.blocks = p.block.tiles;
            const int64_t pairs = ((int64_t)b.seqs * c.heads + XCDS - 1) / XCDS * XCDS;
            const dim3 grid((uint32_t)(pairs * a.blocks), (uint32_t)a.splits);
            // more waves than the 2048 that run at once: those with most keys first, in whichever sequence (a pair for
            // each lane; beyond some rounds the order of one sequence's blocks is enough)
            a.ordered = pairs <= 64 * XCDS && pairs * a.blocks * p.block.waves > 2048 && pairs * a.blocks * p.block.waves <= 8 * 2048;
            // pages of 32 tokens and more hold a whole step: half the address work (3 prompts of up to 1500
            // tokens, 32 heads of 64: 74 us for 85)
            auto run = [&](auto wide, auto waves) {
                constexpr int W = decltype(waves)::value;
                hipLaunchKernelGGL((k_attend_block<D, block_tiles(D), decltype(wide)::value, W>), grid, dim3(64 * W), 0, s, a);
            };
            auto with_pages = [&](auto waves) { c.page_log2 >= 5 ? run(std::true_type{}, waves) : run(std::false_type{}, waves); };
            if (p.block.waves == 1) with_pages(std::integral_constant<int, 1>{});
            if constexpr (D < 256) {
                if (p.block.waves == 2) with_pages(std::integral_constant<int, 2>{});
                if (p.block.waves == 4) with_pages(std::integral_constant<int, 4>{});
            }
            const int64_t rows = (int64_t)b.tokens * q.heads;
            if (a.splits > 16) hipLaunchKernelGGL((k_attend_join<D, 4, false>), dim3((uint32_t)rows), dim3(256), 0, s, a);
            else if (a.splits > 1) hipLaunchKernelGGL((k_attend_join<D, 1, false>), dim3((uint32_t)((rows + 3) / 4)), dim3(256), 0, s, a);
        }
        if (p.rows.on) {
            part(p.rows, ws);
            a.row_tiles = p.rows.tiles;
            a.few = p.rows.few;
            // codes that one row tile reads are read once: they need not stay in the caches (716 MB: 128 us, 138 with them)
            const dim3 grid((uint32_t)a.splits, (uint32_t)(c.heads * a.row_tiles), (uint32_t)b.seqs);
            if (a.row_tiles == 1) hipLaunchKernelGGL((k_attend_rows<D, 2>), grid, dim3(256), 0, s, a);
            else hipLaunchKernelGGL((k_attend_rows<D, 0>), grid, dim3(256), 0, s, a);
            const int64_t rows = (int64_t)b.seqs * c.heads * a.few;
            if (a.splits > 16) hipLaunchKernelGGL((k_attend_join<D, 4, true>), dim3((uint32_t)rows), dim3(256), 0, s, a);
            else if (a.splits > 1) hipLaunchKernelGGL((k_attend_join<D, 1, true>), dim3((uint32_t)((rows + 3) / 4)), dim3(256), 0, s, a);
        }
    };
    if (c.dim == 64) with(std::integral_constant<int, 64>{});
    else if (c.dim == 128) with(std::integral_constant<int, 128>{});
    else with(std::integral_constant<int, 256>{});
    return hipGetLastError();
}

}  // namespace nf4
