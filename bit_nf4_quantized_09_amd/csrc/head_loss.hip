// head_loss.hip -- softmax cross entropy of a vocabulary head without its logits (gfx950).
//
//   z = X W^T,  loss = lse(z) - z_y,  G = dloss (softmax(z) - onehot),  dX = G W,  dW = G^T X
//
// The vocabulary is taken in pieces.  A first pass computes the logits tile by tile and keeps
// of each tile only the maximum and the sum of exponentials of every row, the target's logit
// apart: with S = sum_{v != y} exp(z_v - z_y), loss = log1p(S) and 1 - p_y = S / (1 + S) keep
// their digits where the target has nearly all of the weight (lse - z_y would cancel).  For the gradient each piece's logits are computed
// again, turned into G (bf16, a piece of [M][piece], small enough to stay in the last-level
// cache) in the product's epilogue, and multiplied with the piece of W (dX, accumulated in fp32
// over the pieces) and with X (dW).  Rounding: logits, maxima, sums and accumulators are fp32;
// G is rounded to bf16, the type of the matrix instructions' operands and of the outputs; it
// holds dloss / max|dloss| times p - onehot, and the factor max|dloss| is applied to the fp32
// sums, so that a mean's 1/count does not round the many nearly equal target entries alike.
//
// Products.  256 x 256 output tiles, 8 waves, v_mfma_f32_32x32x16_bf16, contraction in steps
// of 64 through two LDS stages filled by direct loads.  Both products put the token (or, for
// dW, vocabulary) index into the accumulator's columns, so that a lane's 16 accumulators of a
// tile belong to one row of the result: the softmax's sums stay in the lane, and stores take
// four neighbours of a row at once.
#include "bufio.h"
#include "decoder.h"

namespace nf4 {

constexpr int HL_T = 256;                 // output tile, both ways
constexpr int HL_K = 64;                  // contraction step
constexpr int HL_STAGE = HL_T * HL_K * 2; // bytes of one operand's stage: 32 KB
constexpr float LOG2E = 1.4426950408889634f;
constexpr float LN2 = 0.6931471805599453f;

typedef __attribute__((address_space(3))) uint8_t lds_u8;

// Sixteen bytes per lane from memory into LDS at base + 16 * lane, without passing registers.
__device__ __forceinline__ void load_to_lds(__amdgpu_buffer_rsrc_t r, lds_u8* base, uint32_t voff, uint32_t soff) {
    __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (__attribute__((address_space(3))) void*)base, 16, (int)voff, (int)soff, 0, 0);
}

// Rows of 128 bytes (64 values of the contraction): 16-byte chunk c of row r lies at chunk
// c ^ g(r), so that 16 neighbouring rows reading one chunk meet all 64 banks once.
__device__ __forceinline__ int hl_swizzle(int row) { return (row ^ (row >> 3)) & 7; }
__device__ __forceinline__ int hl_off(int row, int chunk) { return row * 128 + ((chunk ^ hl_swizzle(row)) << 4); }

// Rows of 512 bytes (256 columns of one contraction value), read transposed: 32-byte segment
// u of row r lies at u ^ 2 (r & 3), so that the 4 rows x 2 segments of one pass meet all banks.
__device__ __forceinline__ int hl_toff(int row, int col) {
    return row * 512 + (((col >> 4) ^ ((row & 3) << 1)) << 5) + ((col & 15) << 1);
}

typedef short hl_i16x4 __attribute__((ext_vector_type(4)));
__device__ __forceinline__ uint2 hl_read_tr(const uint8_t* p) {
    const hl_i16x4 v = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
        (__attribute__((address_space(3))) hl_i16x4*)(const __attribute__((address_space(3))) uint8_t*)(p));
    return __builtin_bit_cast(uint2, v);
}

// Output tile of a workgroup: neighbours in launch order go to different XCDs, so XCD x gets a
// contiguous run of the tile order (columns of 4 row tiles), whose operands its L2 then shares.
__device__ __forceinline__ bool hl_tile(int wg, int tiles_a, int tiles_b, int& ta, int& tb) {
    const int total = tiles_a * tiles_b, q = total / 8, rem = total % 8;
    const int x = wg % 8, local = wg / 8;
    const int p = x * q + (x < rem ? x : rem) + local;
    if (local >= q + (x < rem ? 1 : 0)) return false;
    const int per = 4 * tiles_b, first = p / per * 4;
    const int g = tiles_a - first < 4 ? tiles_a - first : 4;
    ta = first + p % per % g;
    tb = p % per / g;
    return true;
}

struct HeadArgs {
    const uint16_t* X;        // [M][K]
    const uint16_t* W;        // [V][K]
    int64_t M, K, V;
    const int64_t* targets;
    int64_t ignore;
    int64_t v0;               // first vocabulary row of the launch, and
    int tiles_v, tiles_m;     // its tiles
    float2* part;             // [tile of v][Mp]: maximum and sum of a row, base 2 (statistics)
    float* zy;                // [Mp]: target's logit, base 2
    const float2* rows;       // [Mp]: lse, base 2, and 1 - p of the target (gradient)
    const float* dloss;
    uint32_t* top;            // max|dloss| as bits
    uint16_t* G;              // [Mp][ldg], or null
    uint16_t* Gt;             // [ldg][Mp], or null
    int64_t ldg, Mp;
};

// Logits of a 256 (vocabulary) x 256 (tokens) tile; GRAD false: row statistics, true: G.
template <bool GRAD>
__global__ __launch_bounds__(512)
void k_head_logits(HeadArgs a) {
    extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int h = lane >> 5, rl = lane & 31;
    int tv, tm;
    if (!hl_tile(blockIdx.x, a.tiles_v, a.tiles_m, tv, tm)) return;
    const int64_t v0 = a.v0 + (int64_t)tv * HL_T, m0 = (int64_t)tm * HL_T;
    if (!GRAD && blockIdx.x == 0 && tid == 0) *a.top = 0;      // for k_head_rows
    const int wv = wave >> 2, wm = wave & 3;           // 2 x 4 waves of 128 x 64
    // rows past the end repeat the last one (their results are dropped)
    uint32_t wof[4], xof[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int row = wave * 32 + i * 8 + (lane >> 3);
        const int chunk = (lane & 7) ^ hl_swizzle(row);
        const int64_t rv = v0 + row < a.V ? row : a.V - 1 - v0, rm = m0 + row < a.M ? row : a.M - 1 - m0;
        wof[i] = (uint32_t)(rv * a.K * 2) + chunk * 16;
        xof[i] = (uint32_t)(rm * a.K * 2) + chunk * 16;
    }
    const __amdgpu_buffer_rsrc_t rw = make_rsrc(a.W + v0 * a.K, (a.V - v0) * a.K * 2);
    const __amdgpu_buffer_rsrc_t rx = make_rsrc(a.X + m0 * a.K, (a.M - m0) * a.K * 2);
    auto load = [&](int stage, int step) {
        lds_u8* base = (lds_u8*)lds + stage * 2 * HL_STAGE + wave * 4096;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            load_to_lds(rw, base + i * 1024, wof[i], (uint32_t)step * 128);
            load_to_lds(rx, base + HL_STAGE + i * 1024, xof[i], (uint32_t)step * 128);
        }
    };
    f32x16 acc[4][2];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j) acc[i][j] = f32x16{};
    const int steps = (int)(a.K / HL_K);
    load(0, 0);
    for (int it = 0; it < steps; ++it) {
        asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
        __syncthreads();
        if (it + 1 < steps) load((it + 1) & 1, it + 1);
        const uint8_t* sw = lds + (it & 1) * 2 * HL_STAGE;
        const uint8_t* sx = sw + HL_STAGE;
#pragma unroll
        for (int s = 0; s < 4; ++s) {
            bf16x8 af[4], bf[2];
#pragma unroll
            for (int j = 0; j < 2; ++j) bf[j] = *reinterpret_cast<const bf16x8*>(sx + hl_off(wm * 64 + j * 32 + rl, 2 * s + h));
#pragma unroll
            for (int i = 0; i < 4; ++i) af[i] = *reinterpret_cast<const bf16x8*>(sw + hl_off(wv * 128 + i * 32 + rl, 2 * s + h));
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 2; ++j) acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(af[i], bf[j], acc[i][j], 0, 0, 0);
        }
    }
    // accumulator (i, j, reg): vocabulary row 32 i + 8 (reg / 4) + 4 h + reg % 4 of the wave's 128,
    // token 32 j + rl of its 64
    const int64_t vw = v0 + wv * 128 + 4 * h;
    if constexpr (!GRAD) {
        __syncthreads();
        float2* join = reinterpret_cast<float2*>(lds);          // [2][256]
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const int64_t m = m0 + wm * 64 + j * 32 + rl;
            const int64_t target = m < a.M ? a.targets[m] : -1;
            float top = -INFINITY;
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int r = 0; r < 16; ++r) {
                    const int64_t v = vw + i * 32 + 8 * (r >> 2) + (r & 3);
                    float z = v < a.V ? acc[i][j][r] * LOG2E : -INFINITY;
                    if (v == target && v < a.V) {
                        a.zy[m] = z;
                        z = -INFINITY;
                    }
                    acc[i][j][r] = z;
                    top = fmaxf(top, z);
                }
            float sum = 0.0f;
            const float ref = top > -INFINITY ? top : 0.0f;
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int r = 0; r < 16; ++r) sum += __builtin_amdgcn_exp2f(acc[i][j][r] - ref);
            const float other = __shfl_xor(top, 32), osum = __shfl_xor(sum, 32);
            const float both = fmaxf(top, other), bref = both > -INFINITY ? both : 0.0f;
            sum = sum * __builtin_amdgcn_exp2f(top - bref) + osum * __builtin_amdgcn_exp2f(other - bref);
            if (h == 0) join[wv * 256 + wm * 64 + j * 32 + rl] = make_float2(both, sum);
        }
        __syncthreads();
        if (tid < 256) {
            const float2 p = join[tid], q = join[256 + tid];
            const float both = fmaxf(p.x, q.x), ref = both > -INFINITY ? both : 0.0f;
            const float sum = p.y * __builtin_amdgcn_exp2f(p.x - ref) + q.y * __builtin_amdgcn_exp2f(q.x - ref);
            a.part[((a.v0 / HL_T) + tv) * a.Mp + m0 + tid] = make_float2(both, sum);
        }
    } else {
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const int64_t m = m0 + wm * 64 + j * 32 + rl;
            int64_t target = m < a.M ? a.targets[m] : -1;
            const bool live = m < a.M && target >= 0 && target < a.V && target != a.ignore;
            const float most = __uint_as_float(*a.top);
            const float g = live ? (most > 0.0f ? a.dloss[m] / most : a.dloss[m]) : 0.0f;
            const float2 row = live ? a.rows[m] : make_float2(0.0f, 0.0f);
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int r4 = 0; r4 < 4; ++r4) {
                    const int64_t v = vw + i * 32 + 8 * r4;
                    float y[4];
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        const float p = __builtin_amdgcn_exp2f(acc[i][j][4 * r4 + r] * LOG2E - row.x);
                        y[r] = live && v + r < a.V ? g * (v + r == target ? -row.y : p) : 0.0f;
                    }
                    const uint2 w = make_uint2(pack_bf16x2(y[0], y[1]), pack_bf16x2(y[2], y[3]));
                    if (a.G) *reinterpret_cast<uint2*>(a.G + m * a.ldg + (v - a.v0)) = w;
                    if (a.Gt) {
                        uint16_t* t = a.Gt + (v - a.v0) * a.Mp + m;
                        t[0] = (uint16_t)w.x;
                        t[a.Mp] = (uint16_t)(w.x >> 16);
                        t[2 * a.Mp] = (uint16_t)w.y;
                        t[3 * a.Mp] = (uint16_t)(w.y >> 16);
                    }
                }
        }
    }
}

// lse, loss and 1 - p of the target of each row from its tiles' statistics, and max|dloss|.
__global__ __launch_bounds__(256)
void k_head_rows(const float2* part, const float* zy, const int64_t* targets, int64_t M, int64_t Mp, int64_t V,
                 int64_t ignore, int tiles, const float* dloss, uint32_t* most, float2* rows, float* loss) {
    const int64_t m = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (m >= M) return;
    float top = -INFINITY, sum = 0.0f;
    for (int t = 0; t < tiles; ++t) {
        const float2 p = part[t * Mp + m];
        const float both = fmaxf(top, p.x), ref = both > -INFINITY ? both : 0.0f;
        sum = sum * __builtin_amdgcn_exp2f(top - ref) + p.y * __builtin_amdgcn_exp2f(p.x - ref);
        top = both;
    }
    const int64_t target = targets[m];
    const bool live = target >= 0 && target < V && target != ignore;
    if (!live) {
        if (loss) loss[m] = 0.0f;
        return;
    }
    const float rest = top + log2f(sum), z = zy[m], d = z - rest;   // the other entries' lse, base 2
    const float tail = log1pf(exp2f(-fabsf(d)));
    if (loss) loss[m] = d >= 0.0f ? tail : tail - d * LN2;
    rows[m] = make_float2(fmaxf(z, rest) + tail * LOG2E, 1.0f / (1.0f + exp2f(d)));
    if (dloss) {
        const float g = fabsf(dloss[m]);
        if (g < INFINITY) atomicMax(most, __float_as_uint(g));      // a maximum: any order gives the same
    }
}

struct ProductArgs {
    const uint16_t* A;        // [rows][lda]: contraction along the row
    int64_t lda, rows, out_rows;   // rows of A (all readable), rows written
    const uint16_t* B;        // [P][N]: contraction down the rows
    int64_t P, N;             // contraction values of B (A has zeros past them), columns
    int steps;                // contraction steps of 64: each starts below P
    int tiles_r, tiles_n;
    uint16_t* out;            // bf16 [out_rows][N], or null
    float* sum;               // fp32 [out_rows][N], or null
    int add;                  // 1: add what `sum` holds
    const uint32_t* top;      // factor on `out` (fp32 bits)
};

// C[r][n] = sum_p A[r][p] B[p][n], tiles of 256 rows x 256 columns.
__global__ __launch_bounds__(512)
void k_head_product(ProductArgs a) {
    extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int h = lane >> 5, rl = lane & 31;
    int tr, tn;
    if (!hl_tile(blockIdx.x, a.tiles_r, a.tiles_n, tr, tn)) return;
    const int64_t r0 = (int64_t)tr * HL_T, n0 = (int64_t)tn * HL_T;
    const int wn = wave >> 2, wr = wave & 3;           // 2 x 4 waves of 128 columns x 64 rows
    uint32_t aof[4];
    int brow[4];
    uint32_t bcol[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int row = wave * 32 + i * 8 + (lane >> 3);
        const int64_t ra = r0 + row < a.rows ? row : a.rows - 1 - r0;
        aof[i] = (uint32_t)(ra * a.lda * 2) + (((lane & 7) ^ hl_swizzle(row)) << 4);
        brow[i] = wave * 8 + i * 2 + (lane >> 5);
        const int q = lane & 31;
        const int chunk = (((q >> 1) ^ ((brow[i] & 3) << 1)) << 1) | (q & 1);
        bcol[i] = (uint32_t)(n0 + chunk * 8 < a.N ? chunk * 16 : 0);   // columns past the last: any, dropped
    }
    const __amdgpu_buffer_rsrc_t ra = make_rsrc(a.A + r0 * a.lda, (a.rows - r0) * a.lda * 2);
    auto load = [&](int stage, int step) {
        lds_u8* base = (lds_u8*)lds + stage * 2 * HL_STAGE + wave * 4096;
        const int64_t p0 = (int64_t)step * HL_K;
        const __amdgpu_buffer_rsrc_t rb = make_rsrc(a.B + p0 * a.N + n0, (a.P - p0) * a.N * 2);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            load_to_lds(ra, base + i * 1024, aof[i], (uint32_t)step * 128);
            // contraction rows past the last repeat it: A is zero there
            const int64_t row = p0 + brow[i] < a.P ? brow[i] : a.P - 1 - p0;
            load_to_lds(rb, base + HL_STAGE + i * 1024, (uint32_t)(row * a.N * 2) + bcol[i], 0);
        }
    };
    f32x16 acc[4][2];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j) acc[i][j] = f32x16{};
    const int g = lane >> 4, jl = lane & 15;
    const int trow = 8 * (g >> 1) + (jl >> 2);
    int tof[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) tof[i] = hl_toff(trow, wn * 128 + i * 32 + 16 * (g & 1) + 4 * (jl & 3));
    load(0, 0);
    for (int it = 0; it < a.steps; ++it) {
        asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
        __syncthreads();
        if (it + 1 < a.steps) load((it + 1) & 1, it + 1);
        const uint8_t* sa = lds + (it & 1) * 2 * HL_STAGE;
        const uint8_t* sb = sa + HL_STAGE;
#pragma unroll
        for (int s = 0; s < 4; ++s) {
            bf16x8 bf[4], af[2];
#pragma unroll
            for (int j = 0; j < 2; ++j) af[j] = *reinterpret_cast<const bf16x8*>(sa + hl_off(wr * 64 + j * 32 + rl, 2 * s + h));
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const uint2 lo = hl_read_tr(sb + tof[i] + s * 16 * 512);
                const uint2 hi = hl_read_tr(sb + tof[i] + s * 16 * 512 + 4 * 512);
                bf[i] = __builtin_bit_cast(bf16x8, make_uint4(lo.x, lo.y, hi.x, hi.y));
            }
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 2; ++j) acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(bf[i], af[j], acc[i][j], 0, 0, 0);
        }
    }
    // accumulator (i, j, reg): column 32 i + 8 (reg / 4) + 4 h + reg % 4 of the wave's 128, row 32 j + rl of its 64
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        const int64_t r = r0 + wr * 64 + j * 32 + rl;
        if (r >= a.out_rows) continue;
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int r4 = 0; r4 < 4; ++r4) {
                const int64_t n = n0 + wn * 128 + i * 32 + 8 * r4 + 4 * h;
                if (n >= a.N) continue;
                f32x4 y = {acc[i][j][4 * r4], acc[i][j][4 * r4 + 1], acc[i][j][4 * r4 + 2], acc[i][j][4 * r4 + 3]};
                if (a.add) y += *reinterpret_cast<const f32x4*>(a.sum + r * a.N + n);
                if (a.out) y *= __uint_as_float(*a.top);
                if (a.out)
                    *reinterpret_cast<uint2*>(a.out + r * a.N + n) = make_uint2(pack_bf16x2(y[0], y[1]), pack_bf16x2(y[2], y[3]));
                else
                    *reinterpret_cast<f32x4*>(a.sum + r * a.N + n) = y;
            }
    }
}

// Pieces of the vocabulary and the workspace's layout.
struct HeadPlan {
    int64_t Mp;               // tokens up to whole tiles
    int64_t tiles;            // vocabulary tiles
    int64_t piece;            // vocabulary tiles of a piece
    size_t top, zy, rows, part, G, Gt, sum, bytes;
};

static HeadPlan head_plan(int64_t M, int64_t K, int64_t V, bool dx, bool dw) {
    HeadPlan p{};
    p.Mp = (M + HL_T - 1) / HL_T * HL_T;
    p.tiles = (V + HL_T - 1) / HL_T;
    // a piece of G of at most 64 MB (and its transpose) stays in the 256 MB last-level cache
    const int64_t most = ((int64_t)64 << 20) / (p.Mp > 0 ? p.Mp * HL_T * 2 : 1);
    p.piece = most < 1 ? 1 : (most < p.tiles ? most : p.tiles);
    size_t at = 0;
    auto take = [&](size_t n) {
        const size_t was = at;
        at += (n + 255) & ~(size_t)255;
        return was;
    };
    p.top = take(4);
    p.zy = take((size_t)p.Mp * 4);
    p.rows = take((size_t)p.Mp * sizeof(float2));
    p.part = take((size_t)p.Mp * p.tiles * sizeof(float2));
    p.G = take(dx ? (size_t)p.Mp * p.piece * HL_T * 2 : 0);
    p.Gt = take(dw ? (size_t)p.Mp * p.piece * HL_T * 2 : 0);
    p.sum = take(dx && p.piece < p.tiles ? (size_t)M * K * 4 : 0);
    p.bytes = at;
    return p;
}

size_t head_loss_ws_bytes(int64_t M, int64_t K, int64_t V, bool dx, bool dw) { return head_plan(M, K, V, dx, dw).bytes; }

hipError_t launch_head_loss(const uint16_t* X, int64_t M, int64_t K, const uint16_t* W, int64_t V,
                            const int64_t* targets, int64_t ignore, const float* dloss, float* loss, uint16_t* dX,
                            uint16_t* dW, void* ws, hipStream_t s) {
    const HeadPlan p = head_plan(M, K, V, dX != nullptr, dW != nullptr);
    uint8_t* base = (uint8_t*)ws;
    constexpr int lds = 4 * HL_STAGE;
    for (const void* f : {(const void*)k_head_logits<false>, (const void*)k_head_logits<true>, (const void*)k_head_product}) {
        const hipError_t e = hipFuncSetAttribute(f, hipFuncAttributeMaxDynamicSharedMemorySize, lds);
        if (e != hipSuccess) return e;
    }
    HeadArgs a{};
    a.X = X;
    a.W = W;
    a.M = M;
    a.K = K;
    a.V = V;
    a.targets = targets;
    a.ignore = ignore;
    a.dloss = dloss;
    a.part = (float2*)(base + p.part);
    a.zy = (float*)(base + p.zy);
    a.rows = (float2*)(base + p.rows);
    a.top = (uint32_t*)(base + p.top);
    a.Mp = p.Mp;
    a.tiles_m = (int)(p.Mp / HL_T);
    a.tiles_v = (int)p.tiles;
    auto grid = [](int64_t x, int64_t y) { return dim3((uint32_t)((x * y + 7) / 8 * 8)); };
    hipLaunchKernelGGL(k_head_logits<false>, grid(a.tiles_v, a.tiles_m), dim3(512), lds, s, a);
    hipLaunchKernelGGL(k_head_rows, dim3((uint32_t)((M + 255) / 256)), dim3(256), 0, s, a.part, a.zy, targets, M, p.Mp, V,
                       ignore, (int)p.tiles, dX || dW ? dloss : nullptr, a.top, (float2*)(base + p.rows), loss);
    if (!dX && !dW) return hipGetLastError();
    a.G = dX ? (uint16_t*)(base + p.G) : nullptr;
    a.Gt = dW ? (uint16_t*)(base + p.Gt) : nullptr;
    for (int64_t t0 = 0; t0 < p.tiles; t0 += p.piece) {
        const int64_t n = p.tiles - t0 < p.piece ? p.tiles - t0 : p.piece;
        const int64_t rows = V - t0 * HL_T < n * HL_T ? V - t0 * HL_T : n * HL_T;   // vocabulary rows of the piece
        a.v0 = t0 * HL_T;
        a.tiles_v = (int)n;
        a.ldg = n * HL_T;
        hipLaunchKernelGGL(k_head_logits<true>, grid(a.tiles_v, a.tiles_m), dim3(512), lds, s, a);
        const int tiles_n = (int)((K + HL_T - 1) / HL_T);
        if (dX) {
            const bool last = t0 + n >= p.tiles;
            ProductArgs d{a.G, a.ldg, p.Mp, M, W + a.v0 * K, rows, K, (int)((rows + HL_K - 1) / HL_K), a.tiles_m, tiles_n,
                          last ? dX : nullptr, (float*)(base + p.sum), t0 > 0 ? 1 : 0, a.top};
            hipLaunchKernelGGL(k_head_product, grid(d.tiles_r, d.tiles_n), dim3(512), lds, s, d);
        }
        if (dW) {
            ProductArgs d{a.Gt, p.Mp, a.ldg, rows, X, M, K, (int)((M + HL_K - 1) / HL_K), (int)n, tiles_n, dW + a.v0 * K, nullptr, 0, a.top};
            hipLaunchKernelGGL(k_head_product, grid(d.tiles_r, d.tiles_n), dim3(512), lds, s, d);
        }
    }
    return hipGetLastError();
}

// The gradient of a head that no token reached (a kernel, so that a graph may hold it).
__global__ __launch_bounds__(256)
void k_head_zero(uint4* p, int64_t n) {
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (int64_t)gridDim.x * 256) p[i] = make_uint4(0, 0, 0, 0);
}

hipError_t launch_head_zero(uint16_t* p, int64_t n, hipStream_t s) {
    const int64_t pieces = n / 8, blocks = (pieces + 255) / 256;
    hipLaunchKernelGGL(k_head_zero, dim3((uint32_t)(blocks < 4096 ? blocks : 4096)), dim3(256), 0, s, (uint4*)p, pieces);
    return hipGetLastError();
}

}  // namespace nf4
