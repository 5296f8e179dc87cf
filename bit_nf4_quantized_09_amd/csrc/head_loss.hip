// head_loss.hip -- softmax cross entropy of a vocabulary head, its logits never in memory as such (gfx950).
//
//   z = X W^T,  loss = lse(z) - z_y,  G = dloss (softmax(z) - onehot),  dX = G W,  dW = G^T X
//
// Loss alone: one product computes the logits tile by tile and keeps of each tile only the
// maximum and the sum of exponentials of every row, the target apart: with
// S = sum_{v != y} exp(z_v - z_y), loss = log1p(S) and 1 - p_y = S / (1 + S) keep their digits
// where the target has nearly all of the weight (lse - z_y would cancel).
//
// Loss and dX: one pass over the vocabulary in pieces, two products a piece, like the forward
// of an attention whose keys and values are the rows of W.  The first product's epilogue writes
// E[m][v] = 2^(z - R[m]) in bf16, the target's entry zero, with a running integer reference R[m]
// (base 2) that starts at the target's logit; the second adds E W to fp32 sums; at the end
// dX = dloss (sums 2^R / l - (1 - p_y) W_y), the target's row added in fp32.  bf16 has fp32's
// exponents, so R need not be the maximum: a tile takes a reference of its own only where a
// logit passes R by more than 2^40, and the join after each piece (k_head_join) then brings the
// row's other tiles and sums to the new R by exact powers of two.
//
// With dW, the contraction runs over tokens and needs normalised weights.  Every piece's E is kept,
// as bf16 and the eight bits that follow (up to 1 GB of bf16: half as much again as bf16 logits), and once l is known k_head_turn makes
// G = dloss / max|dloss| (p - onehot) of it, in bf16 and transposed, rounded once; the factor
// max|dloss| is applied to the fp32 sums, so that a mean's 1/count does not round the many nearly
// equal target entries alike.  Beyond 1 GB each piece's logits are computed again instead
// (HEAD_GT): a fourth product (4096 tokens x 32000 x 8192: 6.65 ms, 5.2 to 5.4 with E kept; x 131200 x 4096,
// beyond: 14.2 ms).
//
// Rounding: logits, maxima, sums and accumulators are fp32; E and G are bf16, the type of the
// matrix instructions' operands and of the outputs.
//
// Products.  Tiles of 512 or 256 rows x 128 columns, 4 waves, v_mfma_f32_32x32x16_bf16: one wave per
// SIMD with 256 accumulators, or two with 128 that hide each other's ends.  The long operand (X, E, G^T)
// is private to its wave and comes in fragment order (tile_map.h) straight into registers, two steps
// ahead; X is packed once per call, E and G^T are written in that order by the logits' epilogue and
// by k_head_turn.  The 128-column operand (rows of W, or columns of W or X read transposed) goes through
// four LDS stages filled by direct loads, three steps ahead.  Bound by the matrix instructions at the clock
// that the card holds under them: 2048 tokens x 32000 x 4096, logits and dX: 490 + 490 us, 1100 TFLOP/s
// (440 + 415 before the card is warm); 4096 x 32000 x 8192 with dW: 1280, 1250 and 1190 TFLOP/s.
// (256 x 256 tiles with both operands in LDS, 8 waves of 128 x 64: LDS reads and writes take as
// many cycles as the matrix instructions; 940-1000 TFLOP/s.)
// Grids that such tiles leave mostly empty, and up to 64 tokens, whose time is that of reading W, take
// tiles of 64 tokens (k_head_few, k_head_few_product) or a quarter of a tile a wave (k_head_split).
#include "bufio.h"
#include "decoder.h"
#include "lds_dma.h"
#include "tile_map.h"

namespace nf4 {

constexpr int HL_TM = FUSED_TM;           // rows of a block of the packed operand: 512
constexpr int HL_TN = FUSED_TN;           // columns of an output tile: 128
constexpr int HL_K = 64;                  // contraction step
constexpr int HL_STAGE = HL_TN * HL_K * 2;   // an LDS stage: 16 KB
constexpr float LOG2E = 1.4426950408889634f;
constexpr float LN2 = 0.6931471805599453f;

// Stage of a direct operand: 128 rows of 128 bytes (64 values of the contraction), 16-byte chunk c of
// row r at chunk c ^ g(r), so that 16 neighbouring rows reading one chunk meet all 64 banks once.
__device__ __forceinline__ int hl_swizzle(int row) { return (row ^ (row >> 3)) & 7; }

// Stage of a transposed operand: 64 rows of 256 bytes (128 columns of one contraction value), 32-byte
// segment u of row r at u ^ 2 (r & 3), so that the 4 rows x 2 segments of one pass meet all banks.
__device__ __forceinline__ int hl_toff(int row, int col) {
    return row * 256 + (((col >> 4) ^ ((row & 3) << 1)) << 5) + ((col & 15) << 1);
}

typedef short hl_i16x4 __attribute__((ext_vector_type(4)));
__device__ __forceinline__ uint2 hl_read_tr(const uint8_t* p) {
    const hl_i16x4 v = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
        (__attribute__((address_space(3))) hl_i16x4*)(const __attribute__((address_space(3))) uint8_t*)(p));
    return __builtin_bit_cast(uint2, v);
}

// Output tile of a workgroup: neighbours in launch order go to different XCDs, so XCD x gets a
// contiguous run of the tile order (columns of 2 row tiles), whose operands its L2 then shares.
__device__ __forceinline__ bool hl_tile(int wg, int64_t tiles_m, int64_t tiles_n, int64_t& tm, int64_t& tn) {
    const int64_t total = tiles_m * tiles_n, q = total / XCDS, rem = total % XCDS;
    const int64_t x = wg % XCDS, local = wg / XCDS;
    if (local >= q + (x < rem ? 1 : 0)) return false;
    tile_at(x * q + (x < rem ? x : rem) + local, tiles_m, tiles_n, tm, tn);
    return true;
}

// Bytes of a block in use when `rows` rows of the tile are: 4 KB per 32 rows.
template <int I>
__device__ __forceinline__ int hl_block_bytes(int64_t rows) {
    return __builtin_amdgcn_readfirstlane(rows < 128 * I ? (int)((rows + 31) / 32) * 4096 : 16384 * I);
}
// A tile's part of the first block of its row tile of 512, of `steps` blocks.
__device__ __forceinline__ const uint16_t* hl_blocks(const uint16_t* p, int64_t row, int64_t steps) {
    return p + (row / HL_TM) * steps * (int64_t)(A_BLOCK_BYTES / 2) + (row % HL_TM) * 64;
}

template <int I>
struct HlFrags {
    uint4 f[I][4];            // [row tile i][substep s]
};

template <int I>
__device__ __forceinline__ void hl_landed() {
    if constexpr (I == 4) asm volatile("s_waitcnt vmcnt(36) lgkmcnt(0)" ::: "memory");
    else asm volatile("s_waitcnt vmcnt(20) lgkmcnt(0)" ::: "memory");
}

// The main loop of both products: acc[i][j] += (rows 32 i.. of the wave's 32 I) x (columns 32 j..),
// contraction steps first .. last - 1 (at least one).  SWAP: accumulator columns are the long
// operand's rows.  TRANS: the 128-column operand is read transposed.  `blocks`: the long operand's
// 64 KB blocks of this row tile, `block_bytes` of each in use (rows past the last are zero and are
// not fetched); `dma(stage, step, q)`: fills quarter q of a stage with the other operand.
//
// A step is 8 regions of 2 I matrix instructions.  Region 2 s + half uses the rows of one half (I = 4:
// 2 half, 2 half + 1) of substep s, reloads their fragments for two steps ahead, and (half 0) reads the next
// substep's column fragments; regions 0-3 also start a quarter each of the stage three steps ahead.  The
// barrier stands before the last region, whose matrix instructions hide the next step's first LDS reads.  A
// stage is complete at the barrier before its first read: hl_landed lets fewer loads be out than each wave
// has started since it started that stage's (36 of at least 46 for I = 4, 20 of at least 26 for I = 2).
template <int I, bool SWAP, bool TRANS, typename Dma>
__device__ __forceinline__ void hl_loop(f32x16 (&acc)[I][4], const uint8_t* lds, const uint16_t* blocks, int block_bytes, int first, int last,
                                        int wave, int lane, Dma&& dma) {
    const int h = lane >> 5, rl = lane & 31;
    int off[4];               // LDS offset of this lane's column fragments; + 4096 j (direct), + 4096 s (transposed)
    if constexpr (TRANS) {
        const int g = lane >> 4, jl = lane & 15;
        const int row0 = 8 * (g >> 1) + (jl >> 2);
#pragma unroll
        for (int j = 0; j < 4; ++j) off[j] = hl_toff(row0, j * 32 + 16 * (g & 1) + 4 * (jl & 3));
    } else {
        // row 32 j + rl, chunk 2 s + h: swizzled by g(rl) ^ 4 (j & 1), so (s, j) and (s ^ 2 (j & 1), 0) share a base
#pragma unroll
        for (int s = 0; s < 4; ++s) off[s] = rl * 128 + (((2 * s + h) ^ hl_swizzle(rl)) << 4);
    }
    auto read_b = [&](const uint8_t* stage, int j, int s) -> bf16x8 {
        if constexpr (TRANS) {
            const uint8_t* p = stage + off[j] + s * 16 * 256;
            const uint2 lo = hl_read_tr(p), hi = hl_read_tr(p + 4 * 256);
            return __builtin_bit_cast(bf16x8, make_uint4(lo.x, lo.y, hi.x, hi.y));
        } else {
            return *reinterpret_cast<const bf16x8*>(stage + off[s ^ (2 * (j & 1))] + 4096 * j);
        }
    };
    uint32_t a_voff[I];
#pragma unroll
    for (int i = 0; i < I; ++i) a_voff[i] = (uint32_t)((wave * I + i) * 4096 + lane * 16);
    // (past the last step the range is empty and the fragments are zero: an odd number of steps ends with an idle one)
    auto a_rsrc = [&](int step) {
        return make_rsrc(blocks + (int64_t)(step < last ? step : first) * (A_BLOCK_BYTES / 2), step < last ? block_bytes : 0);
    };
    auto clamp = [&](int step) { return step < last ? step : last - 1; };
    auto load_all = [&](HlFrags<I>& F, int step) {
        const __amdgpu_buffer_rsrc_t rs = a_rsrc(step);
#pragma unroll
        for (int s = 0; s < 4; ++s)
#pragma unroll
            for (int i = 0; i < I; ++i) F.f[i][s] = buf_load16(rs, a_voff[i] + 1024 * s, 0);
    };
    auto mfma = [&](int i, int j, uint4 af, bf16x8 bf) {
        const bf16x8 a = __builtin_bit_cast(bf16x8, af);
        acc[i][j] = SWAP ? __builtin_amdgcn_mfma_f32_32x32x16_bf16(bf, a, acc[i][j], 0, 0, 0)
                         : __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, bf, acc[i][j], 0, 0, 0);
    };
    bf16x8 fb[2][4];
    HlFrags<I> fa0, fa1;
    auto step_body = [&](int it, HlFrags<I>& cur) {
        const int st = (it - first) & 3;
        const uint8_t* now = lds + st * HL_STAGE;
        const uint8_t* next = lds + ((st + 1) & 3) * HL_STAGE;
        const __amdgpu_buffer_rsrc_t rs = a_rsrc(it + 2);
        const int ahead = clamp(it + 3);
#pragma unroll
        for (int rg = 0; rg < 8; ++rg) {
            const int s = rg >> 1, half = rg & 1;
            if (rg == 7) {
                hl_landed<I>();
                __builtin_amdgcn_s_barrier();
                asm volatile("" ::: "memory");
#pragma unroll
                for (int j = 0; j < 4; ++j) fb[0][j] = read_b(next, j, 0);
            } else if (half == 0 && s < 3) {
#pragma unroll
                for (int j = 0; j < 4; ++j) fb[(s & 1) ^ 1][j] = read_b(now, j, s + 1);
            }
            if (rg < 4) dma((st + 3) & 3, ahead, rg);
#pragma unroll
            for (int t = 0; t < 2 * I; ++t) mfma(I / 2 * half + (t >> 2), t & 3, cur.f[I / 2 * half + (t >> 2)][s], fb[s & 1][t & 3]);
#pragma unroll
            for (int q = 0; q < I / 2; ++q) cur.f[I / 2 * half + q][s] = buf_load16(rs, a_voff[I / 2 * half + q] + 1024 * s, 0);
#pragma unroll
            for (int t = 0; t < 2 * I; ++t) {
                __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);                       // matrix
                __builtin_amdgcn_sched_group_barrier(0x002, 8 / I, 0);                   // VALU
                if ((rg == 7 || (half == 0 && s < 3)) && t < 4)
                    __builtin_amdgcn_sched_group_barrier(0x100, TRANS ? 2 : 1, 0);      // LDS reads
                if (t == 2 || (I == 4 && t == 5)) __builtin_amdgcn_sched_group_barrier(0x020, 1, 0);   // loads
            }
            __builtin_amdgcn_sched_barrier(0);
        }
    };
#pragma unroll
    for (int st = 0; st < 3; ++st)
#pragma unroll
        for (int q = 0; q < 4; ++q) dma(st, clamp(first + st), q);
    __builtin_amdgcn_sched_barrier(0);
    load_all(fa0, first);
    load_all(fa1, first + 1);
    __builtin_amdgcn_sched_barrier(0);
    hl_landed<I>();
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
#pragma unroll
    for (int j = 0; j < 4; ++j) fb[0][j] = read_b(lds, j, 0);
    for (int it = first; it < last; it += 2) {
        step_body(it, fa0);
        step_body(it + 1, fa1);
    }
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");      // nothing may land in LDS after the workgroup
}

// X in fragment order (64 KB per 512 rows and 64 values, zeros past row M): one wave per 32 rows and step.
__global__ __launch_bounds__(256)
void k_head_pack(const uint16_t* X, int64_t M, int64_t K, uint16_t* out) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int64_t steps = K / HL_K;
    const int64_t step = blockIdx.x, tm = blockIdx.y >> 2;
    const int i = (int)(blockIdx.y & 3);
    const int64_t row0 = tm * HL_TM + 128 * wave + 32 * i, row = row0 + (lane & 31);
    if (row0 >= M) return;                // no row of these 32 is in use, and none is read
    uint4* block = reinterpret_cast<uint4*>(out + (tm * steps + step) * (A_BLOCK_BYTES / 2));
#pragma unroll
    for (int s = 0; s < 4; ++s) {
        uint4 v = make_uint4(0, 0, 0, 0);
        if (row < M) v = *reinterpret_cast<const uint4*>(X + row * K + step * HL_K + (2 * s + (lane >> 5)) * 8);
        block[1024 * wave + 64 * (4 * i + s) + lane] = v;
    }
}

struct HeadArgs {
    const uint16_t* X;        // [M][K], and
    const uint16_t* Xp;       // in fragment order
    const uint16_t* W;        // [V][K]
    int64_t M, K, V;
    const int64_t* targets;
    int64_t ignore;
    int64_t v0;               // first vocabulary row of the launch, and
    int64_t tiles_v, tiles_m; // its tiles (of 128 or 32 vocabulary rows; of 512 or 256 tokens)
    float2* part;             // [Mp][tiles of v of the launch]: reference and sum of a row, base 2
    float* zy;                // [Mp]: target's logit, base 2 (HEAD_STATS: out)
    const float* ref;         // [Mp]: running reference (HEAD_E)
    const float4* rows;       // [Mp]: lse, base 2; 1 - p of the target; dloss; the target (as bits, -1: none) (HEAD_GT)
    const uint32_t* top;      // max|dloss| as bits (HEAD_GT)
    uint16_t* out;            // E or G^T in fragment order
    uint8_t* low;             // the next eight bits of E's values, in the same order, or null (HEAD_E)
    int64_t out_steps;        // blocks of a row tile of `out`
    int64_t Mp;
};

// What the epilogue of the logits' product leaves: row statistics, exponentials against the running
// reference with their sums, or normalised gradients, transposed.
enum HeadMode { HEAD_STATS, HEAD_E, HEAD_GT };

__device__ __forceinline__ bool head_live(int64_t target, int64_t V, int64_t ignore) {
    return target >= 0 && target < V && target != ignore;
}
constexpr float HEAD_ROOM = 40.0f;        // binades a logit may pass the running reference by
// The factor on G, from max|dloss|: at least the smallest normal number, so that its inverse is finite.
__device__ __forceinline__ float head_scale(const uint32_t* top) { return fmaxf(__uint_as_float(*top), 0x1p-126f); }

// E is kept for dW as bf16 and eight bits more, so that G is rounded once, from a value of 16 bits: the two together
// are the fp32 value's bits with the last eight rounded away.
__device__ __forceinline__ uint32_t head_low(float y, uint32_t kept) {
    const int d = (int)(__float_as_uint(y) - kept + 0x80u) >> 8;
    return (uint32_t)(d < -128 ? -128 : d > 127 ? 127 : d) & 0xFFu;
}
__device__ __forceinline__ float head_both(float kept, uint32_t low) {
    return kept == 0.0f ? 0.0f : __uint_as_float(__float_as_uint(kept) + ((uint32_t)(int32_t)(int8_t)low << 8));
}

// The epilogue of HEAD_STATS and HEAD_E for 32 tokens m0 .. (column rl) and the 32 J vocabulary rows v0 .. of tile
// tv: z[j][reg] is row 32 j + 8 (reg / 4) + 4 h + reg % 4.
template <HeadMode MODE, int J>
__device__ __forceinline__ void head_column(const HeadArgs& a, f32x16* acc, int64_t m0, int64_t v0, int64_t tv, int h, int rl) {
    const int left = (int)(a.V - v0 < 32 * J ? a.V - v0 : 32 * J) - 4 * h;      // this lane's valid rows end
    const int64_t m = m0 + rl;
    const int64_t target = m < a.M ? a.targets[m] : -1;
    const bool live = m < a.M && head_live(target, a.V, a.ignore);
    const int64_t tl = target - v0 - 4 * h;
    const int hit = live && tl >= 0 && tl < 32 * J ? (int)tl : -1;             // the target's row, if this lane's
    float top = -INFINITY;
#pragma unroll
    for (int j = 0; j < J; ++j)
#pragma unroll
        for (int r = 0; r < 16; ++r) {
            const int v = j * 32 + 8 * (r >> 2) + (r & 3);
            float z = acc[j][r] * LOG2E;
            if (v == hit) {
                if (MODE == HEAD_STATS) a.zy[m] = z;
                z = -INFINITY;
            }
            z = v < left ? z : -INFINITY;
            acc[j][r] = z;
            top = fmaxf(top, z);
        }
    top = fmaxf(top, __shfl_xor(top, 32));
    float ref = top > -INFINITY ? top : 0.0f;
    if (MODE == HEAD_E) {
        ref = live ? a.ref[m] : 0.0f;
        if (top > ref + HEAD_ROOM) ref = ceilf(top);          // an integer, like the running one
    }
    // E's blocks of 512 tokens and 64 vocabulary rows: row m's 16-byte chunk of rows v .. v + 7
    const int in = (int)(m0 % HL_TM);
    const int64_t place = MODE == HEAD_E ? (m0 / HL_TM) * a.out_steps * A_BLOCK_BYTES + (in >> 5) * 4096 + rl * 16 + 8 * h : 0;
    float sum = 0.0f;
#pragma unroll
    for (int j = 0; j < J; ++j)
#pragma unroll
        for (int r4 = 0; r4 < 4; ++r4) {
            float y[4];
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                y[r] = __builtin_amdgcn_exp2f(acc[j][4 * r4 + r] - ref);
                if (MODE == HEAD_E && !live) y[r] = 0.0f;
                sum += y[r];
            }
            if (MODE == HEAD_E) {
                const int64_t chunk = ((v0 - a.v0) >> 3) + 4 * j + r4;         // of the row's 16-byte chunks
                const int64_t to = place + (chunk >> 3) * A_BLOCK_BYTES + (chunk & 7) * 512;
                const uint2 e = make_uint2(pack_bf16x2(y[0], y[1]), pack_bf16x2(y[2], y[3]));
                *reinterpret_cast<uint2*>(reinterpret_cast<uint8_t*>(a.out) + to) = e;
                if (a.low)
                    *reinterpret_cast<uint32_t*>(a.low + to / 2) = head_low(y[0], e.x << 16) | head_low(y[1], e.x & 0xFFFF0000u) << 8 |
                                                                   head_low(y[2], e.y << 16) << 16 | head_low(y[3], e.y & 0xFFFF0000u) << 24;
            }
        }
    sum += __shfl_xor(sum, 32);
    if (MODE == HEAD_E && !live) ref = 0.0f;
    if (h == 0 && m < a.Mp) a.part[m * a.tiles_v + tv] = make_float2(MODE == HEAD_E ? ref : top, sum);
}

// Logits of a tile of 128 I tokens x 128 vocabulary rows.
template <HeadMode MODE, int I>
__global__ __launch_bounds__(256) __attribute__((amdgpu_waves_per_eu(I == 4 ? 1 : 2, I == 4 ? 1 : 2)))
void k_head_logits(HeadArgs a) {
    __shared__ __attribute__((aligned(16))) uint8_t lds[4 * HL_STAGE];
    constexpr bool SWAP = MODE != HEAD_GT;
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int h = lane >> 5, rl = lane & 31;
    int64_t tv, tm;
    if (!hl_tile(blockIdx.x, a.tiles_m, a.tiles_v, tm, tv)) return;
    const int64_t v0 = a.v0 + tv * HL_TN, m0 = tm * 128 * I;
    const int steps = __builtin_amdgcn_readfirstlane((int)(a.K / HL_K));
    // a wave fills rows 32 wave .. of a stage, 8 rows a load; rows past V repeat the last (dropped later)
    uint32_t wof[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        const int row = wave * 32 + q * 8 + (lane >> 3);
        const int64_t rv = v0 + row < a.V ? row : a.V - 1 - v0;
        wof[q] = (uint32_t)(rv * a.K * 2) + (((lane & 7) ^ hl_swizzle(row)) << 4);
    }
    const dma_rsrc rw = make_dma_rsrc(a.W + v0 * a.K, (a.V - v0) * a.K * 2);
    const uint32_t mine = lds_address(lds) + wave * 4096;
    f32x16 acc[I][4];
#pragma unroll
    for (int i = 0; i < I; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = f32x16{};
    hl_loop<I, SWAP, false>(acc, lds, hl_blocks(a.Xp, m0, steps), hl_block_bytes<I>(a.M - m0), 0, steps, wave, lane,
                         [&](int stage, int step, int q) {
                             load_to_lds(rw, mine + stage * HL_STAGE + q * 1024, wof[q], (uint32_t)step * 128);
                         });
    if constexpr (MODE == HEAD_GT) {
        // accumulator (i, j, reg): token 32 i + 8 (reg / 4) + 4 h + reg % 4 of the wave's 32 I, vocabulary row 32 j + rl.
        // G^T's block of 512 vocabulary rows and 64 tokens: this tile is wave slice tv % 4 of it.
        const float inv = 1.0f / head_scale(a.top);
#pragma unroll
        for (int i = 0; i < I; ++i) {
            const int64_t mi = m0 + (wave * I + i) * 32;
            uint8_t* block = reinterpret_cast<uint8_t*>(a.out) + ((tv >> 2) * a.out_steps + (mi >> 6)) * A_BLOCK_BYTES +
                             (tv & 3) * 16384 + rl * 16 + 8 * h;
#pragma unroll
            for (int r4 = 0; r4 < 4; ++r4) {
                float4 row[4];
#pragma unroll
                for (int r = 0; r < 4; ++r) row[r] = a.rows[mi + 8 * r4 + 4 * h + r];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int v = (int)v0 + j * 32 + rl;
                    float y[4];
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        const int target = __float_as_int(row[r].w);
                        const float p = __builtin_amdgcn_exp2f(acc[i][j][4 * r4 + r] * LOG2E - row[r].x);
                        y[r] = target >= 0 && v < a.V ? row[r].z * inv * (v == target ? -row[r].y : p) : 0.0f;
                    }
                    *reinterpret_cast<uint2*>(block + 1024 * (4 * j + (i & 1) * 2 + (r4 >> 1)) + 512 * (r4 & 1)) =
                        make_uint2(pack_bf16x2(y[0], y[1]), pack_bf16x2(y[2], y[3]));
                }
            }
        }
        return;
    }
    // accumulator (i, j, reg): token 32 i + rl of the wave's 32 I, vocabulary row 32 j + 8 (reg / 4) + 4 h + reg % 4
#pragma unroll
    for (int i = 0; i < I; ++i) head_column<MODE, 4>(a, acc[i], m0 + (wave * I + i) * 32, v0, tv, h, rl);
}

// Tiles of 64 tokens, for few tokens and for grids that 512-token tiles leave mostly empty.
//
// Logits: a workgroup takes 128 vocabulary rows and 32 NT tokens, each of its four waves 32 of the rows, and streams
// W (whole 128-byte lines of 8 rows a load) and X through three LDS stages, two steps ahead, two workgroups on a
// compute unit.  (One with six stages: as fast up to 64 tokens, 223 us for 179 on 512 x 32000 x 4096.)  Up to 64
// tokens its time is that of reading W, past the caches where nothing reads it again (ONCE): 33 tokens x 32000 x
// 4096: 55 us, 4.8 TB/s.  (W straight into registers, 32 rows a load, meets every line four times: 75 us.)
constexpr int FEW_TOKENS = 64, FEW_TN = 32, FEW_STAGES = 3;
constexpr int few_stage(int nt) { return 16384 + 4096 * nt; }            // bytes: 128 x 64 or 64 x 128 of W, then X or E
constexpr int FEW_JOIN = 65536;           // the product's sums of 32 rows, of each wave
constexpr int few_lds(int nt) { return FEW_STAGES * few_stage(nt) > FEW_JOIN ? FEW_STAGES * few_stage(nt) : FEW_JOIN; }

// Tile of a workgroup, the token blocks of one slice of W on one XCD.
__device__ __forceinline__ bool few_tile(int wg, int64_t blocks, int64_t slices, int64_t& block, int64_t& slice) {
    const int64_t total = blocks * slices, q = total / XCDS, rem = total % XCDS;
    const int64_t x = wg % XCDS, local = wg / XCDS;
    if (local >= q + (x < rem ? 1 : 0)) return false;
    const int64_t at = x * q + (x < rem ? x : rem) + local;
    block = at % blocks;
    slice = at / blocks;
    return true;
}

// Waits until only the 4 + NT loads of the youngest stage are out, and meets the other waves.
template <int NT>
__device__ __forceinline__ void few_landed() {
    if constexpr (NT == 2) asm volatile("s_waitcnt vmcnt(6) lgkmcnt(0)" ::: "memory");
    else asm volatile("s_waitcnt vmcnt(5) lgkmcnt(0)" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
}

template <HeadMode MODE, int NT, bool ONCE>
__global__ __launch_bounds__(256, 2)
void k_head_few(HeadArgs a) {
    extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int h = lane >> 5, rl = lane & 31;
    int64_t block, slice;
    if (!few_tile(blockIdx.x, (a.M + 32 * NT - 1) / (32 * NT), a.tiles_v / 4, block, slice)) return;
    const int64_t b0 = a.v0 + slice * 128, m0 = block * 32 * NT;
    const int steps = __builtin_amdgcn_readfirstlane((int)(a.K / HL_K));
    // a wave fills its own 32 rows of W and 8 NT of X, 8 a load (rows past the end repeat the last: dropped later)
    uint32_t wof[4], xof[NT];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        const int row = wave * 32 + q * 8 + (lane >> 3);
        const int64_t rv = b0 + row < a.V ? row : a.V - 1 - b0;
        wof[q] = (uint32_t)(rv * a.K * 2) + (((lane & 7) ^ hl_swizzle(row)) << 4);
    }
#pragma unroll
    for (int q = 0; q < NT; ++q) {
        const int row = (wave * NT + q) * 8 + (lane >> 3);
        xof[q] = (uint32_t)((m0 + row < a.M ? row : a.M - 1 - m0) * a.K * 2) + (((lane & 7) ^ hl_swizzle(row)) << 4);
    }
    const dma_rsrc rw = make_dma_rsrc(a.W + b0 * a.K, (a.V - b0) * a.K * 2), rx = make_dma_rsrc(a.X + m0 * a.K, (a.M - m0) * a.K * 2);
    const uint32_t base = lds_address(lds);
    auto fill = [&](int stage, int step) {
        const int at = step < steps ? step : steps - 1;
        const uint32_t to = base + stage * few_stage(NT);
#pragma unroll
        for (int q = 0; q < 4; ++q) load_to_lds<ONCE>(rw, to + wave * 4096 + q * 1024, wof[q], (uint32_t)at * 128);
#pragma unroll
        for (int q = 0; q < NT; ++q) load_to_lds(rx, to + 16384 + (wave * NT + q) * 1024, xof[q], (uint32_t)at * 128);
    };
    f32x16 acc[NT];
#pragma unroll
    for (int i = 0; i < NT; ++i) acc[i] = f32x16{};
    int off[4];
#pragma unroll
    for (int s = 0; s < 4; ++s) off[s] = rl * 128 + (((2 * s + h) ^ hl_swizzle(rl)) << 4);      // (row 32 i + rl: swizzled by 4 (i & 1) more)
#pragma unroll
    for (int i = 0; i < FEW_STAGES - 1; ++i) fill(i, i);
    int stage = 0, free = FEW_STAGES - 1;
    for (int it = 0; it < steps; ++it) {
        few_landed<NT>();
        fill(free, it + FEW_STAGES - 1);                                  // the stage that every wave left before the barrier
        const uint8_t* sw = lds + stage * few_stage(NT);
#pragma unroll
        for (int s = 0; s < 4; ++s) {
            const bf16x8 w = *reinterpret_cast<const bf16x8*>(sw + wave * 4096 + off[s ^ (2 * (wave & 1))]);
#pragma unroll
            for (int i = 0; i < NT; ++i) {
                const bf16x8 x = *reinterpret_cast<const bf16x8*>(sw + 16384 + 4096 * i + off[s ^ (2 * (i & 1))]);
                acc[i] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(w, x, acc[i], 0, 0, 0);
            }
        }
        free = stage;
        stage = stage + 1 < FEW_STAGES ? stage + 1 : 0;
    }
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
#pragma unroll
    for (int i = 0; i < NT; ++i) head_column<MODE, 1>(a, &acc[i], m0 + 32 * i, b0 + 32 * wave, slice * 4 + wave, h, rl);
}

// The same for grids that leave most compute units empty: a workgroup takes 32 vocabulary rows and its waves a quarter
// of the contraction each (steps wave, wave + 4, ..), every wave with stages of its own, joined at the end.
constexpr int SPLIT_STAGES = 3;
constexpr int split_stage(int nt) { return 4096 + 4096 * nt; }           // bytes of a wave's: 32 rows of W, then X
constexpr int split_lds(int nt) { return SPLIT_STAGES * 4 * split_stage(nt); }
template <HeadMode MODE, int NT>
__global__ __launch_bounds__(256)
void k_head_split(HeadArgs a) {
    extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int h = lane >> 5, rl = lane & 31;
    int64_t block, tile;
    if (!few_tile(blockIdx.x, (a.M + 32 * NT - 1) / (32 * NT), a.tiles_v, block, tile)) return;
    const int64_t b0 = a.v0 + tile / 4 * 128, m0 = block * 32 * NT;      // (the last slice of 128 has rows, its last tiles may have none)
    const int steps = __builtin_amdgcn_readfirstlane((int)(a.K / HL_K));
    uint32_t wof[4], xof[4 * NT];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        const int row = (int)(tile & 3) * 32 + q * 8 + (lane >> 3);
        const int64_t rv = b0 + row < a.V ? row : a.V - 1 - b0;
        wof[q] = (uint32_t)(rv * a.K * 2) + (((lane & 7) ^ hl_swizzle(row & 31)) << 4);
    }
#pragma unroll
    for (int q = 0; q < 4 * NT; ++q) {
        const int row = q * 8 + (lane >> 3);
        xof[q] = (uint32_t)((m0 + row < a.M ? row : a.M - 1 - m0) * a.K * 2) + (((lane & 7) ^ hl_swizzle(row)) << 4);
    }
    const dma_rsrc rw = make_dma_rsrc(a.W + b0 * a.K, (a.V - b0) * a.K * 2), rx = make_dma_rsrc(a.X + m0 * a.K, (a.M - m0) * a.K * 2);
    const uint8_t* mine = lds + wave * SPLIT_STAGES * split_stage(NT);
    const uint32_t base = lds_address(mine);
    auto fill = [&](int stage, int step) {
        const int at = step < steps ? step : steps - 1;
        const uint32_t to = base + stage * split_stage(NT);
#pragma unroll
        for (int q = 0; q < 4; ++q) load_to_lds(rw, to + q * 1024, wof[q], (uint32_t)at * 128);
#pragma unroll
        for (int q = 0; q < 4 * NT; ++q) load_to_lds(rx, to + 4096 + q * 1024, xof[q], (uint32_t)at * 128);
    };
    f32x16 acc[NT];
#pragma unroll
    for (int i = 0; i < NT; ++i) acc[i] = f32x16{};
    int off[4];
#pragma unroll
    for (int s = 0; s < 4; ++s) off[s] = rl * 128 + (((2 * s + h) ^ hl_swizzle(rl)) << 4);
    fill(0, wave);
    fill(1, wave + 4);
    int stage = 0, free = 2;
    for (int it = wave; it < steps; it += 4) {
        // this stage has landed once only the next one's loads are out
        if constexpr (NT == 2) asm volatile("s_waitcnt vmcnt(12) lgkmcnt(0)" ::: "memory");
        else asm volatile("s_waitcnt vmcnt(8) lgkmcnt(0)" ::: "memory");
        fill(free, it + 8);
        const uint8_t* sw = mine + stage * split_stage(NT);
#pragma unroll
        for (int s = 0; s < 4; ++s) {
            const bf16x8 w = *reinterpret_cast<const bf16x8*>(sw + off[s]);
#pragma unroll
            for (int i = 0; i < NT; ++i) {
                const bf16x8 x = *reinterpret_cast<const bf16x8*>(sw + 4096 + 4096 * i + off[s ^ (2 * (i & 1))]);
                acc[i] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(w, x, acc[i], 0, 0, 0);
            }
        }
        free = stage;
        stage = stage + 1 < SPLIT_STAGES ? stage + 1 : 0;
    }
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    __syncthreads();
    auto cell = [&](int from, int i, int r4) { return reinterpret_cast<f32x4*>(lds + (((from * NT + i) * 4 + r4) << 10) + lane * 16); };
#pragma unroll
    for (int i = 0; i < NT; ++i)
#pragma unroll
        for (int r4 = 0; r4 < 4; ++r4) *cell(wave, i, r4) = f32x4{acc[i][4 * r4], acc[i][4 * r4 + 1], acc[i][4 * r4 + 2], acc[i][4 * r4 + 3]};
    __syncthreads();
    if (wave >= NT) return;
    f32x16 sum;
#pragma unroll
    for (int r4 = 0; r4 < 4; ++r4) {
        f32x4 y = *cell(0, wave, r4);
#pragma unroll
        for (int from = 1; from < 4; ++from) y += *cell(from, wave, r4);
#pragma unroll
        for (int r = 0; r < 4; ++r) sum[4 * r4 + r] = y[r];
    }
    head_column<MODE, 1>(a, &sum, m0 + 32 * wave, a.v0 + tile * 32, tile, h, rl);
}

// A row's loss from its target's logit and the others' log-sum (both base 2): the loss, lse
// (base 2) and 1 - p of the target.  A target's logit of -inf has an infinite loss and p = 0; +inf (an overflow) and NaN
// leave nothing that is known.
struct RowLoss {
    float loss, lse, rest;
};
__device__ __forceinline__ RowLoss row_loss(float z, float others) {
    if (!(z < INFINITY)) return RowLoss{NAN, NAN, NAN};
    const float d = z - others;
    const float tail = log1pf(exp2f(-fabsf(d)));
    return RowLoss{d >= 0.0f ? tail : tail - d * LN2, fmaxf(z, others) + tail * LOG2E, 1.0f / (1.0f + exp2f(d))};
}

// The loss from a row's statistics: a workgroup per row.
__global__ __launch_bounds__(256)
void k_head_rows(const float2* part, const float* zy, const int64_t* targets, int64_t V, int64_t ignore, int tiles, float* loss) {
    __shared__ float2 join[4];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int64_t m = blockIdx.x;
    const float2* p = part + m * tiles;
    // each wave's own reference first
    float top = -INFINITY, sum = 0.0f;
#pragma unroll 4
    for (int t = threadIdx.x; t < tiles; t += 256) top = fmaxf(top, p[t].x);
#pragma unroll
    for (int x = 1; x < 64; x <<= 1) top = fmaxf(top, __shfl_xor(top, x));
    const float ref = top > -INFINITY ? top : 0.0f;
#pragma unroll 4
    for (int t = threadIdx.x; t < tiles; t += 256) sum += p[t].y * __builtin_amdgcn_exp2f(p[t].x - ref);
#pragma unroll
    for (int x = 1; x < 64; x <<= 1) sum += __shfl_xor(sum, x);
    if (lane == 0) join[wave] = make_float2(top, sum);
    __syncthreads();
    if (threadIdx.x != 0) return;
#pragma unroll
    for (int w = 0; w < 4; ++w) top = fmaxf(top, join[w].x);
    const float all = top > -INFINITY ? top : 0.0f;
    sum = 0.0f;
#pragma unroll
    for (int w = 0; w < 4; ++w) sum += join[w].y * __builtin_amdgcn_exp2f(join[w].x - all);
    loss[m] = head_live(targets[m], V, ignore) ? row_loss(zy[m], top + log2f(sum)).loss : 0.0f;
}

// Target logits (base 2) and the first references, one wave per row; the last workgroup: the largest
// finite |dloss| of the rows that count.  With `counted`: X with zeros for the rows that do not count, for dW, whose sums over
// tokens would take a NaN from a row of no weight (0 NaN = NaN).
__global__ __launch_bounds__(256)
void k_head_target(const uint16_t* __restrict__ X, const uint16_t* __restrict__ W, int64_t M, int64_t K, int64_t V, const int64_t* targets,
                   int64_t ignore, float* zy, float* ref, float* total, const float* dloss, uint32_t* top, uint16_t* __restrict__ counted) {
    const int lane = threadIdx.x & 63;
    if (blockIdx.x == gridDim.x - 1) {
        __shared__ float join[4];
        float most = 0.0f;
#pragma unroll 4
        for (int64_t i = threadIdx.x; i < M; i += 256) {
            const float g = fabsf(dloss[i]);
            if (g < INFINITY && head_live(targets[i], V, ignore)) most = fmaxf(most, g);
        }
#pragma unroll
        for (int x = 1; x < 64; x <<= 1) most = fmaxf(most, __shfl_xor(most, x));
        if (lane == 0) join[threadIdx.x >> 6] = most;
        __syncthreads();
        if (threadIdx.x == 0) *top = __float_as_uint(fmaxf(fmaxf(join[0], join[1]), fmaxf(join[2], join[3])));
        return;
    }
    const int64_t m = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
    if (m >= M) return;
    const int64_t target = targets[m];
    float sum = 0.0f;
    uint4* copy = reinterpret_cast<uint4*>(counted + m * K);
    if (head_live(target, V, ignore)) {
        const uint4* x = reinterpret_cast<const uint4*>(X + m * K);
        const uint4* w = reinterpret_cast<const uint4*>(W + target * K);
        // (four vectors at a time: one by one their loads wait for each other)
        for (int64_t i0 = lane; i0 < K / 8; i0 += 256) {
            uint4 xv[4], wv[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int64_t i = i0 + 64 * j;
                xv[j] = wv[j] = make_uint4(0, 0, 0, 0);
                if (i < K / 8) {
                    xv[j] = x[i];
                    wv[j] = w[i];
                }
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                float a[8], b[8];
                if (counted && i0 + 64 * j < K / 8) copy[i0 + 64 * j] = xv[j];
                Vec16<uint16_t>::unpack(xv[j], a);
                Vec16<uint16_t>::unpack(wv[j], b);
#pragma unroll
                for (int u = 0; u < 8; ++u) sum = __fmaf_rn(a[u], b[u], sum);
            }
        }
#pragma unroll
        for (int x = 1; x < 64; x <<= 1) sum += __shfl_xor(sum, x);
    } else if (counted) {
        for (int64_t i = lane; i < K / 8; i += 64) copy[i] = make_uint4(0, 0, 0, 0);
    }
    if (lane == 0) {
        zy[m] = sum * LOG2E;
        ref[m] = fmaxf(rintf(sum * LOG2E), -0x1.fffffep127f);       // (finite for a logit of -inf: any other raises it)
        total[m] = 0.0f;
    }
}

struct JoinArgs {
    const float2* part;       // [Mp][tiles] of the piece: reference and sum
    int tiles, width;         // tiles of the piece, their vocabulary rows
    int64_t M, Mp;
    const int64_t* targets;
    int64_t ignore, V;
    uint16_t* E;              // in fragment order,
    int64_t steps;            // blocks of a row tile
    const float* ref;         // running reference of each row before the piece, and
    float* next;              // after it (the next piece's, where each keeps its own),
    float* total;             // running sum
    float* factor;            // out: factor on the row's sums so far
    const float* zy;
    int last;                 // 1: also the loss and what the gradients need of a row
    const float* dloss;
    float* loss;
    float2* ends;             // out (last): factor on the sums, and on the target's row of W
    float4* rows;             // out (last): see HeadArgs
};

// After a piece: each row's new reference and sum, its tiles brought to that reference.  One
// wave per row (rows that only fill the last tile included).
__global__ __launch_bounds__(256)
void k_head_join(JoinArgs a) {
    const int lane = threadIdx.x & 63;
    const int64_t m = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
    if (m >= a.Mp) return;
    const int64_t target = m < a.M ? a.targets[m] : -1;
    if (m >= a.M || !head_live(target, a.V, a.ignore)) {
        if (lane == 0 && a.last) a.rows[m] = make_float4(0.0f, 0.0f, 0.0f, __int_as_float(-1));
        if (lane == 0 && m < a.M) {
            a.factor[m] = 1.0f;
            if (a.last) {
                if (a.loss) a.loss[m] = 0.0f;
                a.ends[m] = make_float2(0.0f, 0.0f);
            }
        }
        return;
    }
    const float2* part = a.part + m * a.tiles;
    const float old = a.ref[m];
    float now = old;
    for (int t = lane; t < a.tiles; t += 64) now = fmaxf(now, part[t].x);
#pragma unroll
    for (int x = 1; x < 64; x <<= 1) now = fmaxf(now, __shfl_xor(now, x));
    float sum = 0.0f;
    for (int t0 = 0; t0 < a.tiles; t0 += 64) {
        const int t = t0 + lane;
        const float2 p = t < a.tiles ? part[t] : make_float2(now, 0.0f);
        sum += p.y * (p.x == now ? 1.0f : __builtin_amdgcn_exp2f(p.x - now));
        // tiles left below the row's new reference are scaled
        uint64_t todo = __ballot(p.x < now);
        const int in = (int)(m % HL_TM);
        uint8_t* blocks = reinterpret_cast<uint8_t*>(a.E) + (m / HL_TM) * a.steps * A_BLOCK_BYTES + (in >> 5) * 4096 + (in & 31) * 16;
        while (todo) {
            const int b = __ffsll((unsigned long long)todo) - 1;
            todo &= todo - 1;
            const float f = __builtin_amdgcn_exp2f(__shfl(p.x, b) - now);
            // the row's values of the tile, a 16-byte chunk per lane
            if (lane < a.width / 8) {
                const int64_t chunk = (int64_t)(t0 + b) * (a.width / 8) + lane;
                uint4* e = reinterpret_cast<uint4*>(blocks + (chunk >> 3) * A_BLOCK_BYTES + (chunk & 7) * 512);
                float x[8];
                Vec16<uint16_t>::unpack(*e, x);
#pragma unroll
                for (int u = 0; u < 8; ++u) x[u] *= f;
                *e = Vec16<uint16_t>::pack(x);
            }
        }
    }
#pragma unroll
    for (int x = 1; x < 64; x <<= 1) sum += __shfl_xor(sum, x);
    if (lane != 0) return;
    const float f = old == now ? 1.0f : __builtin_amdgcn_exp2f(old - now);
    const float total = a.total[m] * f + sum;
    a.next[m] = now;
    a.total[m] = total;
    a.factor[m] = f;
    if (!a.last) return;
    const float z = a.zy[m], g = a.dloss[m];
    const RowLoss r = row_loss(z, now + log2f(total));
    if (a.loss) a.loss[m] = r.loss;
    a.ends[m] = make_float2(g * __builtin_amdgcn_exp2f(now - r.lse), g * r.rest);
    a.rows[m] = make_float4(r.lse, r.rest, g, __int_as_float((int)target));
}

struct ProductArgs {
    const uint16_t* A;        // in fragment order, `a_steps` blocks of each row tile
    int64_t a_steps, out_rows;
    const uint16_t* B;        // [P][N]: contraction down the rows (A has zeros past P)
    int64_t P, N;
    int steps;                // contraction steps of 64: each starts below P
    int splits;               // parts of the contraction, each with sums of its own
    int64_t tiles_r, tiles_n;
    float* sum;               // fp32 [splits][out_rows][N]
    const float* factor;      // ADD: factor of each row on what `sum` holds
    bool add;                 // ADD, of the tiles of 64 rows
    uint16_t* out;            // OUT_DX, OUT_DW: bf16 [out_rows][N] (splits == 1)
    const uint32_t* top;      // OUT_DW: times head_scale(top)
    const float2* ends;       // OUT_DX: out[r] = ends[r].x * sums - ends[r].y * W[targets[r]]
    const uint16_t* W;
    const int64_t* targets;
    int64_t V, ignore;
};

// Four values of a finished row of dX; u: the target's row of W there.  A row that does not count (live: 0) is zero
// whatever its sums hold.
__device__ __forceinline__ uint2 head_dx4(f32x4 y, float2 row, uint2 u, bool live) {
    if (!live) return make_uint2(0, 0);
    return make_uint2(pack_bf16x2(row.x * y[0] - row.y * bf16_lo(u.x), row.x * y[1] - row.y * bf16_hi(u.x)),
                      pack_bf16x2(row.x * y[2] - row.y * bf16_lo(u.y), row.x * y[3] - row.y * bf16_hi(u.y)));
}

// C[r][n] = sum_p A[r][p] B[p][n], tiles of 128 I rows x 128 columns; ADD: on top of what `sum` holds.
enum ProductOut { OUT_SUM, OUT_DX, OUT_DW };
template <ProductOut OUT, bool ADD, int I>
__global__ __launch_bounds__(256) __attribute__((amdgpu_waves_per_eu(I == 4 ? 1 : 2, I == 4 ? 1 : 2)))
void k_head_product(ProductArgs a) {
    __shared__ __attribute__((aligned(16))) uint8_t lds[4 * HL_STAGE];
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int h = lane >> 5, rl = lane & 31;
    const int split = blockIdx.y;
    int64_t tr, tn;
    if (!hl_tile(blockIdx.x, a.tiles_r, a.tiles_n, tr, tn)) return;
    const int per = (a.steps + a.splits - 1) / a.splits;
    const int first = __builtin_amdgcn_readfirstlane(split * per);
    const int last = __builtin_amdgcn_readfirstlane(first + per < a.steps ? first + per : a.steps);
    const int64_t r0 = tr * 128 * I, n0 = tn * HL_TN;
    const uint32_t mine = lds_address(lds) + wave * 4096;
    // a wave fills rows 16 wave .. of a stage, 4 rows a load; columns past N: any, dropped later
    uint32_t bcol = 0;
    {
        const int q = lane & 15, row = lane >> 4;
        const int chunk = (((q >> 1) ^ (row << 1)) << 1) | (q & 1);
        bcol = (uint32_t)(n0 + chunk * 8 < a.N ? chunk * 16 : 0);
    }
    f32x16 acc[I][4];
#pragma unroll
    for (int i = 0; i < I; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = f32x16{};
    if (first < last)
        hl_loop<I, true, true>(acc, lds, hl_blocks(a.A, r0, a.a_steps), hl_block_bytes<I>(a.out_rows - r0), first, last,
                            wave, lane,
                            [&](int stage, int step, int q) {
                                const int64_t p0 = (int64_t)step * HL_K;
                                const dma_rsrc rb = make_dma_rsrc(a.B + p0 * a.N + n0, (a.P - p0) * a.N * 2);
                                // contraction rows past the last repeat it: A is zero there
                                const int row = wave * 16 + q * 4 + (lane >> 4), most = (int)(a.P - p0 < HL_K ? a.P - p0 : HL_K) - 1;
                                load_to_lds(rb, mine + stage * HL_STAGE + q * 1024,
                                            (uint32_t)((row < most ? row : most) * (int)a.N * 2) + bcol, 0);
                            });
    // accumulator (i, j, reg): row 32 i + rl of the wave's 32 I, column 32 j + 8 (reg / 4) + 4 h + reg % 4.  Each 32
    // rows go through the wave's own quarter of LDS (row r's 16-byte chunk c at c ^ r), so that memory is met in
    // whole rows of 128 columns.
    __syncthreads();
    uint8_t* turn = lds + wave * HL_STAGE;
    float* sums = a.sum + split * a.out_rows * a.N;
    const int chunk = lane & 31;
    const int64_t n = n0 + 4 * chunk;
#pragma unroll
    for (int i = 0; i < I; ++i) {
        const int64_t ri = r0 + (wave * I + i) * 32;
        if (ri >= a.out_rows) break;
        // what the rows are joined with is requested before the turn through LDS
        f32x4 old[16];
        uint2 wy[16];
        float2 end[16];
        uint32_t live = 0;
#pragma unroll
        for (int q = 0; q < 16; ++q) {
            const int64_t r = ri + 2 * q + h;
            const bool in = r < a.out_rows && n < a.N;
            old[q] = f32x4{};
            wy[q] = make_uint2(0, 0);
            end[q] = make_float2(0.0f, 0.0f);
            if (ADD && in) old[q] = *reinterpret_cast<const f32x4*>(sums + r * a.N + n) * a.factor[r];
            if (OUT == OUT_DX && in) {
                const int64_t target = a.targets[r];
                const bool on = head_live(target, a.V, a.ignore);
                live |= (on ? 1u : 0u) << q;
                wy[q] = *reinterpret_cast<const uint2*>(a.W + (on ? target * a.N : 0) + n);
                end[q] = a.ends[r];
            }
        }
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int r4 = 0; r4 < 4; ++r4)
                *reinterpret_cast<f32x4*>(turn + rl * 512 + (((8 * j + 2 * r4 + h) ^ rl) << 4)) =
                    f32x4{acc[i][j][4 * r4], acc[i][j][4 * r4 + 1], acc[i][j][4 * r4 + 2], acc[i][j][4 * r4 + 3]};
#pragma unroll
        for (int q = 0; q < 16; ++q) {
            const int in = 2 * q + h;
            const int64_t r = ri + in;
            f32x4 y = *reinterpret_cast<const f32x4*>(turn + in * 512 + ((chunk ^ in) << 4)) + old[q];
            if (r >= a.out_rows || n >= a.N) continue;
            if constexpr (OUT == OUT_SUM) {
                *reinterpret_cast<f32x4*>(sums + r * a.N + n) = y;
            } else if constexpr (OUT == OUT_DW) {
                y *= head_scale(a.top);
                *reinterpret_cast<uint2*>(a.out + r * a.N + n) = make_uint2(pack_bf16x2(y[0], y[1]), pack_bf16x2(y[2], y[3]));
            } else {
                *reinterpret_cast<uint2*>(a.out + r * a.N + n) = head_dx4(y, end[q], wy[q], live >> q & 1);
            }
        }
    }
}

// The same sums in tiles of 32 NT rows x 128 columns: a step's 64 rows of B go through LDS once, each wave takes 16
// of them for the whole tile, and the four waves' accumulators are added at the end.
template <int NT, ProductOut OUT>
__global__ __launch_bounds__(256, 2)
void k_head_few_product(ProductArgs a) {
    extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int h = lane >> 5, rl = lane & 31;
    const int split = blockIdx.y;
    int64_t block, tn;
    if (!few_tile(blockIdx.x, a.tiles_r, a.tiles_n, block, tn)) return;
    const int per = (a.steps + a.splits - 1) / a.splits;
    const int first = __builtin_amdgcn_readfirstlane(split * per);
    const int last = __builtin_amdgcn_readfirstlane(first + per < a.steps ? first + per : a.steps);
    const int64_t r0 = block * 32 * NT, n0 = tn * HL_TN;
    const uint32_t base = lds_address(lds);
    uint32_t bcol;
    int off[4];
    {
        const int q = lane & 15, row = lane >> 4;
        const int chunk = (((q >> 1) ^ (row << 1)) << 1) | (q & 1);
        bcol = (uint32_t)(n0 + chunk * 8 < a.N ? chunk * 16 : 0);
        const int g = lane >> 4, jl = lane & 15;
        const int row0 = 8 * (g >> 1) + (jl >> 2);
#pragma unroll
        for (int j = 0; j < 4; ++j) off[j] = hl_toff(row0, j * 32 + 16 * (g & 1) + 4 * (jl & 3)) + wave * 16 * 256;
    }
    // the rows' fragments of a block: 4 KB per 32 rows, 1 KB of them a wave's
    const uint8_t* A = reinterpret_cast<const uint8_t*>(a.A) + (r0 / HL_TM) * a.a_steps * A_BLOCK_BYTES + (r0 % HL_TM) * 128;
    auto fill = [&](int stage, int step) {
        const int at = step < last ? step : last - 1;
        const uint32_t to = base + stage * few_stage(NT);
        const int64_t p0 = (int64_t)at * HL_K;
        const dma_rsrc rb = make_dma_rsrc(a.B + p0 * a.N + n0, (a.P - p0) * a.N * 2);
        const dma_rsrc ra = make_dma_rsrc(A + at * (int64_t)A_BLOCK_BYTES, 4096 * NT);
        const int most = (int)(a.P - p0 < HL_K ? a.P - p0 : HL_K) - 1;    // rows past the last repeat it: A is zero there
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const int row = wave * 16 + q * 4 + (lane >> 4);
            load_to_lds(rb, to + wave * 4096 + q * 1024, (uint32_t)((row < most ? row : most) * (int)a.N * 2) + bcol, 0);
        }
#pragma unroll
        for (int i = 0; i < NT; ++i) load_to_lds(ra, to + 16384 + i * 4096 + wave * 1024, (uint32_t)(i * 4096 + wave * 1024 + lane * 16), 0);
    };
    f32x16 acc[NT][4];
#pragma unroll
    for (int i = 0; i < NT; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = f32x16{};
    if (first < last) {
#pragma unroll
        for (int i = 0; i < FEW_STAGES - 1; ++i) fill(i, first + i);
        int stage = 0, free = FEW_STAGES - 1;
        for (int it = first; it < last; ++it) {
            few_landed<NT>();
            fill(free, it + FEW_STAGES - 1);
            const uint8_t* sb = lds + stage * few_stage(NT);
            bf16x8 x[NT];
#pragma unroll
            for (int i = 0; i < NT; ++i) x[i] = *reinterpret_cast<const bf16x8*>(sb + 16384 + i * 4096 + wave * 1024 + lane * 16);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const uint2 lo = hl_read_tr(sb + off[j]), hi = hl_read_tr(sb + off[j] + 4 * 256);
                const bf16x8 w = __builtin_bit_cast(bf16x8, make_uint4(lo.x, lo.y, hi.x, hi.y));
#pragma unroll
                for (int i = 0; i < NT; ++i) acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(w, x[i], acc[i][j], 0, 0, 0);
            }
            free = stage;
            stage = stage + 1 < FEW_STAGES ? stage + 1 : 0;
        }
    }
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    // accumulator (i, j, reg): row 32 i + rl, column 32 j + 8 (reg / 4) + 4 h + reg % 4; wave w finishes columns
    // 32 w .., 32 rows at a time
    auto cell = [&](int from, int j, int r4) { return reinterpret_cast<f32x4*>(lds + (((from * 4 + j) * 4 + r4) << 10) + lane * 16); };
    float* sums = a.sum + split * a.out_rows * a.N;
#pragma unroll
    for (int i = 0; i < NT; ++i) {
        __syncthreads();
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int r4 = 0; r4 < 4; ++r4)
                *cell(wave, j, r4) = f32x4{acc[i][j][4 * r4], acc[i][j][4 * r4 + 1], acc[i][j][4 * r4 + 2], acc[i][j][4 * r4 + 3]};
        __syncthreads();
        const int64_t r = r0 + 32 * i + rl;
#pragma unroll
        for (int r4 = 0; r4 < 4; ++r4) {
            const int64_t n = n0 + 32 * wave + 8 * r4 + 4 * h;
            if (r >= a.out_rows || n >= a.N) continue;
            f32x4 y = *cell(0, wave, r4);
#pragma unroll
            for (int from = 1; from < 4; ++from) y += *cell(from, wave, r4);
            if constexpr (OUT == OUT_DW) {
                y *= head_scale(a.top);
                *reinterpret_cast<uint2*>(a.out + r * a.N + n) = make_uint2(pack_bf16x2(y[0], y[1]), pack_bf16x2(y[2], y[3]));
            } else {
                f32x4* to = reinterpret_cast<f32x4*>(sums + r * a.N + n);
                if (a.add) y += *to * a.factor[r];
                *to = y;
            }
        }
    }
}

// dX from the sums of several parts of the contraction: a thread per four columns.
__global__ __launch_bounds__(256)
void k_head_finish(ProductArgs a, uint16_t* out) {
    const int64_t r = blockIdx.x, n = ((int64_t)blockIdx.y * 256 + threadIdx.x) * 4;
    if (n >= a.N) return;
    const int64_t target = a.targets[r];
    const bool live = head_live(target, a.V, a.ignore);
    const uint2 w = *reinterpret_cast<const uint2*>(a.W + (live ? target * a.N : 0) + n);
    f32x4 y = {};
#pragma unroll 8
    for (int s = 0; s < a.splits; ++s) y += *reinterpret_cast<const f32x4*>(a.sum + (s * a.out_rows + r) * a.N + n);
    *reinterpret_cast<uint2*>(out + r * a.N + n) = head_dx4(y, a.ends[r], w, live);
}

// G^T of a piece from its E: G = dloss / max|dloss| (E 2^(R - lse) - the target's 1 - p), R the reference that the
// piece ended with.  A lane takes 8 vocabulary entries of a token; eight lanes with eight tokens exchange them for
// 8 tokens of an entry each.
struct TurnArgs {
    const uint16_t* E;        // [tokens / 512][steps_v] blocks, and
    const uint8_t* low;       // the eight bits more
    uint16_t* G;              // [vocabulary / 512][steps_m] blocks
    int64_t steps_v, steps_m; // steps of 64 vocabulary rows, of 64 tokens
    int64_t v0, V;
    const float* ref;         // the piece's last references
    const float4* rows;
    const uint32_t* top;
};
__global__ __launch_bounds__(256)
void k_head_turn(TurnArgs a) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    // a wave: 32 tokens x 64 vocabulary entries, 4 KB on both sides
    const int64_t step = (int64_t)blockIdx.x * 4 + wave, m0 = (int64_t)blockIdx.y * 32;
    if (step >= a.steps_v) return;
    const int64_t m = m0 + (lane & 31);
    const float4 row = a.rows[m];
    const int target = __float_as_int(row.w);
    const float inv = 1.0f / head_scale(a.top), f = target >= 0 ? row.z * inv * __builtin_amdgcn_exp2f(a.ref[m] - row.x) : 0.0f;
    const float mine = -row.z * inv * row.y;
    const int64_t in = ((m0 / HL_TM) * a.steps_v + step) * A_BLOCK_BYTES + (m0 % HL_TM) * 128 + lane * 16;
    uint4 e[4];
    uint2 low[4];
#pragma unroll
    for (int s = 0; s < 4; ++s) {
        e[s] = *reinterpret_cast<const uint4*>(reinterpret_cast<const uint8_t*>(a.E) + in + s * 1024);
        low[s] = *reinterpret_cast<const uint2*>(a.low + (in + s * 1024) / 2);
    }
#pragma unroll
    for (int s = 0; s < 4; ++s) {
        const int64_t v = step * HL_K + 16 * s + 8 * (lane >> 5);        // of the piece
        float y[8];
        Vec16<uint16_t>::unpack(e[s], y);
#pragma unroll
        for (int u = 0; u < 8; ++u) {
            y[u] = f * head_both(y[u], (u < 4 ? low[s].x : low[s].y) >> (8 * (u & 3)));
            if (a.v0 + v + u == target) y[u] = mine;
            if (target < 0 || a.v0 + v + u >= a.V) y[u] = 0.0f;
        }
        uint4 g = Vec16<uint16_t>::pack(y);
        // 8 x 8 values of 16 bits across 8 lanes: halves, pairs, and neighbours change places
        {
            const bool up = lane & 4;
            const uint32_t x = __shfl_xor((int)(up ? g.x : g.z), 4), z = __shfl_xor((int)(up ? g.y : g.w), 4);
            g = up ? make_uint4(x, z, g.z, g.w) : make_uint4(g.x, g.y, x, z);
        }
        {
            const bool up = lane & 2;
            const uint32_t x = __shfl_xor((int)(up ? g.x : g.y), 2), z = __shfl_xor((int)(up ? g.z : g.w), 2);
            g = up ? make_uint4(x, g.y, z, g.w) : make_uint4(g.x, x, g.z, z);
        }
        {
            const bool up = lane & 1;
            auto swap = [&](uint32_t own) {
                const uint32_t other = __shfl_xor((int)own, 1);
                return up ? (own & 0xFFFF0000u) | (other >> 16) : (own & 0xFFFFu) | (other << 16);
            };
            g = make_uint4(swap(g.x), swap(g.y), swap(g.z), swap(g.w));
        }
        // this lane's entry, with the tokens of its eight
        const int64_t ve = v + (lane & 7);
        uint8_t* out = reinterpret_cast<uint8_t*>(a.G) + ((ve / HL_TM) * a.steps_m + m0 / HL_K) * A_BLOCK_BYTES + (ve % HL_TM >> 5) * 4096 +
                       ((m0 & 32) >> 3) * 512 + ((lane & 31) >> 3) * 512 + (ve & 31) * 16;
        *reinterpret_cast<uint4*>(out) = g;
    }
}

// Pieces of the vocabulary and the workspace's layout.
struct HeadPlan {
    int64_t Mp;               // tokens up to whole tiles
    bool few;                 // logits by k_head_few, or
    bool split;               // by k_head_split
    int width;                // vocabulary rows of a tile of the logits,
    int64_t rows;             // and its tokens (not few: 256 or 512)
    int64_t piece;            // vocabulary rows of a piece (a multiple of 512: whole row tiles of G^T)
    int64_t pieces;
    bool keep;                // every piece's E is kept until dW
    bool few_dx;              // dX by k_head_few_product
    int splits;               // parts of dX's contraction
    size_t top, zy, ref, total, factor, ends, of_rows, part, Xp, counted, E, low, G, sum, bytes;
    int64_t blocks(int64_t M) const { return M <= 32 ? 1 : (M + 63) / 64; }                   // of 64 tokens (one of 32)
    // tiles of the logits (few: four to a workgroup)
    int64_t tiles(int64_t vocabulary) const { return (vocabulary + 127) / 128 * (few ? 4 : 1); }
    size_t piece_bytes() const { return (size_t)Mp * piece * 2; }
};

constexpr int64_t CUS = 256;
// The time of a product in tiles of 512, 256 and 64 rows, for a step of 64: in units of a 512-row tile's 1.65 us, of
// which a compute unit holds one.  It holds two of the smaller; two of 256 rows take as long as one of 512 (alone:
// 0.9 us), two of 64 rows 0.64 to 0.76 us (alone: 0.42 us).
static double rounds_512(int64_t tiles) { return (double)((tiles + CUS - 1) / CUS); }
static double rounds_pairs(int64_t tiles, double two, double one) {
    const int64_t rest = tiles % (2 * CUS);
    return (double)(tiles / (2 * CUS)) * two + (rest == 0 ? 0.0 : rest <= CUS ? one : two);
}
static double rounds_256(int64_t tiles) { return rounds_pairs(tiles, 1.0, 0.55); }
static double rounds_64(int64_t tiles) { return rounds_pairs(tiles, 0.46, 0.25); }

static HeadPlan head_plan(int64_t M, int64_t K, int64_t V, bool dx, bool dw) {
    HeadPlan p{};
    const bool grad = dx || dw;
    p.Mp = (M + HL_TM - 1) / HL_TM * HL_TM;
    // a piece of E or G^T of at most 128 MB, half of the last-level cache: larger pieces pass over dX's
    // fp32 sums less often (64 MB: 947 us for 2048 tokens x 32000 x 4096, 128 MB: 903 us)
    const int64_t most = ((int64_t)128 << 20) / (p.Mp > 0 ? p.Mp * 2 : 1) / 512 * 512, all = (V + 511) / 512 * 512;
    p.piece = most < 512 ? 512 : (most < all ? most : all);
    p.pieces = V > 0 ? (V + p.piece - 1) / p.piece : 0;
    // dW from the kept E, up to 1 GB of it, instead of from the logits again
    p.keep = dw && p.piece_bytes() * p.pieces <= (size_t)1 << 30;
    // the tiles whose last round over the compute units ends first
    const int64_t slices = ((grad && p.piece < V ? p.piece : V) + HL_TN - 1) / HL_TN;
    const double all_256 = rounds_256(slices * ((M + 255) / 256));
    p.few = M <= FEW_TOKENS || rounds_64(slices * p.blocks(M)) < all_256;
    // a quarter of a tile for each wave's contraction: where four times the tiles still fit the compute units once, or,
    // of a long contraction, twice (33 tokens x 8000 x 2048: 13.5 and 23.1 us; x 16000 x 6144: 41 and 64; x 16000 x 576:
    // 16.7 and 15.5)
    p.split = p.few && slices * p.blocks(M) * 4 <= (K >= 4096 ? 2 * CUS : CUS);
    // over many steps 512-row tiles fetch less for their products and have little to hide at the ends (4096 x 16384 x
    // 8192: 829 and 859 us; 4096 x 32000 x 4096, losses alone: 866 and 818)
    p.rows = K >= 96 * HL_K && rounds_512(slices * (p.Mp / HL_TM)) <= all_256 ? 512 : 256;
    p.width = p.few ? FEW_TN : HL_TN;
    // where dX has too few tiles for the compute units, its contraction is cut into parts
    const int64_t columns = (K + HL_TN - 1) / HL_TN, steps = p.piece / HL_K;
    auto cut = [&](int64_t tiles, int64_t fill, int64_t least, int most) {
        int64_t n = tiles > 0 ? fill / tiles : 1;
        n = n < steps / least ? n : steps / least;
        return (int)(n < 1 ? 1 : n < most ? n : most);
    };
    const int64_t big = p.Mp / HL_TM * columns, small = p.blocks(M) * columns;
    const int big_splits = cut(big, CUS, 16, 8), few_splits = cut(small, 2 * CUS, 4, 64);
    auto per = [&](int splits) { return (double)((steps + splits - 1) / splits); };
    p.few_dx = M <= FEW_TOKENS || rounds_64(small * few_splits) * per(few_splits) < rounds_512(big * big_splits) * per(big_splits);
    p.splits = p.few_dx ? few_splits : big_splits;
    size_t at = 0;
    auto take = [&](size_t n) {
        const size_t was = at;
        at += (n + 255) & ~(size_t)255;
        return was;
    };
    const size_t row = (size_t)p.Mp * 4;
    p.top = take(4);
    p.zy = take(row);
    p.ref = take(row * (p.keep ? p.pieces + 1 : 1));
    p.total = take(row);
    p.factor = take(row);
    p.ends = take(2 * row);
    p.of_rows = take(4 * row);
    p.part = take((size_t)p.Mp * p.tiles(grad && p.piece < V ? p.piece : V) * sizeof(float2));
    p.Xp = take((size_t)p.Mp * K * 2);
    p.counted = take(dw ? (size_t)M * K * 2 : 0);
    p.E = take(grad ? p.piece_bytes() * (p.keep ? p.pieces : 1) : 0);
    p.low = take(p.keep ? p.piece_bytes() / 2 * p.pieces : 0);
    p.G = p.keep ? take(p.piece_bytes()) : p.E;
    p.sum = take(dx && (p.piece < V || p.splits > 1 || p.few_dx) ? (size_t)M * K * 4 * p.splits : 0);
    p.bytes = at;
    return p;
}

size_t head_loss_ws_bytes(int64_t M, int64_t K, int64_t V, bool dx, bool dw) { return head_plan(M, K, V, dx, dw).bytes; }

static dim3 head_grid(int64_t x, int64_t y, int splits = 1) { return dim3((uint32_t)((x * y + 7) / 8 * 8), (uint32_t)splits); }

// f(first vocabulary row, rows, whether it is the last piece)
template <typename F>
static void for_pieces(const HeadPlan& p, int64_t V, F&& f) {
    for (int64_t v0 = 0; v0 < V; v0 += p.piece) f(v0, V - v0 < p.piece ? V - v0 : p.piece, v0 + p.piece >= V);
}

// Tiles of 64 tokens use more LDS than the 64 KB that a kernel has unasked.
template <typename Args>
static void launch_few(void (*kernel)(Args), int bytes, dim3 grid, hipStream_t s, const Args& a) {
    if (hipFuncSetAttribute((const void*)kernel, hipFuncAttributeMaxDynamicSharedMemorySize, bytes) == hipSuccess)
        hipLaunchKernelGGL(kernel, grid, dim3(256), bytes, s, a);       // (an error is met by the caller's hipGetLastError)
}

template <HeadMode MODE>
static void launch_tiles(int64_t rows, HeadArgs& a, hipStream_t s) {
    a.tiles_m = (a.M + rows - 1) / rows;
    const dim3 grid = head_grid(a.tiles_v, a.tiles_m);
    if (rows == 512) hipLaunchKernelGGL((k_head_logits<MODE, 4>), grid, dim3(256), 0, s, a);
    else hipLaunchKernelGGL((k_head_logits<MODE, 2>), grid, dim3(256), 0, s, a);
}

template <HeadMode MODE>
static void launch_logits(const HeadPlan& p, HeadArgs& a, int64_t rows, hipStream_t s) {
    a.tiles_v = p.tiles(rows);
    const dim3 few = head_grid(a.tiles_v / 4, p.blocks(a.M));
    constexpr bool once = MODE == HEAD_STATS;
    const dim3 split = head_grid(a.tiles_v, p.blocks(a.M));
    if (p.split && a.M <= 32) launch_few(k_head_split<MODE, 1>, split_lds(1), split, s, a);
    else if (p.split) launch_few(k_head_split<MODE, 2>, split_lds(2), split, s, a);
    else if (p.few && a.M <= 32) launch_few(k_head_few<MODE, 1, once>, few_lds(1), few, s, a);
    else if (p.few && a.M <= 64) launch_few(k_head_few<MODE, 2, once>, few_lds(2), few, s, a);
    else if (p.few) launch_few(k_head_few<MODE, 2, false>, few_lds(2), few, s, a);
    else launch_tiles<MODE>(p.rows, a, s);
}

hipError_t launch_head_loss(const uint16_t* X, int64_t M, int64_t K, const uint16_t* W, int64_t V,
                            const int64_t* targets, int64_t ignore, const float* dloss, float* loss, uint16_t* dX,
                            uint16_t* dW, void* ws, hipStream_t s) {
    const HeadPlan p = head_plan(M, K, V, dX != nullptr, dW != nullptr);
    uint8_t* base = (uint8_t*)ws;
    const dim3 row_grid((uint32_t)(p.Mp / 4));
    HeadArgs a{};
    uint16_t* Xp = (uint16_t*)(base + p.Xp);
    a.X = X;
    a.Xp = Xp;
    a.W = W;
    a.M = M;
    a.K = K;
    a.V = V;
    a.targets = targets;
    a.ignore = ignore;
    a.part = (float2*)(base + p.part);
    a.zy = (float*)(base + p.zy);
    a.ref = (float*)(base + p.ref);
    a.rows = (float4*)(base + p.of_rows);
    a.top = (uint32_t*)(base + p.top);
    a.out = (uint16_t*)(base + p.E);
    a.Mp = p.Mp;
    if (!p.few || (dW && !p.keep)) hipLaunchKernelGGL(k_head_pack, dim3((uint32_t)(K / HL_K), (uint32_t)(p.Mp / HL_TM * 4)), dim3(256), 0, s, X, M, K, Xp);
    if (!dX && !dW) {
        launch_logits<HEAD_STATS>(p, a, V, s);
        hipLaunchKernelGGL(k_head_rows, dim3((uint32_t)M), dim3(256), 0, s, a.part, a.zy, targets, V, ignore, (int)a.tiles_v, loss);
        return hipGetLastError();
    }
    float* ref = (float*)(base + p.ref);
    float* total = (float*)(base + p.total);
    uint32_t* top = (uint32_t*)(base + p.top);
    uint16_t* counted = dW ? (uint16_t*)(base + p.counted) : nullptr;
    ProductArgs d{};
    d.A = a.out;
    d.N = K;
    d.tiles_n = (K + HL_TN - 1) / HL_TN;
    d.sum = (float*)(base + p.sum);
    d.factor = (float*)(base + p.factor);
    d.ends = (float2*)(base + p.ends);
    d.W = W;
    d.targets = targets;
    d.V = V;
    d.ignore = ignore;
    d.splits = p.splits;
    hipLaunchKernelGGL(k_head_target, dim3((uint32_t)((M + 3) / 4 + 1)), dim3(256), 0, s, X, W, M, K, V, targets, ignore, a.zy,
                       ref, total, dloss, top, counted);
    const int64_t piece_values = (int64_t)(p.piece_bytes() / 2);
    int64_t at = 0;                       // the piece, where each has a place of its own
    for_pieces(p, V, [&](int64_t v0, int64_t rows, bool last) {
        a.v0 = v0;
        a.out = (uint16_t*)(base + p.E) + at * piece_values;
        a.low = p.keep ? base + p.low + at * piece_values : nullptr;
        a.out_steps = (rows + HL_TN - 1) / HL_TN * (HL_TN / HL_K);
        a.ref = ref + at * p.Mp;
        launch_logits<HEAD_E>(p, a, rows, s);
        const JoinArgs j{a.part, (int)a.tiles_v, p.width, M, p.Mp, targets, ignore, V, a.out, a.out_steps, ref + at * p.Mp, ref + (at + p.keep) * p.Mp, total,
                         (float*)(base + p.factor), a.zy, last ? 1 : 0, dloss, loss, (float2*)(base + p.ends), (float4*)(base + p.of_rows)};
        hipLaunchKernelGGL(k_head_join, row_grid, dim3(256), 0, s, j);
        at += p.keep;
        if (!dX) return;
        d.A = a.out;
        d.a_steps = a.out_steps;
        d.out_rows = M;
        d.B = W + v0 * K;
        d.P = rows;
        d.steps = (int)((rows + HL_K - 1) / HL_K);
        d.tiles_r = p.few_dx ? p.blocks(M) : p.Mp / HL_TM;
        d.out = dX;
        d.add = v0 > 0;
        const dim3 grid = head_grid(d.tiles_r, d.tiles_n, d.splits);
        auto run = [&](auto kernel) { hipLaunchKernelGGL(kernel, grid, dim3(256), 0, s, d); };
        if (p.few_dx && M <= 32) launch_few(k_head_few_product<1, OUT_SUM>, few_lds(1), grid, s, d);
        else if (p.few_dx) launch_few(k_head_few_product<2, OUT_SUM>, few_lds(2), grid, s, d);
        else if (last && p.splits == 1) d.add ? run(k_head_product<OUT_DX, true, 4>) : run(k_head_product<OUT_DX, false, 4>);
        else d.add ? run(k_head_product<OUT_SUM, true, 4>) : run(k_head_product<OUT_SUM, false, 4>);
    });
    if (dX && (p.splits > 1 || p.few_dx))
        hipLaunchKernelGGL(k_head_finish, dim3((uint32_t)M, (uint32_t)((K + 1023) / 1024)), dim3(256), 0, s, d, dX);
    if (!dW) return hipGetLastError();
    d.splits = 1;
    d.top = top;
    d.A = (uint16_t*)(base + p.G);
    d.B = counted;
    d.P = M;
    d.steps = (int)((M + HL_K - 1) / HL_K);
    d.a_steps = p.Mp / HL_K;
    at = 0;
    for_pieces(p, V, [&](int64_t v0, int64_t rows, bool) {
        if (p.keep) {
            const TurnArgs t{(uint16_t*)(base + p.E) + at * piece_values, base + p.low + at * piece_values, (uint16_t*)(base + p.G),
                             (rows + HL_TN - 1) / HL_TN * (HL_TN / HL_K), d.a_steps, v0, V, ref + (at + 1) * p.Mp, a.rows, top};
            ++at;
            hipLaunchKernelGGL(k_head_turn, dim3((uint32_t)((t.steps_v + 3) / 4), (uint32_t)(d.steps * 2)), dim3(256), 0, s, t);
        } else {
            a.v0 = v0;
            a.out = (uint16_t*)(base + p.G);
            a.out_steps = d.a_steps;
            a.tiles_v = (rows + HL_TN - 1) / HL_TN;
            launch_tiles<HEAD_GT>(p.rows, a, s);
        }
        d.out_rows = rows;
        // short contractions are mostly ends, which two smaller tiles on a compute unit hide for each other (281 x
        // 37263 x 5504: 354 and 238 us; 4096 x 32000 x 8192: 1790 and 1840)
        int64_t tile = d.steps >= 64 ? 512 : 256;
        const int64_t fine = (rows + 63) / 64;
        if (rounds_64(fine * d.tiles_n) < (tile == 512 ? rounds_512((rows + 511) / 512 * d.tiles_n) : rounds_256((rows + 255) / 256 * d.tiles_n))) tile = 64;
        d.tiles_r = (rows + tile - 1) / tile;
        d.out = dW + v0 * K;
        const dim3 grid = head_grid(d.tiles_r, d.tiles_n);
        if (tile == 64) launch_few(k_head_few_product<2, OUT_DW>, few_lds(2), grid, s, d);
        else if (tile == 512) hipLaunchKernelGGL((k_head_product<OUT_DW, false, 4>), grid, dim3(256), 0, s, d);
        else hipLaunchKernelGGL((k_head_product<OUT_DW, false, 2>), grid, dim3(256), 0, s, d);
    });
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
