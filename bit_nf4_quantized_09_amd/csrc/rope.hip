// rope.hip -- rotary positions of queries and keys, forward and backward (gfx950).
//
// Pair (a, b) of a head at position p becomes magnitude (a cos - b sin, a sin + b cos), the
// angle p * freq; the gradient is the transpose, the same with the angle negated.  Bound by
// HBM: each value is read once and written once.  One workgroup per token (a few tokens: one
// per token and part of its heads) computes the token's cos and sin once into LDS, at most
// 256 pairs, and every thread then rotates two 16-byte vectors at a time of any of the
// token's heads, queries and keys alike.  4096 tokens of 64 + 64 heads of 128 in bf16 (268 MB): 44 us,
// 6.1 TB/s (above a large copy's 4.9, as half of it is still in the last-level cache); 16 tokens: 3.2 us.
#include "decoder.h"

namespace nf4 {

struct RopeArgs {
    RopeView rope;
    const int32_t* positions;
    HeadsView in[2], out[2];
    int heads;                // of both tensors
    int dim;
};

template <typename T, bool INTER, bool VEC>
__global__ __launch_bounds__(256)
void k_rope(RopeArgs a) {
    __shared__ float2 cs[ROPE_MAX_DIM / 2];
    const int64_t t = blockIdx.x;
    rope_fill(a.rope, a.positions[t], cs, threadIdx.x, 256);
    __syncthreads();
    const int per = rope_items<T, VEC>(a.rope.rotary, a.dim);
    const int total = per * a.heads;
    for (int i = blockIdx.y * 256 + threadIdx.x; i < total; i += 256 * gridDim.y) {
        const int h = i / per, c = i - h * per;
        const bool second = h >= a.in[0].heads;
        const HeadsView& x = second ? a.in[1] : a.in[0];
        const HeadsView& y = second ? a.out[1] : a.out[0];
        const int hh = second ? h - a.in[0].heads : h;
        rope_item<T, INTER, VEC>((const T*)x.data + t * x.token_stride + hh * x.head_stride,
                                 (T*)y.data + t * y.token_stride + hh * y.head_stride, c, a.rope, cs);
    }
}

hipError_t launch_rope(const RopeView& rope, const int32_t* positions, int64_t M, int head_dim, bool bf16,
                       const HeadsView* in, const HeadsView* out, int count, hipStream_t s) {
    RopeArgs a{};
    a.rope = rope;
    a.positions = positions;
    a.dim = head_dim;
    const int N = bf16 ? 8 : 4;
    // 16-byte vectors need every head's row aligned and the rotated part in whole items
    bool vec = rope.rotary % (2 * N) == 0 && (head_dim - rope.rotary) % N == 0;
    for (int i = 0; i < 2; ++i) {
        a.in[i] = in[i < count ? i : 0];
        a.out[i] = out[i < count ? i : 0];
        if (i >= count) continue;
        a.heads += in[i].heads;
        for (const HeadsView* v : {&in[i], &out[i]})
            vec = vec && (uintptr_t)v->data % 16 == 0 && v->token_stride % N == 0 && v->head_stride % N == 0;
    }
    const int per = rope.rotary / (vec ? 2 * N : 2) + (head_dim - rope.rotary) / (vec ? N : 1);
    const int64_t rounds = ((int64_t)per * a.heads + 255) / 256;
    // few tokens: their heads are spread over more workgroups, until about 1024 are there
    int64_t parts = M >= 1024 ? 1 : (1024 + M - 1) / M;
    if (parts > rounds) parts = rounds;
    if (parts > 65535) parts = 65535;
    const dim3 grid((uint32_t)M, (uint32_t)parts);
    auto run = [&](auto kernel) { hipLaunchKernelGGL(kernel, grid, dim3(256), 0, s, a); };
    const bool inter = rope.interleaved != 0;
    if (bf16) {
        if (vec) inter ? run(k_rope<uint16_t, true, true>) : run(k_rope<uint16_t, false, true>);
        else inter ? run(k_rope<uint16_t, true, false>) : run(k_rope<uint16_t, false, false>);
    } else {
        if (vec) inter ? run(k_rope<float, true, true>) : run(k_rope<float, false, true>);
        else inter ? run(k_rope<float, true, false>) : run(k_rope<float, false, false>);
    }
    return hipGetLastError();
}

}  // namespace nf4
