// rotary.h -- the rotation of positions, shared by rope.hip and kv_append.hip (internal).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "nf4_common.h"

namespace nf4 {

constexpr int ROPE_MAX_DIM = 512;

// Device view of per-token heads (strides in elements).
struct HeadsView {
    void* data;
    int64_t token_stride, head_stride;
    int heads;
};

struct RopeView {
    const int64_t* freq;
    int rotary;               // rotated values of a head (0: no rotation)
    int interleaved;
    float magnitude;
    float sign;               // -1: turn the other way (the gradient)
};

// cos and sin of position * freq / 2^64 turns.  The product wraps modulo one turn exactly, and its top
// 32 bits are the signed fraction of a turn (error 2^-33), rounded to fp32 (2^-25 of a turn at most).
// v_sin_f32 and v_cos_f32 take turns: within 1.25e-7 over [-1/2, 1/2] (all 2^22 multiples of 2^-22 tried),
// at two instructions for what sincospif takes some sixty.
__device__ __forceinline__ float2 rope_cos_sin(int64_t freq, int position) {
    const uint64_t turn = (uint64_t)freq * (uint64_t)(int64_t)position;
    const float t = (float)(int32_t)(turn >> 32) * 0x1p-32f;
    return make_float2(__builtin_amdgcn_cosf(t), __builtin_amdgcn_sinf(t));
}

// (a, b) turned; the same expression wherever a pair is rotated.  The products are rounded
// apart from their sum (no contraction in this build).
__device__ __forceinline__ float2 rope_turn(float a, float b, float2 cs) {
    return make_float2(a * cs.x - b * cs.y, a * cs.y + b * cs.x);
}

// Sixteen bytes of values in fp32 and back (bf16: 8, round to nearest even; fp32: 4).
template <typename T>
struct Vec16;
template <>
struct Vec16<uint16_t> {
    static constexpr int N = 8;
    static __device__ __forceinline__ void unpack(uint4 w, float* f) {
        f[0] = bf16_lo(w.x); f[1] = bf16_hi(w.x); f[2] = bf16_lo(w.y); f[3] = bf16_hi(w.y);
        f[4] = bf16_lo(w.z); f[5] = bf16_hi(w.z); f[6] = bf16_lo(w.w); f[7] = bf16_hi(w.w);
    }
    static __device__ __forceinline__ uint4 pack(const float* f) {
        return make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                          pack_bf16x2(f[6], f[7]));
    }
    static __device__ __forceinline__ float to_f32(uint16_t v) { return bf16_to_f32(v); }
    static __device__ __forceinline__ uint16_t from_f32(float v) { return f32_to_bf16(v); }
};
template <>
struct Vec16<float> {
    static constexpr int N = 4;
    static __device__ __forceinline__ void unpack(uint4 w, float* f) {
        f[0] = __uint_as_float(w.x); f[1] = __uint_as_float(w.y); f[2] = __uint_as_float(w.z); f[3] = __uint_as_float(w.w);
    }
    static __device__ __forceinline__ uint4 pack(const float* f) {
        return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
    }
    static __device__ __forceinline__ float to_f32(float v) { return v; }
    static __device__ __forceinline__ float from_f32(float v) { return v; }
};

// The cos and sin of one token's pairs into LDS, the magnitude multiplied in.
__device__ __forceinline__ void rope_fill(const RopeView& r, int position, float2* cs, int tid, int threads) {
    for (int i = tid; i < r.rotary / 2; i += threads) {
        const float2 v = rope_cos_sin(r.freq[i], position);
        cs[i] = make_float2(v.x * r.magnitude, v.y * r.sign * r.magnitude);
    }
}

// Work items of one head: VEC rotates N pairs (two 16-byte vectors) per item and copies N
// values per item past the rotated ones; otherwise one pair, or one value, per item.
template <typename T, bool VEC>
__device__ __forceinline__ int rope_items(int rotary, int head_dim) {
    constexpr int N = VEC ? Vec16<T>::N : 1;
    return rotary / (2 * N) + (head_dim - rotary) / N;
}

// Rotates the head at `in` into `out` (item `c` of it), cos and sin in LDS.
template <typename T, bool INTER, bool VEC>
__device__ __forceinline__ void rope_item(const T* in, T* out, int c, const RopeView& r, const float2* cs) {
    constexpr int N = VEC ? Vec16<T>::N : 1;
    const int rot = r.rotary / (2 * N);
    if (c >= rot) {
        const int d = r.rotary + (c - rot) * N;
        if constexpr (VEC) *reinterpret_cast<uint4*>(out + d) = *reinterpret_cast<const uint4*>(in + d);
        else out[d] = in[d];
        return;
    }
    const int first = INTER ? 2 * c * N : c * N;                  // the item's first value, and
    const int second = INTER ? first + N : first + r.rotary / 2;  // that of its second vector
    float x[2 * N];
    if constexpr (VEC) {
        Vec16<T>::unpack(*reinterpret_cast<const uint4*>(in + first), x);
        Vec16<T>::unpack(*reinterpret_cast<const uint4*>(in + second), x + N);
    } else {
        x[0] = Vec16<T>::to_f32(in[first]);
        x[1] = Vec16<T>::to_f32(in[second]);
    }
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const int a = INTER ? 2 * i : i, b = INTER ? 2 * i + 1 : i + N;
        const float2 t = rope_turn(x[a], x[b], cs[c * N + i]);
        x[a] = t.x;
        x[b] = t.y;
    }
    if constexpr (VEC) {
        *reinterpret_cast<uint4*>(out + first) = Vec16<T>::pack(x);
        *reinterpret_cast<uint4*>(out + second) = Vec16<T>::pack(x + N);
    } else {
        out[first] = Vec16<T>::from_f32(x[0]);
        out[second] = Vec16<T>::from_f32(x[1]);
    }
}

}  // namespace nf4
