// rows.h -- eight neighbouring values of a row at a time, of any alignment, and sums over a row's
// threads; shared by block_norm.hip, gradients.hip and logits.hip (internal).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "rotary.h"

namespace nf4 {

// Eight values as they lie in memory.  Rows of odd widths start anywhere: the 16-byte accesses ask for no
// more alignment than a value has (global accesses of this GPU may be unaligned), so that odd widths take
// the same path as whole ones.
template <typename T>
struct Eight {
    uint4 w[sizeof(T) / 2];
};
template <typename T>
struct Loose;
template <>
struct Loose<uint16_t> {
    typedef uint32_t type __attribute__((ext_vector_type(4), aligned(2)));
};
template <>
struct Loose<float> {
    typedef uint32_t type __attribute__((ext_vector_type(4), aligned(4)));
};

// `left` of the eight are there (0 or fewer: none; eight or more: all); the others read as zero.
template <typename T>
__device__ __forceinline__ Eight<T> load_eight(const T* p, int64_t left) {
    constexpr int N = 16 / sizeof(T);
    Eight<T> e;
    if (left >= 8) {
#pragma unroll
        for (int i = 0; i < (int)(sizeof(T) / 2); ++i) e.w[i] = __builtin_bit_cast(uint4, *reinterpret_cast<const typename Loose<T>::type*>(p + i * N));
    } else {
        T v[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = i < left ? p[i] : T(0);
        __builtin_memcpy(&e, v, sizeof(e));
    }
    return e;
}
template <typename T>
__device__ __forceinline__ void store_eight(T* p, int64_t left, const Eight<T>& e) {
    constexpr int N = 16 / sizeof(T);
    if (left >= 8) {
#pragma unroll
        for (int i = 0; i < (int)(sizeof(T) / 2); ++i)
            *reinterpret_cast<typename Loose<T>::type*>(p + i * N) = __builtin_bit_cast(typename Loose<T>::type, e.w[i]);
    } else if (left > 0) {
        T v[8];
        __builtin_memcpy(v, &e, sizeof(e));
#pragma unroll
        for (int i = 0; i < 7; ++i)
            if (i < left) p[i] = v[i];
    }
}
template <typename T>
__device__ __forceinline__ void unpack_eight(const Eight<T>& e, float (&f)[8]) {
#pragma unroll
    for (int i = 0; i < (int)(sizeof(T) / 2); ++i) Vec16<T>::unpack(e.w[i], f + i * (16 / sizeof(T)));
}
template <typename T>
__device__ __forceinline__ Eight<T> pack_eight(const float (&f)[8]) {
    Eight<T> e;
#pragma unroll
    for (int i = 0; i < (int)(sizeof(T) / 2); ++i) e.w[i] = Vec16<T>::pack(f + i * (16 / sizeof(T)));
    return e;
}

// Sum over a wave's 64 lanes, in every lane: four steps inside rows of 16 lanes, then the four rows.
template <int CONTROL>
__device__ __forceinline__ float from_lane(float v) {
    return __uint_as_float((uint32_t)__builtin_amdgcn_mov_dpp((int)__float_as_uint(v), CONTROL, 0xF, 0xF, false));
}
__device__ __forceinline__ float wave_sum(float v) {
    v += from_lane<0xB1>(v);              // quad_perm [1, 0, 3, 2]
    v += from_lane<0x4E>(v);              // quad_perm [2, 3, 0, 1]
    v += from_lane<0x141>(v);             // row_half_mirror
    v += from_lane<0x140>(v);             // row_mirror
    auto row = [&](int lane) { return __uint_as_float((uint32_t)__builtin_amdgcn_readlane((int)__float_as_uint(v), lane)); };
    return (row(0) + row(16)) + (row(32) + row(48));
}

// Sums of N numbers over the WAVES waves that share a row, in all of their threads.  `shared` holds 2 N WAVES numbers;
// the halves take turns, so that one barrier per sum is enough (a half is written again only after the barrier of the
// sum between).
template <int WAVES, int N>
__device__ __forceinline__ void row_sums(float (&v)[N], float* shared, int& turn) {
#pragma unroll
    for (int n = 0; n < N; ++n) v[n] = wave_sum(v[n]);
    if constexpr (WAVES > 1) {
        float* half = shared + turn * N * WAVES;
        if ((threadIdx.x & 63) == 0) {
#pragma unroll
            for (int n = 0; n < N; ++n) half[n * WAVES + (threadIdx.x >> 6)] = v[n];
        }
        __syncthreads();
#pragma unroll
        for (int n = 0; n < N; ++n) {
            float s = half[n * WAVES];
#pragma unroll
            for (int w = 1; w < WAVES; ++w) s += half[n * WAVES + w];
            v[n] = s;
        }
        turn ^= 1;
    }
}

}  // namespace nf4
