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

// (Global memory by its type: a flat access would count among the LDS accesses that a sum waits for, and with it every
// load on its way.)
#define NF4_GLOBAL __attribute__((address_space(1)))
template <typename T>
__device__ __forceinline__ uintptr_t at_value(const T* row, uint32_t at) {
    return (uintptr_t)row + at * (uint32_t)sizeof(T);
}
// STREAM: a nontemporal load, for what is read once.
template <typename T, bool STREAM = false>
__device__ __forceinline__ Eight<T> load_whole(uintptr_t p) {
    Eight<T> e;
#pragma unroll
    for (int i = 0; i < (int)(sizeof(T) / 2); ++i) {
        const NF4_GLOBAL typename Loose<T>::type* at = (const NF4_GLOBAL typename Loose<T>::type*)p + i;
        if constexpr (STREAM) e.w[i] = __builtin_bit_cast(uint4, __builtin_nontemporal_load(at));
        else e.w[i] = __builtin_bit_cast(uint4, *at);
    }
    return e;
}
// The values a place on (down) or back, a zero behind.
template <typename T>
__device__ __forceinline__ void shift_one(Eight<T>& e, bool down) {
    constexpr int D = 2 * sizeof(T);
    uint32_t w[D + 2] = {};
    __builtin_memcpy(w + 1, &e, sizeof(e));
    uint32_t v[D];
#pragma unroll
    for (int i = 0; i < D; ++i) {
        if constexpr (sizeof(T) == 2) v[i] = down ? w[i + 1] >> 16 | w[i + 2] << 16 : w[i + 1] << 16 | w[i] >> 16;
        else v[i] = down ? w[i + 2] : w[i];
    }
    __builtin_memcpy(&e, v, sizeof(e));
}
// Values `at` .. at + 7 of a row of `n` (those past its end read as zero, and are not written).  The row's address is the
// same in all lanes: offsets of 32 bits leave it in scalar registers.  (The loops of a row's last values are loops, for
// their conditions side by side would take the scalar registers.)
template <typename T>
__device__ __forceinline__ Eight<T> load_eight(const T* row, uint32_t at, uint32_t n) {
    const uintptr_t p = at_value(row, at);
    if (at + 8 <= n) return load_whole<T>(p);
    Eight<T> e = {};
#pragma unroll 1
    for (uint32_t i = at < n ? n - at : 0; i > 0; --i) {
        shift_one(e, false);
        const T v = ((const NF4_GLOBAL T*)p)[i - 1];
        uint32_t first = 0;
        __builtin_memcpy(&first, &v, sizeof(T));
        e.w[0].x |= first;
    }
    return e;
}
template <typename T>
__device__ __forceinline__ void store_eight(T* row, uint32_t at, uint32_t n, Eight<T> e) {
    const uintptr_t p = at_value(row, at);
    if (at + 8 <= n) {
#pragma unroll
        for (int i = 0; i < (int)(sizeof(T) / 2); ++i)
            *((NF4_GLOBAL typename Loose<T>::type*)p + i) = __builtin_bit_cast(typename Loose<T>::type, e.w[i]);
    } else {
#pragma unroll 1
        for (uint32_t i = 0; at + i < n; ++i) {
            T v;
            __builtin_memcpy(&v, &e.w[0].x, sizeof(T));
            ((NF4_GLOBAL T*)p)[i] = v;
            shift_one(e, true);
        }
    }
}
// load_eight in two parts for rows of eight values and more, so that nothing waits where the load is started: load_late
// reads eight values that are all there (the row's last ones past its end), settle moves them to their places once they
// are needed.
template <typename T, bool STREAM = false>
__device__ __forceinline__ Eight<T> load_late(const T* row, uint32_t at, uint32_t n) {
    return load_whole<T, STREAM>(at_value(row, at + 8 <= n ? at : n - 8));
}
template <typename T>
__device__ __forceinline__ void settle(Eight<T>& e, uint32_t at, uint32_t n) {
    const uint32_t s = at + 8 <= n ? 0 : at + 8 - n;      // places that the values lie too high
    constexpr int D = 2 * sizeof(T);              // dwords
    uint32_t w[D + 4] = {};
    __builtin_memcpy(w, &e, sizeof(e));
    const uint32_t dwords = s * sizeof(T) / 4;
#pragma unroll
    for (int step = 4; step >= 1; step /= 2)
#pragma unroll
        for (int i = 0; i < D; ++i) w[i] = dwords & step ? w[i + step] : w[i];
    if constexpr (sizeof(T) == 2) {
#pragma unroll
        for (int i = 0; i < D; ++i) w[i] = s & 1 ? w[i] >> 16 | w[i + 1] << 16 : w[i];
    }
#pragma unroll
    for (int i = 0; i < D; ++i) w[i] = s >= 8 ? 0u : w[i];
    __builtin_memcpy(&e, w, sizeof(e));
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

// Sum over a wave's 64 lanes, the same in every lane: four steps inside rows of 16 lanes, then the rows onto the last one.
template <int CONTROL, int ROWS>
__device__ __forceinline__ float from_lane(float v) {
    return __uint_as_float((uint32_t)__builtin_amdgcn_update_dpp(0, (int)__float_as_uint(v), CONTROL, ROWS, 0xF, ROWS == 0xF));
}
__device__ __forceinline__ float wave_sum(float v) {
    v += from_lane<0xB1, 0xF>(v);         // quad_perm [1, 0, 3, 2]
    v += from_lane<0x4E, 0xF>(v);         // quad_perm [2, 3, 0, 1]
    v += from_lane<0x141, 0xF>(v);        // row_half_mirror
    v += from_lane<0x140, 0xF>(v);        // row_mirror
    v += from_lane<0x142, 0xA>(v);        // row_bcast15: rows 0 and 2 onto 1 and 3
    v += from_lane<0x143, 0xC>(v);        // row_bcast31: rows 0 and 1 onto 2 and 3
    return __uint_as_float((uint32_t)__builtin_amdgcn_readlane((int)__float_as_uint(v), 63));
}

// Sums of N numbers over the `waves` waves that share a row (16 at most; GROUP false: one, without a barrier), in all of
// their threads.  `shared` has 2 N quadruples of four, zero at first; the halves take turns, so that one barrier per sum is
// enough (a half is written again only after the barrier of the sum between).  UNIFORM: the sums leave the vector registers
// (gradients of 4096 x 8192, fp32 stream: 124 us, 128 without; where a thread has four vectors of a row, whose registers are
// spilled either way, of 1024 x 32768: 365 and 325).
template <bool GROUP, bool UNIFORM, int N>
__device__ __forceinline__ void row_sums(float (&v)[N], float4* shared, int& turn, int waves) {
#pragma unroll
    for (int n = 0; n < N; ++n) v[n] = wave_sum(v[n]);
    if constexpr (GROUP) {
        float4* half = shared + turn * N * 4;
        if ((threadIdx.x & 63) == 0) {
#pragma unroll
            for (int n = 0; n < N; ++n) reinterpret_cast<float*>(half + n * 4)[threadIdx.x >> 6] = v[n];
        }
        __syncthreads();
#pragma unroll
        for (int n = 0; n < N; ++n) v[n] = 0.0f;
        for (int w = 0; w < waves; w += 4)
#pragma unroll
            for (int n = 0; n < N; ++n) {
                const float4 s = half[n * 4 + (w >> 2)];
                v[n] += (s.x + s.y) + (s.z + s.w);
            }
        if constexpr (UNIFORM)
#pragma unroll
            for (int n = 0; n < N; ++n) v[n] = __uint_as_float((uint32_t)__builtin_amdgcn_readfirstlane((int)__float_as_uint(v[n])));
        turn ^= 1;
    }
}

}  // namespace nf4
