// lds_dma.h -- direct loads from memory into LDS (internal).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace nf4 {

// A buffer descriptor as plain registers.
typedef int dma_rsrc __attribute__((ext_vector_type(4)));
__device__ __forceinline__ dma_rsrc make_dma_rsrc(const void* base, int64_t bytes) {
    const uint64_t p = (uint64_t)base;
    return dma_rsrc{(int)(uint32_t)p, (int)((p >> 32) & 0xFFFF), (int)(bytes < 0x7FFFFFFF ? bytes : 0x7FFFFFFF), 0x00020000};
}

// Sixteen bytes per lane from memory into LDS at `at` + 16 * lane, without passing registers.  In
// assembly, because the compiler makes transposing LDS reads wait for every such load of the
// builtin's kind, whichever part of LDS it fills; the kernels that use it wait for it themselves
// (s_waitcnt vmcnt).  The compiler counts the loads it knows of, so its own waits with these among
// them are only stricter.  It puts no wait states inside or right before a string of assembly, so
// the string has its own: the load reads M0, which needs one after the scalar write, and its scalar
// operands may come from a vector instruction (v_readfirstlane), which needs five.  The scalar write
// counts as one of these and s_nop 3 as four; they pass behind the matrix instructions in flight.
// NT: nontemporal, for what is read once.
template <bool NT = false>
__device__ __forceinline__ void load_to_lds(dma_rsrc r, uint32_t at, uint32_t voff, uint32_t soff) {
    if constexpr (NT)
        asm volatile("s_mov_b32 m0, %0\n\ts_nop 3\n\tbuffer_load_dwordx4 %1, %2, %3 offen nt lds" ::"s"(at), "v"(voff), "s"(r), "s"(soff) : "memory", "m0");
    else
        asm volatile("s_mov_b32 m0, %0\n\ts_nop 3\n\tbuffer_load_dwordx4 %1, %2, %3 offen lds" ::"s"(at), "v"(voff), "s"(r), "s"(soff) : "memory", "m0");
}
__device__ __forceinline__ uint32_t lds_address(const void* p) {
    return (uint32_t)(uintptr_t)(__attribute__((address_space(3))) const uint8_t*)(p);
}

}  // namespace nf4
