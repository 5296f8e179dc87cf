// status.h -- the thread's last error and status helpers of the C entry points (internal to
// the library; defined in api.hip).
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include <string>

#include "../../include/qlora_nf4.h"

namespace nf4 {

nf4_status fail(nf4_status st, const std::string& msg);
nf4_status hip_status(hipError_t e, const char* where);
nf4_status out_of_memory() noexcept;      // NF4_ERR_HIP, and says so

// Nothing may leave a C entry point but a status: what throws here is the host's memory.
template <typename F>
nf4_status guarded(F&& f) noexcept {
    try {
        return f();
    } catch (...) {
        return out_of_memory();
    }
}
inline bool aligned(const void* p, size_t a) { return ((uintptr_t)p % a) == 0; }
inline size_t align256(size_t x) { return (x + 255) & ~(size_t)255; }

}  // namespace nf4
