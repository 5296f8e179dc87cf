// overlap.h -- whether two operands share memory.  Host code, free of HIP.
#pragma once

#include <stddef.h>
#include <stdint.h>

namespace nf4 {

// Rows of `width` bytes, `stride` bytes from one to the next.  128 bits: strides and counts come from the caller, and their
// products need not fit 64.  (Rows one behind the other are one row, and so is a row that stands for all.)
struct Memory {
    typedef __int128 Wide;
    Wide at = 0, rows = 0, stride = 0, width = 0, end = 0;
    Memory() {}
    Memory(const void* p, int64_t n, int64_t step, int64_t row_width, int elem)
        : at((Wide)(uintptr_t)p), rows(p ? n : 0), stride((Wide)step * elem), width((Wide)row_width * elem) {
        if (rows > 1 && stride == width) width *= rows, rows = 1;
        if (rows > 1 && stride == 0) rows = 1;
        end = at + (rows - 1) * stride + width;
    }
    Memory(const void* p, size_t bytes) : Memory(p, 1, 0, (int64_t)bytes, 1) {}
    bool empty() const { return rows < 1 || width < 1; }
    // whether a row of them meets the bytes from .. to - 1: the first row that ends past `from` does, or none
    bool meets(Wide from, Wide to) const {
        const Wide row = from < at + width ? 0 : rows == 1 ? 1 : (from - at - width) / stride + 1;
        return row < rows && at + row * stride < to;
    }
};

// Operands that lie side by side in the rows of one buffer do not meet, although their ranges do.
inline bool share_memory(const Memory& a, const Memory& b) {
    typedef Memory::Wide Wide;
    if (a.end <= b.at || b.end <= a.at || a.empty() || b.empty()) return false;
    if (a.rows == 1) return b.meets(a.at, a.end);
    if (b.rows == 1) return a.meets(b.at, b.end);
    if (a.stride == b.stride && a.width <= a.stride && b.width <= b.stride) {
        // every row of b lies as far behind a row of a: only that one and the next can meet it
        const Memory& first = a.at <= b.at ? a : b;
        const Memory& later = a.at <= b.at ? b : a;
        const Wide row = (later.at - first.at) / first.stride, past = (later.at - first.at) % first.stride;
        return (row < first.rows && past < first.width) || (row + 1 < first.rows && past + later.width > first.stride);
    }
    const Memory& few = a.rows <= b.rows ? a : b;
    const Memory& many = a.rows <= b.rows ? b : a;
    for (Wide i = 0; i < few.rows; ++i)
        if (many.meets(few.at + i * few.stride, few.at + i * few.stride + few.width)) return true;
    return false;
}

}  // namespace nf4
