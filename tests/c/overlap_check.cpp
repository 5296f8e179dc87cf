// Host check of overlap.h over many small operands: whether two of them share a byte, against a mark on each of their bytes.
// Prints "<pairs> <failures>".
#include <cstdio>
#include <cstdlib>
#include <initializer_list>
#include <vector>

#include "overlap.h"

using namespace nf4;

struct Rows {
    int at, rows, stride, width, elem;
    Memory memory() const { return Memory((const void*)(uintptr_t)(4096 + at), rows, stride, width, elem); }
    std::vector<bool> bytes() const {
        std::vector<bool> v(4096);
        for (int i = 0; i < rows; ++i)
            for (int j = 0; j < width * elem; ++j) v[at + i * stride * elem + j] = true;
        return v;
    }
};

int main() {
    long long pairs = 0, bad = 0;
    srand(1);
    auto below = [](int n) { return rand() % n; };
    auto draw = [&](int stride) {
        Rows r;
        r.elem = below(2) ? 2 : 4;
        r.rows = 1 + below(8);
        r.width = 1 + below(12);
        r.stride = stride >= r.width ? stride : below(8) == 0 ? 0 : r.width + below(3) * below(12);
        r.at = below(400);
        return r;
    };
    for (int i = 0; i < 300000; ++i) {
        const int common = below(2) ? 12 + below(14) : 0;
        Rows a = draw(common), b = draw(common);
        if (common && below(2)) b.elem = a.elem;              // rows of one buffer
        const std::vector<bool> x = a.bytes(), y = b.bytes();
        bool want = false;
        for (size_t j = 0; j < x.size(); ++j) want = want || (x[j] && y[j]);
        ++pairs;
        if (share_memory(a.memory(), b.memory()) != want || share_memory(b.memory(), a.memory()) != want) ++bad;
    }
    // nothing shares memory with nothing, and sizes whose products pass 64 bits are held
    const Memory none, huge((const void*)4096, 0x7FFFFFFF, INT64_MAX, INT64_MAX / 2, 4), one((const void*)(1 << 20), 16);
    bad += share_memory(none, one) + share_memory(one, none) + !share_memory(huge, one) + !share_memory(one, huge) + share_memory(Memory(nullptr, 5, 8, 8, 4), one);
    printf("%lld %lld\n", pairs, bad);
    return 0;
}
