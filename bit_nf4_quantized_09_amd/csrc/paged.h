// paged.h -- places of a batch's tokens in the paged cache, shared by kv_append.hip and
// kv_attention.hip (internal).
#pragma once

#include "decoder.h"

namespace nf4 {

// The sequence of packed token t: the last b with starts[b] <= t.  Every lane of the wave
// gets it; each round reads 64 evenly spaced starts, one per lane (one round up to 64
// sequences, two up to 4096).
__device__ __forceinline__ int sequence_of(const int32_t* starts, int seqs, int t, int lane) {
    int lo = 0, n = seqs;
    while (n > 1) {
        const int step = (n + 63) >> 6;
        const int at = lo + lane * step;
        const bool before = lane * step < n && starts[at] <= t;
        int hits = __popcll(__ballot(before));
        hits = hits < 1 ? 1 : hits;
        const int next = (hits - 1) * step;
        lo += next;
        n = n - next < step ? n - next : step;
    }
    return __builtin_amdgcn_readfirstlane(lo);
}

// The new tokens begin .. begin + count - 1 of a sequence, from its two starts.  Starts are device data that no host check
// has seen: whatever they say, the tokens are among the batch's.
struct NewTokens {
    int begin, count;
};
__device__ __forceinline__ NewTokens new_tokens(const BatchView& b, int start, int end) {
    const int from = start < 0 ? 0 : (start < b.tokens ? start : b.tokens);
    const int to = end < from ? from : (end < b.tokens ? end : b.tokens);
    return NewTokens{from, to - from};
}

// Position of the new token `i` places on from a sequence's length.  A length near 2^31 wraps round to a negative position,
// which is left out like any negative one (and 2^31 - 256 is past every table).
__device__ __forceinline__ int position_at(int length, int i) { return (int)((uint32_t)length + (uint32_t)i); }

// Page of the pool that holds positions p .. of a sequence, or -1 if the sequence has none there.
__device__ __forceinline__ int page_of(const CacheView& c, const BatchView& b, int seq, int page_index) {
    if (page_index < 0 || page_index >= b.table_width) return -1;
    const int page = b.table[seq * b.table_stride + page_index];
    return page >= 0 && page < c.pages ? page : -1;
}

}  // namespace nf4
