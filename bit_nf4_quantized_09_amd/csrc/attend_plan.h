// attend_plan.h -- how attention over the paged cache is launched: which kernels, the chunks their keys
// are split into and the workspace of the chunks' parts.  Host code, free of HIP.
#pragma once

#include <stddef.h>
#include <stdint.h>

#include "tile_map.h"

namespace nf4 {

constexpr int KV_STEP = 32;               // keys of a step
constexpr int KV_WAVES = 4;               // waves of k_attend_rows
constexpr int KV_FEW = 32;                // rows of a (sequence, kv head) that count as few
constexpr int KV_WHOLE = 1 << 30;         // the longest chunk (a longer sequence's few chunks are taken in turn)

// A call's sizes: max_new and max_length as the caller states them.
struct AttendShape {
    int dim, kv_heads;
    int64_t seqs, tokens, heads, max_new, max_length;
    bool window = false;                  // max_length is a window's keys, which the sequences that it cuts fill
};
constexpr int64_t ATTEND_PAIRS = (int64_t)1 << 25;        // (sequence, kv head) pairs of a call at most: one wave each, of 2^32 threads

// One kernel's part of a call: its chunks and where its parts lie.
struct AttendPart {
    bool on;
    int tiles, chunk, splits;             // row tiles (blocks) launched per (sequence, kv head)
    size_t slots, bytes;                  // row slots; workspace
    int waves;                            // k_attend_block: waves that share a block's keys
    int few;                              // k_attend_rows: rows of a (sequence, kv head) that have slots
};
struct AttendPlan {
    AttendPart rows, block;
};
// (3 prompts of up to 1500 tokens behind 1100 cached, 32 heads of 128: one tile 213 us, two 131, four, past the
// registers, 570; of 256: one tile 355, two 1281; of 64: two tiles 92, four 96)
constexpr int block_tiles(int dim) { return dim == 256 ? 1 : 2; }     // CT
constexpr int block_rows(int dim) { return block_tiles(dim) * 16; }

// k_attend_rows reads the keys once per 16 rows and splits them over many workgroups; k_attend_block
// reads them once per block_rows rows and decodes them once per block_tiles tiles.  A batch whose sequences all bring
// up to 32 rows per kv head needs the first alone, one of equal longer ones the second alone; any other
// may hold both kinds, and each kernel takes its own, unless there is so little to read that two launches more cost
// more than the tiles that a few rows leave empty (27 sequences of up to 494 keys and 11 tokens, 8 heads of 64: 36 us
// with both kernels, 24 with one).
// (17 to 32 rows by k_attend_block instead: 55 us for 49 with 8 sequences of up to 8000 keys and 4 tokens, 8 groups of
// 8 heads of 256, 31 for 19 with heads of 64.)
// Chunks: for k_attend_rows about 4096 workgroups (some rounds of three or four on each compute unit, so that a
// ragged batch's last chunks end together) at the stated lengths, but chunks of 1024 keys where 1024 workgroups are left
// then, for a workgroup's start, end and join cost as much as some 200 keys (two sequences of 120001 keys, 8 kv
// heads: chunks of 512 keys 82 us, 1024 76; of 24 sequences of up to 4096, 64 heads: 1536 keys 128 us, half of that 130, twice 191),
// and of at least 256 keys; up to 768 keys stay whole, for the join's launch costs more (4 sequences of up to 600 keys,
// heads of 128: 7.0 us, 8.9 in chunks; of up to 900: 9.0 and 9.0, heads of 256 14.4 and 11.9).  For k_attend_block, where there are fewer blocks than waves that run at once, two or four
// waves share a block's keys (4 prompts of up to 534 tokens, 8 heads of 64: 12.5 us, 22.5 alone; 2 of 1277, 16 heads of
// 128: 31 and 35; but 3 of 1500, 32 heads: 134 and 127, and heads of 256, whose parts are as large as a step's
// work: 24 and 10 for 3 of 76 tokens), and chunks only where there are still fewer than 1024 waves, one for
// each SIMD: of 128 keys a wave at least where most of the keys were there before (27 sequences of up to 494 keys
// and 11 tokens: 15 us, 24 with 512), of 512 for prompts, whose early rows see few keys but are joined like the
// others (one prompt of 252 behind 1370 keys, 8 heads of 256: 70 us with 128, 49 with 512).
// A window makes the sequences that it cuts equally long, so that workgroups come in rounds: window_splits takes the chunks,
// all of one size, for which an estimate is least: rounds of three workgroups on a compute unit (one with heads of 256), each
// as long as a wave's steps take one after the other (1.1 us) or the round's bytes at 6 TB/s, and 5 us for a join.  24
// sequences, window of 4096, 64 heads on 8: 39 us with whole windows, 42 with a round of four chunks, 48 with one and a half of
// six; window of 1024: 14 us whole, 20 to 22 with two chunks; of 8192: 72 whole, 80 with two.  (Eight waves to a
// workgroup instead of chunks: no faster, one sequence, window of 1000: 13.3 us, 11.8 with chunks.)
// Sequences that the window does not cut stay ragged, and then the call waits for a long chunk's few waves: chunks of
// KV_SERIAL keys at most (80 us of a wave's steps), or of an eighth of the window where that is longer, and no more of
// them than workgroups are wanted without a window, for most may find nothing to do.  48 sequences of 500 to 60000 keys,
// 64 heads on 8, window of 50000: 347 us, 412 in the chunks of the estimate alone; one of 60000 and 47 of 200: 75 and
// 345; 16 of 131072, which a window of 65536 cuts all: 343 and 316.
constexpr int64_t KV_SERIAL = 72 * KV_WAVES * KV_STEP, KV_ROUNDS = 4096;
inline int64_t window_splits(const AttendShape& a, int64_t groups) {
    auto held = [](int64_t v, int64_t low, int64_t high) { return v < low ? low : v > high ? high : v; };
    const int64_t first = held((a.max_length + KV_SERIAL - 1) / KV_SERIAL, 1, 8);
    const int64_t most = held(held(a.max_length / (KV_WAVES * KV_STEP), 1, KV_ROUNDS / groups), first, 64);
    const int64_t at_once = 256 * (a.dim == 256 ? 1 : 3);
    int64_t best = first;
    double least = 0;
    for (int64_t s = first; s <= most; ++s) {
        const int64_t steps = (a.max_length + s * KV_STEP - 1) / (s * KV_STEP), workgroups = groups * s;
        const double wave = 1.1 * (double)((steps + KV_WAVES - 1) / KV_WAVES);
        const double bytes = (double)(workgroups < at_once ? workgroups : at_once) * (double)steps * (KV_STEP * 2.0) * a.dim / 6e6;
        const double cost = (double)((workgroups + at_once - 1) / at_once) * (wave > bytes ? wave : bytes) + (s > 1 ? 5.0 : 0.0);
        if (s == first || cost < least) best = s, least = cost;
    }
    return best;
}
constexpr int64_t BLOCK_ALONE = 1024 * 512;
inline AttendPlan attend_plan(const AttendShape& a) {
    AttendPlan p{};
    // no sequence brings more tokens than the batch (a capacity in its place would launch for rows that are not there)
    const int64_t max_new = a.max_new < a.tokens ? a.max_new : a.tokens, max_length = a.max_length;
    const int64_t most_rows = max_new * (a.heads / a.kv_heads), keys = a.seqs * a.kv_heads * max_length;
    p.rows.on = most_rows <= KV_FEW || (a.tokens != a.seqs * max_new && keys > BLOCK_ALONE);
    p.block.on = most_rows > KV_FEW;
    auto chunks = [&](AttendPart& q, int64_t keys, int64_t unit, int64_t least, size_t slots) {
        int64_t chunk = (keys + unit - 1) / unit * unit;
        chunk = chunk < least ? least : (chunk > KV_WHOLE ? KV_WHOLE : chunk);
        const int64_t splits = (max_length + chunk - 1) / chunk;
        q.chunk = (int)chunk;
        q.splits = (int)(splits < 1 ? 1 : (splits < 1024 ? splits : 1024));
        q.slots = slots;
        q.bytes = q.splits > 1 ? (slots * q.splits * (a.dim + 2) * sizeof(float) + 255) & ~(size_t)255 : 0;
    };
    if (p.rows.on) {
        const int64_t r = most_rows < KV_FEW ? most_rows : KV_FEW;
        p.rows.few = (int)r;
        p.rows.tiles = (int)((r + 15) / 16);
        const int64_t groups = a.seqs * a.kv_heads * p.rows.tiles, wide = keys * p.rows.tiles / 1024;
        const int64_t least = max_length <= 768 ? 768 : wide < 256 ? 256 : wide < 1024 ? wide / 128 * 128 : 1024;
        const size_t slots = (size_t)(a.seqs * a.kv_heads * r);
        if (a.window) {
            const int64_t s = window_splits(a, groups);
            chunks(p.rows, (max_length + s - 1) / s, KV_STEP, KV_STEP, slots);
        } else {
            chunks(p.rows, max_length * groups / 4096, KV_WAVES * KV_STEP, least, slots);
        }
    }
    if (p.block.on) {
        const int64_t rows = block_rows(a.dim);
        int64_t blocks = (most_rows + rows - 1) / rows;
        const int64_t pairs = (a.seqs * a.kv_heads + XCDS - 1) / XCDS * XCDS, most = (int64_t)1 << 24;      // (waves launched)
        const int64_t groups = (a.tokens * a.heads + rows - 1) / rows;
        const int waves = p.block.waves = a.dim == 256 || max_length < 256 || groups >= 2048 || 4 * pairs > most ? 1 : groups >= 1024 ? 2 : 4;
        blocks = blocks < most / (pairs * waves) ? blocks : most / (pairs * waves);      // (a workgroup takes several beyond that)
        p.block.tiles = (int)(blocks < 1 ? 1 : blocks);
        // one chunk, of whatever length: no row has a slot for a part
        if (groups * waves >= 1024) p.block.chunk = KV_WHOLE, p.block.splits = 1;
        else chunks(p.block, max_length * groups * waves / 1024, KV_STEP, (16 * max_new <= max_length ? 128 : 512) * waves, (size_t)(a.tokens * a.heads));
    }
    return p;
}

// The shape of a call with a window: its keys side by side are the sequence as far as the launches are concerned (a
// block's rows and the window's start up to a whole step reach further).  A window that cuts no sequence of the stated
// length is planned like none (48 sequences of 500 to 60000 keys, 64 heads on 8, window of 2^20: 325 us, none 317, as a window 450).
inline int64_t sink_span(int64_t sinks) { return (sinks + KV_STEP - 1) / KV_STEP * KV_STEP; }
inline AttendShape window_shape(AttendShape a, int64_t window, int64_t sinks) {
    const int64_t most = sink_span(sinks) + window + block_rows(a.dim) + KV_STEP;
    a.window = window + sinks < a.max_length;
    if (most < a.max_length) a.max_length = most;
    return a;
}

}  // namespace nf4
