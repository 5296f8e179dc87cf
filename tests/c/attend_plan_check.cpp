// Host check of attention's launches (attend_plan.h) over many sizes: where a row's keys are split between workgroups,
// every row that a kernel may take has a slot for its parts inside the planned workspace, which holds no more, and chunks hold whole steps; a
// launch stays below 2^32 threads along each dimension; and more new tokens than the batch has change nothing.
// Prints "<sizes> <failures>".
#include <cstdio>
#include <initializer_list>

#include "attend_plan.h"

using namespace nf4;

static int64_t sizes = 0, bad = 0;

static void fail(const AttendShape& a, const char* what) {
    if (++bad <= 10)
        printf("dim %d kv_heads %d seqs %lld tokens %lld heads %lld max_new %lld max_length %lld: %s\n", a.dim, a.kv_heads,
               (long long)a.seqs, (long long)a.tokens, (long long)a.heads, (long long)a.max_new, (long long)a.max_length, what);
}

static void check_part(const AttendShape& a, const AttendPart& q, int64_t slots, int64_t step) {
    if (q.chunk < 1 || q.chunk > KV_WHOLE || q.chunk % step) fail(a, "chunk");
    if (q.splits < 1 || q.splits > 1024) fail(a, "splits");
    if (q.tiles < 1) fail(a, "tiles");
    if (q.splits == 1) return;
    if ((int64_t)q.slots < slots) fail(a, "rows without a slot");
    const size_t need = (size_t)slots * q.splits * (a.dim + 2) * 4;
    if (q.bytes < need) fail(a, "workspace");
    if (q.bytes >= need + 256) fail(a, "workspace that no row uses");
}

static void check(const AttendShape& a) {
    ++sizes;
    const AttendPlan p = attend_plan(a);
    if (!p.rows.on && !p.block.on) fail(a, "no kernel");
    if (p.rows.on) {
        const int64_t rows = (a.max_new < a.tokens ? a.max_new : a.tokens) * (a.heads / a.kv_heads);
        check_part(a, p.rows, a.seqs * a.kv_heads * (rows < KV_FEW ? rows : KV_FEW), KV_WAVES * KV_STEP);
    }
    if (p.block.on) {
        check_part(a, p.block, a.tokens * a.heads, KV_STEP);
        if (p.block.waves != 1 && p.block.waves != 2 && p.block.waves != 4) fail(a, "waves");
        const int64_t pairs = (a.seqs * a.kv_heads + XCDS - 1) / XCDS * XCDS;
        if (pairs * p.block.tiles * 64 * p.block.waves >= (int64_t)1 << 32) fail(a, "threads of the prompts' kernel");
    }
    AttendShape held = a;
    held.max_new = a.max_new < a.tokens ? a.max_new : a.tokens;
    const AttendPlan h = attend_plan(held);
    auto same = [](const AttendPart& x, const AttendPart& y) {
        return x.on == y.on && x.tiles == y.tiles && x.chunk == y.chunk && x.splits == y.splits && x.bytes == y.bytes && x.waves == y.waves && x.few == y.few;
    };
    if (!same(p.rows, h.rows) || !same(p.block, h.block)) fail(a, "more new tokens than the batch has");
}

int main() {
    for (int dim : {64, 128, 256})
        for (int kv : {1, 8, 64, 4096})
            for (int64_t group : {1, 3, 8})
                for (int64_t seqs : {1, 5, 64, 65535})
                    for (int64_t tokens : {int64_t(1), seqs, 7 * seqs, int64_t(4096), int64_t(1) << 20})
                        for (int64_t max_new : {int64_t(1), int64_t(9), int64_t(1500), int64_t(1) << 20, (int64_t(1) << 23) - 1})
                            for (int64_t length : {int64_t(1), int64_t(700), int64_t(5000), int64_t(131072), int64_t(1) << 24,
                                                   (int64_t(1) << 24) + 1, int64_t(1) << 30, int64_t(0x7FFFFFFF)})
                                // (what the entry point lets through)
                                if (tokens * kv * group < (1 << 26) && max_new * group < (1 << 30) && seqs * kv <= ATTEND_PAIRS)
                                    check(AttendShape{dim, kv, seqs, tokens, kv * group, max_new, length});
    printf("%lld %lld\n", (long long)sizes, (long long)bad);
    return 0;
}
