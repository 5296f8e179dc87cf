// Host check of how long a window's chunks are (attend_plan.h): a sequence that the window does not cut may be the only long one
// of its batch, so no workgroup's waves take more than KV_SERIAL keys one after the other, or an eighth of the window; no more
// workgroups are asked for than without a window, but for those that this takes; and a window that cuts nothing is planned like none.
// Prints "<sizes> <failures>".
#include <cstdio>
#include <initializer_list>

#include "attend_plan.h"

using namespace nf4;

static bool same(const AttendPart& x, const AttendPart& y) {
    return x.on == y.on && x.tiles == y.tiles && x.chunk == y.chunk && x.splits == y.splits && x.bytes == y.bytes && x.waves == y.waves && x.few == y.few;
}

int main() {
    int64_t sizes = 0, bad = 0;
    for (int dim : {64, 128, 256})
        for (int kv : {1, 8, 32})
            for (int64_t group : {1, 8})
                for (int64_t seqs : {1, 2, 16, 24, 48, 3000})
                    for (int64_t tokens : {1, 2, 700})
                        for (int64_t length : {200, 4097, 32832, 60001, 131073, 1000000})
                            for (int64_t window : {1, 500, 4096, 8192, 16384, 50000, 65536, 200000, 0x7FFFFFFF})
                                for (int64_t sinks : {0, 4, 300}) {
                                    if (seqs * tokens * kv * group >= (1 << 26)) continue;
                                    ++sizes;
                                    const AttendShape a{dim, kv, seqs, seqs * tokens, kv * group, tokens, length};
                                    const AttendPlan p = attend_plan(window_shape(a, window, sinks));
                                    bool good = true;
                                    if (window + sinks >= length) {
                                        const AttendPlan q = attend_plan(a);
                                        good = same(p.rows, q.rows) && same(p.block, q.block);
                                    } else if (p.rows.on) {
                                        const int64_t keys = window + sinks + 128 < length ? window + sinks + 128 : length;
                                        const int64_t most = keys / 8 > KV_SERIAL ? keys / 8 : KV_SERIAL, groups = seqs * kv * p.rows.tiles;
                                        good = p.rows.chunk <= most + KV_STEP;
                                        good = good && (p.rows.splits <= (keys + KV_SERIAL - 1) / KV_SERIAL || groups * p.rows.splits <= 4096 + groups);
                                    }
                                    bad += good ? 0 : 1;
                                }
    printf("%lld %lld\n", (long long)sizes, (long long)bad);
    return 0;
}
