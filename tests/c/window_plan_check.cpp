// Host check of the launches of attention with a window (attend_plan.h) over many sizes: chunks hold whole steps and cover
// the window's keys, and every row that is split has a slot for its parts inside the planned workspace.  Prints
// "<sizes> <failures>".
#include <cstdio>
#include <initializer_list>

#include "attend_plan.h"

using namespace nf4;

int main() {
    int64_t sizes = 0, bad = 0;
    for (int dim : {64, 128, 256})
        for (int kv : {1, 8, 64, 4096})
            for (int64_t group : {1, 3, 8, 32})
                for (int64_t seqs : {1, 5, 24, 65535})
                    for (int64_t tokens : {seqs, 3 * seqs, 700 * seqs})
                        for (int64_t length : {int64_t(1), int64_t(33), int64_t(700), int64_t(1121), int64_t(4191), int64_t(131072), int64_t(1) << 30, int64_t(0x7FFFFFFF)}) {
                            const int64_t max_new = tokens / seqs;
                            if (tokens * kv * group >= (1 << 26) || seqs * kv > ATTEND_PAIRS) continue;
                            ++sizes;
                            const AttendPlan p = attend_plan(AttendShape{dim, kv, seqs, tokens, kv * group, max_new, length, true});
                            const AttendPart& q = p.rows;
                            const int64_t rows = max_new * group < KV_FEW ? max_new * group : KV_FEW;
                            bool good = p.rows.on || p.block.on;
                            if (q.on) {
                                good = good && q.chunk >= KV_STEP && q.chunk <= KV_WHOLE && q.chunk % KV_STEP == 0 && q.splits >= 1 && q.splits <= 65;
                                good = good && (int64_t)q.chunk * q.splits >= (length < KV_WHOLE ? length : KV_WHOLE);
                                const size_t need = (size_t)(seqs * kv * rows) * q.splits * (dim + 2) * 4;
                                good = good && (q.splits == 1 ? q.bytes == 0 : q.bytes >= need && q.bytes < need + 256);
                            }
                            bad += good ? 0 : 1;
                        }
    printf("%lld %lld\n", (long long)sizes, (long long)bad);
    return 0;
}
