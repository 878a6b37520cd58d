// Every launch that the norm's backward vector kernel may be given, for every
// width up to past the widest it takes: enough shared memory for at least one
// row in flight, and for the sums that the CTA's rows leave at the end.
#include <cstdio>

#include "rms_norm_plan.h"

using namespace fp8q;

int main() {
    long plans = 0, bad = 0;
    for (int es = 2; es <= 4; es += 2)
        for (int streams = 2; streams <= 3; ++streams)
            for (int shift = 0; shift < 2; ++shift)
                for (int64_t n = 1; n <= 21000; ++n) {
                    const int epv = 16 / es;
                    if (!shift && n % epv) continue;
                    const BwdPlan b = bwd_plan(es, n, shift != 0, streams);
                    if (b.k == 0) continue;                      // another kernel takes it
                    ++plans;
                    const int64_t nvec = shift ? (n + 2 * epv - 2) / epv : n / epv;
                    const int64_t stage = int64_t{streams} * b.k * 16 * b.tpr * b.rows;
                    const bool ok = (b.k == 1 || b.k == 2 || b.k == 4 || b.k == 8) && b.k * epv <= 32 &&
                                    b.tpr % 32 == 0 && b.tpr > 0 && int64_t{b.tpr} * b.k >= nvec &&
                                    b.rows >= 1 && b.tpr * b.rows <= bwd_threads(b.k * epv) &&
                                    b.rows * ((b.tpr + 31) / 32) <= 32 &&
                                    (b.ctas == 1 || b.ctas == 2) &&
                                    b.stages >= 1 && b.stages <= kBwdMaxStages && b.smem == b.stages * stage &&
                                    int64_t{b.smem} * b.ctas <= kSmemPerSm &&
                                    b.smem >= 4 * n;             // the rows' sums, fp32
                    if (!ok && bad++ < 8)
                        std::printf("es %d n %lld shift %d streams %d: k %d tpr %d rows %d ctas %d stages %d smem %d\n", es,
                                    static_cast<long long>(n), shift, streams, b.k, b.tpr, b.rows, b.ctas, b.stages, b.smem);
                }
    if (bad) {
        std::printf("%ld of %ld launches bad\n", bad, plans);
        return 1;
    }
    std::printf("ok: %ld launches\n", plans);
    return 0;
}
