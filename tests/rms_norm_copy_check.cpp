// Every 16-byte copy of the norm's backward kernel for rows that are no
// multiple of 16 bytes, for the widths that it takes: on a 16-byte boundary,
// inside the tensor, and with all that it holds of its row.
#include <cstdio>

#include "rms_norm_plan.h"

using namespace fp8q;

int main() {
    long copies = 0, bad = 0;
    for (int es = 2; es <= 4; es += 2)
        for (int n = 1; n <= 40; ++n) {
            if (bwd_plan(es, n, true, 2).k == 0) continue;                 // another kernel takes it
            for (int64_t m = 1; m <= 40; ++m)
                for (int64_t row = 0; row < m; ++row) {
                    const int epv = 16 / es, off = static_cast<int>(row * n % epv);
                    for (int at = -off; at < n; at += epv) {               // the vectors' first columns
                        const int64_t first = row * n + at;
                        const int bytes = copy_bytes(row, m, at, n, es);
                        const int64_t end = first + bytes / es, want = (at + epv < n ? at + epv : n) + row * n;
                        ++copies;
                        const bool ok = first >= 0 && first * es % 16 == 0 && bytes >= 0 && bytes <= 16 && bytes % es == 0 &&
                                        end <= m * n && end >= want;
                        if (!ok && bad++ < 8)
                            std::printf("es %d m %lld n %d row %lld column %d: %d bytes, %lld elements left\n", es,
                                        static_cast<long long>(m), n, static_cast<long long>(row), at, bytes,
                                        static_cast<long long>(m * n - first));
                    }
                }
        }
    if (bad) {
        std::printf("%ld of %ld copies bad\n", bad, copies);
        return 1;
    }
    std::printf("ok: %ld copies\n", copies);
    return 0;
}
