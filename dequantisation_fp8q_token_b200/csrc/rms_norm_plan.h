// rms_norm_plan.h -- how the norm's backward vector kernel (rms_norm.cu) is
// launched and how far its copies reach: plain arithmetic on sizes, apart from
// the kernel so that it can be swept without a GPU.
#pragma once

#include <stdint.h>

#ifdef __CUDACC__
#define FP8Q_HOST_DEVICE __host__ __device__ __forceinline__
#else
#define FP8Q_HOST_DEVICE inline
#endif

namespace fp8q {

constexpr int kBwdMaxStages = 4;
constexpr int kSmemPerSm = 222 * 1024;     // dynamic shared memory that CTAs of one SM may share here

// Threads of a CTA at most, and registers a thread that its bounds leave: up to
// 8 elements of a row a thread 512 and 64, up to 16 448 and 72 (two CTAs an
// SM), for more 640 and 96.
constexpr int bwd_threads(int elems) { return elems <= 8 ? 512 : elems <= 16 ? 448 : 640; }
constexpr int bwd_min_ctas(int elems) { return elems <= 16 ? 2 : 1; }
constexpr int bwd_regs(int elems) { return elems <= 8 ? 64 : elems <= 16 ? 72 : 96; }

struct BwdPlan {
    int k;          // 16-byte vectors a thread holds of a row; 0: no such launch
    int tpr;        // threads of a row
    int rows;       // rows of a CTA
    int ctas;       // CTAs an SM
    int stages;     // rows in flight
    int smem;       // bytes of a CTA: stages x streams x k x 16 x tpr x rows
};

// n elements of es bytes a row, in the tensors' own vectors (`shift`) or the
// row's; streams: tensors that are read (dy, r and perhaps dres).
inline BwdPlan bwd_plan(int es, int64_t n, bool shift, int streams) {
    const int epv = 16 / es, kmax = 32 / epv;              // 32 elements of a row per thread at most
    if (shift && n < epv) return {};       // a vector would hold more rows than two, and end past the tensor with any
    const int64_t nvec = shift ? (n + 2 * epv - 2) / epv : n / epv;
    for (int k = 1; k <= kmax; k *= 2) {
        const int threads = bwd_threads(k * epv);
        if (nvec > static_cast<int64_t>(threads) * k) continue;
        BwdPlan b = {};
        b.tpr = static_cast<int>(((nvec + k - 1) / k + 31) / 32 * 32);
        // as many rows as there are threads and, with one row of each in flight, memory for: fp32 rows
        // of 9217 to 10240 columns in three streams leave threads for two and memory for one
        const int row = streams * k * 16 * b.tpr;
        if (row > kSmemPerSm) return {};                   // no smaller with other k
        b.rows = threads / b.tpr < kSmemPerSm / row ? threads / b.tpr : kSmemPerSm / row;
        const int stage = row * b.rows;
        // two CTAs an SM where their registers and two stages each fit, else one
        b.ctas = 2 * bwd_regs(k * epv) * b.tpr * b.rows <= 65536 && kSmemPerSm / 2 >= 2 * stage ? 2 : 1;
        const int per_cta = kSmemPerSm / b.ctas;
        b.stages = per_cta / stage < kBwdMaxStages ? per_cta / stage : kBwdMaxStages;
        b.smem = b.stages * stage;
        b.k = k;
        return b;
    }
    return {};
}

// Bytes of the 16 at column `at` of a row that its tensor holds.  Rows are at
// least a vector long (bwd_plan), so only the last one's last vector ends past it.
FP8Q_HOST_DEVICE int copy_bytes(int64_t row, int64_t m, int at, int n, int es) {
    return row == m - 1 && at + 16 / es > n ? (n - at) * es : 16;
}

}  // namespace fp8q
