// gated_mm.cu -- the first half of a gated feed-forward block on fp8 operands,
// in one kernel: both projections, the activation and the product, and (fine
// scales) the cast of the result to 1 x 128 fp8 groups.
//
//   gate = A Wg^T, up = A Wu^T          A [M][K], Wg and Wu [I][K], fp8 codes
//   h    = gate * sigmoid(p(gate)) * up
//          silu: p(g) = g;  gelu (tanh form): p(g) = 2 sqrt(2/pi) (g + 0.044715 g^3)
// with per-tensor scales (gate = acc * fl(sa * sg)) or fine-grained ones (the
// fold of scaled_mm.cu).  gate and up stay fp32 until h is rounded, once.
//
// A tile is 128 columns of h: its B operand is 128 rows of Wg followed by the
// same 128 rows of Wu, so one M 128 x N 256 MMA per k step gives a thread's
// row of gate and of up side by side in TMEM and neither leaves the SM.  128
// columns are also one block of the weights' scales and one group of the
// output's.  Roles, ring, accumulators and bounded waits are those of
// scaled_mm.cu: warp 0 copies (TMA), warp 1 issues the MMAs, warps 2-9 fold,
// activate and store.
//
// Kernels and their forms:
//   gated_mm_kernel, persistent   128 x (128 + 128) tiles (kWide; kRagged where
//     the output's rows are not multiples of 32 bytes);
//   gated_mm_kernel, kCluster     when the tiles would fill at most half of
//     the SMs (few rows, a narrow I): the CTAs of a cluster split the k axis
//     of one tile, each leaves its sums in its shared memory, and each then
//     reads the parts of its share of the rows through distributed shared
//     memory, adds them in rank order and finishes those rows;
//   gated_mm_kernel, kDup2, kDup4 fine scales, at most 64 or 32 rows, clusters:
//     the A tile holds the rows 2 or 4 times over, so that every warp's TMEM
//     lanes hold them and each folds 1 / DUP of the columns;
//   gated_mm_kernel, kFew16, 32   fine scales, at most 16 or 32 rows, a tile
//     for each SM: the operands change places (the weights' 128 rows are the
//     MMA's M, the rows of A its N), so that no power goes into rows that there
//     are not, and a warp folds one column of gate or of up per lane;
//   gated_pair_kernel             per-tensor scales, many tiles: 256 rows on
//     CTA pairs (tcgen05.mma.cta_group::2), the even CTA loading the tile's
//     rows of Wg and the odd one its rows of Wu.
#include <atomic>
#include <cstring>
#include <type_traits>

#include "gated_device.cuh"
#include "mm_device.cuh"

namespace fp8q {
namespace mm {

constexpr int kHN = 128;                          // columns of h per tile
constexpr int kBN = 2 * kHN;                      // rows of B: gate's, then up's
constexpr int kATileBytes = BM * BK;
constexpr int kHalfBBytes = kHN * BK;
constexpr int kRing = 4;                          // stages (48 KB each)
constexpr int kAccs = kTmemCols / kBN;            // accumulators
constexpr int kHalf = kHN / 2;                    // columns of h one epilogue warp owns
constexpr int kOutQuant = 3;                      // OUT: kF32, kF16, kBF16 or codes
constexpr int kMaxSplit = 8;                      // CTAs of a cluster (the portable limit)
constexpr int kPartPitch = kBN + 4;               // floats of a row of exchanged sums (16 bytes off a bank period)
constexpr int kStagePitch = 17;                   // words of a row in an epilogue warp's staging area (an odd number)
constexpr int kStageBytes = 32 * kStagePitch * 4;
constexpr int kGatedSmemBytes = kRing * (kATileBytes + 2 * kHalfBBytes) + 1024 /* alignment */ + 256 /* barriers */ +
                                kEpiWarps * kStageBytes;
static_assert(BM * kPartPitch * 4 <= kRing * (kATileBytes + 2 * kHalfBBytes), "the exchange fits in the ring");

// What a launch of gated_mm_kernel is compiled for.  The persistent forms have
// every register of a fold thread in use, and code for the others would spill
// some of them: 4096 x 18432 x 7168 to fp8 takes 1080 us, and took 1200 in a
// build with 48 bytes of spills.
enum { kWide, kRagged, kCluster, kDup2, kDup4, kFew16, kFew32 };

struct GatedParams {
    int M, I, num_kb;
    int tiles_m, tiles_n;
    const float* sa;            // per-tensor: [1]; fine-grained: [M][ld]
    const float* sg;            // per-tensor: [1]; fine-grained: [ceil(I/128)][ld]
    const float* su;
    int ld;                     // k-blocks
    void* h;                    // [M][I] of the output type
    void* gu;                   // null or [M][2 I] of the output type: gate, then up (per-tensor scales)
    uint8_t* q;                 // [M][I] codes
    float* sinv;                // [M][ceil(I/128)]
    int groups;                 // ceil(I/128)
    int align_h, align_gu, align_q;   // 32, 16, 4 or 1: what bases and row pitches (and up's offset) are multiples of
    int fmt, rule;              // of the codes
    int act;
    int a_rows;                 // rows of A's TMA box
    int split;                  // CTAs that share a tile's k axis
    uint32_t* status;
    uint64_t wait_limit_ns;
};

// act(g) * u
__device__ __forceinline__ float silu_mul(float g, float u) {
    return __fmul_rn(__fmul_rn(g, sigmoid_approx(g)), u);
}
__device__ __forceinline__ float gelu_mul(float g, float u) {
    return __fmul_rn(__fmul_rn(g, sigmoid_approx(gelu_exponent(g))), u);
}
template <int N>
__device__ __forceinline__ void activate(const float (&g)[N], const float (&u)[N], int act, float (&h)[N]) {
    if (act == FP8Q_ACT_SILU) {
#pragma unroll
        for (int i = 0; i < N; ++i) h[i] = silu_mul(g[i], u[i]);
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i) h[i] = gelu_mul(g[i], u[i]);
    }
}

// N consecutive columns of one row (`row`: its first element), columns below `cols` only.
// align: the bytes that bases and row pitches are multiples of (32, 16 or less).
template <int YT, int N>
__device__ __forceinline__ void store_cols(typename OutT<YT>::T* row, int col0, int cols, int align, const float (&v)[N]) {
    constexpr int PER = YT == kF32 ? 8 : 16;         // elements of 32 bytes
#pragma unroll
    for (int c = 0; c < N / PER; ++c) {
        const int col = col0 + c * PER;
        if (align >= 16 && col + PER <= cols) {
            uint32_t w[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                if constexpr (YT == kF32) w[i] = __float_as_uint(v[c * PER + i]);
                else w[i] = pack2<YT>(v[c * PER + 2 * i], v[c * PER + 2 * i + 1]);
            }
            if (align >= 32) {
                st_v8(row + col, w);
            } else {
                st_v4(row + col, make_uint4(w[0], w[1], w[2], w[3]));
                st_v4(row + col + PER / 2, make_uint4(w[4], w[5], w[6], w[7]));
            }
        } else {
#pragma unroll
            for (int i = 0; i < PER; ++i) {
                if (col + i < cols) {
                    if constexpr (YT == kF32) row[col + i] = v[c * PER + i];
                    else if constexpr (YT == kF16) row[col + i] = __float2half_rn(v[c * PER + i]);
                    else row[col + i] = __float2bfloat16_rn(v[c * PER + i]);
                }
            }
        }
    }
}

// 16 columns of one row whose base and pitch are multiples of 32 bytes, so that a vector of its
// columns is whole or not there
template <int YT>
__device__ __forceinline__ void store_cols_wide(typename OutT<YT>::T* row, int col0, int cols, const float (&v)[16]) {
    constexpr int PER = YT == kF32 ? 8 : 16;         // elements of 32 bytes
#pragma unroll
    for (int c = 0; c < 16 / PER; ++c) {
        uint32_t w[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            if constexpr (YT == kF32) w[i] = __float_as_uint(v[c * PER + i]);
            else w[i] = pack2<YT>(v[c * PER + 2 * i], v[c * PER + 2 * i + 1]);
        }
        if (col0 + c * PER < cols) st_v8(row + col0 + c * PER, w);
    }
}
// 16 columns of a warp's 32 rows where no vector may be stored: through the
// warp's staging area, so that lanes then write neighbouring elements (half a
// warp a row) instead of one column of 32 rows.  row0: the warp's first row.
template <int YT>
__device__ __forceinline__ void store_cols_staged(typename OutT<YT>::T* base, int64_t pitch, int row0, int rows, int col0,
                                                  int cols, const float (&v)[16], float* stage) {
    const int lane = threadIdx.x & 31;
    __syncwarp();
#pragma unroll
    for (int i = 0; i < 16; ++i) stage[lane * kStagePitch + i] = v[i];
    __syncwarp();
    const int col = col0 + (lane & 15);
#pragma unroll 4
    for (int r = lane >> 4; r < 32; r += 2) {
        if (row0 + r < rows && col < cols) {
            const float f = stage[r * kStagePitch + (lane & 15)];
            typename OutT<YT>::T* d = base + (row0 + r) * pitch + col;
            if constexpr (YT == kF32) *d = f;
            else if constexpr (YT == kF16) *d = __float2half_rn(f);
            else *d = __float2bfloat16_rn(f);
        }
    }
}

// the largest magnitude of the first `cols` values
template <int N> __device__ __forceinline__ uint32_t absmax_below(const float (&v)[N], int cols) {
    uint32_t a = 0u;                                 // magnitude bits: a NaN stays the maximum
#pragma unroll
    for (int i = 0; i < N; ++i)
        if (i < cols) a = max(a, __float_as_uint(v[i]) & 0x7FFFFFFFu);
    return a;
}
// the per-token cast's scales of a group
__device__ __forceinline__ void group_scales(uint32_t amax_bits, int fmt, int rule, float& scale, float& sinv) {
    float amax = __uint_as_float(amax_bits);
    if (amax < 1e-4f) amax = 1e-4f;
    scale = fmt == kE4M3 ? scale_from_amax<kE4M3>(amax, rule) : scale_from_amax<kE5M2>(amax, rule);
    sinv = fmt == kE4M3 ? scale_inv_from_amax<kE4M3>(amax, rule) : scale_inv_from_amax<kE5M2>(amax, rule);
}
__device__ __forceinline__ uint32_t encode4(const float* v, float scale, int fmt) {
    const float a = __fmul_rn(v[0], scale), b = __fmul_rn(v[1], scale);
    const float c = __fmul_rn(v[2], scale), d = __fmul_rn(v[3], scale);
    return fmt == kE4M3 ? enc4<kE4M3>(a, b, c, d) : enc4<kE5M2>(a, b, c, d);
}

// ---------------------------------------------------------------------------
// one CTA per tile, or a cluster per tile that splits its k axis
// ---------------------------------------------------------------------------
__device__ __forceinline__ float4 ld_cluster16(uint32_t a) {
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0,%1,%2,%3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(a) : "memory");
    return v;
}

template <bool FINE, int OUT, int MODE>
__global__ void __launch_bounds__(kThreads, 1)
gated_mm_kernel(const __grid_constant__ CUtensorMap map_a, const __grid_constant__ CUtensorMap map_g,
                const __grid_constant__ CUtensorMap map_u, const GatedParams p, const uint32_t idesc) {
    constexpr int YT = OUT == kOutQuant ? kBF16 : OUT;
    constexpr int DUP = MODE == kDup4 ? 4 : MODE == kDup2 ? 2 : 1;
    constexpr bool kSingle = MODE >= kCluster;       // one tile per CTA or cluster, finished by exchange
    constexpr int kCols = kHalf / DUP;               // columns of gate, and of up, that a thread folds
    constexpr bool kFew = MODE >= kFew16;
    constexpr int kRows = MODE == kFew16 ? 16 : 32;  // kFew: rows of A (N)
    using T = typename OutT<YT>::T;
    extern __shared__ uint8_t smem_raw[];
    __shared__ int s_abort;
    __shared__ uint32_t s_amax[2][2][BM];            // [tile parity][column half][row]
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t* sA = smem;
    uint8_t* sB = smem + kRing * kATileBytes;
    uint64_t* bars = reinterpret_cast<uint64_t*>(sB + kRing * 2 * kHalfBBytes);
    float* stage_base = reinterpret_cast<float*>(reinterpret_cast<uint8_t*>(bars) + 256);
    // bars: full[kRing], empty[kRing], tfull[kAccs], tempty[kAccs], drain, amax[4]
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 2 * kRing + 2 * kAccs + 1 + 4);
    const uint32_t full0 = smem_u32(bars), empty0 = full0 + 8 * kRing;
    const uint32_t tfull0 = empty0 + 8 * kRing, tempty0 = tfull0 + 8 * kAccs;
    const uint32_t drain_bar = tempty0 + 8 * kAccs, amax0 = drain_bar + 8;
    volatile int* abort = &s_abort;

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        s_abort = 0;
        for (int s = 0; s < kRing; ++s) {
            mbar_init(full0 + 8 * s, 1);
            mbar_init(empty0 + 8 * s, 1);
        }
        for (int b = 0; b < kAccs; ++b) {
            mbar_init(tfull0 + 8 * b, 1);
            mbar_init(tempty0 + 8 * b, kEpiWarps);
        }
        mbar_init(drain_bar, 1);
        for (int i = 0; i < 4; ++i) mbar_init(amax0 + 8 * i, 2);    // the two warps of a quarter's rows
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        prefetch_tensormap(&map_a);
        prefetch_tensormap(&map_g);
        prefetch_tensormap(&map_u);
    }
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;"
                     :: "r"(smem_u32(tmem_slot)), "r"(kTmemCols) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem_base = *tmem_slot;

    pdl_begin();

    const int tiles = p.tiles_m * p.tiles_n;
    const int split = kSingle ? p.split : 1;
    const int rank = split > 1 ? static_cast<int>(pair::cta_rank()) : 0;
    const int first = blockIdx.x / split, stride = gridDim.x / split;
    // this CTA's k-blocks
    const int kb0 = kSingle ? static_cast<int>(static_cast<int64_t>(p.num_kb) * rank / split) : 0;
    const int kb1 = kSingle ? static_cast<int>(static_cast<int64_t>(p.num_kb) * (rank + 1) / split) : p.num_kb;
    uint32_t fail = 0;
    // epilogue: this thread's row, kCols columns of gate then as many of up, or (kFew) its column of
    // gate or of up for every row of A, as fp32 pairs
    float2 accum[kFew ? kRows / 2 : kCols];
    // its row and first column within the tile; a warp may read TMEM lanes 32 * (warp % 4) .. + 31
    auto row_of = [&] { return (DUP == 1 ? warp & 3 : DUP == 2 ? warp & 1 : 0) * 32 + lane; };
    auto col_of = [&] { return ((warp - 2) >> 2) * kHalf + (DUP == 1 ? 0 : DUP == 2 ? (warp & 3) >> 1 : warp & 3) * kCols; };

    if (warp == 0) {
        // ------------------------------------------------------------ producer
        if (lane == 0) {
            int stage = 0;
            uint32_t phase = 0;
            int64_t issued = 0;
            for (int t = first; t < tiles && !fail; t += stride) {
                int mb, nb;
                tile_coords(t, p.tiles_m, p.tiles_n, mb, nb);
                for (int kb = kb0; kb < kb1; ++kb) {
                    if (!mbar_wait(empty0 + 8 * stage, phase ^ 1u, abort, p.wait_limit_ns)) { fail = kTimeoutProducer; break; }
                    const uint32_t fb = full0 + 8 * stage;
                    mbar_arrive_expect_tx(fb, static_cast<uint32_t>((DUP * p.a_rows + kBN) * BK));
#pragma unroll
                    for (int d = 0; d < DUP; ++d)
                        tma_load_2d(smem_u32(sA + stage * kATileBytes + d * (kATileBytes / DUP)), &map_a, kb * BK, mb * BM, fb);
                    tma_load_2d(smem_u32(sB + stage * 2 * kHalfBBytes), &map_g, kb * BK, nb * kHN, fb);
                    tma_load_2d(smem_u32(sB + stage * 2 * kHalfBBytes + kHalfBBytes), &map_u, kb * BK, nb * kHN, fb);
                    ++issued;
                    if (++stage == kRing) { stage = 0; phase ^= 1u; }
                }
            }
            if (fail) *abort = 1;
            // every copy this thread issued has landed before the ring is reused or the CTA exits
            for (int s = 0; s < kRing; ++s) {
                const bool used = s < stage || issued >= kRing;
                if (used && !mbar_wait_drain(full0 + 8 * s, s < stage ? phase : phase ^ 1u, p.wait_limit_ns)) fail |= kTimeoutDrain;
            }
        }
    } else if (warp == 1) {
        // ------------------------------------------------------------ MMA issuer
        if (lane == 0) {
            int stage = 0;
            uint32_t phase = 0;
            int acc = 0;
            uint32_t acc_phase = 0;
            for (int t = first; t < tiles && !fail; t += stride) {
                if (kb0 == kb1) continue;
                for (int kb = kb0; kb < kb1; ++kb) {
                    if (FINE || kb == kb0) {
                        if (!mbar_wait(tempty0 + 8 * acc, acc_phase ^ 1u, abort, p.wait_limit_ns)) { fail = kTimeoutMma; break; }
                        tc_fence_after();
                    }
                    if (!mbar_wait(full0 + 8 * stage, phase, abort, p.wait_limit_ns)) { fail = kTimeoutMma; break; }
                    tc_fence_after();
                    const uint32_t a0 = smem_u32(sA + stage * kATileBytes), b0 = smem_u32(sB + stage * 2 * kHalfBBytes);
#pragma unroll
                    for (int j = 0; j < BK / 32; ++j) {
                        const uint32_t d = tmem_base + static_cast<uint32_t>(acc * kBN);
                        const uint64_t a = smem_desc_sw128(a0 + 32 * j), b = smem_desc_sw128(b0 + 32 * j);
                        if constexpr (kFew) {
                            mma_f8f6f4(d, b, a, idesc, j > 0);
                            mma_f8f6f4(d + kHN, smem_desc_sw128(b0 + kHalfBBytes + 32 * j), a, idesc, j > 0);
                        } else {
                            mma_f8f6f4(d, a, b, idesc, FINE ? (j > 0) : (kb > kb0 || j > 0));
                        }
                    }
                    mma_commit(empty0 + 8 * stage);
                    if (++stage == kRing) { stage = 0; phase ^= 1u; }
                    if (FINE || kb + 1 == kb1) {
                        mma_commit(tfull0 + 8 * acc);
                        if (++acc == kAccs) { acc = 0; acc_phase ^= 1u; }
                    }
                }
            }
            if (fail) *abort = 1;
            // every tensor-core operation this thread issued has completed
            mma_commit(drain_bar);
            if (!mbar_wait_drain(drain_bar, 0, p.wait_limit_ns)) fail |= kTimeoutDrain;
        }
    } else {
        // ------------------------------------------------------------ epilogue
        const int quarter = warp & 3, half = (warp - 2) >> 2;
        const int trow = row_of(), tcol = col_of();
        const uint32_t lane_addr = static_cast<uint32_t>(quarter * 32) << 16;
        float* stage_area = stage_base + (warp - 2) * (kStageBytes / 4);
        int acc = 0;
        uint32_t acc_phase = 0, amax_phase = 0;
        float sg_all = 0.0f, su_all = 0.0f;
        if (!FINE) {
            const float sa = __ldg(p.sa);
            sg_all = __fmul_rn(sa, __ldg(p.sg));
            su_all = __fmul_rn(sa, __ldg(p.su));
        }
        for (int t = first; t < tiles && !fail; t += stride) {
            int mb, nb;
            tile_coords(t, p.tiles_m, p.tiles_n, mb, nb);
            const int row = mb * BM + trow;
            const bool row_ok = row < p.M;
            const bool warp_rows_live = row - lane < p.M;
#pragma unroll
            for (int i = 0; i < (kFew ? kRows / 2 : kCols); ++i) accum[i] = make_float2(0.0f, 0.0f);
            if constexpr (kFew) {
                // lane l: the scale of row l times the block's; all of them go through the warp's
                // staging area, one k-block's while the one before may still be read
                const float* sb = (half == 0 ? p.sg : p.su) + static_cast<int64_t>(nb) * p.ld;
                const float* sa = p.sa + static_cast<int64_t>(lane < p.M ? lane : p.M - 1) * p.ld;
                float sa_next = 0.0f, sb_next = 0.0f;
                if (kb0 < kb1) {
                    sa_next = __ldg(sa + kb0);
                    sb_next = __ldg(sb + kb0);
                }
                for (int kb = kb0; kb < kb1; ++kb) {
                    float* slot = stage_area + (kb & 1) * kRows;
                    if (lane < kRows) slot[lane] = __fmul_rn(sa_next, sb_next);
                    if (kb + 1 < kb1) {
                        sa_next = __ldg(sa + kb + 1);
                        sb_next = __ldg(sb + kb + 1);
                    }
                    __syncwarp();
                    const bool ok = __all_sync(0xFFFFFFFFu, mbar_wait(tfull0 + 8 * acc, acc_phase, abort, p.wait_limit_ns));
                    if (!ok) { fail = kTimeoutEpilogue; break; }
                    tc_fence_after();
                    const uint32_t addr = tmem_base + lane_addr + static_cast<uint32_t>(acc * kBN + half * kHN);
                    uint32_t r[kRows];
                    if constexpr (kRows == 16) {
                        tmem_ld16_async(addr, r);
                        tmem_wait16(r);
                    } else {
                        tmem_ld32_async(addr, r);
                        tmem_wait32(r);
                    }
#pragma unroll
                    for (int i = 0; i < kRows / 4; ++i) {
                        const float4 sc = *reinterpret_cast<const float4*>(slot + 4 * i);
                        accum[2 * i] = __ffma2_rn(make_float2(__uint_as_float(r[4 * i]), __uint_as_float(r[4 * i + 1])),
                                                  make_float2(sc.x, sc.y), accum[2 * i]);
                        accum[2 * i + 1] = __ffma2_rn(make_float2(__uint_as_float(r[4 * i + 2]), __uint_as_float(r[4 * i + 3])),
                                                      make_float2(sc.z, sc.w), accum[2 * i + 1]);
                    }
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(tempty0 + 8 * acc);
                    if (++acc == kAccs) { acc = 0; acc_phase ^= 1u; }
                }
                if (fail) break;
            } else if constexpr (FINE) {
                // rows past M fold with the last row's scales; nothing reads their sums
                const float* sa_next = p.sa + static_cast<int64_t>(row_ok ? row : p.M - 1) * p.ld + kb0;
                const float* sg_next = p.sg + static_cast<int64_t>(nb) * p.ld + kb0;
                const float* su_next = p.su + static_cast<int64_t>(nb) * p.ld + kb0;
                float sa = 0.0f, sg = 0.0f, su = 0.0f;
                if (kb0 < kb1) {
                    sa = __ldg(sa_next);
                    sg = __ldg(sg_next);
                    su = __ldg(su_next);
                }
                for (int kb = kb0; kb < kb1; ++kb) {
                    const float g1 = __fmul_rn(sa, sg), u1 = __fmul_rn(sa, su);
                    if (kb + 1 < kb1) {
                        sa = __ldg(++sa_next);
                        sg = __ldg(++sg_next);
                        su = __ldg(++su_next);
                    }
                    const bool ok = __all_sync(0xFFFFFFFFu, mbar_wait(tfull0 + 8 * acc, acc_phase, abort, p.wait_limit_ns));
                    if (!ok) { fail = kTimeoutEpilogue; break; }
                    tc_fence_after();
                    if (warp_rows_live) {
                        // chunks of 16 columns of gate, then as many of up; the load of the
                        // next chunk is in flight while one is folded in (two in flight take the
                        // same time: the loads' throughput beside the MMAs is the bound)
                        constexpr int kChunks = kCols / 16;
                        const uint32_t addr = tmem_base + lane_addr + static_cast<uint32_t>(acc * kBN + tcol);
                        const float2 g2 = make_float2(g1, g1), u2 = make_float2(u1, u1);
                        uint32_t r0[16], r1[16];
                        tmem_ld16_async(addr, r0);
                        tmem_wait16(r0);
#pragma unroll
                        for (int c = 0; c < 2 * kChunks; ++c) {
                            uint32_t (&cur)[16] = (c & 1) ? r1 : r0;
                            uint32_t (&nxt)[16] = (c & 1) ? r0 : r1;
                            const int n = c + 1;
                            if (n < 2 * kChunks)
                                tmem_ld16_async(addr + static_cast<uint32_t>(n < kChunks ? 16 * n : kHN + 16 * (n - kChunks)), nxt);
#pragma unroll
                            for (int i = 0; i < 8; ++i)
                                accum[c * 8 + i] = __ffma2_rn(make_float2(__uint_as_float(cur[2 * i]),
                                                                          __uint_as_float(cur[2 * i + 1])),
                                                              c < kChunks ? g2 : u2, accum[c * 8 + i]);
                            if (n < 2 * kChunks) tmem_wait16(nxt);
                        }
                    }
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(tempty0 + 8 * acc);
                    if (++acc == kAccs) { acc = 0; acc_phase ^= 1u; }
                }
                if (fail) break;
            } else if (kb0 < kb1) {
                const bool ok = __all_sync(0xFFFFFFFFu, mbar_wait(tfull0 + 8 * acc, acc_phase, abort, p.wait_limit_ns));
                if (!ok) { fail = kTimeoutEpilogue; break; }
                tc_fence_after();
                if (warp_rows_live) {
                    const uint32_t addr = tmem_base + lane_addr + static_cast<uint32_t>(acc * kBN + tcol);
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        uint32_t r[32];
                        tmem_ld32_async(addr + static_cast<uint32_t>(c < 2 ? 32 * c : kHN + 32 * (c - 2)), r);
                        tmem_wait32(r);
                        const float s = c < 2 ? sg_all : su_all;
#pragma unroll
                        for (int i = 0; i < 16; ++i)
                            accum[c * 16 + i] = make_float2(__fmul_rn(__uint_as_float(r[2 * i]), s),
                                                            __fmul_rn(__uint_as_float(r[2 * i + 1]), s));
                    }
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(tempty0 + 8 * acc);
                if (++acc == kAccs) { acc = 0; acc_phase ^= 1u; }
            }
            if (kSingle || !warp_rows_live) continue;      // a single tile is finished below
            if constexpr (!kSingle) {
            const int col0 = nb * kHN + tcol;
            // 16 columns at a time, the activated values over gate's registers
#pragma unroll
            for (int c = 0; c < kHalf / 16; ++c) {
                float g[16], u[16], h[16];
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    g[2 * i] = accum[8 * c + i].x;
                    g[2 * i + 1] = accum[8 * c + i].y;
                    u[2 * i] = accum[kHalf / 2 + 8 * c + i].x;
                    u[2 * i + 1] = accum[kHalf / 2 + 8 * c + i].y;
                }
                activate(g, u, p.act, h);
                if constexpr (OUT == kOutQuant) {
#pragma unroll
                    for (int i = 0; i < 8; ++i) accum[8 * c + i] = make_float2(h[2 * i], h[2 * i + 1]);
                } else {
                    auto put = [&](void* out, int64_t pitch, int align, const float (&v)[16]) {
                        T* base = static_cast<T*>(out);
                        if constexpr (MODE == kWide) {
                            if (row_ok) store_cols_wide<YT>(base + row * pitch, col0 + 16 * c, p.I, v);
                        } else if (align >= 16) {
                            if (row_ok) store_cols<YT>(base + row * pitch, col0 + 16 * c, p.I, align, v);
                        } else {
                            store_cols_staged<YT>(base, pitch, row - lane, p.M, col0 + 16 * c, p.I, v, stage_area);
                        }
                    };
                    put(p.h, p.I, p.align_h, h);
                    if (!FINE && p.gu) {
                        put(p.gu, 2 * static_cast<int64_t>(p.I), p.align_gu, g);
                        put(static_cast<T*>(p.gu) + p.I, 2 * static_cast<int64_t>(p.I), p.align_gu, u);
                    }
                }
            }
            if constexpr (OUT == kOutQuant) {
                // the group's amax: this warp's half and, through shared memory, the other
                // warp's.  Two buffers in turn: a warp is at most one tile ahead.  Columns past I
                // are zeros times the scales, which is a NaN where those are infinite: left out.
                uint32_t mine = 0u;                      // magnitude bits: a NaN stays the maximum
                const int cols = p.I - col0;             // of this warp's half that there are
                if (cols >= kHalf) {
#pragma unroll
                    for (int i = 0; i < kHalf / 2; ++i)
                        mine = max(mine, max(__float_as_uint(accum[i].x) & 0x7FFFFFFFu, __float_as_uint(accum[i].y) & 0x7FFFFFFFu));
                } else {
#pragma unroll
                    for (int i = 0; i < kHalf / 2; ++i) {
                        if (2 * i < cols) mine = max(mine, __float_as_uint(accum[i].x) & 0x7FFFFFFFu);
                        if (2 * i + 1 < cols) mine = max(mine, __float_as_uint(accum[i].y) & 0x7FFFFFFFu);
                    }
                }
                s_amax[amax_phase][half][trow] = mine;
                __syncwarp();
                if (lane == 0) mbar_arrive(amax0 + 8 * quarter);
                const bool ok = __all_sync(0xFFFFFFFFu, mbar_wait(amax0 + 8 * quarter, amax_phase, abort, p.wait_limit_ns));
                if (!ok) { fail = kTimeoutEpilogue; break; }
                float scale, sinv;
                group_scales(max(mine, s_amax[amax_phase][half ^ 1][trow]), p.fmt, p.rule, scale, sinv);
                amax_phase ^= 1u;
                if (row_ok && half == 0) p.sinv[static_cast<int64_t>(row) * p.groups + nb] = sinv;
                auto word = [&](int i) {             // codes 4 i .. 4 i + 3
                    const float v[4] = {accum[2 * i].x, accum[2 * i].y, accum[2 * i + 1].x, accum[2 * i + 1].y};
                    return encode4(v, scale, p.fmt);
                };
                if constexpr (MODE == kWide) {
                    uint8_t* qrow = p.q + static_cast<int64_t>(row) * p.I + col0;
#pragma unroll
                    for (int c = 0; c < kHalf / 32; ++c) {
                        uint32_t w[8];
#pragma unroll
                        for (int i = 0; i < 8; ++i) w[i] = word(8 * c + i);
                        if (row_ok && col0 + 32 * c < p.I) st_v8(qrow + 32 * c, w);
                    }
                } else {
                    // as store_cols_staged: half a warp writes a row's 64 codes, as words where they
                    // are aligned, else 16 bytes at a time
                    uint32_t* area = reinterpret_cast<uint32_t*>(stage_area);
                    __syncwarp();
                    auto stage_words = [&](auto e4m3) {
#pragma unroll
                        for (int i = 0; i < kHalf / 4; ++i) {
                            const float a = __fmul_rn(accum[2 * i].x, scale), b = __fmul_rn(accum[2 * i].y, scale);
                            const float c = __fmul_rn(accum[2 * i + 1].x, scale), d = __fmul_rn(accum[2 * i + 1].y, scale);
                            const uint32_t w = decltype(e4m3)::value ? enc4<kE4M3>(a, b, c, d) : enc4<kE5M2>(a, b, c, d);
                            asm volatile("st.shared.b32 [%0], %1;" :: "r"(smem_u32(area + lane * kStagePitch + i)), "r"(w) : "memory");
                        }
                    };
                    if (p.fmt == kE4M3) stage_words(std::true_type());
                    else stage_words(std::false_type());
                    __syncwarp();
                    const int l = lane & 15, rows = p.M - (row - lane);       // of this warp
                    uint8_t* q0 = p.q + static_cast<int64_t>(row - lane) * p.I + col0;
                    if (p.align_q >= 4) {
#pragma unroll 8
                        for (int r = lane >> 4; r < 32; r += 2) {
                            const uint32_t w = area[r * kStagePitch + l];
                            if (r < rows && col0 + 4 * l < p.I) st_u32(q0 + static_cast<int64_t>(r) * p.I + 4 * l, w);
                        }
                    } else {
#pragma unroll 2
                        for (int r = lane >> 4; r < 32; r += 2) {
                            const uint8_t* codes = reinterpret_cast<const uint8_t*>(area + r * kStagePitch);
#pragma unroll
                            for (int c = 0; c < kHalf; c += 16)
                                if (r < rows && col0 + c + l < p.I) q0[static_cast<int64_t>(r) * p.I + c + l] = codes[c + l];
                        }
                    }
                }
            }
            }
        }
        if (fail && lane == 0) *abort = 1;
    }

    if constexpr (kSingle) {
        // The one tile of this CTA or cluster: rank r finishes rows [r * share, (r + 1) * share)
        // of the live ones.  A warp that has folded this CTA's last k-block has seen its last MMA
        // and, before that, its last copy complete, so the ring holds nothing and takes the sums,
        // row by row.
        int mb, nb;
        tile_coords(first, p.tiles_m, p.tiles_n, mb, nb);
        const int live = min(BM, p.M - mb * BM);
        const int share = (live + split - 1) / split;
        const int trow = row_of(), tcol = col_of();
        float* parts = reinterpret_cast<float*>(smem);
        if (warp >= 2 && !fail) {
            if constexpr (kFew) {
                float* dst = parts + ((warp - 2) >> 2) * kHN + (warp & 3) * 32 + lane;
#pragma unroll
                for (int r = 0; r < kRows; ++r)
                    if (r < live) dst[r * kPartPitch] = r % 2 ? accum[r / 2].y : accum[r / 2].x;
            } else if (trow < live) {
                float* dst = parts + trow * kPartPitch + tcol;
#pragma unroll
                for (int i = 0; i < kCols / 2; ++i)
                    *reinterpret_cast<float4*>(dst + (i < kCols / 4 ? 4 * i : kHN + 4 * (i - kCols / 4))) =
                        make_float4(accum[2 * i].x, accum[2 * i].y, accum[2 * i + 1].x, accum[2 * i + 1].y);
            }
        }
        __syncwarp();
        if (split > 1) pair::cluster_sync();
        else __syncthreads();
        // no CTA leaves while another may still read its sums: each warp arrives once it has read
        // all that it will, and waits at the end
        bool arrived = split == 1;
        const int mine = min(share, live - rank * share);         // rows of this rank
        for (int r = warp - 2; r < mine && warp >= 2; r += kEpiWarps) {
            // lane l: columns 4 l .. 4 l + 3, the ranks' sums added in rank order.  One row at a
            // time: two or four in flight made the code larger and the kernel slower (128 x 2048 x
            // 7168: 16.0 against 16.9 us; 1 x 2048 x 7168: 10.1 against 10.3).
            const uint32_t at = smem_u32(smem) + 4u * static_cast<uint32_t>((rank * share + r) * kPartPitch + 4 * lane);
            float4 a[kMaxSplit], b[kMaxSplit];
#pragma unroll
            for (int s = 0; s < kMaxSplit; ++s) {
                if (s < split) {
                    uint32_t src = at;
                    if (split > 1) asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(src) : "r"(at), "r"(s));
                    a[s] = ld_cluster16(src);
                    b[s] = ld_cluster16(src + 4u * kHN);
                }
            }
            float g[4] = {0.0f, 0.0f, 0.0f, 0.0f}, u[4] = {0.0f, 0.0f, 0.0f, 0.0f}, h[4];
#pragma unroll
            for (int s = 0; s < kMaxSplit; ++s) {
                if (s < split) {
                    g[0] += a[s].x; g[1] += a[s].y; g[2] += a[s].z; g[3] += a[s].w;
                    u[0] += b[s].x; u[1] += b[s].y; u[2] += b[s].z; u[3] += b[s].w;
                }
            }
            if (!arrived && r + kEpiWarps >= mine) {
                __syncwarp();
                // the operands: not before the loads have returned
                asm volatile("barrier.cluster.arrive.release.aligned;"
                             :: "f"(g[0]), "f"(g[1]), "f"(g[2]), "f"(g[3]), "f"(u[0]), "f"(u[1]), "f"(u[2]), "f"(u[3])
                             : "memory");
                arrived = true;
            }
            activate(g, u, p.act, h);
            const int64_t row = static_cast<int64_t>(mb) * BM + rank * share + r;
            const int col = nb * kHN + 4 * lane;
            if constexpr (OUT != kOutQuant) {
                auto put = [&](void* base, int64_t o, int align, const float (&v)[4]) {
                    T* d = static_cast<T*>(base) + o;
                    if (align >= 16 && col + 4 <= p.I) {
                        if constexpr (YT == kF32) st_v4(d, make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]),
                                                                      __float_as_uint(v[2]), __float_as_uint(v[3])));
                        else st_v2(d, make_uint2(pack2<YT>(v[0], v[1]), pack2<YT>(v[2], v[3])));
                        return;
                    }
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        if (col + i >= p.I) break;
                        if constexpr (YT == kF32) d[i] = v[i];
                        else if constexpr (YT == kF16) d[i] = __float2half_rn(v[i]);
                        else d[i] = __float2bfloat16_rn(v[i]);
                    }
                };
                put(p.h, row * p.I + col, p.align_h, h);
                if (!FINE && p.gu) {
                    put(p.gu, row * 2 * p.I + col, p.align_gu, g);
                    put(p.gu, row * 2 * p.I + p.I + col, p.align_gu, u);
                }
            } else {
                uint32_t amax = absmax_below(h, p.I - col);
#pragma unroll
                for (int off = 16; off > 0; off >>= 1) amax = max(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, off));
                float scale, sinv;
                group_scales(amax, p.fmt, p.rule, scale, sinv);
                if (lane == 0) p.sinv[row * p.groups + nb] = sinv;
                const uint32_t w = encode4(h, scale, p.fmt);
                uint8_t* d = p.q + row * p.I + col;
                if (p.align_q >= 4 && col + 4 <= p.I) {
                    st_u32(d, w);
                } else {
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        if (col + i < p.I) d[i] = static_cast<uint8_t>(w >> (8 * i));
                }
            }
        }
        if (!arrived) {
            __syncwarp();
            asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
        }
    }

    if (fail && p.status && lane == 0) atomicOr(p.status, fail);
    tc_fence_before();
    if (kSingle && split > 1) {
        __syncwarp();
        asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
    }
    __syncthreads();
    tc_fence_after();
    if (warp == 1) {
        __syncwarp();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" :: "r"(tmem_base), "r"(kTmemCols)
                     : "memory");
    }
}

// ---------------------------------------------------------------------------
// CTA pairs (per-tensor scales): 256 rows x 128 columns of h per pair, the
// protocol of scaled_mm.cu's pair kernel.  The pair's B operand is split by
// its rows: the even CTA holds the tile's 128 rows of Wg and the odd one its
// 128 rows of Wu, so columns 0..127 of the N 256 accumulator (128 rows of it
// in each CTA's TMEM) are gate and 128..255 up.
// ---------------------------------------------------------------------------
namespace pair {

constexpr int kGatedStages = 6;
constexpr int kGatedSmem = kGatedStages * (kATileBytes + kHalfBBytes) + 1024 + 256;

template <int YT>
__global__ void __launch_bounds__(kThreads, 1)
gated_pair_kernel(const __grid_constant__ CUtensorMap map_a, const __grid_constant__ CUtensorMap map_g,
                  const __grid_constant__ CUtensorMap map_u, const GatedParams p, const uint32_t idesc) {
    using T = typename OutT<YT>::T;
    extern __shared__ uint8_t smem_raw[];
    __shared__ int s_abort;
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t* sA = smem;
    uint8_t* sB = smem + kGatedStages * kATileBytes;
    uint64_t* bars = reinterpret_cast<uint64_t*>(sB + kGatedStages * kHalfBBytes);
    // bars: full[], empty[], tfull[kAccs], tempty[kAccs], drain
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 2 * kGatedStages + 2 * kAccs + 1);
    const uint32_t full0 = smem_u32(bars), empty0 = full0 + 8 * kGatedStages;
    const uint32_t tfull0 = empty0 + 8 * kGatedStages, tempty0 = tfull0 + 8 * kAccs;
    const uint32_t drain_bar = tempty0 + 8 * kAccs;
    volatile int* abort = &s_abort;

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = cta_rank();
    const bool leader = rank == 0;
    if (threadIdx.x == 0) {
        s_abort = 0;
        for (int s = 0; s < kGatedStages; ++s) {
            mbar_init(full0 + 8 * s, 1);           // the leader's expect-tx arrival, bytes of both CTAs
            mbar_init(empty0 + 8 * s, 1);          // the leader's commit
        }
        for (int b = 0; b < kAccs; ++b) {
            mbar_init(tfull0 + 8 * b, 1);                // the leader's commit
            mbar_init(tempty0 + 8 * b, 2 * kEpiWarps);   // every epilogue warp of both CTAs (leader's copy)
        }
        mbar_init(drain_bar, 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        prefetch_tensormap(&map_a);
        prefetch_tensormap(leader ? &map_g : &map_u);
    }
    __syncwarp();
    cluster_sync();                                // the peer's barriers exist before anything signals them
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;"
                     :: "r"(smem_u32(tmem_slot)), "r"(kTmemCols) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem_base = *tmem_slot;

    pdl_begin();

    const int tiles = p.tiles_m * p.tiles_n;
    const int pair_id = blockIdx.x >> 1, pairs = gridDim.x >> 1;
    uint32_t fail = 0;

    if (warp == 0) {
        // ------------------------------------------------------------ producer (both CTAs)
        if (lane == 0) {
            const CUtensorMap* map_b = leader ? &map_g : &map_u;
            int stage = 0;
            uint32_t phase = 0;
            int64_t issued = 0;
            for (int t = pair_id; t < tiles && !fail; t += pairs) {
                int mb, nb;
                tile_coords(t, p.tiles_m, p.tiles_n, mb, nb);
                for (int kb = 0; kb < p.num_kb; ++kb) {
                    if (!mbar_wait(empty0 + 8 * stage, phase ^ 1u, abort, p.wait_limit_ns)) { fail = kTimeoutProducer; break; }
                    const uint32_t fb = full0 + 8 * stage;
                    if (leader) mbar_arrive_expect_tx(fb, static_cast<uint32_t>(2 * (kATileBytes + kHalfBBytes)));
                    tma_load_2d_pair(smem_u32(sA + stage * kATileBytes), &map_a, kb * BK,
                                     mb * 2 * BM + static_cast<int>(rank) * BM, fb);
                    tma_load_2d_pair(smem_u32(sB + stage * kHalfBBytes), map_b, kb * BK, nb * kHN, fb);
                    ++issued;
                    if (++stage == kGatedStages) { stage = 0; phase ^= 1u; }
                }
            }
            if (fail) *abort = 1;
            // every stage this CTA filled has been consumed by the pair's MMAs
            for (int s = 0; s < kGatedStages; ++s) {
                const bool used = s < stage || issued >= kGatedStages;
                if (used && !mbar_wait_drain(empty0 + 8 * s, s < stage ? phase : phase ^ 1u, p.wait_limit_ns))
                    fail |= kTimeoutDrain;
            }
        }
    } else if (warp == 1) {
        // ------------------------------------------------------------ MMA issuer (leader only)
        if (lane == 0 && leader) {
            int stage = 0;
            uint32_t phase = 0;
            int acc = 0;
            uint32_t acc_phase = 0;
            for (int t = pair_id; t < tiles && !fail; t += pairs) {
                if (p.num_kb == 0) continue;
                if (!mbar_wait(tempty0 + 8 * acc, acc_phase ^ 1u, abort, p.wait_limit_ns)) { fail = kTimeoutMma; break; }
                tc_fence_after();
                for (int kb = 0; kb < p.num_kb; ++kb) {
                    if (!mbar_wait(full0 + 8 * stage, phase, abort, p.wait_limit_ns)) { fail = kTimeoutMma; break; }
                    tc_fence_after();
                    const uint32_t a0 = smem_u32(sA + stage * kATileBytes), b0 = smem_u32(sB + stage * kHalfBBytes);
#pragma unroll
                    for (int j = 0; j < BK / 32; ++j)
                        mma_pair(tmem_base + static_cast<uint32_t>(acc * kBN), smem_desc_sw128(a0 + 32 * j),
                                 smem_desc_sw128(b0 + 32 * j), idesc, (kb > 0 || j > 0));
                    commit_both(empty0 + 8 * stage);
                    if (++stage == kGatedStages) { stage = 0; phase ^= 1u; }
                }
                if (fail) break;
                commit_both(tfull0 + 8 * acc);
                if (++acc == kAccs) { acc = 0; acc_phase ^= 1u; }
            }
            if (fail) *abort = 1;
            commit_local(drain_bar);
            if (!mbar_wait_drain(drain_bar, 0, p.wait_limit_ns)) fail |= kTimeoutDrain;
        }
    } else {
        // ------------------------------------------------------------ epilogue (both CTAs)
        const int quarter = warp & 3;
        const int half = (warp - 2) >> 2;
        const uint32_t lane_addr = static_cast<uint32_t>(quarter * 32) << 16;
        int acc = 0;
        uint32_t acc_phase = 0;
        const float sa = __ldg(p.sa);
        const float sg = __fmul_rn(sa, __ldg(p.sg)), su = __fmul_rn(sa, __ldg(p.su));
        for (int t = pair_id; t < tiles && !fail; t += pairs) {
            int mb, nb;
            tile_coords(t, p.tiles_m, p.tiles_n, mb, nb);
            const int row = mb * 2 * BM + static_cast<int>(rank) * BM + quarter * 32 + lane;
            if (p.num_kb > 0) {
                const bool ok = __all_sync(0xFFFFFFFFu, mbar_wait(tfull0 + 8 * acc, acc_phase, abort, p.wait_limit_ns));
                if (!ok) { fail = kTimeoutEpilogue; break; }
                tc_fence_after();
            }
            const uint32_t addr = tmem_base + lane_addr + static_cast<uint32_t>(acc * kBN + half * kHalf);
#pragma unroll
            for (int c = 0; c < kHalf / 32; ++c) {
                uint32_t r0[32], r1[32];
                if (p.num_kb > 0) {
                    tmem_ld32_async(addr + 32 * c, r0);
                    tmem_ld32_async(addr + kHN + 32 * c, r1);
                    tmem_wait32(r0);
                    tmem_wait32(r1);
                } else {
#pragma unroll
                    for (int i = 0; i < 32; ++i) r0[i] = r1[i] = 0u;
                }
                const int col0 = nb * kHN + half * kHalf + 32 * c;
                float g[32], u[32], h[32];
#pragma unroll
                for (int i = 0; i < 32; ++i) {
                    g[i] = __fmul_rn(__uint_as_float(r0[i]), sg);
                    u[i] = __fmul_rn(__uint_as_float(r1[i]), su);
                }
                activate(g, u, p.act, h);
                if (row < p.M && col0 < p.I) {
                    store_cols<YT>(static_cast<T*>(p.h) + static_cast<int64_t>(row) * p.I, col0, p.I, p.align_h, h);
                    if (p.gu) {
                        T* grow = static_cast<T*>(p.gu) + static_cast<int64_t>(row) * 2 * p.I;
                        store_cols<YT>(grow, col0, p.I, p.align_gu, g);
                        store_cols<YT>(grow + p.I, col0, p.I, p.align_gu, u);
                    }
                }
            }
            if (p.num_kb > 0) {
                tc_fence_before();
                __syncwarp();
                if (lane == 0) arrive_leader(tempty0 + 8 * acc);
                if (++acc == kAccs) { acc = 0; acc_phase ^= 1u; }
            }
        }
        if (fail && lane == 0) *abort = 1;
    }

    if (fail && p.status && lane == 0) atomicOr(p.status, fail);
    // neither CTA leaves (or frees TMEM) while the other may still signal its
    // barriers or the pair's MMAs may still write its TMEM
    tc_fence_before();
    __syncthreads();
    cluster_sync();
    tc_fence_after();
    if (warp == 1) {
        __syncwarp();
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" :: "r"(tmem_base), "r"(kTmemCols)
                     : "memory");
    }
}

}  // namespace pair

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------
namespace {

// clusters of `size` CTAs of `kernel` that fit on the current device at once (asked once per device)
template <typename Kernel>
int clusters_that_fit(Kernel kernel, cudaLaunchConfig_t cfg, int size, std::atomic<int>* cache) {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) dev = -1;
    const bool cached = dev >= 0 && dev < 64;
    if (cached) {
        const int v = cache[dev].load(std::memory_order_relaxed);
        if (v > 0) return v;
    }
    cfg.gridDim = dim3(size);
    int fit = 0;
    if (cudaOccupancyMaxActiveClusters(&fit, kernel, &cfg) != cudaSuccess || fit < 1) fit = sm_count() / (size + 1);
    if (fit < 1) fit = 1;
    if (cached) cache[dev].store(fit, std::memory_order_relaxed);
    return fit;
}

template <bool FINE, int OUT, int MODE>
cudaError_t launch_gated_mode(const CUtensorMap& ma, const CUtensorMap& mg, const CUtensorMap& mu, GatedParams& p,
                              uint32_t idesc, cudaStream_t s) {
    auto kernel = gated_mm_kernel<FINE, OUT, MODE>;
    const cudaError_t e = allow_smem(kernel, kGatedSmemBytes);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = kGatedSmemBytes;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = FP8Q_PDL;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    attr[1].val.clusterDim.x = p.split;
    cfg.numAttrs = p.split > 1 ? 2 : 1;
    const int tiles = p.tiles_m * p.tiles_n;
    const int ctas = p.split > 1 ? tiles * p.split : (tiles < sm_count() ? tiles : sm_count());
    cfg.gridDim = dim3(static_cast<unsigned>(ctas));
    return cudaLaunchKernelEx(&cfg, kernel, ma, mg, mu, p, idesc);
}

// The form for few rows of fine-scaled operands.  Where clusters share tiles, a fold's time is the
// latency of its TMEM loads, and copies of the rows share those out among all warps (64 x 2048 x 7168:
// 13.2 us, 14.0 without; with the operands swapped 14.7, since an MMA of few columns takes as long as
// one of 256).  Where each SM has a tile, HBM sets the time and the power cap HBM's neighbours: with
// the operands swapped 1 x 18432 x 7168 runs for seconds at 44.5 us and 1957 MHz, with copies at 51.5
// and 1537.
enum class Few { kNo, kCopy2, kCopy4, kSwap16, kSwap32 };
Few few_rows(int64_t M, int64_t tiles_n) {
    if (M > 64 || tiles_n > sm_count()) return Few::kNo;
    const bool shared = 2 * tiles_n <= sm_count();
    if (M > 32) return shared ? Few::kCopy2 : Few::kNo;
    return shared ? Few::kCopy4 : M <= 16 ? Few::kSwap16 : Few::kSwap32;
}

// clusters of `size` CTAs of the kernel's shape that fit on the device at once
int split_fit(int size) {
    static std::atomic<int> fit[kMaxSplit + 1][64];
    auto kernel = gated_mm_kernel<true, kOutQuant, kCluster>;
    if (allow_smem(kernel, kGatedSmemBytes) != cudaSuccess) return 1;
    cudaLaunchConfig_t cfg = {};
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = kGatedSmemBytes;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = size;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return clusters_that_fit(kernel, cfg, size, fit[size]);
}

// Split the k axis over the CTAs of a cluster where that is estimated to be faster: a tile
// whose k axis one SM walks alone streams its weights at that SM's rate while others idle.
// In ns, from runs of 512 to 2048 columns over every split: a k-block takes 480 (fine scales),
// 380 (fine scales, DUP) or 330.  A cluster's barriers and its first rows take 1500, and each
// row that a CTA reads parts of 37 (14 bytes a clock through distributed shared memory).  An
// undivided tile's own epilogue takes 1200, or (DUP) 550 for each eight rows.
// Undivided and at the best split, us: 64 x 1024 x 1024 10.9 and 7.0 (4 CTAs), 100 x 1024 x 1024
// 8.4 and 8.9 (4), 128 x 512 x 2048 12.0 and 10.0 (8), 1 x 2048 x 7168 25.5 and 10.2 (6).
int choose_split(const GatedParams& p, int64_t per_kb, bool dup) {
    const int tiles = p.tiles_m * p.tiles_n, rows = p.M < BM ? p.M : BM;
    int split = 1;
    int64_t best = per_kb * p.num_kb + (dup ? 550 * ((rows + 7) / 8) : 1200);
    for (int c = 2; c <= kMaxSplit && c <= p.num_kb && static_cast<int64_t>(tiles) * c <= sm_count(); ++c) {
        const int64_t cost = per_kb * ((p.num_kb + c - 1) / c) + 1500 + 37LL * rows * (c - 1) / c;
        if (cost >= best || tiles > split_fit(c)) continue;
        best = cost;
        split = c;
    }
    return split;
}

template <bool FINE, int OUT>
cudaError_t launch_gated(const CUtensorMap& ma, const CUtensorMap& mg, const CUtensorMap& mu, GatedParams& p,
                         uint32_t idesc, cudaStream_t s) {
    if constexpr (FINE) {
        const Few few = few_rows(p.M, p.tiles_n);
        if (few != Few::kNo) {
            p.split = choose_split(p, 380, true);
            return few == Few::kSwap16 ? launch_gated_mode<FINE, OUT, kFew16>(ma, mg, mu, p, idesc, s)
                 : few == Few::kSwap32 ? launch_gated_mode<FINE, OUT, kFew32>(ma, mg, mu, p, idesc, s)
                 : few == Few::kCopy4 ? launch_gated_mode<FINE, OUT, kDup4>(ma, mg, mu, p, idesc, s)
                                      : launch_gated_mode<FINE, OUT, kDup2>(ma, mg, mu, p, idesc, s);
        }
    }
    p.split = choose_split(p, FINE ? 480 : 330, false);
    if (p.split > 1) return launch_gated_mode<FINE, OUT, kCluster>(ma, mg, mu, p, idesc, s);
    const bool wide = OUT == kOutQuant ? p.align_q >= 32 : p.align_h >= 32 && (!p.gu || p.align_gu >= 32);
    return wide ? launch_gated_mode<FINE, OUT, kWide>(ma, mg, mu, p, idesc, s)
                : launch_gated_mode<FINE, OUT, kRagged>(ma, mg, mu, p, idesc, s);
}

template <int YT>
cudaError_t launch_gated_pair(const CUtensorMap& ma, const CUtensorMap& mg, const CUtensorMap& mu, const GatedParams& p,
                              uint32_t idesc, cudaStream_t s) {
    auto kernel = pair::gated_pair_kernel<YT>;
    const cudaError_t e = allow_smem(kernel, pair::kGatedSmem);
    if (e != cudaSuccess) return e;
    static std::atomic<int> fit[64];
    cudaLaunchConfig_t cfg = {};
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = pair::kGatedSmem;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 2;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = FP8Q_PDL;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    const int tiles = p.tiles_m * p.tiles_n, most = clusters_that_fit(kernel, cfg, 2, fit);
    cfg.gridDim = dim3(static_cast<unsigned>(2 * (tiles < most ? tiles : most)));
    return cudaLaunchKernelEx(&cfg, kernel, ma, mg, mu, p, idesc);
}

}  // namespace
}  // namespace mm

fp8q_status launch_gated_mm(const GatedProblem& g, cudaStream_t s) {
    using namespace mm;
    const int64_t M = g.M, I = g.I, K = g.K;
    // CTA pairs (256-row tiles, per-tensor scales) under the rule of scaled_mm.cu:
    // when the tiles give two CTAs each to nine tenths of the SMs
    const int64_t tall_tiles = ((M + 2 * BM - 1) / (2 * BM)) * ((I + kHN - 1) / kHN);
    const bool pairs = !g.fine && M >= 2 * BM && tall_tiles * 20 >= 9LL * sm_count();
    // fewer than 128 rows: only they (rounded up to 16, a valid N of swapped operands) are loaded
    const Few few = g.fine ? few_rows(M, (I + kHN - 1) / kHN) : Few::kNo;
    const bool swapped = few == Few::kSwap16 || few == Few::kSwap32;
    const int a_rows = M >= BM ? BM : static_cast<int>((M + 15) / 16 * 16);
    CUtensorMap ma, mg, mu;
    memset(&ma, 0, sizeof(ma));
    memset(&mg, 0, sizeof(mg));
    memset(&mu, 0, sizeof(mu));
    if (K > 0 && (!make_map(&ma, g.a, M, K, a_rows) || !make_map(&mg, g.w_gate, I, K, kHN) ||
                  !make_map(&mu, g.w_up, I, K, kHN)))
        return FP8Q_ERR_CUDA;
    GatedParams p = {};
    p.M = static_cast<int>(M);
    p.I = static_cast<int>(I);
    p.num_kb = static_cast<int>((K + BK - 1) / BK);
    p.tiles_m = static_cast<int>((M + (pairs ? 2 * BM : BM) - 1) / (pairs ? 2 * BM : BM));
    p.tiles_n = static_cast<int>((I + kHN - 1) / kHN);
    p.sa = g.sa;
    p.sg = g.s_gate;
    p.su = g.s_up;
    p.ld = p.num_kb;
    p.h = g.h;
    p.gu = g.gate_up;
    p.q = g.q;
    p.sinv = g.sinv;
    p.groups = p.tiles_n;
    const int eb = g.yt == kF32 ? 4 : 2;
    auto align_of = [](const void* base, int64_t pitch) {
        const uint64_t bits = reinterpret_cast<uintptr_t>(base) | static_cast<uint64_t>(pitch);
        return bits % 32 == 0 ? 32 : bits % 16 == 0 ? 16 : bits % 4 == 0 ? 4 : 1;
    };
    p.align_h = align_of(g.h, I * eb);
    p.align_gu = align_of(g.gate_up, I * eb);
    p.align_q = align_of(g.q, I);
    p.fmt = g.fmt;
    p.rule = g.rule;
    p.act = g.act;
    p.a_rows = a_rows;
    p.status = g.status;
    p.wait_limit_ns = kWaitLimitNs;
    cudaError_t e;
    if (pairs) {
        // M 256 (128 rows per CTA), N 256
        const uint32_t idesc = (instr_desc(g.fa, g.fb, kBN) & ~(0x1Fu << 24)) | (static_cast<uint32_t>(2 * BM >> 4) << 24);
        e = g.yt == kF32 ? launch_gated_pair<kF32>(ma, mg, mu, p, idesc, s)
          : g.yt == kF16 ? launch_gated_pair<kF16>(ma, mg, mu, p, idesc, s)
                         : launch_gated_pair<kBF16>(ma, mg, mu, p, idesc, s);
        return cuda_status(e);
    }
    const uint32_t idesc = swapped ? instr_desc(g.fb, g.fa, a_rows) : instr_desc(g.fa, g.fb, kBN);
    if (g.q) e = launch_gated<true, kOutQuant>(ma, mg, mu, p, idesc, s);
    else if (g.fine)
        e = g.yt == kF32 ? launch_gated<true, kF32>(ma, mg, mu, p, idesc, s)
          : g.yt == kF16 ? launch_gated<true, kF16>(ma, mg, mu, p, idesc, s)
                         : launch_gated<true, kBF16>(ma, mg, mu, p, idesc, s);
    else
        e = g.yt == kF32 ? launch_gated<false, kF32>(ma, mg, mu, p, idesc, s)
          : g.yt == kF16 ? launch_gated<false, kF16>(ma, mg, mu, p, idesc, s)
                         : launch_gated<false, kBF16>(ma, mg, mu, p, idesc, s);
    return cuda_status(e);
}

}  // namespace fp8q
