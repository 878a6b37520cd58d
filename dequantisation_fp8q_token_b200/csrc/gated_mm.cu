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
// Three kernels' worth of shapes:
//   gated_mm_kernel, no cluster   persistent, 128 x (128 + 128) tiles;
//   gated_mm_kernel, clusters     when the tiles would fill at most half of
//     the SMs (few rows, a narrow I): the CTAs of a cluster split the k axis
//     of one tile, then each sums the parts of its share of the rows through
//     distributed shared memory, in rank order, and finishes those rows;
//   gated_pair_kernel             per-tensor scales, many tiles: 256 rows on
//     CTA pairs (tcgen05.mma.cta_group::2), the even CTA loading the tile's
//     rows of Wg and the odd one its rows of Wu.
#include <cstring>

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
constexpr int kGatedSmemBytes = kRing * (kATileBytes + 2 * kHalfBBytes) + 1024 /* alignment */ + 256 /* barriers */;
static_assert(BM * kPartPitch * 4 <= kRing * (kATileBytes + 2 * kHalfBBytes), "the exchange fits in the ring");

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
    int align_h, align_gu, align_q;   // 32, 16 or 1: what bases and row pitches (and up's offset) are multiples of
    int fmt, rule;              // of the codes
    int act;
    int stage_tx;               // bytes one stage's TMA boxes bring
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

template <int N> __device__ __forceinline__ uint32_t absmax_of(const float (&v)[N]) {
    uint32_t a = 0u;                                 // magnitude bits: a NaN stays the maximum
#pragma unroll
    for (int i = 0; i < N; ++i) a = max(a, __float_as_uint(v[i]) & 0x7FFFFFFFu);
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
template <bool FINE, int OUT>
__global__ void __launch_bounds__(kThreads, 1)
gated_mm_kernel(const __grid_constant__ CUtensorMap map_a, const __grid_constant__ CUtensorMap map_g,
                const __grid_constant__ CUtensorMap map_u, const GatedParams p, const uint32_t idesc) {
    constexpr int YT = OUT == kOutQuant ? kBF16 : OUT;
    using T = typename OutT<YT>::T;
    extern __shared__ uint8_t smem_raw[];
    __shared__ int s_abort;
    __shared__ uint32_t s_amax[2][2][BM];            // [tile parity][column half][row]
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t* sA = smem;
    uint8_t* sB = smem + kRing * kATileBytes;
    uint64_t* bars = reinterpret_cast<uint64_t*>(sB + kRing * 2 * kHalfBBytes);
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
    const int rank = p.split > 1 ? static_cast<int>(pair::cta_rank()) : 0;
    const int first = blockIdx.x / p.split, stride = gridDim.x / p.split;
    // this CTA's k-blocks
    const int kb0 = static_cast<int>(static_cast<int64_t>(p.num_kb) * rank / p.split);
    const int kb1 = static_cast<int>(static_cast<int64_t>(p.num_kb) * (rank + 1) / p.split);
    uint32_t fail = 0;
    // epilogue: this thread's row, 64 columns of gate then 64 of up, as fp32 pairs
    float2 accum[kHalf];

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
                    mbar_arrive_expect_tx(fb, static_cast<uint32_t>(p.stage_tx));
                    tma_load_2d(smem_u32(sA + stage * kATileBytes), &map_a, kb * BK, mb * BM, fb);
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
                    for (int j = 0; j < BK / 32; ++j)
                        mma_f8f6f4(tmem_base + static_cast<uint32_t>(acc * kBN), smem_desc_sw128(a0 + 32 * j),
                                   smem_desc_sw128(b0 + 32 * j), idesc, FINE ? (j > 0) : (kb > kb0 || j > 0));
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
        const int quarter = warp & 3;                 // TMEM lanes this warp may read
        const int half = (warp - 2) >> 2;             // which 64 columns of h
        const uint32_t lane_addr = static_cast<uint32_t>(quarter * 32) << 16;
        int acc = 0;
        uint32_t acc_phase = 0, amax_phase = 0;
        float sg = 0.0f, su = 0.0f;
        if (!FINE) {
            const float sa = __ldg(p.sa);
            sg = __fmul_rn(sa, __ldg(p.sg));
            su = __fmul_rn(sa, __ldg(p.su));
        }
        for (int t = first; t < tiles && !fail; t += stride) {
            int mb, nb;
            tile_coords(t, p.tiles_m, p.tiles_n, mb, nb);
            const int trow = quarter * 32 + lane;
            const int row = mb * BM + trow;
            const bool row_ok = row < p.M;
            const bool warp_rows_live = row - lane < p.M;
#pragma unroll
            for (int i = 0; i < kHalf; ++i) accum[i] = make_float2(0.0f, 0.0f);
            if (FINE) {
                const float* sa_row = p.sa + static_cast<int64_t>(row_ok ? row : 0) * p.ld;
                const float* sg_row = p.sg + static_cast<int64_t>(nb) * p.ld;
                const float* su_row = p.su + static_cast<int64_t>(nb) * p.ld;
                float sa_next = 0.0f, sg_next = 0.0f, su_next = 0.0f;
                if (kb0 < kb1) {
                    sa_next = row_ok ? __ldg(sa_row + kb0) : 0.0f;
                    sg_next = __ldg(sg_row + kb0);
                    su_next = __ldg(su_row + kb0);
                }
                for (int kb = kb0; kb < kb1; ++kb) {
                    const float g1 = __fmul_rn(sa_next, sg_next), u1 = __fmul_rn(sa_next, su_next);
                    if (kb + 1 < kb1) {
                        sa_next = row_ok ? __ldg(sa_row + kb + 1) : 0.0f;
                        sg_next = __ldg(sg_row + kb + 1);
                        su_next = __ldg(su_row + kb + 1);
                    }
                    const bool ok = __all_sync(0xFFFFFFFFu, mbar_wait(tfull0 + 8 * acc, acc_phase, abort, p.wait_limit_ns));
                    if (!ok) { fail = kTimeoutEpilogue; break; }
                    tc_fence_after();
                    if (warp_rows_live) {
                        // four chunks of 16 columns of gate, then four of up; the load of the
                        // next chunk is in flight while one is folded in
                        const uint32_t addr = tmem_base + lane_addr + static_cast<uint32_t>(acc * kBN + half * kHalf);
                        const float2 g2 = make_float2(g1, g1), u2 = make_float2(u1, u1);
                        uint32_t r0[16], r1[16];
                        tmem_ld16_async(addr, r0);
                        tmem_wait16(r0);
#pragma unroll
                        for (int c = 0; c < 8; ++c) {
                            uint32_t (&cur)[16] = (c & 1) ? r1 : r0;
                            uint32_t (&nxt)[16] = (c & 1) ? r0 : r1;
                            const int n = c + 1;
                            if (n < 8) tmem_ld16_async(addr + static_cast<uint32_t>(n < 4 ? 16 * n : kHN + 16 * (n - 4)), nxt);
#pragma unroll
                            for (int i = 0; i < 8; ++i)
                                accum[c * 8 + i] = __ffma2_rn(make_float2(__uint_as_float(cur[2 * i]),
                                                                          __uint_as_float(cur[2 * i + 1])),
                                                              c < 4 ? g2 : u2, accum[c * 8 + i]);
                            if (n < 8) tmem_wait16(nxt);
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
                    const uint32_t addr = tmem_base + lane_addr + static_cast<uint32_t>(acc * kBN + half * kHalf);
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        uint32_t r[32];
                        tmem_ld32_async(addr + static_cast<uint32_t>(c < 2 ? 32 * c : kHN + 32 * (c - 2)), r);
                        tmem_wait32(r);
                        const float s = c < 2 ? sg : su;
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
            if (p.split > 1 || !warp_rows_live) continue;      // a cluster finishes its one tile below
            const int col0 = nb * kHN + half * kHalf;
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
                } else if (row_ok) {
                    store_cols<YT>(static_cast<T*>(p.h) + static_cast<int64_t>(row) * p.I, col0 + 16 * c, p.I, p.align_h, h);
                    if (!FINE && p.gu) {
                        T* grow = static_cast<T*>(p.gu) + static_cast<int64_t>(row) * 2 * p.I;
                        store_cols<YT>(grow, col0 + 16 * c, p.I, p.align_gu, g);
                        store_cols<YT>(grow + p.I, col0 + 16 * c, p.I, p.align_gu, u);
                    }
                }
            }
            if constexpr (OUT == kOutQuant) {
                // the group's amax: this warp's half and, through shared memory, the other
                // warp's.  Two buffers in turn: a warp is at most one tile ahead.
                uint32_t mine = 0u;                      // magnitude bits: a NaN stays the maximum
#pragma unroll
                for (int i = 0; i < kHalf / 2; ++i)
                    mine = max(mine, max(__float_as_uint(accum[i].x) & 0x7FFFFFFFu, __float_as_uint(accum[i].y) & 0x7FFFFFFFu));
                s_amax[amax_phase][half][trow] = mine;
                __syncwarp();
                if (lane == 0) mbar_arrive(amax0 + 8 * quarter);
                const bool ok = __all_sync(0xFFFFFFFFu, mbar_wait(amax0 + 8 * quarter, amax_phase, abort, p.wait_limit_ns));
                if (!ok) { fail = kTimeoutEpilogue; break; }
                float scale, sinv;
                group_scales(max(mine, s_amax[amax_phase][half ^ 1][trow]), p.fmt, p.rule, scale, sinv);
                amax_phase ^= 1u;
                if (row_ok) {
                    if (half == 0) p.sinv[static_cast<int64_t>(row) * p.groups + nb] = sinv;
                    uint8_t* qrow = p.q + static_cast<int64_t>(row) * p.I;
#pragma unroll
                    for (int c = 0; c < kHalf / 32; ++c) {
                        uint32_t w[8];
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            const float v[4] = {accum[16 * c + 2 * i].x, accum[16 * c + 2 * i].y,
                                                accum[16 * c + 2 * i + 1].x, accum[16 * c + 2 * i + 1].y};
                            w[i] = encode4(v, scale, p.fmt);
                        }
                        const int col = col0 + 32 * c;
                        if (p.align_q >= 32 && col + 32 <= p.I) {
                            st_v8(qrow + col, w);
                        } else if (p.align_q >= 16 && col + 32 <= p.I) {
                            st_v4(qrow + col, make_uint4(w[0], w[1], w[2], w[3]));
                            st_v4(qrow + col + 16, make_uint4(w[4], w[5], w[6], w[7]));
                        } else {
#pragma unroll
                            for (int i = 0; i < 32; ++i)
                                if (col + i < p.I) qrow[col + i] = static_cast<uint8_t>(w[i / 4] >> (8 * (i % 4)));
                        }
                    }
                }
            }
        }
        if (fail && lane == 0) *abort = 1;
    }

    if (p.split > 1) {
        // The cluster's one tile: rank r finishes rows [r * share, (r + 1) * share) of the live
        // ones.  Every CTA's copies and MMAs are done (drained above), so once all have arrived
        // the rings hold nothing: each thread writes its row's sums into the owner's ring.
        int mb, nb;
        tile_coords(first, p.tiles_m, p.tiles_n, mb, nb);
        const int live = min(BM, p.M - mb * BM);
        const int share = (live + p.split - 1) / p.split;
        __syncwarp();
        pair::cluster_sync();
        if (warp >= 2) {
            const int trow = (warp & 3) * 32 + lane, half = (warp - 2) >> 2;
            if (trow < live) {
                const int owner = trow / share;
                // [source rank][row of the owner's share][gate 0..127, up 0..127]
                const uint32_t local = smem_u32(smem) +
                    4u * static_cast<uint32_t>((rank * share + trow - owner * share) * kPartPitch + half * kHalf);
                uint32_t dst;
                asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(dst) : "r"(local), "r"(owner));
#pragma unroll
                for (int i = 0; i < kHalf / 2; ++i) {
                    const uint32_t at = dst + (i < kHalf / 4 ? 16u * i : 4u * kHN + 16u * (i - kHalf / 4));
                    asm volatile("st.shared::cluster.v4.f32 [%0], {%1,%2,%3,%4};"
                                 :: "r"(at), "f"(accum[2 * i].x), "f"(accum[2 * i].y), "f"(accum[2 * i + 1].x),
                                    "f"(accum[2 * i + 1].y) : "memory");
                }
            }
        }
        __syncwarp();
        pair::cluster_sync();
        if (warp >= 2) {
            const float* parts = reinterpret_cast<const float*>(smem);
            for (int r = warp - 2; r < share && rank * share + r < live; r += kEpiWarps) {
                const int row = mb * BM + rank * share + r;
                // lane l: columns 4 l .. 4 l + 3, the ranks' sums added in rank order
                float g[4] = {0.0f, 0.0f, 0.0f, 0.0f}, u[4] = {0.0f, 0.0f, 0.0f, 0.0f}, h[4];
                for (int s = 0; s < p.split; ++s) {
                    const float* src = parts + static_cast<int64_t>(s * share + r) * kPartPitch;
                    const float4 a = *reinterpret_cast<const float4*>(src + 4 * lane);
                    const float4 b = *reinterpret_cast<const float4*>(src + kHN + 4 * lane);
                    g[0] += a.x; g[1] += a.y; g[2] += a.z; g[3] += a.w;
                    u[0] += b.x; u[1] += b.y; u[2] += b.z; u[3] += b.w;
                }
                activate(g, u, p.act, h);
                const int col = nb * kHN + 4 * lane;
                if constexpr (OUT != kOutQuant) {
                    auto put = [&](void* base, int64_t at, const float (&v)[4]) {
                        T* d = static_cast<T*>(base) + at;
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            if (col + i >= p.I) break;
                            if constexpr (YT == kF32) d[i] = v[i];
                            else if constexpr (YT == kF16) d[i] = __float2half_rn(v[i]);
                            else d[i] = __float2bfloat16_rn(v[i]);
                        }
                    };
                    put(p.h, static_cast<int64_t>(row) * p.I + col, h);
                    if (!FINE && p.gu) {
                        put(p.gu, static_cast<int64_t>(row) * 2 * p.I + col, g);
                        put(p.gu, static_cast<int64_t>(row) * 2 * p.I + p.I + col, u);
                    }
                } else {
                    uint32_t a = absmax_of(h);
#pragma unroll
                    for (int off = 16; off > 0; off >>= 1) a = max(a, __shfl_xor_sync(0xFFFFFFFFu, a, off));
                    float scale, sinv;
                    group_scales(a, p.fmt, p.rule, scale, sinv);
                    if (lane == 0) p.sinv[static_cast<int64_t>(row) * p.groups + nb] = sinv;
                    const uint32_t w = encode4(h, scale, p.fmt);
                    uint8_t* d = p.q + static_cast<int64_t>(row) * p.I + col;
                    if (p.align_q >= 16 && col + 4 <= p.I) st_u32(d, w);
                    else
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            if (col + i < p.I) d[i] = static_cast<uint8_t>(w >> (8 * i));
                }
            }
        }
    }

    if (fail && p.status && lane == 0) atomicOr(p.status, fail);
    tc_fence_before();
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

template <bool FINE, int OUT>
cudaError_t launch_gated(const CUtensorMap& ma, const CUtensorMap& mg, const CUtensorMap& mu, GatedParams& p,
                         uint32_t idesc, cudaStream_t s) {
    auto kernel = gated_mm_kernel<FINE, OUT>;
    static std::atomic<bool> allowed[64];
    const cudaError_t e = allow_smem(kernel, kGatedSmemBytes, allowed);
    if (e != cudaSuccess) return e;
    static std::atomic<int> fit[4][64];
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
    const int tiles = p.tiles_m * p.tiles_n;
    // Split the k axis over as many CTAs as leave every tile its own cluster, at
    // least two k-blocks each: a tile whose k axis one SM walks alone streams its
    // weights at that SM's rate while the others idle.
    p.split = 1;
    cfg.numAttrs = 2;
    for (int c = kMaxSplit, i = 3; c > 1; c /= 2, --i) {
        if (p.num_kb < 2 * c || static_cast<int64_t>(tiles) * c > sm_count()) continue;
        attr[1].val.clusterDim.x = c;
        if (tiles > clusters_that_fit(kernel, cfg, c, fit[i])) continue;
        p.split = c;
        break;
    }
    if (p.split == 1) cfg.numAttrs = 1;
    const int ctas = p.split > 1 ? tiles * p.split : (tiles < sm_count() ? tiles : sm_count());
    cfg.gridDim = dim3(static_cast<unsigned>(ctas));
    return cudaLaunchKernelEx(&cfg, kernel, ma, mg, mu, p, idesc);
}

template <int YT>
cudaError_t launch_gated_pair(const CUtensorMap& ma, const CUtensorMap& mg, const CUtensorMap& mu, const GatedParams& p,
                              uint32_t idesc, cudaStream_t s) {
    auto kernel = pair::gated_pair_kernel<YT>;
    static std::atomic<bool> allowed[64];
    const cudaError_t e = allow_smem(kernel, pair::kGatedSmem, allowed);
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
    // fewer than 128 rows: only they (rounded up to 16) are loaded, see scaled_mm.cu
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
        return bits % 32 == 0 ? 32 : bits % 16 == 0 ? 16 : 1;
    };
    p.align_h = align_of(g.h, I * eb);
    p.align_gu = align_of(g.gate_up, I * eb);
    p.align_q = align_of(g.q, I);
    p.fmt = g.fmt;
    p.rule = g.rule;
    p.act = g.act;
    p.stage_tx = (a_rows + kBN) * BK;
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
    const uint32_t idesc = instr_desc(g.fa, g.fb, kBN);
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
