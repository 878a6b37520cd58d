// rms_norm.cu -- root-mean-square norm with the residual's addition, its
// cast to 1 x G fp8 groups, and its backward pass.
//
//   r[i][c]  = T(x[i][c] + residual[i][c])          (r = x without a residual)
//   rstd[i]  = 1 / sqrt(mean_c r[i][c]^2 + eps)
//   y[i][c]  = r[i][c] * rstd[i] * w[c]              (fp32; stored as T, cast to fp8, or both)
//   backward, with t = dy * w and xhat = r * rstd:
//     dx[i][c] = rstd[i] * (t - xhat * mean_c(t * xhat)) + dres[i][c]
//     dw[c]    = sum_i dy[i][c] * xhat[i][c]
// The norm is that of the stored sum r, which is what the next layer adds to
// and what the backward pass is given, so the gradient is that of the value
// computed.  Every sum is fp32; y is rounded once, to T or to fp8.
#include "fp8q_device.cuh"
#include "fp8q_internal.h"

namespace fp8q {
namespace {

// ---------------------------------------------------------------------------
// vectors of VB bytes of type XT as fp32 values
// ---------------------------------------------------------------------------
template <int XT, int VB> struct VecOf { static constexpr int EPV = VB / ElemBytes<XT>::value; };

// Plain (coherent) loads: the sum may be written over x or the residual.
template <int VB>
__device__ __forceinline__ Vec<VB> load_vec_plain(const void* p) {
    Vec<VB> v;
    if constexpr (VB == 32)
        asm volatile("ld.global.L1::no_allocate.v8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                     : "=r"(v.w[0]), "=r"(v.w[1]), "=r"(v.w[2]), "=r"(v.w[3]), "=r"(v.w[4]), "=r"(v.w[5]),
                       "=r"(v.w[6]), "=r"(v.w[7]) : "l"(p));
    else
        asm volatile("ld.global.L1::no_allocate.v4.b32 {%0,%1,%2,%3}, [%4];"
                     : "=r"(v.w[0]), "=r"(v.w[1]), "=r"(v.w[2]), "=r"(v.w[3]) : "l"(p));
    return v;
}
template <int VB>
__device__ __forceinline__ void store_vec(void* p, const Vec<VB>& v) {
    if constexpr (VB == 32) st_v8(p, v.w);
    else st_v4(p, make_uint4(v.w[0], v.w[1], v.w[2], v.w[3]));
}
template <int XT, int VB>
__device__ __forceinline__ void unpack(const Vec<VB>& v, float (&f)[VecOf<XT, VB>::EPV]) {
#pragma unroll
    for (int i = 0; i < VB / 4; ++i) {
        if constexpr (XT == kF32) f[i] = __uint_as_float(v.w[i]);
        else widen2<XT>(v.w[i], f[2 * i], f[2 * i + 1]);
    }
}
template <int XT, int VB>
__device__ __forceinline__ Vec<VB> pack(const float (&f)[VecOf<XT, VB>::EPV]) {
    Vec<VB> v;
#pragma unroll
    for (int i = 0; i < VB / 4; ++i) {
        if constexpr (XT == kF32) v.w[i] = __float_as_uint(f[i]);
        else v.w[i] = pack2<XT>(f[2 * i], f[2 * i + 1]);
    }
    return v;
}
// N consecutive elements of the weight (16-byte aligned; kept in L1, every row reads them)
template <int WT, int N>
__device__ __forceinline__ void load_weight(const uint8_t* __restrict__ w, int64_t e, float (&f)[N]) {
    constexpr int WS = ElemBytes<WT>::value;
#pragma unroll
    for (int j = 0; j < N * WS / 16; ++j) {
        const uint4 t = __ldg(reinterpret_cast<const uint4*>(w + e * WS) + j);
        Vec<16> v;
        v.w[0] = t.x; v.w[1] = t.y; v.w[2] = t.z; v.w[3] = t.w;
        float g[VecOf<WT, 16>::EPV];
        unpack<WT, 16>(v, g);
#pragma unroll
        for (int i = 0; i < VecOf<WT, 16>::EPV; ++i) f[j * VecOf<WT, 16>::EPV + i] = g[i];
    }
}
template <int XT> __device__ __forceinline__ void elem_store(uint8_t* p, float f) {
    if constexpr (XT == kF32) *reinterpret_cast<float*>(p) = f;
    else if constexpr (XT == kF16) *reinterpret_cast<__half*>(p) = __float2half_rn(f);
    else *reinterpret_cast<__nv_bfloat16*>(p) = __float2bfloat16_rn(f);
}
// T(f) as an fp32 value
template <int XT> __device__ __forceinline__ float round_to(float f) {
    if constexpr (XT == kF32) return f;
    else if constexpr (XT == kF16) return __half2float(__float2half_rn(f));
    else return __bfloat162float(__float2bfloat16_rn(f));
}

__device__ __forceinline__ float rstd_of(float sumsq, int64_t n, float eps) {
    return __frcp_rn(__fsqrt_rn(__fadd_rn(__fdiv_rn(sumsq, static_cast<float>(n)), eps)));
}
__device__ __forceinline__ float warp_sum(float s) {
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, off);
    return s;
}
// Sum over the blockDim.x threads of this thread's row (a multiple of 32), in a
// fixed order; `sh` holds 32 floats per row.  One __syncthreads when a row
// spans several warps.
__device__ __forceinline__ float row_sum(float s, float* sh) {
    s = warp_sum(s);
    const int nw = blockDim.x >> 5;
    if (nw > 1) {
        float* mine = sh + 32 * threadIdx.y;
        if ((threadIdx.x & 31) == 0) mine[threadIdx.x >> 5] = s;
        __syncthreads();
        // every warp adds the partial sums itself: lane l takes partial l
        s = warp_sum((threadIdx.x & 31) < nw ? mine[threadIdx.x & 31] : 0.0f);
    }
    return s;
}

struct GroupScale { float scale, sinv; };
__device__ __forceinline__ GroupScale group_scale(uint32_t amax_bits, int fmt, int rule) {
    float amax = __uint_as_float(amax_bits);
    if (amax < 1e-4f) amax = 1e-4f;      // the per-token cast's clamp; a NaN amax stays NaN
    GroupScale g;
    g.scale = fmt == kE4M3 ? scale_from_amax<kE4M3>(amax, rule) : scale_from_amax<kE5M2>(amax, rule);
    g.sinv = fmt == kE4M3 ? scale_inv_from_amax<kE4M3>(amax, rule) : scale_inv_from_amax<kE5M2>(amax, rule);
    return g;
}

struct FwdParams {
    const uint8_t* x;
    const uint8_t* res;        // or null
    uint8_t* res_out;          // where the sum goes (null without a residual)
    const uint8_t* w;
    uint8_t* y;                // or null
    uint8_t* q;                // or null
    float* sinv;
    float* rstd;               // or null
    int64_t m, n;
    float eps;
    int group;                 // G
    int lanes;                 // vector kernel: lanes that hold one group
    int fmt, rule;
};

// ---------------------------------------------------------------------------
// Forward, vector kernel.  blockDim = (threads of a row, rows of the CTA); a
// row's vectors stay in registers from the load to the cast, so each input
// byte is read once.  Vector k of thread t covers elements
// (k * blockDim.x + t) * EPV ..: consecutive lanes hold consecutive vectors
// and blockDim.x is a multiple of 32, so a group of G elements is `lanes`
// consecutive lanes of one warp and its amax takes log2(lanes) shuffles.
// Bound by HBM (the arithmetic is ~10 operations an element).
// ---------------------------------------------------------------------------
template <int XT, int WT, int VB, int K>
__global__ void __launch_bounds__(1024)
rms_norm_vec_kernel(const FwdParams p) {
    constexpr int ES = ElemBytes<XT>::value;
    constexpr int EPV = VB / ES;
    __shared__ float sh[32 * 8];
    pdl_trigger();
    pdl_wait();
    const int64_t row = static_cast<int64_t>(blockIdx.x) * blockDim.y + threadIdx.y;
    const bool live = row < p.m;
    const int nvec = static_cast<int>(p.n / EPV);
    const int64_t base = row * p.n;
    Vec<VB> v[K], u[K];
#pragma unroll
    for (int k = 0; k < K; ++k) {
        const int i = threadIdx.x + k * blockDim.x;
        if (live && i < nvec) {
            v[k] = load_vec_plain<VB>(p.x + (base + static_cast<int64_t>(i) * EPV) * ES);
            if (p.res) u[k] = load_vec_plain<VB>(p.res + (base + static_cast<int64_t>(i) * EPV) * ES);
        }
    }
    float f[K][EPV];
    float s = 0.0f;
#pragma unroll
    for (int k = 0; k < K; ++k) {
        const int i = threadIdx.x + k * blockDim.x;
        if (live && i < nvec) {
            unpack<XT, VB>(v[k], f[k]);
            if (p.res) {
                float g[EPV];
                unpack<XT, VB>(u[k], g);
#pragma unroll
                for (int j = 0; j < EPV; ++j) f[k][j] = __fadd_rn(f[k][j], g[j]);
                v[k] = pack<XT, VB>(f[k]);
                store_vec<VB>(p.res_out + (base + static_cast<int64_t>(i) * EPV) * ES, v[k]);
                if constexpr (XT != kF32) unpack<XT, VB>(v[k], f[k]);   // the stored sum is what is normed
            }
#pragma unroll
            for (int j = 0; j < EPV; ++j) s = __fmaf_rn(f[k][j], f[k][j], s);
        } else {
#pragma unroll
            for (int j = 0; j < EPV; ++j) f[k][j] = 0.0f;
        }
    }
    s = row_sum(s, sh);
    const float rstd = rstd_of(s, p.n, p.eps);
    if (live && p.rstd && threadIdx.x == 0) p.rstd[row] = rstd;
#pragma unroll
    for (int k = 0; k < K; ++k) {
        const int i = threadIdx.x + k * blockDim.x;
        if (live && i < nvec) {
            float w[EPV];
            load_weight<WT, EPV>(p.w, static_cast<int64_t>(i) * EPV, w);
#pragma unroll
            for (int j = 0; j < EPV; ++j) f[k][j] = __fmul_rn(__fmul_rn(f[k][j], rstd), w[j]);
            if (p.y) store_vec<VB>(p.y + (base + static_cast<int64_t>(i) * EPV) * ES, pack<XT, VB>(f[k]));
        }
    }
    if (!p.q) return;
    const int64_t gpr = p.n / p.group;
#pragma unroll
    for (int k = 0; k < K; ++k) {
        const int i = threadIdx.x + k * blockDim.x;
        uint32_t a = 0u;          // magnitude bits: a NaN stays the maximum
#pragma unroll
        for (int j = 0; j < EPV; ++j) a = max(a, __float_as_uint(f[k][j]) & 0x7FFFFFFFu);
        for (int off = p.lanes >> 1; off > 0; off >>= 1) a = max(a, __shfl_xor_sync(0xFFFFFFFFu, a, off));
        if (live && i < nvec) {
            const GroupScale g = group_scale(a, p.fmt, p.rule);
            uint32_t c[EPV / 4];
#pragma unroll
            for (int j = 0; j < EPV / 4; ++j) {
                const float e0 = __fmul_rn(f[k][4 * j], g.scale), e1 = __fmul_rn(f[k][4 * j + 1], g.scale);
                const float e2 = __fmul_rn(f[k][4 * j + 2], g.scale), e3 = __fmul_rn(f[k][4 * j + 3], g.scale);
                c[j] = p.fmt == kE4M3 ? enc4<kE4M3>(e0, e1, e2, e3) : enc4<kE5M2>(e0, e1, e2, e3);
            }
            uint8_t* dst = p.q + base + static_cast<int64_t>(i) * EPV;
            if constexpr (EPV == 16) st_v4(dst, make_uint4(c[0], c[1], c[2], c[3]));
            else if constexpr (EPV == 8) st_v2(dst, make_uint2(c[0], c[1]));
            else st_u32(dst, c[0]);
            if ((i & (p.lanes - 1)) == 0) p.sinv[row * gpr + i / p.lanes] = g.sinv;
        }
    }
}

// Forward for every other layout (any width, any group that divides it,
// element-aligned pointers, rows too long for registers): one CTA per row,
// which reads the row again (from L2) for each of the three steps.  The sum
// is read back from res_out, so res_out may be x or the residual itself.
template <int XT, int WT>
__global__ void __launch_bounds__(256)
rms_norm_generic_kernel(const FwdParams p) {
    constexpr int ES = ElemBytes<XT>::value, WS = ElemBytes<WT>::value;
    __shared__ float sh[32];
    pdl_begin();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nw = blockDim.x >> 5;
    for (int64_t row = blockIdx.x; row < p.m; row += gridDim.x) {
        const int64_t base = row * p.n;
        float s = 0.0f;
        for (int64_t c = threadIdx.x; c < p.n; c += blockDim.x) {
            float f = elem_load<XT>(p.x + (base + c) * ES);
            if (p.res) {
                f = round_to<XT>(__fadd_rn(f, elem_load<XT>(p.res + (base + c) * ES)));
                elem_store<XT>(p.res_out + (base + c) * ES, f);
            }
            s = __fmaf_rn(f, f, s);
        }
        const float rstd = rstd_of(row_sum(s, sh), p.n, p.eps);
        __syncthreads();                   // res_out is complete, and sh may be written again
        if (p.rstd && threadIdx.x == 0) p.rstd[row] = rstd;
        const uint8_t* r = p.res ? p.res_out : p.x;
        auto value = [&](int64_t c) {
            return __fmul_rn(__fmul_rn(elem_load<XT>(r + (base + c) * ES), rstd), elem_load<WT>(p.w + c * WS));
        };
        if (!p.q) {
            for (int64_t c = threadIdx.x; c < p.n; c += blockDim.x) elem_store<XT>(p.y + (base + c) * ES, value(c));
            continue;
        }
        const int64_t gpr = p.n / p.group;
        for (int64_t g = warp; g < gpr; g += nw) {
            uint32_t a = 0u;
            for (int c = lane; c < p.group; c += 32)
                a = max(a, __float_as_uint(value(g * p.group + c)) & 0x7FFFFFFFu);
#pragma unroll
            for (int off = 16; off > 0; off >>= 1) a = max(a, __shfl_xor_sync(0xFFFFFFFFu, a, off));
            const GroupScale gs = group_scale(a, p.fmt, p.rule);
            if (lane == 0) p.sinv[row * gpr + g] = gs.sinv;
            for (int c = lane; c < p.group; c += 32) {
                const float f = value(g * p.group + c);
                const float e = __fmul_rn(f, gs.scale);
                const uint32_t code = p.fmt == kE4M3 ? enc2<kE4M3>(e, 0.0f) : enc2<kE5M2>(e, 0.0f);
                p.q[base + g * p.group + c] = static_cast<uint8_t>(code & 0xFFu);
                if (p.y) elem_store<XT>(p.y + (base + g * p.group + c) * ES, f);
            }
        }
    }
}

// ---------------------------------------------------------------------------
// Backward, vector kernel.  Each CTA walks rows blockIdx.x * R + ty, + grid *
// R, ...; every thread owns the same K vectors of each row, so its part of dw
// stays in registers until the end and goes to the CTA's row of `part`
// (summed in a fixed order by the second kernel: no atomics).  A thread
// copies its own 16-byte vectors of dy, r and dres into its own slots of
// shared memory (cp.async, `stages` rows ahead), so a row's loads are in
// flight while earlier rows are reduced, and no barrier guards the slots.
// ---------------------------------------------------------------------------
struct BwdParams {
    const uint8_t* dy;
    const uint8_t* r;
    const uint8_t* w;
    const float* rstd;
    const uint8_t* dres;       // or null
    uint8_t* dx;
    float* part;               // [gridDim.x][n], or null when dw is not wanted
    int64_t m, n;
    int stages;
};

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" :: "r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// wait until at most `pending` of this thread's groups are in flight
__device__ __forceinline__ void cp_async_wait(int pending) {
    if (pending >= 3) asm volatile("cp.async.wait_group 3;" ::: "memory");
    else if (pending == 2) asm volatile("cp.async.wait_group 2;" ::: "memory");
    else if (pending == 1) asm volatile("cp.async.wait_group 1;" ::: "memory");
    else asm volatile("cp.async.wait_group 0;" ::: "memory");
}
__device__ __forceinline__ Vec<16> ld_shared16(uint32_t a) {
    Vec<16> v;
    asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(v.w[0]), "=r"(v.w[1]), "=r"(v.w[2]), "=r"(v.w[3]) : "r"(a) : "memory");
    return v;
}

constexpr int kBwdMaxThreads = 640;
constexpr int kBwdMaxStages = 4;

template <int XT, int WT, int K>
__global__ void __launch_bounds__(kBwdMaxThreads)
rms_norm_bwd_vec_kernel(const BwdParams p) {
    constexpr int ES = ElemBytes<XT>::value;
    constexpr int EPV = 16 / ES;
    extern __shared__ __align__(16) uint8_t slots[];
    __shared__ float sh[2][32 * 8];
    pdl_trigger();
    pdl_wait();
    const int tpr = blockDim.x, rows = blockDim.y;
    const int tid = threadIdx.y * tpr + threadIdx.x, nthreads = tpr * rows;
    const int nvec = static_cast<int>(p.n / EPV);
    const int streams = p.dres ? 3 : 2;
    const int64_t step = static_cast<int64_t>(gridDim.x) * rows;
    const int64_t first = static_cast<int64_t>(blockIdx.x) * rows + threadIdx.y;
    const int64_t iters = p.m > static_cast<int64_t>(blockIdx.x) * rows
                              ? (p.m - static_cast<int64_t>(blockIdx.x) * rows + step - 1) / step : 0;
    const uint32_t slot0 = static_cast<uint32_t>(__cvta_generic_to_shared(slots)) + 16 * tid;
    // slot (stage, stream, k) of this thread
    auto slot = [&](int stage, int stream, int k) {
        return slot0 + static_cast<uint32_t>(16 * nthreads) * ((stage * streams + stream) * K + k);
    };
    auto fetch = [&](int64_t it, int stage) {
        const int64_t row = first + it * step;
        if (it < iters && row < p.m) {
#pragma unroll
            for (int k = 0; k < K; ++k) {
                const int i = threadIdx.x + k * tpr;
                if (i < nvec) {
                    const int64_t o = (row * p.n + static_cast<int64_t>(i) * EPV) * ES;
                    cp_async16(slot(stage, 0, k), p.dy + o);
                    cp_async16(slot(stage, 1, k), p.r + o);
                    if (streams == 3) cp_async16(slot(stage, 2, k), p.dres + o);
                }
            }
        }
        cp_async_commit();
    };
    for (int st = 0; st < p.stages; ++st) fetch(st, st);

    float w[K][EPV], acc[K][EPV];
#pragma unroll
    for (int k = 0; k < K; ++k) {
        const int i = threadIdx.x + k * tpr;
#pragma unroll
        for (int j = 0; j < EPV; ++j) acc[k][j] = w[k][j] = 0.0f;
        if (i < nvec) load_weight<WT, EPV>(p.w, static_cast<int64_t>(i) * EPV, w[k]);
    }
    const float inv_n = __fdiv_rn(1.0f, static_cast<float>(p.n));
    int stage = 0;
    for (int64_t it = 0; it < iters; ++it) {
        const int64_t row = first + it * step;
        const bool live = row < p.m;
        const float rstd = live ? __ldg(p.rstd + row) : 0.0f;
        cp_async_wait(p.stages - 1);
        float s = 0.0f;
#pragma unroll
        for (int k = 0; k < K; ++k) {
            if (live && static_cast<int>(threadIdx.x + k * tpr) < nvec) {
                float dy[EPV], r[EPV];
                unpack<XT, 16>(ld_shared16(slot(stage, 0, k)), dy);
                unpack<XT, 16>(ld_shared16(slot(stage, 1, k)), r);
#pragma unroll
                for (int j = 0; j < EPV; ++j) s = __fmaf_rn(__fmul_rn(dy[j], w[k][j]), __fmul_rn(r[j], rstd), s);
            }
        }
        // two sets of partial sums in turn: the next row's may be written while
        // a slow warp still reads this row's
        const float mean = __fmul_rn(row_sum(s, sh[it & 1]), inv_n);
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const int i = threadIdx.x + k * tpr;
            if (live && i < nvec) {
                float dy[EPV], r[EPV], o[EPV], d[EPV];
                unpack<XT, 16>(ld_shared16(slot(stage, 0, k)), dy);
                unpack<XT, 16>(ld_shared16(slot(stage, 1, k)), r);
                if (streams == 3) unpack<XT, 16>(ld_shared16(slot(stage, 2, k)), d);
#pragma unroll
                for (int j = 0; j < EPV; ++j) {
                    const float xhat = __fmul_rn(r[j], rstd);
                    acc[k][j] = __fmaf_rn(dy[j], xhat, acc[k][j]);
                    o[j] = __fmul_rn(rstd, __fmaf_rn(-xhat, mean, __fmul_rn(dy[j], w[k][j])));
                    if (streams == 3) o[j] = __fadd_rn(o[j], d[j]);
                }
                store_vec<16>(p.dx + (row * p.n + static_cast<int64_t>(i) * EPV) * ES, pack<XT, 16>(o));
            }
        }
        fetch(it + p.stages, stage);
        if (++stage == p.stages) stage = 0;
    }
    cp_async_wait(0);
    if (!p.part) return;
    // the CTA's rows of accumulators, added in row order through shared memory
    if (rows > 1) {
        float* sum = reinterpret_cast<float*>(slots);     // [nvec * EPV], free now
        for (int y = rows - 1; y >= 0; --y) {
            __syncthreads();
            if (threadIdx.y == y) {
#pragma unroll
                for (int k = 0; k < K; ++k) {
                    const int i = threadIdx.x + k * tpr;
                    if (i < nvec)
#pragma unroll
                        for (int j = 0; j < EPV; ++j) {
                            if (y < rows - 1) acc[k][j] += sum[i * EPV + j];
                            sum[i * EPV + j] = acc[k][j];
                        }
                }
            }
        }
        if (threadIdx.y != 0) return;
    }
#pragma unroll
    for (int k = 0; k < K; ++k) {
        const int i = threadIdx.x + k * tpr;
        if (i < nvec) {
            float* dst = p.part + static_cast<int64_t>(blockIdx.x) * p.n + static_cast<int64_t>(i) * EPV;
#pragma unroll
            for (int j = 0; j < EPV / 4; ++j)
                st_v4(dst + 4 * j, make_uint4(__float_as_uint(acc[k][4 * j]), __float_as_uint(acc[k][4 * j + 1]),
                                              __float_as_uint(acc[k][4 * j + 2]), __float_as_uint(acc[k][4 * j + 3])));
        }
    }
}

// dw[c] = WT(sum over p of part[p][c]): 32 columns per CTA, the rows of `part`
// split over 16 warps, each summed in ascending order, then the 16 sums in order
template <int WT>
__global__ void __launch_bounds__(512)
rms_norm_dw_kernel(const float* __restrict__ part, int parts, int64_t n, uint8_t* __restrict__ dw) {
    pdl_begin();
    __shared__ float sh[16][33];
    const int64_t c = static_cast<int64_t>(blockIdx.x) * 32 + threadIdx.x;
    float s = 0.0f;
    if (c < n)
        for (int i = threadIdx.y; i < parts; i += 16) s += part[static_cast<int64_t>(i) * n + c];
    sh[threadIdx.y][threadIdx.x] = s;
    __syncthreads();
    if (threadIdx.y == 0 && c < n) {
        for (int i = 1; i < 16; ++i) s += sh[i][threadIdx.x];
        elem_store<WT>(dw + c * ElemBytes<WT>::value, s);
    }
}

// Backward for every other layout: one CTA per row for dx ...
template <int XT, int WT>
__global__ void __launch_bounds__(256)
rms_norm_bwd_dx_kernel(const BwdParams p) {
    constexpr int ES = ElemBytes<XT>::value, WS = ElemBytes<WT>::value;
    __shared__ float sh[32];
    pdl_begin();
    const float inv_n = __fdiv_rn(1.0f, static_cast<float>(p.n));
    for (int64_t row = blockIdx.x; row < p.m; row += gridDim.x) {
        const int64_t base = row * p.n;
        const float rstd = __ldg(p.rstd + row);
        float s = 0.0f;
        for (int64_t c = threadIdx.x; c < p.n; c += blockDim.x)
            s = __fmaf_rn(__fmul_rn(elem_load<XT>(p.dy + (base + c) * ES), elem_load<WT>(p.w + c * WS)),
                          __fmul_rn(elem_load<XT>(p.r + (base + c) * ES), rstd), s);
        const float mean = __fmul_rn(row_sum(s, sh), inv_n);
        __syncthreads();
        for (int64_t c = threadIdx.x; c < p.n; c += blockDim.x) {
            const float t = __fmul_rn(elem_load<XT>(p.dy + (base + c) * ES), elem_load<WT>(p.w + c * WS));
            const float xhat = __fmul_rn(elem_load<XT>(p.r + (base + c) * ES), rstd);
            float o = __fmul_rn(rstd, __fmaf_rn(-xhat, mean, t));
            if (p.dres) o = __fadd_rn(o, elem_load<XT>(p.dres + (base + c) * ES));
            elem_store<XT>(p.dx + (base + c) * ES, o);
        }
    }
}
// ... and 256 columns x one slice of the rows per CTA for the partial sums of dw
template <int XT>
__global__ void __launch_bounds__(256)
rms_norm_bwd_part_kernel(const BwdParams p, int64_t rows_per_part) {
    constexpr int ES = ElemBytes<XT>::value;
    pdl_begin();
    const int64_t c = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
    if (c >= p.n) return;
    const int64_t r0 = static_cast<int64_t>(blockIdx.y) * rows_per_part;
    const int64_t r1 = r0 + rows_per_part < p.m ? r0 + rows_per_part : p.m;
    float s = 0.0f;
    for (int64_t row = r0; row < r1; ++row)
        s = __fmaf_rn(elem_load<XT>(p.dy + (row * p.n + c) * ES),
                      __fmul_rn(elem_load<XT>(p.r + (row * p.n + c) * ES), __ldg(p.rstd + row)), s);
    p.part[static_cast<int64_t>(blockIdx.y) * p.n + c] = s;
}

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------
bool aligned_to(const void* p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }
int round32(int64_t v) { return static_cast<int>((v + 31) / 32 * 32); }

template <int XT, int WT, int VB, int K>
fp8q_status run_fwd_vec(const FwdParams& p, cudaStream_t s) {
    constexpr int EPV = VB / ElemBytes<XT>::value;
    const int64_t nvec = p.n / EPV;
    const int tpr = round32((nvec + K - 1) / K);
    const int rows = tpr >= 256 ? 1 : (256 / tpr < 8 ? 256 / tpr : 8);
    const int64_t grid = (p.m + rows - 1) / rows;
    return cuda_status(launch_kernel(rms_norm_vec_kernel<XT, WT, VB, K>, dim3(static_cast<unsigned>(grid)),
                                     dim3(tpr, rows), s, p));
}

template <int XT, int WT>
fp8q_status run_fwd(const FwdParams& p0, cudaStream_t s) {
    constexpr int ES = ElemBytes<XT>::value;
    FwdParams p = p0;
    // vector bytes that the width, the pointers and the group allow
    int vb = 0;
    for (int b = 32; b >= 16 && !vb; b -= 16) {
        const int epv = b / ES;
        const int64_t nvec = p.n / epv;
        bool ok = (p.n * ES) % b == 0 && aligned_to(p.x, b) && aligned_to(p.res, b) && aligned_to(p.res_out, b) &&
                  aligned_to(p.y, b) && aligned_to(p.w, 16) && nvec <= 1024 * 4 && (b == 16 || ES == 4 || nvec <= 1024 * 2);
        if (ok && p.q) {
            const int lanes = p.group / epv;
            ok = p.group % epv == 0 && lanes >= 1 && lanes <= 32 && (lanes & (lanes - 1)) == 0 && aligned_to(p.q, epv);
            p.lanes = lanes;
        }
        if (ok) vb = b;
    }
    if (!vb) {
        const int64_t cap = static_cast<int64_t>(sm_count()) * 8;
        return cuda_status(launch_kernel(rms_norm_generic_kernel<XT, WT>,
                                         dim3(static_cast<unsigned>(p.m < cap ? p.m : cap)), dim3(256), s, p));
    }
    const int64_t nvec = p.n * ES / vb;
    if (vb == 32) {
        if (nvec <= 1024) return run_fwd_vec<XT, WT, 32, 1>(p, s);
        if (nvec <= 2048) return run_fwd_vec<XT, WT, 32, 2>(p, s);
        if constexpr (XT == kF32) return run_fwd_vec<XT, WT, 32, 4>(p, s);
        return FP8Q_ERR_CUDA;      // not reached: 16-bit rows of more vectors take 16-byte ones
    }
    if (nvec <= 256) return run_fwd_vec<XT, WT, 16, 1>(p, s);
    if (nvec <= 2048) return run_fwd_vec<XT, WT, 16, 2>(p, s);
    return run_fwd_vec<XT, WT, 16, 4>(p, s);
}

// rows of partial sums of dw that a call may write
int64_t bwd_parts(int64_t m) {
    const int64_t cap = 2LL * sm_count();
    return m < cap ? m : cap;
}

template <int WT>
fp8q_status run_dw(const float* part, int64_t parts, int64_t n, void* dw, cudaStream_t s) {
    return cuda_status(launch_kernel(rms_norm_dw_kernel<WT>, dim3(static_cast<unsigned>((n + 31) / 32)), dim3(32, 16), s,
                                     part, static_cast<int>(parts), n, static_cast<uint8_t*>(dw)));
}

constexpr int kSmemPerSm = 222 * 1024;     // dynamic shared memory that CTAs of one SM may share here

template <int XT, int WT, int K>
fp8q_status run_bwd_vec(const BwdParams& p0, int64_t* parts, cudaStream_t s) {
    constexpr int EPV = 16 / ElemBytes<XT>::value;
    BwdParams p = p0;
    const int64_t nvec = p.n / EPV;
    const int tpr = round32((nvec + K - 1) / K);
    const int rows = tpr >= 256 ? 1 : (256 / tpr < 8 ? 256 / tpr : 8);
    const int stage = (p.dres ? 3 : 2) * K * 16 * tpr * rows;
    // two CTAs on an SM where each can have two stages, else one
    const int per_cta = kSmemPerSm / 2 >= 2 * stage ? kSmemPerSm / 2 : kSmemPerSm;
    p.stages = per_cta / stage < kBwdMaxStages ? per_cta / stage : kBwdMaxStages;
    const int smem = p.stages * stage;
    auto kernel = rms_norm_bwd_vec_kernel<XT, WT, K>;
    static std::atomic<bool> allowed[64];
    const cudaError_t e = allow_smem(kernel, kSmemPerSm, allowed);
    if (e != cudaSuccess) return cuda_status(e);
    const int64_t cap = (per_cta == kSmemPerSm ? 1LL : 2LL) * sm_count(), want = (p.m + rows - 1) / rows;
    *parts = want < cap ? want : cap;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(*parts));
    cfg.blockDim = dim3(tpr, rows);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = FP8Q_PDL;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cuda_status(cudaLaunchKernelEx(&cfg, kernel, p));
}

template <int XT, int WT>
fp8q_status run_bwd(const BwdParams& p, void* dw, cudaStream_t s) {
    constexpr int ES = ElemBytes<XT>::value;
    constexpr int EPV = 16 / ES;
    constexpr int KMAX = 32 / EPV;         // 32 elements of a row per thread at most
    const int64_t nvec = p.n / EPV;
    const int streams = p.dres ? 3 : 2;
    const bool vec = (p.n * ES) % 16 == 0 && aligned_to(p.dy, 16) && aligned_to(p.r, 16) && aligned_to(p.dres, 16) &&
                     aligned_to(p.dx, 16) && aligned_to(p.w, 16) && aligned_to(p.part, 16) &&
                     nvec <= static_cast<int64_t>(kBwdMaxThreads) * KMAX &&
                     streams * KMAX * 16LL * round32((nvec + KMAX - 1) / KMAX) <= kSmemPerSm;
    int64_t parts = 0;
    fp8q_status st;
    if (p.m == 0) {
        st = FP8Q_OK;
    } else if (vec) {
        if (nvec <= 512) st = run_bwd_vec<XT, WT, 1>(p, &parts, s);
        else if (nvec <= 1024) st = run_bwd_vec<XT, WT, 2>(p, &parts, s);
        else if (nvec <= 2048 || KMAX == 4) st = run_bwd_vec<XT, WT, 4>(p, &parts, s);
        else st = run_bwd_vec<XT, WT, KMAX>(p, &parts, s);
    } else {
        const int64_t cap = static_cast<int64_t>(sm_count()) * 8;
        st = cuda_status(launch_kernel(rms_norm_bwd_dx_kernel<XT, WT>,
                                       dim3(static_cast<unsigned>(p.m < cap ? p.m : cap)), dim3(256), s, p));
        if (st == FP8Q_OK && p.part) {
            const int64_t want = bwd_parts(p.m), per = (p.m + want - 1) / want;
            parts = (p.m + per - 1) / per;
            st = cuda_status(launch_kernel(rms_norm_bwd_part_kernel<XT>,
                                           dim3(static_cast<unsigned>((p.n + 255) / 256), static_cast<unsigned>(parts)),
                                           dim3(256), s, p, per));
        }
    }
    if (st != FP8Q_OK || !dw) return st;
    return run_dw<WT>(p.part, parts, p.n, dw, s);
}

}  // namespace

size_t rms_norm_bwd_workspace(int64_t m, int64_t n) {
    return static_cast<size_t>(bwd_parts(m)) * static_cast<size_t>(n) * sizeof(float);
}

fp8q_status launch_rms_norm(const void* x, int xt, const void* res, void* res_out, const void* w, int wt, int64_t m,
                            int64_t n, float eps, int group, int fmt, int rule, void* y, uint8_t* q, float* sinv,
                            float* rstd, cudaStream_t s) {
    FwdParams p = {};
    p.x = static_cast<const uint8_t*>(x);
    p.res = static_cast<const uint8_t*>(res);
    p.res_out = static_cast<uint8_t*>(res_out);
    p.w = static_cast<const uint8_t*>(w);
    p.y = static_cast<uint8_t*>(y);
    p.q = q;
    p.sinv = sinv;
    p.rstd = rstd;
    p.m = m;
    p.n = n;
    p.eps = eps;
    p.group = group;
    p.lanes = 1;
    p.fmt = fmt;
    p.rule = rule;
    if (xt == kF32) return run_fwd<kF32, kF32>(p, s);
    if (xt == kF16) return wt == kF32 ? run_fwd<kF16, kF32>(p, s) : run_fwd<kF16, kF16>(p, s);
    return wt == kF32 ? run_fwd<kBF16, kF32>(p, s) : run_fwd<kBF16, kBF16>(p, s);
}

fp8q_status launch_rms_norm_bwd(const void* dy, const void* r, int xt, const void* w, int wt, const float* rstd,
                                const void* dres, int64_t m, int64_t n, void* dx, void* dw, float* part,
                                cudaStream_t s) {
    BwdParams p = {};
    p.dy = static_cast<const uint8_t*>(dy);
    p.r = static_cast<const uint8_t*>(r);
    p.w = static_cast<const uint8_t*>(w);
    p.rstd = rstd;
    p.dres = static_cast<const uint8_t*>(dres);
    p.dx = static_cast<uint8_t*>(dx);
    p.part = dw ? part : nullptr;
    p.m = m;
    p.n = n;
    if (xt == kF32) return run_bwd<kF32, kF32>(p, dw, s);
    if (xt == kF16) return wt == kF32 ? run_bwd<kF16, kF32>(p, dw, s) : run_bwd<kF16, kF16>(p, dw, s);
    return wt == kF32 ? run_bwd<kBF16, kF32>(p, dw, s) : run_bwd<kBF16, kBF16>(p, dw, s);
}

}  // namespace fp8q
