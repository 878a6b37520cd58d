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
#include "rms_norm_plan.h"

#include <type_traits>

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
// A vector's elements as pairs of fp32 values.  The kernels compute in packed
// fp32 operations: with 16-bit rows the instructions issued, not the bytes,
// are what a row's time goes into.
template <int XT, int VB>
__device__ __forceinline__ void unpack(const Vec<VB>& v, float2 (&f)[VecOf<XT, VB>::EPV / 2]) {
#pragma unroll
    for (int i = 0; i < VecOf<XT, VB>::EPV / 2; ++i) {
        if constexpr (XT == kF32) f[i] = make_float2(__uint_as_float(v.w[2 * i]), __uint_as_float(v.w[2 * i + 1]));
        else widen2<XT>(v.w[i], f[i].x, f[i].y);
    }
}
template <int XT, int VB>
__device__ __forceinline__ Vec<VB> pack(const float2 (&f)[VecOf<XT, VB>::EPV / 2]) {
    Vec<VB> v;
#pragma unroll
    for (int i = 0; i < VecOf<XT, VB>::EPV / 2; ++i) {
        if constexpr (XT == kF32) {
            v.w[2 * i] = __float_as_uint(f[i].x);
            v.w[2 * i + 1] = __float_as_uint(f[i].y);
        } else {
            v.w[i] = pack2<XT>(f[i].x, f[i].y);
        }
    }
    return v;
}
// N consecutive elements of the weight as stored (16-byte aligned; kept in L1,
// every row reads them), and their values
template <int WT, int N> struct Weights { uint4 v[N * ElemBytes<WT>::value / 16]; };
template <int WT, int N>
__device__ __forceinline__ Weights<WT, N> load_weights(const uint8_t* __restrict__ w, int e) {
    Weights<WT, N> r;
    const uint4* src = reinterpret_cast<const uint4*>(w + static_cast<int64_t>(e) * ElemBytes<WT>::value);
#pragma unroll
    for (int j = 0; j < N * ElemBytes<WT>::value / 16; ++j) r.v[j] = __ldg(src + j);
    return r;
}
// the same from any place and alignment; zeros for elements outside the row's 0 .. n - 1
template <int WT, int N>
__device__ __forceinline__ Weights<WT, N> load_weights_any(const uint8_t* w, int e, int n) {
    using Bits = std::conditional_t<ElemBytes<WT>::value == 4, uint32_t, uint16_t>;
    Weights<WT, N> r;
    uint32_t* out = reinterpret_cast<uint32_t*>(r.v);
    constexpr int PER = 4 / ElemBytes<WT>::value;         // elements of a register
#pragma unroll
    for (int j = 0; j < N / PER; ++j) {
        out[j] = 0u;
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const int c = e + j * PER + i;
            if (c >= 0 && c < n) out[j] |= static_cast<uint32_t>(reinterpret_cast<const Bits*>(w)[c]) << (16 * i);
        }
    }
    return r;
}
template <int WT, int N>
__device__ __forceinline__ void unpack_weights(const Weights<WT, N>& r, float2 (&f)[N / 2]) {
    constexpr int PER = VecOf<WT, 16>::EPV / 2;        // pairs of 16 bytes
#pragma unroll
    for (int j = 0; j < N / 2 / PER; ++j) {
        Vec<16> v;
        v.w[0] = r.v[j].x; v.w[1] = r.v[j].y; v.w[2] = r.v[j].z; v.w[3] = r.v[j].w;
        float2 g[PER];
        unpack<WT, 16>(v, g);
#pragma unroll
        for (int i = 0; i < PER; ++i) f[j * PER + i] = g[i];
    }
}
__device__ __forceinline__ float2 both(float v) { return make_float2(v, v); }
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

// 1 / sqrt(sumsq / n + eps): rsqrtf is within 2^-22.9, which is 2.2 roundings of fp32
__device__ __forceinline__ float rstd_of(float sumsq, float inv_n, float eps) {
    return rsqrtf(__fadd_rn(__fmul_rn(sumsq, inv_n), eps));
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
template <int FMT> __device__ __forceinline__ GroupScale group_scale(float amax, int rule) {
    if (amax < 1e-4f) amax = 1e-4f;      // the per-token cast's clamp; a NaN amax stays NaN
    return {scale_from_amax<FMT>(amax, rule), scale_inv_from_amax<FMT>(amax, rule)};
}
// the larger magnitude of the three (m >= 0), NaN where one is NaN
__device__ __forceinline__ float max_abs(float m, float2 v) {
    float d;
    asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(m), "f"(v.x), "f"(v.y));
    return d;
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
    float eps, inv_n;
    int group;                 // G
    int lanes_log2;            // vector kernel: lanes that hold one group
    int fmt, rule;
};

// ---------------------------------------------------------------------------
// Forward, vector kernel.  blockDim = (threads of a row, rows of the CTA); a
// row's vectors stay in registers from the load to the cast, so each input
// byte is read once.  Vector k of thread t covers elements
// (k * blockDim.x + t) * EPV ..: consecutive lanes hold consecutive vectors
// and blockDim.x is a multiple of 32, so a group of G elements is 2^lanes_log2
// consecutive lanes of one warp and its amax takes lanes_log2 shuffles.
// FMT: kE4M3 or kE5M2 (codes, and y if it is wanted too), or kNoCast (y only).
// bf16 4096 x 7168 with a residual: 36.3 us to y (99% of the measured copy
// bandwidth), 33.1 us to e4m3 (95%); without one, where half the bytes move,
// 21.4 us (84%) and 22.4 us (60%): there the instructions are the bound, of
// which the group's amax, its two divisions and the cast add half again (20
// against 14 million at that size).  A persistent form that kept rows in
// flight in a shared-memory ring took 44 and 59 us: its 16-byte vectors double
// the work per group.
// ---------------------------------------------------------------------------
constexpr int kNoCast = 2;

template <int XT, int WT, int VB, int K, int FMT>
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
    const int64_t at = base + static_cast<int64_t>(threadIdx.x) * EPV;      // of vector 0
    const int pitch = blockDim.x * EPV;                                     // from vector k to k + 1
    bool has[K];
#pragma unroll
    for (int k = 0; k < K; ++k) has[k] = live && static_cast<int>(threadIdx.x + k * blockDim.x) < nvec;
    Vec<VB> v[K], u[K];
    // one vector a thread: its weights are on their way too (more would not stay in registers)
    Weights<WT, EPV> wv;
#pragma unroll
    for (int k = 0; k < K; ++k) {
        if (has[k]) {
            v[k] = load_vec_plain<VB>(p.x + (at + k * pitch) * ES);
            if (p.res) u[k] = load_vec_plain<VB>(p.res + (at + k * pitch) * ES);
            if (K == 1) wv = load_weights<WT, EPV>(p.w, threadIdx.x * EPV);
        }
    }
    float2 f[K][EPV / 2];
    float2 sum = both(0.0f);
#pragma unroll
    for (int k = 0; k < K; ++k) {
        if (has[k]) {
            unpack<XT, VB>(v[k], f[k]);
            if (p.res) {
                float2 g[EPV / 2];
                unpack<XT, VB>(u[k], g);
#pragma unroll
                for (int j = 0; j < EPV / 2; ++j) f[k][j] = __fadd2_rn(f[k][j], g[j]);
                v[k] = pack<XT, VB>(f[k]);
                store_vec<VB>(p.res_out + (at + k * pitch) * ES, v[k]);
                if constexpr (XT != kF32) unpack<XT, VB>(v[k], f[k]);   // the stored sum is what is normed
            }
#pragma unroll
            for (int j = 0; j < EPV / 2; ++j) sum = __ffma2_rn(f[k][j], f[k][j], sum);
        } else {
#pragma unroll
            for (int j = 0; j < EPV / 2; ++j) f[k][j] = both(0.0f);
        }
    }
    const float rstd = rstd_of(row_sum(__fadd_rn(sum.x, sum.y), sh), p.inv_n, p.eps);
    if (live && p.rstd && threadIdx.x == 0) p.rstd[row] = rstd;
#pragma unroll
    for (int k = 0; k < K; ++k) {
        if (has[k]) {
            float2 w[EPV / 2];
            if (K > 1) wv = load_weights<WT, EPV>(p.w, threadIdx.x * EPV + k * pitch);
            unpack_weights<WT, EPV>(wv, w);
#pragma unroll
            for (int j = 0; j < EPV / 2; ++j) f[k][j] = __fmul2_rn(__fmul2_rn(f[k][j], both(rstd)), w[j]);
            if (FMT == kNoCast || p.y) store_vec<VB>(p.y + (at + k * pitch) * ES, pack<XT, VB>(f[k]));
        }
    }
    if constexpr (FMT != kNoCast) {
        const int64_t gpr = p.n / p.group;
#pragma unroll
        for (int k = 0; k < K; ++k) {
            float a = 0.0f;
#pragma unroll
            for (int j = 0; j < EPV / 2; ++j) a = max_abs(a, f[k][j]);
            uint32_t bits = __float_as_uint(a) & 0x7FFFFFFFu;        // a NaN stays the maximum
            for (int off = (1 << p.lanes_log2) >> 1; off > 0; off >>= 1)
                bits = max(bits, __shfl_xor_sync(0xFFFFFFFFu, bits, off));
            if (has[k]) {
                const GroupScale g = group_scale<FMT>(__uint_as_float(bits), p.rule);
                uint32_t c[EPV / 4];
#pragma unroll
                for (int j = 0; j < EPV / 4; ++j) {
                    const float2 lo = __fmul2_rn(f[k][2 * j], both(g.scale)), hi = __fmul2_rn(f[k][2 * j + 1], both(g.scale));
                    c[j] = enc4<FMT>(lo.x, lo.y, hi.x, hi.y);
                }
                uint8_t* dst = p.q + at + k * pitch;
                if constexpr (EPV == 16) st_v4(dst, make_uint4(c[0], c[1], c[2], c[3]));
                else if constexpr (EPV == 8) st_v2(dst, make_uint2(c[0], c[1]));
                else st_u32(dst, c[0]);
                const int i = threadIdx.x + k * blockDim.x;
                if ((i & ((1 << p.lanes_log2) - 1)) == 0) p.sinv[row * gpr + (i >> p.lanes_log2)] = g.sinv;
            }
        }
    }
}

// Forward to y for tensors that are not at 16-byte addresses, up to 8192
// columns: the vector kernel's plan with single elements (element k of thread
// t is k * blockDim.x + t), so a row is still read once and a thread's loads
// are in flight together.  Bound by the load and store instructions.  One
// element past a 16-byte address, the generic kernel's time after it: bf16 with
// a residual 16384 x 1001 45.5 us (112), 4096 x 2048 24.6 (50.3), 4096 x 7168
// 124 (159); 16384 x 100 without one 6.5 (29.0); fp32 600 x 2048 6.9 (10.3).
template <int XT, int WT, int K>
__global__ void __launch_bounds__(512)
rms_norm_elem_kernel(const FwdParams p) {
    constexpr int ES = ElemBytes<XT>::value, WS = ElemBytes<WT>::value;
    __shared__ float sh[32 * 8];
    pdl_begin();
    const int64_t row = static_cast<int64_t>(blockIdx.x) * blockDim.y + threadIdx.y;
    const bool live = row < p.m;
    const int64_t base = (live ? row : p.m - 1) * p.n;
    const int last = static_cast<int>(p.n) - 1, tpr = blockDim.x;
    float f[K];
    // every load unconditional, so that all are in flight: past the end, the last element again
#pragma unroll
    for (int k = 0; k < K; ++k) f[k] = elem_load<XT>(p.x + (base + min(static_cast<int>(threadIdx.x) + k * tpr, last)) * ES);
    if (p.res) {
        float g[K];
#pragma unroll
        for (int k = 0; k < K; ++k)
            g[k] = elem_load<XT>(p.res + (base + min(static_cast<int>(threadIdx.x) + k * tpr, last)) * ES);
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const int c = threadIdx.x + k * tpr;
            f[k] = round_to<XT>(__fadd_rn(f[k], g[k]));
            if (live && c <= last) elem_store<XT>(p.res_out + (base + c) * ES, f[k]);
        }
    }
    float s = 0.0f;
#pragma unroll
    for (int k = 0; k < K; ++k) {
        f[k] = static_cast<int>(threadIdx.x) + k * tpr <= last ? f[k] : 0.0f;
        s = __fmaf_rn(f[k], f[k], s);
    }
    const float rstd = rstd_of(row_sum(s, sh), p.inv_n, p.eps);
    if (live && p.rstd && threadIdx.x == 0) p.rstd[row] = rstd;
#pragma unroll
    for (int k = 0; k < K; ++k) {
        const int c = threadIdx.x + k * tpr;
        f[k] = __fmul_rn(__fmul_rn(f[k], rstd), elem_load<WT>(p.w + min(c, last) * WS));
        if (live && c <= last) elem_store<XT>(p.y + (base + c) * ES, f[k]);
    }
}

// Forward to y for rows that are no multiple of 16 bytes (and weights
// anywhere): the tensors' own aligned vectors, so a row starts `off` elements
// inside its first one.  A vector that holds elements of another row as well
// is read and written by elements, so no row touches another's.  The weights
// come one by one from L1.  With a residual bf16 4096 x 7169 60.0 us (0.60 of
// the copy bandwidth), 16384 x 1001 29.4, fp32 5060 x 5690 73.6 (0.95); single
// elements throughout took 122, 45.9 and 121.
template <int XT, int WT, int K>
__global__ void __launch_bounds__(1024)
rms_norm_shift_kernel(const FwdParams p) {
    constexpr int ES = ElemBytes<XT>::value;
    constexpr int EPV = 16 / ES;
    __shared__ float sh[32 * 8];
    pdl_begin();
    const int64_t row = static_cast<int64_t>(blockIdx.x) * blockDim.y + threadIdx.y;
    const bool live = row < p.m;
    const int64_t base = row * p.n;
    const int n = static_cast<int>(p.n), off = static_cast<int>(base & (EPV - 1));
    const int at = static_cast<int>(threadIdx.x) * EPV - off, pitch = blockDim.x * EPV;    // columns
    auto has = [&](int k) { return live && at + k * pitch < n; };
    auto edge = [&](int k) { return at + k * pitch < 0 || at + k * pitch + EPV > n; };
    auto load = [&](const uint8_t* t, int k) {
        if (!edge(k)) return load_vec_plain<16>(t + (base + at + k * pitch) * ES);
        const uint4 w = load_weights_any<XT, EPV>(t + base * ES, at + k * pitch, n).v[0];
        Vec<16> v;
        v.w[0] = w.x; v.w[1] = w.y; v.w[2] = w.z; v.w[3] = w.w;
        return v;
    };
    auto store = [&](uint8_t* t, int k, const Vec<16>& v) {
        uint8_t* dst = t + (base + at + k * pitch) * ES;
        if (!edge(k)) {
            store_vec<16>(dst, v);
            return;
        }
#pragma unroll
        for (int j = 0; j < EPV; ++j) {
            const int c = at + k * pitch + j;
            if (c < 0 || c >= n) continue;
            if constexpr (ES == 4) *reinterpret_cast<uint32_t*>(dst + 4 * j) = v.w[j];
            else *reinterpret_cast<uint16_t*>(dst + 2 * j) = static_cast<uint16_t>(v.w[j / 2] >> (16 * (j & 1)));
        }
    };
    Vec<16> v[K], u[K];
#pragma unroll
    for (int k = 0; k < K; ++k) {
        if (has(k)) {
            v[k] = load(p.x, k);
            if (p.res) u[k] = load(p.res, k);
        }
    }
    float2 f[K][EPV / 2];
    float2 sum = both(0.0f);
#pragma unroll
    for (int k = 0; k < K; ++k) {
#pragma unroll
        for (int j = 0; j < EPV / 2; ++j) f[k][j] = both(0.0f);
        if (has(k)) {
            unpack<XT, 16>(v[k], f[k]);
            if (p.res) {
                float2 g[EPV / 2];
                unpack<XT, 16>(u[k], g);
#pragma unroll
                for (int j = 0; j < EPV / 2; ++j) f[k][j] = __fadd2_rn(f[k][j], g[j]);
                v[k] = pack<XT, 16>(f[k]);
                store(p.res_out, k, v[k]);
                if constexpr (XT != kF32) unpack<XT, 16>(v[k], f[k]);   // the stored sum is what is normed
            }
#pragma unroll
            for (int j = 0; j < EPV / 2; ++j) sum = __ffma2_rn(f[k][j], f[k][j], sum);
        }
    }
    const float rstd = rstd_of(row_sum(__fadd_rn(sum.x, sum.y), sh), p.inv_n, p.eps);
    if (live && p.rstd && threadIdx.x == 0) p.rstd[row] = rstd;
#pragma unroll
    for (int k = 0; k < K; ++k) {
        if (has(k)) {
            float2 w[EPV / 2];
            unpack_weights<WT, EPV>(load_weights_any<WT, EPV>(p.w, at + k * pitch, n), w);
#pragma unroll
            for (int j = 0; j < EPV / 2; ++j) f[k][j] = __fmul2_rn(__fmul2_rn(f[k][j], both(rstd)), w[j]);
            store(p.y, k, pack<XT, 16>(f[k]));
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
        const float rstd = rstd_of(row_sum(s, sh), p.inv_n, p.eps);
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
            const float amax = __uint_as_float(a);
            const GroupScale gs = p.fmt == kE4M3 ? group_scale<kE4M3>(amax, p.rule) : group_scale<kE5M2>(amax, p.rule);
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
// bf16 4096 x 7168 with a residual: 40.3 us for dx (89% of the measured copy
// bandwidth), 44.0 with dw.
// SHIFT, for rows of 16 bytes and more that are no multiple of them (and weights anywhere): the
// tensors' own aligned vectors, so a row starts `off` elements inside its first
// one.  A thread's vectors lie at the same columns in each of its rows when the
// rows between them are a multiple of 16 bytes together, which the grid sees
// to; what a first or last vector holds of the neighbouring rows is set to
// zero in its slot, and such a vector's dx is stored by elements.  With a
// residual and dw fp16 4096 x 4001 39.8 us and 1600 x 18001 78.6, bf16 16384 x
// 1001 41.5, fp32 5060 x 5690 95.6 (73% of the copy bandwidth), against 96.3,
// 174, 69.6 and 199 with single elements in two passes; bf16 4096 x 7169 82.7
// (145), where the row's last vector makes a thread hold four (4096 x 7001
// 58.6).
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
    float inv_n;
    int stages;
};

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" :: "r"(dst), "l"(src) : "memory");
}
// the first `bytes` of the 16, zeros after them
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, int bytes) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" :: "r"(dst), "l"(src), "r"(bytes) : "memory");
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

template <int BYTES> __device__ __forceinline__ void st_shared_zero(uint32_t a) {
    if constexpr (BYTES == 4) asm volatile("st.shared.b32 [%0], %1;" :: "r"(a), "r"(0) : "memory");
    else asm volatile("st.shared.b16 [%0], %1;" :: "r"(a), "h"(static_cast<uint16_t>(0)) : "memory");
}

// elements of a row that a thread holds
template <int XT, int K> struct BwdElems { static constexpr int N = K * 16 / ElemBytes<XT>::value; };

template <int XT, int WT, int K, bool SHIFT>
__global__ void __launch_bounds__(bwd_threads(BwdElems<XT, K>::N), bwd_min_ctas(BwdElems<XT, K>::N))
rms_norm_bwd_vec_kernel(const BwdParams p) {
    constexpr int ES = ElemBytes<XT>::value;
    constexpr int EPV = 16 / ES;
    extern __shared__ __align__(16) uint8_t slots[];
    __shared__ float sh[2][32 * 16];
    pdl_trigger();
    pdl_wait();
    const int tpr = blockDim.x, rows = blockDim.y;
    const int tid = threadIdx.y * tpr + threadIdx.x;
    const int streams = p.dres ? 3 : 2;
    const int64_t step = static_cast<int64_t>(gridDim.x) * rows;
    const int64_t first = static_cast<int64_t>(blockIdx.x) * rows + threadIdx.y;
    const int n = static_cast<int>(p.n);
    // SHIFT: elements of the row's first vector that are the row's before it;
    // the same for all of a thread's rows, as step * n is a multiple of EPV
    const int off = SHIFT ? static_cast<int>(first * n & (EPV - 1)) : 0;
    const int nvec = SHIFT ? (n + off + EPV - 1) / EPV : n / EPV;
    // rows left for this CTA's first thread row, which has the most
    const int iters = p.m > first - threadIdx.y ? static_cast<int>((p.m - (first - threadIdx.y) + step - 1) / step) : 0;
    const uint32_t slot0 = static_cast<uint32_t>(__cvta_generic_to_shared(slots)) + 16 * tid;
    const uint32_t plane = 16 * tpr * rows;              // one vector of every thread
    // slot (stage, stream, k) of this thread
    auto slot = [&](int stage, int stream, int k) { return slot0 + plane * ((stage * streams + stream) * K + k); };
    const int at = static_cast<int>(threadIdx.x) * EPV - off;               // of vector 0 in a row
    const int pitch = tpr * EPV;
    bool in_row[K];
#pragma unroll
    for (int k = 0; k < K; ++k) in_row[k] = static_cast<int>(threadIdx.x + k * tpr) < nvec;
    // vector k holds elements of another row, or of none
    auto edge = [&](int k) { return SHIFT && (at + k * pitch < 0 || at + k * pitch + EPV > n); };
    auto inside = [&](int k, int j) { return at + k * pitch + j >= 0 && at + k * pitch + j < n; };
    bool edges = false;
#pragma unroll
    for (int k = 0; k < K; ++k) edges |= in_row[k] && edge(k);
    auto fetch = [&](int64_t row, int stage) {
        if (row < p.m) {
            const int64_t o = (row * p.n + at) * ES;
#pragma unroll
            for (int k = 0; k < K; ++k) {
                if (SHIFT && in_row[k]) {
                    const int bytes = copy_bytes(row, p.m, at + k * pitch, n, ES);
                    cp_async16(slot(stage, 0, k), p.dy + o + k * pitch * ES, bytes);
                    cp_async16(slot(stage, 1, k), p.r + o + k * pitch * ES, bytes);
                    if (streams == 3) cp_async16(slot(stage, 2, k), p.dres + o + k * pitch * ES, bytes);
                } else if (in_row[k]) {
                    cp_async16(slot(stage, 0, k), p.dy + o + k * pitch * ES);
                    cp_async16(slot(stage, 1, k), p.r + o + k * pitch * ES);
                    if (streams == 3) cp_async16(slot(stage, 2, k), p.dres + o + k * pitch * ES);
                }
            }
        }
        cp_async_commit();
    };
    for (int st = 0; st < p.stages; ++st) fetch(first + st * step, st);

    Weights<WT, EPV> wv[K];
    float2 acc[K][EPV / 2];
#pragma unroll
    for (int k = 0; k < K; ++k) {
#pragma unroll
        for (int j = 0; j < EPV / 2; ++j) acc[k][j] = both(0.0f);
        if constexpr (SHIFT) wv[k] = load_weights_any<WT, EPV>(p.w, at + k * pitch, n);
        else wv[k] = load_weights<WT, EPV>(p.w, in_row[k] ? at + k * pitch : 0);
    }
    int stage = 0;
    int64_t row = first;
    for (int it = 0; it < iters; ++it, row += step) {
        const bool live = row < p.m;
        const float rstd = live ? __ldg(p.rstd + row) : 0.0f;
        cp_async_wait(p.stages - 1);
        if (SHIFT && edges) {                  // zeros for what is not the row's
#pragma unroll
            for (int k = 0; k < K; ++k) {
                if (!in_row[k] || !edge(k)) continue;
                for (int j = 0; j < EPV; ++j) {
                    if (inside(k, j)) continue;
                    st_shared_zero<ES>(slot(stage, 0, k) + j * ES);
                    st_shared_zero<ES>(slot(stage, 1, k) + j * ES);
                }
            }
        }
        // sum of t * r, t = dy * w: the row's mean of t * xhat over n / rstd
        float2 sum = both(0.0f);
#pragma unroll
        for (int k = 0; k < K; ++k) {
            if (live && in_row[k]) {
                float2 dy[EPV / 2], r[EPV / 2], w[EPV / 2];
                unpack<XT, 16>(ld_shared16(slot(stage, 0, k)), dy);
                unpack<XT, 16>(ld_shared16(slot(stage, 1, k)), r);
                unpack_weights<WT, EPV>(wv[k], w);
#pragma unroll
                for (int j = 0; j < EPV / 2; ++j) sum = __ffma2_rn(__fmul2_rn(dy[j], w[j]), r[j], sum);
            }
        }
        // two sets of partial sums in turn: the next row's may be written while
        // a slow warp still reads this row's
        const float total = row_sum(__fadd_rn(sum.x, sum.y), sh[it & 1]);
        const float mean = __fmul_rn(__fmul_rn(total, p.inv_n), rstd);      // of t * xhat
#pragma unroll
        for (int k = 0; k < K; ++k) {
            if (live && in_row[k]) {
                float2 dy[EPV / 2], r[EPV / 2], w[EPV / 2], o[EPV / 2];
                if (streams == 3) {
                    unpack<XT, 16>(ld_shared16(slot(stage, 2, k)), o);
                } else {
#pragma unroll
                    for (int j = 0; j < EPV / 2; ++j) o[j] = both(0.0f);
                }
                unpack<XT, 16>(ld_shared16(slot(stage, 0, k)), dy);
                unpack<XT, 16>(ld_shared16(slot(stage, 1, k)), r);
                unpack_weights<WT, EPV>(wv[k], w);
#pragma unroll
                for (int j = 0; j < EPV / 2; ++j) {
                    const float2 xhat = __fmul2_rn(r[j], both(rstd));
                    acc[k][j] = __ffma2_rn(dy[j], xhat, acc[k][j]);
                    o[j] = __ffma2_rn(__ffma2_rn(xhat, both(-mean), __fmul2_rn(dy[j], w[j])), both(rstd), o[j]);
                }
                uint8_t* dx = p.dx + (row * p.n + at + k * pitch) * ES;
                if (edge(k)) {
#pragma unroll
                    for (int j = 0; j < EPV / 2; ++j) {
                        if (inside(k, 2 * j)) elem_store<XT>(dx + 2 * j * ES, o[j].x);
                        if (inside(k, 2 * j + 1)) elem_store<XT>(dx + (2 * j + 1) * ES, o[j].y);
                    }
                } else {
                    store_vec<16>(dx, pack<XT, 16>(o));
                }
            }
        }
        fetch(row + p.stages * step, stage);
        if (++stage == p.stages) stage = 0;
    }
    cp_async_wait(0);
    if (!p.part) return;
    if constexpr (SHIFT) {
        // thread rows start at different places: by columns, the threads' sums in row order
        float* total = reinterpret_cast<float*>(slots);           // [n], free after the barrier
        for (int y = rows - 1; y >= 0; --y) {
            __syncthreads();
            if (threadIdx.y == y) {
#pragma unroll
                for (int k = 0; k < K; ++k) {
                    if (!in_row[k]) continue;
                    float v[EPV];                                 // the loads first: none waits for a store
#pragma unroll
                    for (int j = 0; j < EPV; ++j)
                        v[j] = y < rows - 1 ? total[max(0, min(at + k * pitch + j, n - 1))] : 0.0f;
#pragma unroll
                    for (int j = 0; j < EPV; ++j) {
                        const float a = j & 1 ? acc[k][j / 2].y : acc[k][j / 2].x;
                        if (inside(k, j)) total[at + k * pitch + j] = __fadd_rn(a, v[j]);
                    }
                }
            }
        }
        __syncthreads();
        for (int c = tid; c < n; c += tpr * rows) p.part[static_cast<int64_t>(blockIdx.x) * n + c] = total[c];
        return;
    }
    // the CTA's rows of accumulators, added in row order through shared memory
    if (rows > 1) {
        float2* total = reinterpret_cast<float2*>(slots);     // [nvec * EPV / 2], free now
        for (int y = rows - 1; y >= 0; --y) {
            __syncthreads();
            if (threadIdx.y == y) {
#pragma unroll
                for (int k = 0; k < K; ++k) {
                    if (in_row[k])
#pragma unroll
                        for (int j = 0; j < EPV / 2; ++j) {
                            float2* t = total + (at + k * pitch) / 2 + j;
                            if (y < rows - 1) acc[k][j] = __fadd2_rn(acc[k][j], *t);
                            *t = acc[k][j];
                        }
                }
            }
        }
        if (threadIdx.y != 0) return;
    }
#pragma unroll
    for (int k = 0; k < K; ++k) {
        if (in_row[k]) {
            float* dst = p.part + static_cast<int64_t>(blockIdx.x) * p.n + at + k * pitch;
#pragma unroll
            for (int j = 0; j < EPV / 4; ++j)
                st_v4(dst + 4 * j, make_uint4(__float_as_uint(acc[k][2 * j].x), __float_as_uint(acc[k][2 * j].y),
                                              __float_as_uint(acc[k][2 * j + 1].x), __float_as_uint(acc[k][2 * j + 1].y)));
        }
    }
}

// dw[c] = WT(sum over p of part[p][c]), in a fixed order.  32 columns per CTA,
// four a thread, and 64 of the rows at a time, five loads of each thread in
// flight: all of the at most 2 * 160 rows of partial sums at once (2.4 us for
// 296 rows of 7168, against 3.2 us with single columns and 16 rows at a time).
// Widths that are no multiple of 4 take the single columns.
constexpr int kDwRows = 64, kDwLoads = 5;
template <int WT>
__global__ void __launch_bounds__(512)
rms_norm_dw_kernel(const float* __restrict__ part, int parts, int64_t n, uint8_t* __restrict__ dw) {
    pdl_begin();
    __shared__ float4 sh[kDwRows][9];
    const int64_t c = static_cast<int64_t>(blockIdx.x) * 32 + 4 * threadIdx.x;
    float4 s = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    if (c < n) {
        for (int i0 = threadIdx.y; i0 < parts; i0 += kDwRows * kDwLoads) {
            Vec<16> v[kDwLoads];
#pragma unroll
            for (int j = 0; j < kDwLoads; ++j) {
                const int i = i0 + kDwRows * j;
                if (i < parts) v[j] = load_vec_plain<16>(part + static_cast<int64_t>(i) * n + c);
                else v[j].w[0] = v[j].w[1] = v[j].w[2] = v[j].w[3] = 0u;
            }
#pragma unroll
            for (int j = 0; j < kDwLoads; ++j) {
                s.x += __uint_as_float(v[j].w[0]);
                s.y += __uint_as_float(v[j].w[1]);
                s.z += __uint_as_float(v[j].w[2]);
                s.w += __uint_as_float(v[j].w[3]);
            }
        }
    }
    sh[threadIdx.y][threadIdx.x] = s;
    for (int half = kDwRows / 2; half > 0; half /= 2) {
        __syncthreads();
        if (threadIdx.y < half) {
            const float4 t = sh[threadIdx.y + half][threadIdx.x];
            s.x += t.x; s.y += t.y; s.z += t.z; s.w += t.w;
            sh[threadIdx.y][threadIdx.x] = s;
        }
    }
    if (threadIdx.y == 0 && c < n) {
        const float v[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) elem_store<WT>(dw + (c + j) * ElemBytes<WT>::value, v[j]);
    }
}
constexpr int kDwSingles = 10;
template <int WT>
__global__ void __launch_bounds__(512)
rms_norm_dw_generic_kernel(const float* part, int parts, int64_t n, uint8_t* __restrict__ dw) {
    pdl_begin();
    __shared__ float sh[16][33];
    const int64_t c = static_cast<int64_t>(blockIdx.x) * 32 + threadIdx.x;
    float s = 0.0f;
    if (c < n) {
        for (int i0 = threadIdx.y; i0 < parts; i0 += 16 * kDwSingles) {
            float v[kDwSingles];
#pragma unroll
            for (int j = 0; j < kDwSingles; ++j)                // all in flight: past the end, the last again
                v[j] = part[static_cast<int64_t>(min(i0 + 16 * j, parts - 1)) * n + c];
#pragma unroll
            for (int j = 0; j < kDwSingles; ++j)
                if (i0 + 16 * j < parts) s += v[j];
        }
    }
    sh[threadIdx.y][threadIdx.x] = s;
    __syncthreads();
    if (threadIdx.y == 0 && c < n) {
        for (int i = 1; i < 16; ++i) s += sh[i][threadIdx.x];
        elem_store<WT>(dw + c * ElemBytes<WT>::value, s);
    }
}

// Backward, dx, for tensors that are not at 16-byte addresses, up to 4096
// columns, and for rows narrower than a vector: as the forward's, one element at
// a time, dy and r read once.  One element past a 16-byte address, bf16 with a
// residual, the kernel below after it: 16384 x 1001 48.4 us (67.2), 4096 x 2048
// 24.6 (31.1); at the widest, 4096 x 4096, it loses: 75.0 (60.7).
template <int XT, int WT, int K>
__global__ void __launch_bounds__(512)
rms_norm_bwd_elem_kernel(const BwdParams p) {
    constexpr int ES = ElemBytes<XT>::value, WS = ElemBytes<WT>::value;
    __shared__ float sh[32 * 8];
    pdl_begin();
    const int64_t row = static_cast<int64_t>(blockIdx.x) * blockDim.y + threadIdx.y;
    const bool live = row < p.m;
    const int64_t base = (live ? row : p.m - 1) * p.n;
    const int last = static_cast<int>(p.n) - 1, tpr = blockDim.x;
    const float rstd = __ldg(p.rstd + (live ? row : p.m - 1));
    float t[K], x[K], d[K];
#pragma unroll
    for (int k = 0; k < K; ++k) {
        const int64_t e = base + min(static_cast<int>(threadIdx.x) + k * tpr, last);
        t[k] = elem_load<XT>(p.dy + e * ES);
        x[k] = elem_load<XT>(p.r + e * ES);
        d[k] = 0.0f;
    }
    if (p.dres) {
#pragma unroll
        for (int k = 0; k < K; ++k)
            d[k] = elem_load<XT>(p.dres + (base + min(static_cast<int>(threadIdx.x) + k * tpr, last)) * ES);
    }
    float s = 0.0f;
#pragma unroll
    for (int k = 0; k < K; ++k) {
        const int c = threadIdx.x + k * tpr;
        t[k] = __fmul_rn(t[k], elem_load<WT>(p.w + min(c, last) * WS));
        x[k] = __fmul_rn(x[k], rstd);
        if (c <= last) s = __fmaf_rn(t[k], x[k], s);
    }
    const float mean = __fmul_rn(row_sum(s, sh), p.inv_n);
#pragma unroll
    for (int k = 0; k < K; ++k) {
        const int c = threadIdx.x + k * tpr;
        const float o = __fadd_rn(__fmul_rn(rstd, __fmaf_rn(-x[k], mean, t[k])), d[k]);
        if (live && c <= last) elem_store<XT>(p.dx + (base + c) * ES, o);
    }
}

// Backward for every other layout: one CTA per row for dx ...
template <int XT, int WT>
__global__ void __launch_bounds__(256)
rms_norm_bwd_dx_kernel(const BwdParams p) {
    constexpr int ES = ElemBytes<XT>::value, WS = ElemBytes<WT>::value;
    __shared__ float sh[32];
    pdl_begin();
    for (int64_t row = blockIdx.x; row < p.m; row += gridDim.x) {
        const int64_t base = row * p.n;
        const float rstd = __ldg(p.rstd + row);
        float s = 0.0f;
        for (int64_t c = threadIdx.x; c < p.n; c += blockDim.x)
            s = __fmaf_rn(__fmul_rn(elem_load<XT>(p.dy + (base + c) * ES), elem_load<WT>(p.w + c * WS)),
                          __fmul_rn(elem_load<XT>(p.r + (base + c) * ES), rstd), s);
        const float mean = __fmul_rn(row_sum(s, sh), p.inv_n);
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
// ... and COLS columns x one slice of the rows per CTA, 256 / COLS rows at a
// time, for the partial sums of dw: 256 columns, or 32 up to 512, where 256 leave
// many threads without one.  With dx, one element past a 16-byte address, 32 and
// 256 columns: bf16 16384 x 100 13.9 and 20.7 us, 16384 x 500 31.4 and 33.3, with
// a residual 4096 x 1000 26.0 and 20.9, 4096 x 7168 179 and 143.
template <int XT, int COLS>
__global__ void __launch_bounds__(256)
rms_norm_bwd_part_kernel(const BwdParams p, int64_t rows_per_part) {
    constexpr int ES = ElemBytes<XT>::value;
    constexpr int ROWS = 256 / COLS;
    __shared__ float sh[ROWS][COLS + 1];
    pdl_begin();
    const int64_t c = static_cast<int64_t>(blockIdx.x) * COLS + threadIdx.x;
    const int64_t r0 = static_cast<int64_t>(blockIdx.y) * rows_per_part;
    const int64_t r1 = r0 + rows_per_part < p.m ? r0 + rows_per_part : p.m;
    float s = 0.0f;
    if (c < p.n) {
        for (int64_t row = r0 + threadIdx.y; row < r1; row += ROWS)
            s = __fmaf_rn(elem_load<XT>(p.dy + (row * p.n + c) * ES),
                          __fmul_rn(elem_load<XT>(p.r + (row * p.n + c) * ES), __ldg(p.rstd + row)), s);
    }
    sh[threadIdx.y][threadIdx.x] = s;
    __syncthreads();
    if (threadIdx.y == 0 && c < p.n) {
        for (int i = 1; i < ROWS; ++i) s += sh[i][threadIdx.x];
        p.part[static_cast<int64_t>(blockIdx.y) * p.n + c] = s;
    }
}

// ---------------------------------------------------------------------------
// Backward, few rows, in one launch: dw needs the forward's rstd only, so some
// CTAs take rows (dx) and the others columns (dw: 8 threads of V elements, 32
// rows at a time), each reading dy and r for itself, which are in L2 by then.
// No workspace.  Latency bound: bf16 300 x 7168 6.8 us against 9.6 in
// two launches through partial sums, 512 x 18432 19.0 against 26.4.  V: elements
// of a 16-byte vector, or 1 for layouts that have none (with a residual, two
// launches after it: bf16 1 x 1001 2.9 us (5.2), 200 x 1001 3.7 (6.2), fp32 512 x
// 999 5.9 (7.8), bf16 512 x 7169 20.0 (20.1), 512 x 4097 14.7 (12.5), and 512 x 1024
// at an odd address 5.9 (7.6)).
// ---------------------------------------------------------------------------
constexpr int kSmallRows = 512;

template <int XT, int V>
__device__ __forceinline__ void load_elems(const uint8_t* p, int64_t e, float (&f)[V]) {
    if constexpr (V == 1) {
        f[0] = elem_load<XT>(p + e * ElemBytes<XT>::value);
    } else {
        const uint4 t = *reinterpret_cast<const uint4*>(p + e * ElemBytes<XT>::value);
        Vec<16> v;
        v.w[0] = t.x; v.w[1] = t.y; v.w[2] = t.z; v.w[3] = t.w;
        float2 g[V / 2];
        unpack<XT, 16>(v, g);
#pragma unroll
        for (int i = 0; i < V / 2; ++i) {
            f[2 * i] = g[i].x;
            f[2 * i + 1] = g[i].y;
        }
    }
}

template <int XT, int WT, int V>
__global__ void __launch_bounds__(256)
rms_norm_bwd_small_kernel(const BwdParams p, uint8_t* __restrict__ dw, const int row_ctas) {
    constexpr int ES = ElemBytes<XT>::value, WS = ElemBytes<WT>::value;
    constexpr int kCols = 8 * V;
    __shared__ float sh[32 * 8];
    __shared__ float cols[32][kCols + 1];
    pdl_begin();
    if (static_cast<int>(blockIdx.x) < row_ctas) {
        const int64_t row = static_cast<int64_t>(blockIdx.x) * blockDim.y + threadIdx.y, base = row * p.n;
        const bool live = row < p.m;
        const int64_t nvec = live ? p.n / V : 0;
        const float rstd = live ? __ldg(p.rstd + row) : 0.0f;
        auto weights = [&](int64_t i, float (&w)[V]) {
            if constexpr (V == 1) {
                w[0] = elem_load<WT>(p.w + i * WS);
            } else {
                float2 g[V / 2];
                unpack_weights<WT, V>(load_weights<WT, V>(p.w, static_cast<int>(i * V)), g);
#pragma unroll
                for (int j = 0; j < V / 2; ++j) {
                    w[2 * j] = g[j].x;
                    w[2 * j + 1] = g[j].y;
                }
            }
        };
        float s = 0.0f;
#pragma unroll 2
        for (int64_t i = threadIdx.x; i < nvec; i += blockDim.x) {
            float dy[V], r[V], w[V];
            load_elems<XT, V>(p.dy, base + i * V, dy);
            load_elems<XT, V>(p.r, base + i * V, r);
            weights(i, w);
#pragma unroll
            for (int j = 0; j < V; ++j) s = __fmaf_rn(__fmul_rn(dy[j], w[j]), __fmul_rn(r[j], rstd), s);
        }
        const float mean = __fmul_rn(row_sum(s, sh), p.inv_n);
#pragma unroll 2
        for (int64_t i = threadIdx.x; i < nvec; i += blockDim.x) {
            float dy[V], r[V], w[V], d[V], o[V];
            load_elems<XT, V>(p.dy, base + i * V, dy);
            load_elems<XT, V>(p.r, base + i * V, r);
            if (p.dres) load_elems<XT, V>(p.dres, base + i * V, d);
            weights(i, w);
#pragma unroll
            for (int j = 0; j < V; ++j) {
                o[j] = __fmul_rn(rstd, __fmaf_rn(-__fmul_rn(r[j], rstd), mean, __fmul_rn(dy[j], w[j])));
                if (p.dres) o[j] = __fadd_rn(o[j], d[j]);
            }
            if constexpr (V == 1) {
                elem_store<XT>(p.dx + (base + i) * ES, o[0]);
            } else {
                float2 g[V / 2];
#pragma unroll
                for (int j = 0; j < V / 2; ++j) g[j] = make_float2(o[2 * j], o[2 * j + 1]);
                store_vec<16>(p.dx + (base + i * V) * ES, pack<XT, 16>(g));
            }
        }
        return;
    }
    const int tid = threadIdx.y * blockDim.x + threadIdx.x, lane = tid & 7, group = tid >> 3;
    const int64_t c = (static_cast<int64_t>(blockIdx.x) - row_ctas) * kCols + lane * V;
    float acc[V];
#pragma unroll
    for (int j = 0; j < V; ++j) acc[j] = 0.0f;
    if (c < p.n) {
#pragma unroll 4
        for (int row = group; row < static_cast<int>(p.m); row += 32) {
            float dy[V], r[V];
            load_elems<XT, V>(p.dy, row * p.n + c, dy);
            load_elems<XT, V>(p.r, row * p.n + c, r);
            const float rstd = __ldg(p.rstd + row);
#pragma unroll
            for (int j = 0; j < V; ++j) acc[j] = __fmaf_rn(dy[j], __fmul_rn(r[j], rstd), acc[j]);
        }
    }
#pragma unroll
    for (int j = 0; j < V; ++j) cols[group][lane * V + j] = acc[j];
    for (int half = 16; half > 0; half /= 2) {
        __syncthreads();
        if (group < half) {
#pragma unroll
            for (int j = 0; j < V; ++j) {
                acc[j] += cols[group + half][lane * V + j];
                cols[group][lane * V + j] = acc[j];
            }
        }
    }
    if (group == 0 && c < p.n) {
#pragma unroll
        for (int j = 0; j < V; ++j) elem_store<WT>(dw + (c + j) * WS, acc[j]);
    }
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
    auto kernel = !p.q ? rms_norm_vec_kernel<XT, WT, VB, K, kNoCast>
                : p.fmt == kE4M3 ? rms_norm_vec_kernel<XT, WT, VB, K, kE4M3> : rms_norm_vec_kernel<XT, WT, VB, K, kE5M2>;
    return cuda_status(launch_kernel(kernel, dim3(static_cast<unsigned>(grid)), dim3(tpr, rows), s, p));
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
            p.lanes_log2 = ilog2c(lanes);
        }
        if (ok) vb = b;
    }
    const int64_t nshift = (p.n + 2 * (16 / ES) - 2) / (16 / ES);
    if (!vb && !p.q && nshift <= 1024 * 4 && aligned_to(p.x, 16) && aligned_to(p.res, 16) && aligned_to(p.res_out, 16) &&
        aligned_to(p.y, 16)) {
        const int k = nshift <= 256 ? 1 : nshift <= 2048 ? 2 : 4;
        const int tpr = round32((nshift + k - 1) / k), rows = tpr >= 256 ? 1 : 256 / tpr < 8 ? 256 / tpr : 8;
        const dim3 grid(static_cast<unsigned>((p.m + rows - 1) / rows)), block(tpr, rows);
        return cuda_status(k == 1   ? launch_kernel(rms_norm_shift_kernel<XT, WT, 1>, grid, block, s, p)
                           : k == 2 ? launch_kernel(rms_norm_shift_kernel<XT, WT, 2>, grid, block, s, p)
                                    : launch_kernel(rms_norm_shift_kernel<XT, WT, 4>, grid, block, s, p));
    }
    if (!vb && !p.q && p.n <= 8192) {
        const int k = p.n <= 4096 ? 8 : 16;
        const int tpr = round32((p.n + k - 1) / k), rows = tpr >= 256 ? 1 : 256 / tpr < 8 ? 256 / tpr : 8;
        const dim3 grid(static_cast<unsigned>((p.m + rows - 1) / rows)), block(tpr, rows);
        return cuda_status(k == 8 ? launch_kernel(rms_norm_elem_kernel<XT, WT, 8>, grid, block, s, p)
                                  : launch_kernel(rms_norm_elem_kernel<XT, WT, 16>, grid, block, s, p));
    }
    if (!vb) {
        const int64_t cap = static_cast<int64_t>(sm_count()) * 8;
        return cuda_status(launch_kernel(rms_norm_generic_kernel<XT, WT>,
                                         dim3(static_cast<unsigned>(p.m < cap ? p.m : cap)), dim3(256), s, p));
    }
    const int64_t nvec = p.n * ES / vb;
    if (vb == 32) {
        // One vector a thread has the shorter latency; two leave room for more and smaller CTAs
        // an SM, whose rows then overlap better: bf16 7168 wide to fp8, 300 rows 5.0 and 5.4 us,
        // 1000 rows 11.2 and 10.7, 4096 rows 38.8 and 33.1.  Four were slower (39.3).
        const bool many = p.m >= 3LL * sm_count();
        if (nvec <= 256 || (nvec <= 1024 && !many)) return run_fwd_vec<XT, WT, 32, 1>(p, s);
        if (nvec <= 2048) return run_fwd_vec<XT, WT, 32, 2>(p, s);
        if constexpr (XT == kF32) return run_fwd_vec<XT, WT, 32, 4>(p, s);
        return FP8Q_ERR_CUDA;      // not reached: 16-bit rows of more vectors take 16-byte ones
    }
    if (nvec <= 256) return run_fwd_vec<XT, WT, 16, 1>(p, s);
    if (nvec <= 2048) return run_fwd_vec<XT, WT, 16, 2>(p, s);
    return run_fwd_vec<XT, WT, 16, 4>(p, s);
}

// rows of partial sums of dw that a call of more than kSmallRows rows may write
int64_t bwd_parts(int64_t m) {
    const int64_t cap = 2LL * sm_count();
    return m < cap ? m : cap;
}

template <int WT>
fp8q_status run_dw(const float* part, int64_t parts, int64_t n, void* dw, cudaStream_t s) {
    const dim3 grid(static_cast<unsigned>((n + 31) / 32));
    uint8_t* out = static_cast<uint8_t*>(dw);
    if (n % 4 == 0 && aligned_to(part, 16))
        return cuda_status(launch_kernel(rms_norm_dw_kernel<WT>, grid, dim3(8, kDwRows), s, part, static_cast<int>(parts),
                                         n, out));
    return cuda_status(launch_kernel(rms_norm_dw_generic_kernel<WT>, grid, dim3(32, 16), s, part, static_cast<int>(parts),
                                     n, out));
}

template <int XT, int WT, int K, bool SHIFT>
fp8q_status run_bwd_vec(const BwdParams& p0, const BwdPlan& plan, int64_t* parts, cudaStream_t s) {
    constexpr int EPV = 16 / ElemBytes<XT>::value;
    BwdParams p = p0;
    p.stages = plan.stages;
    auto kernel = rms_norm_bwd_vec_kernel<XT, WT, K, SHIFT>;
    const cudaError_t e = allow_smem(kernel, kSmemPerSm);
    if (e != cudaSuccess) return cuda_status(e);
    const int64_t cap = static_cast<int64_t>(plan.ctas) * sm_count(), want = (p.m + plan.rows - 1) / plan.rows;
    *parts = want < cap ? want : cap;
    if (SHIFT && want > cap) {          // several turns: each moves a thread by a multiple of EPV elements
        int64_t turn = EPV;
        while (turn > 1 && (turn / 2) * plan.rows * p.n % EPV == 0) turn /= 2;
        if (cap < turn) return FP8Q_ERR_CUDA;      // not reached: every such GPU has more SMs
        *parts = cap - cap % turn;
    }
    return cuda_status(launch_kernel_smem(kernel, dim3(static_cast<unsigned>(*parts)), dim3(plan.tpr, plan.rows), plan.smem,
                                          s, p));
}

template <int XT, int WT, bool SHIFT>
fp8q_status run_bwd_vec_k(const BwdParams& p, const BwdPlan& plan, int64_t* parts, cudaStream_t s) {
    if (plan.k == 1) return run_bwd_vec<XT, WT, 1, SHIFT>(p, plan, parts, s);
    if (plan.k == 2) return run_bwd_vec<XT, WT, 2, SHIFT>(p, plan, parts, s);
    if constexpr (XT == kF32)
        if (plan.k == 8) return run_bwd_vec<XT, WT, 8, SHIFT>(p, plan, parts, s);
    return run_bwd_vec<XT, WT, 4, SHIFT>(p, plan, parts, s);
}

template <int XT, int WT, int V>
fp8q_status run_bwd_small(const BwdParams& p, void* dw, cudaStream_t s) {
    const int64_t nvec = p.n / V;
    const int tpr = nvec > 128 ? 256 : nvec > 64 ? 128 : nvec > 32 ? 64 : 32, rows = 256 / tpr;
    const int row_ctas = static_cast<int>((p.m + rows - 1) / rows);
    const int64_t col_ctas = dw ? (p.n + 8 * V - 1) / (8 * V) : 0;
    return cuda_status(launch_kernel(rms_norm_bwd_small_kernel<XT, WT, V>, dim3(static_cast<unsigned>(row_ctas + col_ctas)),
                                     dim3(tpr, rows), s, p, static_cast<uint8_t*>(dw), row_ctas));
}

template <int XT, int WT>
fp8q_status run_bwd(const BwdParams& p, void* dw, cudaStream_t s) {
    constexpr int ES = ElemBytes<XT>::value;
    constexpr int EPV = 16 / ES;
    const bool wide = (p.n * ES) % 16 == 0 && aligned_to(p.dy, 16) && aligned_to(p.r, 16) && aligned_to(p.dres, 16) &&
                      aligned_to(p.dx, 16) && aligned_to(p.w, 16);
    if (p.m > 0 && p.m <= kSmallRows)             // with dw or without: the same dx
        return wide ? run_bwd_small<XT, WT, EPV>(p, dw, s) : run_bwd_small<XT, WT, 1>(p, dw, s);
    // rows that are no multiple of 16 bytes but as long, and weights anywhere: the same vectors, shifted
    const bool shift = !(wide && aligned_to(p.part, 16));
    const BwdPlan plan = bwd_plan(ES, p.n, shift, p.dres ? 3 : 2);
    const bool vec = plan.k != 0 && aligned_to(p.dy, 16) && aligned_to(p.r, 16) && aligned_to(p.dres, 16) &&
                     aligned_to(p.dx, 16);
    int64_t parts = 0;
    fp8q_status st;
    if (p.m == 0) {
        st = FP8Q_OK;
    } else if (vec) {
        st = shift ? run_bwd_vec_k<XT, WT, true>(p, plan, &parts, s) : run_bwd_vec_k<XT, WT, false>(p, plan, &parts, s);
    } else {
        const int64_t cap = static_cast<int64_t>(sm_count()) * 8;
        if (p.n <= 4096) {
            constexpr int k = 8;
            const int tpr = round32((p.n + k - 1) / k), rows = tpr >= 256 ? 1 : 256 / tpr < 8 ? 256 / tpr : 8;
            const dim3 grid(static_cast<unsigned>((p.m + rows - 1) / rows)), block(tpr, rows);
            st = cuda_status(launch_kernel(rms_norm_bwd_elem_kernel<XT, WT, k>, grid, block, s, p));
        } else {
            st = cuda_status(launch_kernel(rms_norm_bwd_dx_kernel<XT, WT>,
                                           dim3(static_cast<unsigned>(p.m < cap ? p.m : cap)), dim3(256), s, p));
        }
        if (st == FP8Q_OK && p.part) {
            const int cols = p.n <= 512 ? 32 : 256;
            const int64_t want = bwd_parts(p.m), per = (p.m + want - 1) / want;
            parts = (p.m + per - 1) / per;
            const dim3 grid(static_cast<unsigned>((p.n + cols - 1) / cols), static_cast<unsigned>(parts));
            st = cuda_status(cols == 32
                                 ? launch_kernel(rms_norm_bwd_part_kernel<XT, 32>, grid, dim3(32, 8), s, p, per)
                                 : launch_kernel(rms_norm_bwd_part_kernel<XT, 256>, grid, dim3(256), s, p, per));
        }
    }
    if (st != FP8Q_OK || !dw) return st;
    return run_dw<WT>(p.part, parts, p.n, dw, s);
}

}  // namespace

size_t rms_norm_bwd_workspace(int64_t m, int64_t n) {
    return m <= kSmallRows ? 0 : static_cast<size_t>(bwd_parts(m)) * static_cast<size_t>(n) * sizeof(float);
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
    p.lanes_log2 = 0;
    p.inv_n = 1.0f / static_cast<float>(n);
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
    p.inv_n = 1.0f / static_cast<float>(n);
    if (xt == kF32) return run_bwd<kF32, kF32>(p, dw, s);
    if (xt == kF16) return wt == kF32 ? run_bwd<kF16, kF32>(p, dw, s) : run_bwd<kF16, kF16>(p, dw, s);
    return wt == kF32 ? run_bwd<kBF16, kF32>(p, dw, s) : run_bwd<kBF16, kBF16>(p, dw, s);
}

}  // namespace fp8q
