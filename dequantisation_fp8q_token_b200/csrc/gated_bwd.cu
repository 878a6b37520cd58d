// gated_bwd.cu -- the elementwise part of a gated feed-forward block's
// backward pass, with the per-tensor fp8 cast that the products after it take.
//
//   s = sigmoid(p(gate)), act(g) = g * s
//   d_gate = dh * up * s * (1 + gate * (1 - s) * p'(gate))
//   d_up   = dh * gate * s
//   [d_gate | d_up] [M][2 I] cast with one scale (ColossalAI cast_to_fp8: a
//   zero or NaN amax is replaced by 1, scale = FMAX / amax, scale_inv = 1 / scale)
//
// Two passes, as the per-tensor cast (quant_scaled.cu): the amax is known only
// once every element is, so pass 1 computes the gradients for their maximum
// alone and pass 2 computes them again for the cast.  That moves 14 bytes per
// element of dh for 16-bit types; writing the gradients in between would move
// 16 and round them once more.  Pass 2 walks the rows from the end, where
// pass 1 left its last inputs in L2.
#include "fp8q_device.cuh"
#include "fp8q_internal.h"

namespace fp8q {
namespace {

constexpr int kThreads = 256;

// gradients of gate and up for one element.  1 - s is taken where it keeps its
// digits; where s (1 - s) is 0 the curvature term is 0 whatever p' is.
__device__ __forceinline__ void gated_grad(float dh, float g, float u, int act, float& dg, float& du) {
    float p = g, dp = 1.0f;
    if (act != FP8Q_ACT_SILU) {
        const float g2 = __fmul_rn(g, g);
        p = __fmul_rn(__fmul_rn(1.5957691216057308f, g), __fmaf_rn(0.044715f, g2, 1.0f));
        dp = __fmul_rn(1.5957691216057308f, __fmaf_rn(0.134145f, g2, 1.0f));
    }
    const float e = __expf(-p);
    const float s = __fdividef(1.0f, __fadd_rn(1.0f, e));
    const float om = e < 1.0f ? __fmul_rn(e, s) : __fsub_rn(1.0f, s);
    const float so = __fmul_rn(s, om);
    const float d = so == 0.0f ? s : __fmaf_rn(__fmul_rn(g, so), dp, s);
    dg = __fmul_rn(__fmul_rn(dh, u), d);
    du = __fmul_rn(dh, __fmul_rn(g, s));
}

template <int XT, int VB> struct Elems { static constexpr int N = VB / ElemBytes<XT>::value; };
template <int XT, int VB>
__device__ __forceinline__ void widen(const Vec<VB>& v, float (&f)[Elems<XT, VB>::N]) {
#pragma unroll
    for (int i = 0; i < VB / 4; ++i) {
        if constexpr (XT == kF32) f[i] = __uint_as_float(v.w[i]);
        else widen2<XT>(v.w[i], f[2 * i], f[2 * i + 1]);
    }
}

struct BwdArgs {
    const uint8_t* dh;
    const uint8_t* gu;
    int64_t I;
    int64_t nvec;             // vectors of dh in all
    uint32_t vpr;             // vectors of a row of dh
    int act;
};
// vector v of dh: its first element in dh, and in gate_up (whose rows are twice as long)
__device__ __forceinline__ void place(const BwdArgs& a, int64_t v, int epv, int64_t& e_dh, int64_t& e_gate) {
    const int64_t row = a.nvec <= 0x7FFFFFFFLL ? static_cast<int64_t>(static_cast<uint32_t>(v) / a.vpr) : v / a.vpr;
    e_dh = v * epv;
    e_gate = e_dh + row * a.I;
}

template <int XT, int VB>
__global__ void __launch_bounds__(kThreads)
gated_amax_kernel(const BwdArgs a, uint32_t* __restrict__ partials) {
    constexpr int ES = ElemBytes<XT>::value, N = Elems<XT, VB>::N;
    __shared__ uint32_t sh[kThreads / 32];
    pdl_begin();
    // vectors from keep_from on stay in L2 for pass 2 (three streams)
    const int64_t keep_from = a.nvec - kL2KeepBytes / (3 * VB);
    const uint64_t keep = l2_evict_last_policy(), drop = l2_evict_first_policy();
    uint32_t m = 0u;
    for (int64_t v = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x; v < a.nvec;
         v += static_cast<int64_t>(gridDim.x) * kThreads) {
        int64_t ed, eg;
        place(a, v, N, ed, eg);
        const uint64_t pol = v >= keep_from ? keep : drop;
        float d[N], g[N], u[N];
        const Vec<VB> vd = load_vec_policy<VB>(a.dh + ed * ES, pol);
        const Vec<VB> vg = load_vec_policy<VB>(a.gu + eg * ES, pol);
        const Vec<VB> vu = load_vec_policy<VB>(a.gu + (eg + a.I) * ES, pol);
        widen<XT, VB>(vd, d);
        widen<XT, VB>(vg, g);
        widen<XT, VB>(vu, u);
#pragma unroll
        for (int i = 0; i < N; ++i) {
            float dg, du;
            gated_grad(d[i], g[i], u[i], a.act, dg, du);
            m = max(m, max(__float_as_uint(dg) & 0x7FFFFFFFu, __float_as_uint(du) & 0x7FFFFFFFu));
        }
    }
    m = block_max_u32(m, sh);
    if (threadIdx.x == 0) partials[blockIdx.x] = m;
}

template <int N, int FMT, bool FIX>
__device__ __forceinline__ void encode_vec(const float (&v)[N], float scale, uint8_t* dst) {
    uint32_t c[N / 4];
#pragma unroll
    for (int i = 0; i < N / 4; ++i) {
        const float e0 = __fmul_rn(v[4 * i], scale), e1 = __fmul_rn(v[4 * i + 1], scale);
        const float e2 = __fmul_rn(v[4 * i + 2], scale), e3 = __fmul_rn(v[4 * i + 3], scale);
        c[i] = FIX ? (enc2_sem<FMT, true>(e0, e1) | (enc2_sem<FMT, true>(e2, e3) << 16)) : enc4<FMT>(e0, e1, e2, e3);
    }
    if constexpr (N == 16) st_v4(dst, make_uint4(c[0], c[1], c[2], c[3]));
    else if constexpr (N == 8) st_v2(dst, make_uint2(c[0], c[1]));
    else st_u32(dst, c[0]);
}

template <int XT, int FMT, int VB>
__global__ void __launch_bounds__(kThreads)
gated_cast_kernel(const BwdArgs a, const uint32_t* __restrict__ partials, int nparts, uint8_t* __restrict__ q,
                  float* __restrict__ sinv, int rule) {
    constexpr int ES = ElemBytes<XT>::value, N = Elems<XT, VB>::N;
    __shared__ uint32_t sh;
    pdl_begin();
    float amax;
    bool fix;
    const float scale = colossal_scale<FMT>(reduce_partials(partials, nparts, &sh), amax, fix, rule);
    if (blockIdx.x == 0 && threadIdx.x == 0) *sinv = __fdiv_rn(1.0f, scale);
    const uint64_t drop = l2_evict_first_policy();
    for (int64_t t = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x; t < a.nvec;
         t += static_cast<int64_t>(gridDim.x) * kThreads) {
        int64_t ed, eg;
        place(a, a.nvec - 1 - t, N, ed, eg);
        float d[N], g[N], u[N];
        const Vec<VB> vd = load_vec_policy<VB>(a.dh + ed * ES, drop);
        const Vec<VB> vg = load_vec_policy<VB>(a.gu + eg * ES, drop);
        const Vec<VB> vu = load_vec_policy<VB>(a.gu + (eg + a.I) * ES, drop);
        widen<XT, VB>(vd, d);
        widen<XT, VB>(vg, g);
        widen<XT, VB>(vu, u);
#pragma unroll
        for (int i = 0; i < N; ++i) {
            float dg, du;
            gated_grad(d[i], g[i], u[i], a.act, dg, du);
            g[i] = dg;
            u[i] = du;
        }
        if (!fix) {
            encode_vec<N, FMT, false>(g, scale, q + eg);
            encode_vec<N, FMT, false>(u, scale, q + eg + a.I);
        } else {
            encode_vec<N, FMT, true>(g, scale, q + eg);
            encode_vec<N, FMT, true>(u, scale, q + eg + a.I);
        }
    }
}

// any width, element-aligned pointers: one element at a time, both passes
template <int XT>
__global__ void __launch_bounds__(kThreads)
gated_amax_generic_kernel(const BwdArgs a, int64_t numel, uint32_t* __restrict__ partials) {
    constexpr int ES = ElemBytes<XT>::value;
    __shared__ uint32_t sh[kThreads / 32];
    pdl_begin();
    uint32_t m = 0u;
    for (int64_t e = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x; e < numel;
         e += static_cast<int64_t>(gridDim.x) * kThreads) {
        const int64_t eg = e + e / a.I * a.I;
        float dg, du;
        gated_grad(elem_load<XT>(a.dh + e * ES), elem_load<XT>(a.gu + eg * ES), elem_load<XT>(a.gu + (eg + a.I) * ES),
                   a.act, dg, du);
        m = max(m, max(__float_as_uint(dg) & 0x7FFFFFFFu, __float_as_uint(du) & 0x7FFFFFFFu));
    }
    m = block_max_u32(m, sh);
    if (threadIdx.x == 0) partials[blockIdx.x] = m;
}
template <int XT, int FMT>
__global__ void __launch_bounds__(kThreads)
gated_cast_generic_kernel(const BwdArgs a, int64_t numel, const uint32_t* __restrict__ partials, int nparts,
                          uint8_t* __restrict__ q, float* __restrict__ sinv, int rule) {
    constexpr int ES = ElemBytes<XT>::value;
    __shared__ uint32_t sh;
    pdl_begin();
    float amax;
    bool fix;
    const float scale = colossal_scale<FMT>(reduce_partials(partials, nparts, &sh), amax, fix, rule);
    if (blockIdx.x == 0 && threadIdx.x == 0) *sinv = __fdiv_rn(1.0f, scale);
    for (int64_t e = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x; e < numel;
         e += static_cast<int64_t>(gridDim.x) * kThreads) {
        const int64_t eg = e + e / a.I * a.I;
        float dg, du;
        gated_grad(elem_load<XT>(a.dh + e * ES), elem_load<XT>(a.gu + eg * ES), elem_load<XT>(a.gu + (eg + a.I) * ES),
                   a.act, dg, du);
        const uint32_t c = enc2_sem<FMT, true>(__fmul_rn(dg, scale), __fmul_rn(du, scale));
        q[eg] = static_cast<uint8_t>(c & 0xFFu);
        q[eg + a.I] = static_cast<uint8_t>(c >> 8);
    }
}

int grid_for(int64_t items) {
    const int64_t want = (items + kThreads - 1) / kThreads, cap = static_cast<int64_t>(sm_count()) * 8;
    const int64_t most = cap < kMaxPartials ? cap : kMaxPartials;
    return static_cast<int>(want < most ? want : most);
}

template <int XT, int FMT, int VB>
fp8q_status run_vec(BwdArgs a, int64_t numel, uint8_t* q, float* sinv, uint32_t* partials, int rule, cudaStream_t s) {
    a.nvec = numel / Elems<XT, VB>::N;
    a.vpr = static_cast<uint32_t>(a.I / Elems<XT, VB>::N);
    const int grid = grid_for(a.nvec);
    cudaError_t e = launch_kernel(gated_amax_kernel<XT, VB>, dim3(grid), dim3(kThreads), s, a, partials);
    if (e != cudaSuccess) return cuda_status(e);
    return cuda_status(launch_kernel(gated_cast_kernel<XT, FMT, VB>, dim3(grid), dim3(kThreads), s, a,
                                     static_cast<const uint32_t*>(partials), grid, q, sinv, rule));
}

template <int XT, int FMT>
fp8q_status run(const BwdArgs& a, int64_t numel, uint8_t* q, float* sinv, uint32_t* partials, int rule, cudaStream_t s) {
    constexpr int ES = ElemBytes<XT>::value;
    auto fits = [&](int vb) {
        return a.I % (vb / ES) == 0 && reinterpret_cast<uintptr_t>(a.dh) % vb == 0 &&
               reinterpret_cast<uintptr_t>(a.gu) % vb == 0 && reinterpret_cast<uintptr_t>(q) % (vb / ES) == 0;
    };
    if (fits(32)) return run_vec<XT, FMT, 32>(a, numel, q, sinv, partials, rule, s);
    if (fits(16)) return run_vec<XT, FMT, 16>(a, numel, q, sinv, partials, rule, s);
    const int grid = grid_for(numel);
    cudaError_t e = launch_kernel(gated_amax_generic_kernel<XT>, dim3(grid), dim3(kThreads), s, a, numel, partials);
    if (e != cudaSuccess) return cuda_status(e);
    return cuda_status(launch_kernel(gated_cast_generic_kernel<XT, FMT>, dim3(grid), dim3(kThreads), s, a, numel,
                                     static_cast<const uint32_t*>(partials), grid, q, sinv, rule));
}

}  // namespace

fp8q_status launch_gated_bwd(const void* dh, const void* gate_up, int xt, int64_t M, int64_t I, int act, int fmt,
                             int rule, uint8_t* q, float* sinv, uint32_t* partials, cudaStream_t s) {
    BwdArgs a = {};
    a.dh = static_cast<const uint8_t*>(dh);
    a.gu = static_cast<const uint8_t*>(gate_up);
    a.I = I;
    a.act = act;
    const int64_t numel = M * I;
    if (fmt == kE4M3)
        return xt == kF32 ? run<kF32, kE4M3>(a, numel, q, sinv, partials, rule, s)
             : xt == kF16 ? run<kF16, kE4M3>(a, numel, q, sinv, partials, rule, s)
                          : run<kBF16, kE4M3>(a, numel, q, sinv, partials, rule, s);
    return xt == kF32 ? run<kF32, kE5M2>(a, numel, q, sinv, partials, rule, s)
         : xt == kF16 ? run<kF16, kE5M2>(a, numel, q, sinv, partials, rule, s)
                      : run<kBF16, kE5M2>(a, numel, q, sinv, partials, rule, s);
}

}  // namespace fp8q
