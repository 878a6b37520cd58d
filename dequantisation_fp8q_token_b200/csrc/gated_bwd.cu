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
#include "gated_device.cuh"
#include "per_tensor_device.cuh"
#include "fp8q_internal.h"

namespace fp8q {
namespace {

constexpr int kThreads = 256;

// Gradients of gate and up for two elements, in packed fp32 operations where
// there are any (half the issue slots; the two MUFU operations an element are
// what is left).  With a = gate * s, act' = s + a (1 - s) p'.  1 - s is 0 where
// |p| is large, so p' takes a capped square, which cannot overflow.
template <bool GELU>
__device__ __forceinline__ void gated_grad2(float2 dh, float2 g, float2 u, float2& dg, float2& du) {
    float2 s, om;
    if constexpr (GELU) s = make_float2(sigmoid_approx(gelu_exponent(g.x)), sigmoid_approx(gelu_exponent(g.y)));
    else s = make_float2(sigmoid_approx(g.x), sigmoid_approx(g.y));
    const float2 a = __fmul2_rn(g, s);
    om = __ffma2_rn(s, make_float2(-1.0f, -1.0f), make_float2(1.0f, 1.0f));
    if constexpr (GELU) {
        const float2 g2 = __fmul2_rn(g, g);
        const float2 dp = __ffma2_rn(make_float2(fminf(g2.x, 1e12f), fminf(g2.y, 1e12f)),
                                     make_float2(0.2140644488f, 0.2140644488f),        // 2 sqrt(2/pi) * 3 * 0.044715
                                     make_float2(1.5957691216f, 1.5957691216f));
        om = __fmul2_rn(om, dp);
    }
    dg = __fmul2_rn(__fmul2_rn(dh, u), __ffma2_rn(a, om, s));
    du = __fmul2_rn(dh, a);
}
// magnitude maximum of three values, keeping NaN
__device__ __forceinline__ float max3_abs(float a, float b, float c) {
    float d;
    asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}

template <int XT, int VB> struct Elems { static constexpr int N = VB / ElemBytes<XT>::value; };
// pair i of a vector
template <int XT, int VB>
__device__ __forceinline__ float2 pair_of(const Vec<VB>& v, int i) {
    if constexpr (XT == kF32) return make_float2(__uint_as_float(v.w[2 * i]), __uint_as_float(v.w[2 * i + 1]));
    float2 f;
    if constexpr (XT != kF32) widen2<XT>(v.w[i], f.x, f.y);
    return f;
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

template <int XT, int VB, bool GELU>
__global__ void __launch_bounds__(kThreads)
gated_amax_kernel(const BwdArgs a, uint32_t* __restrict__ partials) {
    constexpr int ES = ElemBytes<XT>::value, N = Elems<XT, VB>::N;
    __shared__ uint32_t sh[kThreads / 32];
    pdl_begin();
    // vectors from keep_from on stay in L2 for pass 2 (three streams)
    const int64_t keep_from = a.nvec - kL2KeepBytes / (3 * VB);
    const uint64_t keep = l2_evict_last_policy(), drop = l2_evict_first_policy();
    float m = 0.0f;
    for (int64_t v = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x; v < a.nvec;
         v += static_cast<int64_t>(gridDim.x) * kThreads) {
        int64_t ed, eg;
        place(a, v, N, ed, eg);
        const uint64_t pol = v >= keep_from ? keep : drop;
        const Vec<VB> vd = load_vec_policy<VB>(a.dh + ed * ES, pol);
        const Vec<VB> vg = load_vec_policy<VB>(a.gu + eg * ES, pol);
        const Vec<VB> vu = load_vec_policy<VB>(a.gu + (eg + a.I) * ES, pol);
#pragma unroll
        for (int i = 0; i < N / 2; ++i) {
            float2 dg, du;
            gated_grad2<GELU>(pair_of<XT, VB>(vd, i), pair_of<XT, VB>(vg, i), pair_of<XT, VB>(vu, i), dg, du);
            m = max3_abs(m, dg.x, du.x);
            m = max3_abs(m, dg.y, du.y);
        }
    }
    const uint32_t bits = block_max_u32(__float_as_uint(m) & 0x7FFFFFFFu, sh);
    if (threadIdx.x == 0) partials[blockIdx.x] = bits;
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

template <int XT, int FMT, int VB, bool GELU>
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
        const Vec<VB> vd = load_vec_policy<VB>(a.dh + ed * ES, drop);
        const Vec<VB> vg = load_vec_policy<VB>(a.gu + eg * ES, drop);
        const Vec<VB> vu = load_vec_policy<VB>(a.gu + (eg + a.I) * ES, drop);
        float g[N], u[N];
#pragma unroll
        for (int i = 0; i < N / 2; ++i) {
            float2 dg, du;
            gated_grad2<GELU>(pair_of<XT, VB>(vd, i), pair_of<XT, VB>(vg, i), pair_of<XT, VB>(vu, i), dg, du);
            g[2 * i] = dg.x;
            g[2 * i + 1] = dg.y;
            u[2 * i] = du.x;
            u[2 * i + 1] = du.y;
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
__device__ __forceinline__ void gated_grad(float dh, float g, float u, int act, float& dg, float& du) {
    float2 a, b;
    if (act == FP8Q_ACT_SILU) gated_grad2<false>(make_float2(dh, 0.0f), make_float2(g, 0.0f), make_float2(u, 0.0f), a, b);
    else gated_grad2<true>(make_float2(dh, 0.0f), make_float2(g, 0.0f), make_float2(u, 0.0f), a, b);
    dg = a.x;
    du = b.x;
}
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

template <int XT, int FMT, int VB, bool GELU>
fp8q_status run_vec(BwdArgs a, int64_t numel, uint8_t* q, float* sinv, uint32_t* partials, int rule, cudaStream_t s) {
    a.nvec = numel / Elems<XT, VB>::N;
    a.vpr = static_cast<uint32_t>(a.I / Elems<XT, VB>::N);
    const int grid = grid_for(a.nvec);
    cudaError_t e = launch_kernel(gated_amax_kernel<XT, VB, GELU>, dim3(grid), dim3(kThreads), s, a, partials);
    if (e != cudaSuccess) return cuda_status(e);
    return cuda_status(launch_kernel(gated_cast_kernel<XT, FMT, VB, GELU>, dim3(grid), dim3(kThreads), s, a,
                                     static_cast<const uint32_t*>(partials), grid, q, sinv, rule));
}

template <int XT, int FMT>
fp8q_status run(const BwdArgs& a, int64_t numel, uint8_t* q, float* sinv, uint32_t* partials, int rule, cudaStream_t s) {
    constexpr int ES = ElemBytes<XT>::value;
    auto fits = [&](int vb) {
        return a.I % (vb / ES) == 0 && reinterpret_cast<uintptr_t>(a.dh) % vb == 0 &&
               reinterpret_cast<uintptr_t>(a.gu) % vb == 0 && reinterpret_cast<uintptr_t>(q) % (vb / ES) == 0;
    };
    const bool gelu = a.act == FP8Q_ACT_GELU_TANH;
    if (fits(32))
        return gelu ? run_vec<XT, FMT, 32, true>(a, numel, q, sinv, partials, rule, s)
                    : run_vec<XT, FMT, 32, false>(a, numel, q, sinv, partials, rule, s);
    if (fits(16))
        return gelu ? run_vec<XT, FMT, 16, true>(a, numel, q, sinv, partials, rule, s)
                    : run_vec<XT, FMT, 16, false>(a, numel, q, sinv, partials, rule, s);
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
