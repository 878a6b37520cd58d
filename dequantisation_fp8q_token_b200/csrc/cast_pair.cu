// cast_pair.cu -- the per-tensor casts of two tensors at once, which is what a
// product's operands need.  The arithmetic is quant_scaled.cu's, bit for bit:
// an amax pass that leaves one maximum per CTA, then a cast pass; here each
// pass is one launch, whose first CTAs take one tensor and the others the
// other.  For whole aligned vectors of 16 MB together at most, where the launches
// are what a cast costs (bf16 300 x 1024 and 768 x 1024: 5.3 us, two casts 9.3; 300 x
// 4096 and 2048 x 4096, 19 MB: 13.5 either way); others are cast one after the other.
#include "per_tensor_device.cuh"
#include "fp8q_internal.h"

namespace fp8q {
namespace {

constexpr int kThreads = 256;
constexpr int kVB = 16;
constexpr int kHalfPartials = kMaxPartials / 2;        // per tensor
constexpr int64_t kPairBytes = 16 << 20;

struct Pair {
    const uint8_t* x[2];
    uint8_t* q[2];
    float* sinv[2];
    int64_t nvec[2];
    int ctas[2];
};

template <int XT>
__global__ void __launch_bounds__(kThreads)
pair_amax_kernel(const Pair p, uint32_t* __restrict__ partials) {
    __shared__ uint32_t sh[kThreads / 32];
    pdl_begin();
    const int which = static_cast<int>(blockIdx.x) >= p.ctas[0], cta = blockIdx.x - which * p.ctas[0];
    const uint8_t* x = p.x[which];
    const int64_t stride = static_cast<int64_t>(p.ctas[which]) * kThreads, nvec = p.nvec[which];
    uint32_t m = 0u;
#pragma unroll 4
    for (int64_t i = static_cast<int64_t>(cta) * kThreads + threadIdx.x; i < nvec; i += stride) {
        const uint4 t = ld_stream_v4(x + i * kVB);
        Vec<kVB> v;
        v.w[0] = t.x; v.w[1] = t.y; v.w[2] = t.z; v.w[3] = t.w;
        m = absmax2<XT>(m, vec_absmax<XT, kVB>(v));
    }
    const uint32_t bits = block_max_u32(absmax_bits<XT>(m), sh);
    if (threadIdx.x == 0) partials[which * kHalfPartials + cta] = bits;
}

template <int XT, int FMT>
__global__ void __launch_bounds__(kThreads)
pair_cast_kernel(const Pair p, const uint32_t* __restrict__ partials, const int rule) {
    __shared__ uint32_t sh;
    pdl_begin();
    const int which = static_cast<int>(blockIdx.x) >= p.ctas[0], cta = blockIdx.x - which * p.ctas[0];
    float amax;
    bool fix;
    const float scale = colossal_scale<FMT>(reduce_partials(partials + which * kHalfPartials, p.ctas[which], &sh), amax,
                                            fix, rule);
    if (cta == 0 && threadIdx.x == 0) *p.sinv[which] = __fdiv_rn(1.0f, scale);
    const uint8_t* x = p.x[which];
    uint8_t* q = p.q[which];
    const int64_t stride = static_cast<int64_t>(p.ctas[which]) * kThreads, nvec = p.nvec[which];
#pragma unroll 4
    for (int64_t i = static_cast<int64_t>(cta) * kThreads + threadIdx.x; i < nvec; i += stride) {
        const uint4 t = ld_stream_v4(x + i * kVB);
        Vec<kVB> v;
        v.w[0] = t.x; v.w[1] = t.y; v.w[2] = t.z; v.w[3] = t.w;
        constexpr int EPV = kVB / ElemBytes<XT>::value;
        if (!fix) encode_store_vec<XT, FMT, kVB, false>(v, scale, q + i * EPV);
        else encode_store_vec<XT, FMT, kVB, true>(v, scale, q + i * EPV);
    }
}

template <int XT, int FMT>
fp8q_status run(const Pair& p, uint32_t* partials, int rule, cudaStream_t s) {
    const dim3 grid(static_cast<unsigned>(p.ctas[0] + p.ctas[1]));
    const cudaError_t e = launch_kernel(pair_amax_kernel<XT>, grid, dim3(kThreads), s, p, partials);
    if (e != cudaSuccess) return cuda_status(e);
    return cuda_status(launch_kernel(pair_cast_kernel<XT, FMT>, grid, dim3(kThreads), s, p,
                                     static_cast<const uint32_t*>(partials), rule));
}

}  // namespace

fp8q_status launch_per_tensor_pair(const void* const (&x)[2], const int64_t (&numel)[2], uint8_t* const (&q)[2],
                                   float* const (&sinv)[2], int xt, int fmt, uint32_t* partials, int rule,
                                   cudaStream_t s) {
    const int es = xt == kF32 ? 4 : 2, epv = kVB / es;
    Pair p = {};
    bool together = (numel[0] + numel[1]) * es <= kPairBytes;
    for (int i = 0; i < 2; ++i) {
        p.x[i] = static_cast<const uint8_t*>(x[i]);
        p.q[i] = q[i];
        p.sinv[i] = sinv[i];
        p.nvec[i] = numel[i] / epv;
        const int64_t want = (p.nvec[i] + 4 * kThreads - 1) / (4 * kThreads);
        p.ctas[i] = static_cast<int>(want < kHalfPartials ? want : kHalfPartials);
        together = together && numel[i] % epv == 0 && reinterpret_cast<uintptr_t>(x[i]) % kVB == 0 &&
                   reinterpret_cast<uintptr_t>(q[i]) % epv == 0;
    }
    if (!together) {
        for (int i = 0; i < 2; ++i) {
            const fp8q_status st = launch_per_tensor(x[i], xt, numel[i], fmt, q[i], sinv[i], partials, rule, s);
            if (st != FP8Q_OK) return st;
        }
        return FP8Q_OK;
    }
    if (fmt == kE4M3)
        return xt == kF32 ? run<kF32, kE4M3>(p, partials, rule, s)
             : xt == kF16 ? run<kF16, kE4M3>(p, partials, rule, s) : run<kBF16, kE4M3>(p, partials, rule, s);
    return xt == kF32 ? run<kF32, kE5M2>(p, partials, rule, s)
         : xt == kF16 ? run<kF16, kE5M2>(p, partials, rule, s) : run<kBF16, kE5M2>(p, partials, rule, s);
}

}  // namespace fp8q
