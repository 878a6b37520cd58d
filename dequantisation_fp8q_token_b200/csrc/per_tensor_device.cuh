// per_tensor_device.cuh -- device code of the casts with one scale per tensor
// (quant_scaled.cu, gated_bwd.cu).
#pragma once

#include "fp8q_device.cuh"

namespace fp8q {

// ---------------------------------------------------------------------------
// per-tensor casts: an amax pass that leaves per-CTA partial maxima, and a
// cast pass that reduces them and re-reads the tensor's tail from L2
// ---------------------------------------------------------------------------
#ifndef FP8Q_PT_L2_KEEP_MB
#define FP8Q_PT_L2_KEEP_MB 80
#endif
constexpr int64_t kL2KeepBytes = (int64_t)FP8Q_PT_L2_KEEP_MB << 20;  // well inside the 126 MB L2

__device__ __forceinline__ uint32_t block_max_u32(uint32_t m, uint32_t* sh) {
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, off));
    const int warp = threadIdx.x >> 5;
    if ((threadIdx.x & 31) == 0) sh[warp] = m;
    __syncthreads();
    m = 0u;
    const int nw = blockDim.x >> 5;
    for (int w = 0; w < nw; ++w) m = max(m, sh[w]);
    return m;
}

// magnitude-bits maximum of the amax pass's partials (every thread gets it)
__device__ __forceinline__ uint32_t reduce_partials(const uint32_t* __restrict__ partials, int nparts,
                                                    uint32_t* sh) {
    if (threadIdx.x < 32) {
        uint32_t m = 0u;
        for (int p = threadIdx.x; p < nparts; p += 32) m = max(m, __ldcg(partials + p));
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, off));
        if (threadIdx.x == 0) *sh = m;
    }
    __syncthreads();
    return *sh;
}

// ColossalAI scale rule from an fp32 magnitude-bits amax.  `fix` is set when
// the hardware's saturating encode could differ from the non-saturating
// reference: a NaN amax (replaced by 1, so NaN/Inf elements and overflow can
// occur) or a scale that overflowed to Inf (amax < FMAX / FLT_MAX).
template <int FMT>
__device__ __forceinline__ float colossal_scale(uint32_t amax_bits, float& amax_out, bool& fix, int rule) {
    const float a = __uint_as_float(amax_bits);
    const float amax = a > 0.0f ? a : 1.0f;
    const float scale = scale_from_amax<FMT>(amax, rule);
    fix = (amax_bits > 0x7F800000u) || isinf(scale);
    amax_out = amax;
    return scale;
}

}  // namespace fp8q
