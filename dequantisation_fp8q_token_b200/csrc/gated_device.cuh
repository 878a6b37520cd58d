// gated_device.cuh -- the activations of a gated feed-forward block, which its
// forward (gated_mm.cu) and backward (gated_bwd.cu) kernels share.
#pragma once

#include "fp8q_device.cuh"

namespace fp8q {

// act(g) = g * sigmoid(p(g)), p(g) = g (SiLU) or
// 2 sqrt(2 / pi) (g + 0.044715 g^3) (GELU, tanh form)
//
// 1 / (1 + 2^(-p log2 e)) with the hardware's exponential and reciprocal (2 and
// 1 ulp), whose small results flush to zero: e^-p below 2^-126 leaves 1, above
// 2^126 leaves 0.  The exponent is rounded to fp32 before the exponential, so
// e^-p is off by up to some |p| roundings more: what p's own last bit moves it
// by, which a longer exponent would leave.  Far negative p show it in an fp32
// result alone (p = -80: 4e-6, relative); 16 bits and fp8 do not hold it.
__device__ __forceinline__ float sigmoid_approx(float p) {
    float e, r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(__fmul_rn(p, -1.4426950408889634f)));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(__fadd_rn(1.0f, e)));
    return r;
}
__device__ __forceinline__ float gelu_exponent(float g) {
    return __fmul_rn(__fmul_rn(1.5957691216057308f, g), __fmaf_rn(__fmul_rn(0.044715f, g), g, 1.0f));
}

}  // namespace fp8q
