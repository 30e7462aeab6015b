// fp8mp_gate.cuh -- the gate of the gated feed-forward block, h = act(g) u, and
// its gradient. Not part of the ABI.
//
// Both activations are g times a logistic function of z(g):
//   SiLU         act(g) = g / (1 + exp(-g))                         z = g
//   GELU (tanh)  act(g) = g (1 + tanh(s (g + c g^3))) / 2
//                       = g / (1 + exp(-z)),   z = 2 s (g + c g^3),
//                  s = sqrt(2 / pi), c = 0.044715
// so with p = 1 / (1 + exp(-z)): act = g p, act' = p + g p (1 - p) z'(g).
// exp and the quotient are CUDA's fast ones (a few ulp): the results are
// rounded to bf16 or FP8 next, and the amax is good to 2^-20.
#pragma once

#include "fp8mp_internal.cuh"

namespace fp8mp {

constexpr float kGelu1 = 1.59576912f;    // 2 sqrt(2 / pi)
constexpr float kGelu3 = 0.0713548163f;  // that times 0.044715

template <int ACT>
__device__ __forceinline__ float gate_exp(float g) {
    if constexpr (ACT == FP8MP_SILU)
        return __expf(-g);
    else
        return __expf(-g * fmaf(kGelu3 * g, g, kGelu1));
}

// act(g)
template <int ACT>
__device__ __forceinline__ float gate_act(float g) {
    return __fdividef(g, 1.0f + gate_exp<ACT>(g));
}

// act(g) and act'(g)
template <int ACT>
__device__ __forceinline__ void gate_act_grad(float g, float &a, float &da) {
    const float p = __fdividef(1.0f, 1.0f + gate_exp<ACT>(g));
    a = g * p;
    const float dz = ACT == FP8MP_SILU ? 1.0f : fmaf(3.0f * kGelu3 * g, g, kGelu1);
    da = fmaf(a * (1.0f - p), dz, p);
}

}  // namespace fp8mp
