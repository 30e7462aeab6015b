// fp8mp_gate.cuh -- the gate of the gated feed-forward block, h = act(g) u, and
// its gradient. Not part of the ABI.
//
// Both activations are g times a logistic function of z(g):
//   SiLU         act(g) = g / (1 + exp(-g))                         z = g
//   GELU (tanh)  act(g) = g (1 + tanh(s (g + c g^3))) / 2
//                       = g / (1 + exp(-z)),   z = 2 s (g + c g^3),
//                  s = sqrt(2 / pi), c = 0.044715
// so with p = 1 / (1 + exp(-z)): act = g p, act' = p + g p (1 - p) z'(g).
// exp2 and the reciprocal are the hardware's approximations (2 ulp each), the
// exponent is rounded once: p is good to (4 + 1.2 |z|) 2^-23 of itself, which a
// contraction's accumulation (1e-5 sum |a b|) hides. The results are rounded to bf16
// or FP8 next; the amax has that error and no other. The rest is done on pairs.
#pragma once

#include "fp8mp_f32x2.cuh"
#include "fp8mp_internal.cuh"

namespace fp8mp {

constexpr float kLog2e = 1.44269504f;
constexpr float kGelu1 = 1.59576912f;   // 2 sqrt(2 / pi)
constexpr float kGelu3 = 0.0713548163f; // that times 0.044715

// p of two values.
template <int ACT>
__device__ __forceinline__ uint64_t gate_logistic(uint64_t g) {
    uint64_t x;  // -z log2(e)
    if constexpr (ACT == FP8MP_SILU)
        x = f2_mul(g, f2_same(-kLog2e));
    else
        x = f2_mul(g, f2_fma(f2_mul(g, g), f2_same(-kLog2e * kGelu3), f2_same(-kLog2e * kGelu1)));
    float x0, x1, e0, e1, d0, d1, p0, p1;
    f2_split(x, x0, x1);
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e0) : "f"(x0));
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e1) : "f"(x1));
    f2_split(f2_add(f2_pack(e0, e1), f2_same(1.0f)), d0, d1);
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(p0) : "f"(d0));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(p1) : "f"(d1));
    return f2_pack(p0, p1);
}

// act(g)
template <int ACT>
__device__ __forceinline__ uint64_t gate_act(uint64_t g) {
    return f2_mul(g, gate_logistic<ACT>(g));
}

// act(g) and act'(g)
template <int ACT>
__device__ __forceinline__ void gate_act_grad(uint64_t g, uint64_t &a, uint64_t &da) {
    const uint64_t p = gate_logistic<ACT>(g);
    a = f2_mul(g, p);
    const uint64_t slope = f2_mul(a, f2_fma(p, f2_same(-1.0f), f2_same(1.0f)));
    if constexpr (ACT == FP8MP_SILU) {
        da = f2_add(slope, p);
    } else {
        // g^2 stays finite: where it would not, p is 0 or 1 and the slope 0
        float s0, s1;
        f2_split(f2_mul(g, g), s0, s1);
        da = f2_fma(slope, f2_fma(f2_pack(fminf(s0, 0x1p60f), fminf(s1, 0x1p60f)), f2_same(3.0f * kGelu3),
                                  f2_same(kGelu1)), p);
    }
}

// dg = dh u act'(g) and du = dh act(g) of four elements, as E5M2 codes under
// `scale`; g and u as bf16 pairs. |dg| and |du| join the running maximum (NaN
// left out).
template <int ACT>
__device__ __forceinline__ void gate_grad_codes(const uint64_t (&dh)[2], const uint32_t (&g)[2], const uint32_t (&u)[2],
                                                uint64_t scale, uint32_t &qg, uint32_t &qu, float &am) {
    float sg[4], su[4];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        uint64_t a, da;
        gate_act_grad<ACT>(f2_from_bits(g[k] << 16, g[k] & 0xFFFF0000u), a, da);
        const uint64_t dg = f2_mul(f2_mul(dh[k], f2_from_bits(u[k] << 16, u[k] & 0xFFFF0000u)), da);
        const uint64_t du = f2_mul(dh[k], a);
        float x0, x1, y0, y1;
        f2_split(dg, x0, x1);
        f2_split(du, y0, y1);
        am = fmaxf(fmaxf(am, fmaxf(fabsf(x0), fabsf(x1))), fmaxf(fabsf(y0), fabsf(y1)));
        f2_split(f2_mul(dg, scale), sg[2 * k], sg[2 * k + 1]);
        f2_split(f2_mul(du, scale), su[2 * k], su[2 * k + 1]);
    }
    qg = cvt_quad_probed<FP8MP_E5M2>(sg[0], sg[1], sg[2], sg[3]);
    qu = cvt_quad_probed<FP8MP_E5M2>(su[0], su[1], su[2], su[3]);
}

}  // namespace fp8mp
