// fp8mp_f32x2.cuh -- pairs of fp32 values in one 64-bit register (low lane
// first) and the two-lane fp32 arithmetic of sm_100-class GPUs: each lane is
// one IEEE operation, bit-identical to the scalar one. Not part of the ABI.
#pragma once

#include <cstdint>

namespace fp8mp {

__device__ __forceinline__ uint64_t f2_from_bits(uint32_t lo, uint32_t hi) {
    uint64_t d;
    asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "r"(lo), "r"(hi));
    return d;
}
__device__ __forceinline__ uint64_t f2_pack(float lo, float hi) {
    return f2_from_bits(__float_as_uint(lo), __float_as_uint(hi));
}
__device__ __forceinline__ uint64_t f2_same(float x) { return f2_pack(x, x); }
__device__ __forceinline__ void f2_split(uint64_t v, float &lo, float &hi) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}
__device__ __forceinline__ uint64_t f2_mul(uint64_t a, uint64_t b) {
    uint64_t d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ uint64_t f2_add(uint64_t a, uint64_t b) {
    uint64_t d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ uint64_t f2_fma(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
}
// A product that is rounded before it joins a sum: mul.f32x2 and a following
// add.f32x2 are contracted into one fma, whatever their .rn says, where the
// scalar instructions are not. (The sign of a zero product is lost.)
__device__ __forceinline__ uint64_t f2_mul_apart(uint64_t a, uint64_t b) { return f2_fma(a, b, 0ull); }
// f2_fma, rounded towards zero.
__device__ __forceinline__ uint64_t f2_fma_rz(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t d;
    asm("fma.rz.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
}

}  // namespace fp8mp
