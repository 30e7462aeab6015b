// fp8mp_pieces.cuh -- eight consecutive elements ("a piece") of a bf16 or fp32
// row in registers, as the row-wise kernels move them: 16- or 32-byte loads and
// stores, values in pairs of fp32. Not part of the ABI.
#pragma once

#include <atomic>

#include "fp8mp_f32x2.cuh"
#include "fp8mp_internal.cuh"

namespace fp8mp {

constexpr int kPiece = 8;

// 16 bytes from global to shared memory, past L1 and the registers.
__device__ __forceinline__ void cp_async_16(uint32_t to, const void *from) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to), "l"(from) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// A kernel may have its shared memory, from the first call on a device on.
template <typename K>
cudaError_t allow_smem(K *kernel, int bytes, std::atomic<bool> (&ready)[64], int device) {
    std::atomic<bool> &mine = ready[device & 63];
    if (mine.load(std::memory_order_acquire)) return cudaSuccess;
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e == cudaSuccess) mine.store(true, std::memory_order_release);
    return e;
}

template <bool BF16>
struct Piece {
    uint32_t w[BF16 ? 4 : 8];
    // Elements 2 i and 2 i + 1.
    __device__ __forceinline__ uint64_t pair(int i) const {
        if constexpr (BF16) return f2_from_bits(w[i] << 16, w[i] & 0xFFFF0000u);
        else return f2_from_bits(w[2 * i], w[2 * i + 1]);
    }
};

// Piece `i` of an array; read once. 32 bytes move as one access where they may, so
// that a warp's covers whole lines.
template <bool BF16>
__device__ __forceinline__ Piece<BF16> load_piece(const void *x, int64_t i) {
    Piece<BF16> r;
    const uint4 *p = reinterpret_cast<const uint4 *>(x) + (BF16 ? i : 2 * i);
    if constexpr (!BF16) {
        if ((reinterpret_cast<uintptr_t>(p) & 31u) == 0) {
            asm volatile("ld.global.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                         : "=r"(r.w[0]), "=r"(r.w[1]), "=r"(r.w[2]), "=r"(r.w[3]), "=r"(r.w[4]), "=r"(r.w[5]),
                           "=r"(r.w[6]), "=r"(r.w[7])
                         : "l"(p)
                         : "memory");
            return r;
        }
    }
#pragma unroll
    for (int j = 0; j < (BF16 ? 1 : 2); ++j) {
        const uint4 v = __ldcs(p + j);
        r.w[4 * j] = v.x;
        r.w[4 * j + 1] = v.y;
        r.w[4 * j + 2] = v.z;
        r.w[4 * j + 3] = v.w;
    }
    return r;
}

__device__ __forceinline__ uint32_t bf16_pair(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

// Four pairs rounded to the array's type.
template <bool BF16>
__device__ __forceinline__ Piece<BF16> round_piece(const uint64_t (&v)[4]) {
    Piece<BF16> r;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        float lo, hi;
        f2_split(v[i], lo, hi);
        if constexpr (BF16) {
            r.w[i] = bf16_pair(lo, hi);
        } else {
            r.w[2 * i] = __float_as_uint(lo);
            r.w[2 * i + 1] = __float_as_uint(hi);
        }
    }
    return r;
}

template <bool BF16>
__device__ __forceinline__ void store_piece(void *x, int64_t i, const Piece<BF16> &r) {
    uint4 *p = reinterpret_cast<uint4 *>(x) + (BF16 ? i : 2 * i);
    if constexpr (!BF16) {
        if ((reinterpret_cast<uintptr_t>(p) & 31u) == 0) {
            asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(r.w[0]), "r"(r.w[1]),
                         "r"(r.w[2]), "r"(r.w[3]), "r"(r.w[4]), "r"(r.w[5]), "r"(r.w[6]), "r"(r.w[7])
                         : "memory");
            return;
        }
    }
#pragma unroll
    for (int j = 0; j < (BF16 ? 1 : 2); ++j)
        p[j] = make_uint4(r.w[4 * j], r.w[4 * j + 1], r.w[4 * j + 2], r.w[4 * j + 3]);
}

// The same with the type known at run time (uniform over the launch).
__device__ __forceinline__ void store_rounded(void *x, int64_t i, const uint64_t (&v)[4], bool bf16) {
    if (bf16) store_piece<true>(x, i, round_piece<true>(v));
    else store_piece<false>(x, i, round_piece<false>(v));
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

}  // namespace fp8mp
