// fp8mp_mma.cuh -- what the kernels that run tcgen05 MMAs on FP8 tiles share:
// the tile constants, the PTX of TMA, tensor memory and MMA, the shared-memory
// descriptors, and the order in which a persistent grid takes its tiles.
// Not part of the ABI.
#pragma once

#include "fp8mp_async.cuh"

namespace fp8mp {

constexpr int BK = 128;           // bytes of k per stage = one 128-byte swizzle row
constexpr int UMMA_K = 32;        // k of one kind::f8f6f4 MMA (32 bytes)
constexpr int TILE_N = 256;       // output columns per tile (TMEM columns per accumulator)
constexpr int ROWS_A = 128;       // rows of A each CTA stages (TMEM lanes)

// ------------------------------------------------------------ PTX wrappers

// Arrive on an mbarrier given by its shared::cluster address (any CTA of the cluster).
__device__ __forceinline__ void mbar_arrive_cluster(uint32_t cluster_addr) {
    asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr) : "memory");
}

// TMA 2-D tile load into this CTA's shared memory; completion is counted on
// the mbarrier at shared::cluster address `bar` (with PAIR it may sit in the
// peer CTA of the pair).
template <bool PAIR>
__device__ __forceinline__ void tma_load_2d(uint32_t dst, const CUtensorMap *map, uint32_t bar, int32_t c0,
                                            int32_t c1) {
    if constexpr (PAIR)
        asm volatile(
            "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes"
            " [%0], [%1, {%3, %4}], [%2];" ::"r"(dst),
            "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(c0), "r"(c1)
            : "memory");
    else
        asm volatile(
            "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes"
            " [%0], [%1, {%3, %4}], [%2];" ::"r"(dst),
            "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(c0), "r"(c1)
            : "memory");
}
// TMA 2-D tile store from this CTA's shared memory (rows / columns outside
// the tensor are not written), tracked as a bulk async-group of the thread.
__device__ __forceinline__ void tma_store_2d(const CUtensorMap *map, uint32_t src, int32_t c0, int32_t c1) {
    asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.bulk_group [%0, {%2, %3}], [%1];" ::"l"(
                     reinterpret_cast<uint64_t>(map)),
                 "r"(src), "r"(c0), "r"(c1)
                 : "memory");
}
__device__ __forceinline__ void bulk_commit_group() { asm volatile("cp.async.bulk.commit_group;" ::: "memory"); }
// Waits until at most one bulk group of this thread still reads shared memory.
__device__ __forceinline__ void bulk_wait_read_le1() { asm volatile("cp.async.bulk.wait_group.read 1;" ::: "memory"); }
// Waits until every bulk group of this thread has completed.
__device__ __forceinline__ void bulk_wait_all() { asm volatile("cp.async.bulk.wait_group 0;" ::: "memory"); }
// Orders this thread's generic-proxy shared-memory writes before later async-proxy reads (TMA).
__device__ __forceinline__ void fence_proxy_async_smem() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }
__device__ __forceinline__ void st_shared_v4(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}

template <bool PAIR>
__device__ __forceinline__ void tmem_alloc(uint32_t slot, uint32_t ncols) {
    if constexpr (PAIR)
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(slot), "r"(ncols)
                     : "memory");
    else
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(slot), "r"(ncols)
                     : "memory");
}
template <bool PAIR>
__device__ __forceinline__ void tmem_relinquish() {
    if constexpr (PAIR)
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    else
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
}
template <bool PAIR>
__device__ __forceinline__ void tmem_dealloc(uint32_t taddr, uint32_t ncols) {
    if constexpr (PAIR)
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(ncols) : "memory");
    else
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(ncols) : "memory");
}
__device__ __forceinline__ void tc_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }

template <bool PAIR>
__device__ __forceinline__ void umma_f8f6f4(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                            uint32_t accumulate) {
    if constexpr (PAIR)
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "setp.ne.b32 p, %4, 0;\n\t"
            "tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
            "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
            : "memory");
    else
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "setp.ne.b32 p, %4, 0;\n\t"
            "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
            "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
            : "memory");
}
// Arrive once on `bar` when all MMAs this thread issued so far complete: in
// this CTA (PAIR = false), or at the same offset in both CTAs of the pair.
template <bool PAIR>
__device__ __forceinline__ void umma_commit_all(uint32_t bar) {
    if constexpr (PAIR) {
        const uint16_t mask = 0x3;
        asm volatile(
            "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
                bar),
            "h"(mask)
            : "memory");
    } else {
        asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar)
                     : "memory");
    }
}
// Arrive once on this CTA's `bar` when the MMAs issued so far complete.
template <bool PAIR>
__device__ __forceinline__ void umma_commit_local(uint32_t bar) {
    if constexpr (PAIR)
        asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar)
                     : "memory");
    else
        asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar)
                     : "memory");
}

// 32 consecutive fp32 columns of this warp's 32 TMEM lanes (lane i of the
// warp gets TMEM lane base+i); the wait is in the same asm so the registers
// are valid when it returns.
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, uint32_t (&r)[32]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
          "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]),
          "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]),
          "=r"(r[30]), "=r"(r[31])
        : "r"(taddr)
        : "memory");
}

// Shared-memory matrix descriptor of a K-major operand tile stored as rows of
// 128 bytes with the 128-byte swizzle (the layout TMA writes with
// CU_TENSOR_MAP_SWIZZLE_128B): 8-row atoms of 1024 bytes stacked along M/N.
__device__ __forceinline__ uint64_t sw128_kmajor_desc(uint32_t saddr) {
    uint64_t d = 0;
    d |= static_cast<uint64_t>((saddr & 0x3FFFFu) >> 4);  // start address, bits 0-13
    d |= static_cast<uint64_t>(1u) << 16;                 // leading byte offset (unused here), bits 16-29
    d |= static_cast<uint64_t>(1024u >> 4) << 32;         // stride byte offset: one 8-row atom, bits 32-45
    d |= static_cast<uint64_t>(1u) << 46;                 // descriptor version for tcgen05, bits 46-47
    d |= static_cast<uint64_t>(2u) << 61;                 // swizzle mode: 128 bytes, bits 61-63
    return d;
}

// Shared-memory matrix descriptor of an MN-major operand tile: one
// 128-byte row of 128 M/N elements per k (the layout TMA writes for a box
// whose inner dimension runs along M/N, with CU_TENSOR_MAP_SWIZZLE_128B),
// 8-row atoms of 1024 bytes stacked along k. The stride byte offset is the
// step between those 8-row groups along k; the leading byte offset is the
// step between 128-element atoms along M/N (a 256-wide tile is staged as
// two 128-wide halves `lbo` bytes apart; a 128-wide tile has one atom).
__device__ __forceinline__ uint64_t sw128_mnmajor_desc(uint32_t saddr, uint32_t lbo) {
    uint64_t d = 0;
    d |= static_cast<uint64_t>((saddr & 0x3FFFFu) >> 4);  // start address, bits 0-13
    d |= static_cast<uint64_t>(lbo >> 4) << 16;           // leading byte offset: next M/N atom, bits 16-29
    d |= static_cast<uint64_t>(1024u >> 4) << 32;         // stride byte offset: next 8 k-rows, bits 32-45
    d |= static_cast<uint64_t>(1u) << 46;                 // descriptor version for tcgen05, bits 46-47
    d |= static_cast<uint64_t>(2u) << 61;                 // swizzle mode: 128 bytes, bits 61-63
    return d;
}

// The tcgen05 instruction descriptor of a kind::f8f6f4 MMA of m x n outputs.
constexpr uint32_t make_idesc(int fmt_a, int fmt_b, int m, int n, int a_mn, int b_mn) {
    return (1u << 4)                                // accumulator: f32
           | (static_cast<uint32_t>(fmt_a) << 7)    // A: 0 = E4M3, 1 = E5M2
           | (static_cast<uint32_t>(fmt_b) << 10)   // B: 0 = E4M3, 1 = E5M2
           | (static_cast<uint32_t>(a_mn) << 15)    // A: 0 = K-major, 1 = MN-major
           | (static_cast<uint32_t>(b_mn) << 16)    // B: 0 = K-major, 1 = MN-major
           | (static_cast<uint32_t>(n >> 3) << 17)  // N / 8
           | (static_cast<uint32_t>(m >> 4) << 24); // M / 16
}

// ------------------------------------------------------------- tile order

// Host: how a persistent grid's raster is grouped (see the definitions).
int raster_group(int64_t kc, int tile_m);
int raster_columns(int64_t rows_a, int64_t rows_b, int64_t kc, int tiles_m, int tiles_n, int gm);

// Tile of round `r` for cluster `c` of `nc`: one tile per cluster per round,
// dealt forwards in even rounds and backwards in odd ones (serpentine). With
// the tiles sorted by contraction length, longest first, the clusters that
// got the last long tiles get the first short ones, which keeps the
// per-cluster sums of k-blocks within one short tile of each other.
__device__ __forceinline__ int serpentine_tile(int r, int c, int nc) {
    return r * nc + ((r & 1) ? nc - 1 - c : c);
}
// Tile index -> (row-block of A, row-block of B), grouped so that the CTAs
// working at the same time share group_m A panels and a few B panels in L2
// (row-block fastest within a group); with group_n > 0 the other way round:
// groups of group_n B panels, column-block fastest, every A panel streamed
// past them once per group.
__device__ __forceinline__ void tile_coords(int t, int tiles_m, int tiles_n, int group_m, int group_n, int &mb,
                                            int &nb) {
    if (group_n > 0) {
        const int group = group_n * tiles_m;
        const int g = t / group;
        const int first = g * group_n;
        const int gn = min(tiles_n - first, group_n);
        const int local = t - g * group;
        nb = first + local % gn;
        mb = local / gn;
        return;
    }
    const int group = group_m * tiles_n;
    const int g = t / group;
    const int first = g * group_m;
    const int gm = min(tiles_m - first, group_m);
    const int local = t - g * group;
    mb = first + local % gm;
    nb = local / gm;
}

// ---------------------------------------------------------------- values

// A bf16 pair with an all-ones exponent field in either half (Inf or NaN).
__device__ __forceinline__ bool has_nonfinite_bf16x2(uint32_t w) {
    const uint32_t t = (w & 0x7F807F80u) ^ 0x7F807F80u;
    return (t & 0xFFFFu) == 0u || (t >> 16) == 0u;
}

// max |v[j]| over 16 values as a pairwise tree (depth 4 instead of a chain
// of 16); fmaxf ignores a NaN operand, so the result is the max of the
// non-NaN |v| (or NaN when all are NaN, which fmaxf(am, .) then ignores).
__device__ __forceinline__ float abs_max16(const float (&v)[16]) {
    float t[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) t[j] = fmaxf(fabsf(v[2 * j]), fabsf(v[2 * j + 1]));
#pragma unroll
    for (int j = 0; j < 4; ++j) t[j] = fmaxf(t[2 * j], t[2 * j + 1]);
    return fmaxf(fmaxf(t[0], t[1]), fmaxf(t[2], t[3]));
}

__device__ __forceinline__ uint32_t pack_bf16x2(float a, float b) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&h);
}

// ------------------------------------------------------------- host side

// An FP8 operand: outer rows of `inner` bytes, dense; boxes of box_outer rows x
// 128 bytes under the 128-byte swizzle. Bytes outside the tensor are read as 0.
inline int make_operand_tmap(CUtensorMap *map, const void *ptr, uint64_t inner, uint64_t outer, uint32_t box_outer) {
    auto enc = tensor_map_encoder();
    if (enc == nullptr) return fail(FP8MP_ERR_LAUNCH, "cuTensorMapEncodeTiled is not available");
    const cuuint64_t dims[2] = {inner, outer};
    const cuuint64_t strides[1] = {inner};
    const cuuint32_t box[2] = {static_cast<cuuint32_t>(BK), box_outer};
    const cuuint32_t estr[2] = {1, 1};
    const CUresult r = enc(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void *>(ptr), dims, strides, box, estr,
                           CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                           CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r != CUDA_SUCCESS) return fail(FP8MP_ERR_LAUNCH, "cuTensorMapEncodeTiled failed (%d)", static_cast<int>(r));
    return FP8MP_OK;
}

}  // namespace fp8mp
