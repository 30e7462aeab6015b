// gated.cu -- the gated feed-forward block on the FP8 tensor cores:
//   forward   g = X8 Wg^T s, u = X8 Wu^T s, h = act(g) u in one launch;
//   dgrad     dh = dY8 Wd8 s, dg = dh u act'(g), du = dh act(g) in one launch;
//   gate      dg and du from a high-precision dh (an HBM-bound pass).
//
// The GEMM side is the persistent tcgen05 pipeline of gemm.cu: one CTA per SM
// (or a cluster of two on 256-row tiles), warp 0 the TMA producer, warp 1 the
// MMA issuer, the others the epilogue, two TMEM accumulators so that a tile's
// epilogue runs beside the next tile's MMAs. What differs is what a tile is
// and what its epilogue does:
//
//   forward: the 256 accumulator columns are 128 gate columns and the same 128
//     up columns (a pair's even CTA stages the gate rows of W8, its odd CTA
//     the up rows; one CTA alone both), so g and u of one element meet in one
//     thread and h never leaves the SM in more than its 8 (or 16) bits. The
//     pre-activations go out as bf16 only when the backward pass wants them.
//   dgrad: 256 columns of dh; the epilogue takes the tile's g and u (bf16) from a
//     ring that a warp of its own fills, and writes the E5M2 codes of dg and du.
//     dh itself is never stored: against a GEMM that writes it in bf16 and a pass
//     that reads it back that is 4 bytes per element less traffic.
//
// Roundings: the sums are the MMA's fp32 accumulators (good to 1e-5 sum |a b|),
// everything up to the output is fp32. h and the gradients' codes are FP8 because
// the next GEMM reads FP8, g and u bf16 because they are the largest tensors that
// training keeps. A few codes in a million (8 at a contraction of 4096, 1 at 256)
// are the neighbour of what exact sums would give.
//
// Both are bound by the tensor cores at training sizes (an epilogue of a few
// dozen instructions per element hides behind a contraction of 4096), and by
// their output traffic at short contractions.
#include <algorithm>
#include <atomic>
#include <cstdlib>
#include <cstring>
#include <mutex>

#include "fp8mp_gate.cuh"
#include "fp8mp_mma.cuh"

namespace fp8mp {

__device__ unsigned int g_gated_timeout_flag = 0;

namespace {

constexpr uint32_t TMEM_COLS = 2 * TILE_N;

enum Mode { FWD = 0, DGRAD = 1 };

// A CTA's warps and shared memory.
//
// Forward: four epilogue warps go from tensor memory to global memory through
// registers, each lane a row, in whole 32-byte sectors; shared memory is left to
// the operand ring, whose depth counts for more (16384 x 4096 -> 14336: 1085 us
// with 7 stages for a pair; 1156 with 5 and staging boxes for TMA stores, 1217
// with 4). Now 1045-1064 us where the board's power allows it, 3.6 PFLOP/s; the plain
// GEMM of that size takes 1030-1056. (A relaxed arrival on the accumulators' barrier
// is level with the release there: 1045-1064 us both, three runs each in turn.)
//
// Dgrad: the epilogue does more per element and waits for g and u, which come
// from DRAM; a warp alone on its scheduler is too slow for that (371-386 us for
// 8192 x 4096 x 14336, 279 for the GEMM alone), and so are loads by the lanes
// themselves, 32 rows apart (410-480 us). So eight warps work, two to a quarter
// of the rows, and one more feeds them chunks of 64 columns of g and u by TMA
// through a ring of two: 306-369 us, by the power the board allows. The MMA warp
// then waits for its operands 35 % of the time, as g, u and the codes (0.7 GB)
// share their way; without that traffic the launch takes 268 us.
template <bool PAIR, int MODE>
struct Cfg {
    static constexpr int TILE_M = PAIR ? 256 : 128;
    static constexpr int TILE_COLS = MODE == FWD ? 128 : 256;  // columns of h (dh) per tile
    static constexpr int ROWS_B = PAIR ? 128 : 256;
    static constexpr int STAGES = MODE == FWD ? (PAIR ? 7 : 4) : (PAIR ? 5 : 3);
    static constexpr int EPI_WARPS = MODE == FWD ? 4 : 8;
    static constexpr int THREADS = 64 + 32 * EPI_WARPS + (MODE == FWD ? 0 : 32);
    static constexpr int A_BYTES = ROWS_A * BK;
    static constexpr int STAGE_BYTES = A_BYTES + ROWS_B * BK;
    static constexpr int TX_BYTES = PAIR ? 2 * STAGE_BYTES : STAGE_BYTES;
    static constexpr int GU_OFFSET = STAGES * STAGE_BYTES;
    static constexpr int GU_BOX = 128 * 128;  // 128 rows of 64 bf16
    static constexpr int GU_CHUNKS = MODE == FWD ? 0 : 2;
    static constexpr int BAR_OFFSET = GU_OFFSET + GU_CHUNKS * 2 * GU_BOX;
    static constexpr int NUM_BARS = 2 * STAGES + 5 + 2 * GU_CHUNKS;
    static constexpr int SLOT_OFFSET = BAR_OFFSET + NUM_BARS * 8;
    static constexpr int FLAG_OFFSET = SLOT_OFFSET + 8;
    static constexpr int SMEM_ALLOC = FLAG_OFFSET + 8 + 1024;
    static constexpr uint32_t TEMPTY_COUNT = PAIR ? 2 * EPI_WARPS : EPI_WARPS;
    static_assert(STAGE_BYTES % 1024 == 0, "swizzle atoms need 1 KB alignment");
    static_assert(SMEM_ALLOC <= 232448, "shared memory budget");
};

struct GatedParams {
    CUtensorMap ta;        // A: the rows (tokens), K-major
    CUtensorMap tb0, tb1;  // forward: the gate and the up rows of W8; dgrad: Wd8 (both)
    CUtensorMap tg, tu;    // dgrad: the halves of the pre-activations
    uint16_t *gu;          // forward: the pre-activations, when they are wanted
    void *out;             // forward: h; dgrad: the codes of dg and du
    int wide;              // 32-byte stores: gu (and a bf16 h), or the codes' halves, lie on such boundaries
    int rows, cols, num_kb;
    int tiles_m, tiles_n, num_tiles, group_m, group_n;
    uint32_t idesc;
    const float *sinv_a, *sinv_b;
    const float *out_scale;
    float *out_amax;
};

__device__ __forceinline__ bool wait_bounded(uint32_t bar, uint32_t parity, volatile int *abort_flag) {
    return fp8mp::wait_bounded(bar, parity, abort_flag, &g_gated_timeout_flag);
}

__device__ __forceinline__ uint4 ld_shared_v4(uint32_t addr) {
    uint4 v;
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "r"(addr)
                 : "memory");
    return v;
}

// 32 bytes to a 32-byte boundary in one store.
__device__ __forceinline__ void store_32_bytes(void *p, const uint32_t (&w)[8]) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(w[0]), "r"(w[1]), "r"(w[2]),
                 "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                 : "memory");
}
// 16 bf16 values (32 bytes): in one store where they lie on a 32-byte boundary.
__device__ __forceinline__ void store_bf16x16(uint16_t *p, bool wide, const uint32_t (&w)[8]) {
    if (wide) {
        store_32_bytes(p, w);
    } else {
        *reinterpret_cast<uint4 *>(p) = make_uint4(w[0], w[1], w[2], w[3]);
        *(reinterpret_cast<uint4 *>(p) + 1) = make_uint4(w[4], w[5], w[6], w[7]);
    }
}

// A forward tile, by one warp: this lane's row, 32 columns of g and u at a time
// (`acc`: the accumulator's column 0 of the warp's lanes). Columns past F and
// rows past M hold zeros (the operands' zero fill), whose h is 0: they need no
// mask in the amax, and are not stored.
template <int ACT, bool H_FP8>
__device__ __forceinline__ float forward_tile(const GatedParams &P, uint32_t acc, int row, int col0, float scale,
                                              float h_scale) {
    float am = 0.0f;
    const bool row_ok = row < P.rows;
    const int64_t f = P.cols;
    uint16_t *g_row = P.gu + static_cast<int64_t>(row) * 2 * f;
#pragma unroll 1
    for (int c = 0; c < 128; c += 32) {
        if (col0 + c >= P.cols) break;
        uint32_t rg[32], ru[32];
        tmem_ld32(acc + static_cast<uint32_t>(c), rg);
        tmem_ld32(acc + static_cast<uint32_t>(128 + c), ru);
#pragma unroll
        for (int o = 0; o < 2; ++o) {  // 16 columns each
            const int col = col0 + c + 16 * o;
            const bool ok = row_ok && col < P.cols;
            uint32_t wg[8], wu[8], wh[8];
#pragma unroll
            for (int k = 0; k < 4; ++k) {  // four columns
                float y[4];
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const int at = 16 * o + 4 * k + 2 * j;
                    const uint64_t g = f2_mul(f2_from_bits(rg[at], rg[at + 1]), f2_same(scale));
                    const uint64_t u = f2_mul(f2_from_bits(ru[at], ru[at + 1]), f2_same(scale));
                    const uint64_t h = f2_mul(gate_act<ACT>(g), u);
                    float v0, v1;
                    f2_split(g, v0, v1);
                    wg[2 * k + j] = pack_bf16x2(v0, v1);
                    f2_split(u, v0, v1);
                    wu[2 * k + j] = pack_bf16x2(v0, v1);
                    f2_split(h, v0, v1);
                    am = fmaxf(am, fmaxf(fabsf(v0), fabsf(v1)));
                    if constexpr (H_FP8)
                        f2_split(f2_mul(h, f2_same(h_scale)), y[2 * j], y[2 * j + 1]);
                    else
                        wh[2 * k + j] = pack_bf16x2(v0, v1);
                }
                if constexpr (H_FP8) wh[k] = cvt_quad_probed<FP8MP_E4M3>(y[0], y[1], y[2], y[3]);
            }
            if (!ok) continue;
            if (P.gu != nullptr) {
                store_bf16x16(g_row + col, P.wide, wg);
                store_bf16x16(g_row + f + col, P.wide, wu);
            }
            if constexpr (H_FP8)
                *reinterpret_cast<uint4 *>(static_cast<uint8_t *>(P.out) + row * f + col) =
                    make_uint4(wh[0], wh[1], wh[2], wh[3]);
            else
                store_bf16x16(static_cast<uint16_t *>(P.out) + row * f + col, P.wide, wh);
        }
    }
    return am;
}

// 32 columns of a dgrad tile: dg and du of this lane's row from the accumulator
// (at `acc`) and its g and u, the 16-byte pieces `piece` .. `piece` + 3 of row
// `r` in boxes of 128-byte rows under the 128-byte swizzle.
template <int ACT>
__device__ __forceinline__ float dgrad_columns(const GatedParams &P, uint32_t acc, uint32_t box_g, uint32_t box_u,
                                               int r, int piece, int row, int col, float scale, float out_scale) {
    float am = 0.0f;
    uint32_t rd[32];
    tmem_ld32(acc, rd);
    uint8_t *out = static_cast<uint8_t *>(P.out) + static_cast<int64_t>(row) * 2 * P.cols + col;
    uint32_t qg[8], qu[8];
#pragma unroll
    for (int o = 0; o < 2; ++o) {  // 16 columns each
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const uint32_t at = static_cast<uint32_t>(r * 128 + (((piece + 2 * o + h) ^ (r & 7)) << 4));
            const uint4 gw = ld_shared_v4(box_g + at), uw = ld_shared_v4(box_u + at);
            const uint32_t g[2][2] = {{gw.x, gw.y}, {gw.z, gw.w}}, u[2][2] = {{uw.x, uw.y}, {uw.z, uw.w}};
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const int i = 16 * o + 8 * h + 4 * k;
                const uint64_t dh[2] = {f2_mul(f2_from_bits(rd[i], rd[i + 1]), f2_same(scale)),
                                        f2_mul(f2_from_bits(rd[i + 2], rd[i + 3]), f2_same(scale))};
                gate_grad_codes<ACT>(dh, g[k], u[k], f2_same(out_scale), qg[4 * o + 2 * h + k], qu[4 * o + 2 * h + k],
                                     am);
            }
        }
    }
    if (row < P.rows && P.wide && col < P.cols) {  // (wide: P.cols is a multiple of 32)
        store_32_bytes(out, qg);
        store_32_bytes(out + P.cols, qu);
    } else if (row < P.rows) {
#pragma unroll
        for (int o = 0; o < 2; ++o)
            if (col + 16 * o < P.cols) {
                *reinterpret_cast<uint4 *>(out + 16 * o) =
                    make_uint4(qg[4 * o], qg[4 * o + 1], qg[4 * o + 2], qg[4 * o + 3]);
                *reinterpret_cast<uint4 *>(out + P.cols + 16 * o) =
                    make_uint4(qu[4 * o], qu[4 * o + 1], qu[4 * o + 2], qu[4 * o + 3]);
            }
    }
    return am;
}

// Chunks of 64 columns of a dgrad tile that exist for a CTA.
__device__ __forceinline__ int dgrad_chunks(const GatedParams &P, int cta_row0, int col0) {
    return cta_row0 < P.rows ? min(4, (P.cols - col0 + 63) / 64) : 0;
}

template <bool PAIR, int MODE, int ACT, bool H_FP8>
__global__ void __launch_bounds__(Cfg<PAIR, MODE>::THREADS, 1) gated_kernel(const __grid_constant__ GatedParams P) {
    using C = Cfg<PAIR, MODE>;
    extern __shared__ uint8_t smem_raw[];
    uint32_t base = smem_u32(smem_raw);
    const uint32_t pad = (1024u - (base & 1023u)) & 1023u;
    uint8_t *smem = smem_raw + pad;
    base += pad;

    const uint32_t bar0 = base + C::BAR_OFFSET;
    auto full_bar = [&](int s) { return bar0 + 8u * s; };
    auto empty_bar = [&](int s) { return bar0 + 8u * (C::STAGES + s); };
    auto tfull_bar = [&](int a) { return bar0 + 8u * (2 * C::STAGES + a); };
    auto tempty_bar = [&](int a) { return bar0 + 8u * (2 * C::STAGES + 2 + a); };
    const uint32_t drain_bar = bar0 + 8u * (2 * C::STAGES + 4);
    auto gu_full = [&](int b) { return bar0 + 8u * (2 * C::STAGES + 5 + b); };  // dgrad
    auto gu_empty = [&](int b) { return bar0 + 8u * (2 * C::STAGES + 5 + C::GU_CHUNKS + b); };
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + C::SLOT_OFFSET);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(smem + C::FLAG_OFFSET);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = PAIR ? cluster_ctarank() : 0u;  // 0 = the CTA that issues the MMAs
    const int cluster_id = PAIR ? static_cast<int>(blockIdx.x >> 1) : static_cast<int>(blockIdx.x);
    const int num_clusters = PAIR ? static_cast<int>(gridDim.x >> 1) : static_cast<int>(gridDim.x);

    if (threadIdx.x == 0) {
        for (int s = 0; s < C::STAGES; ++s) {
            mbar_init(full_bar(s), 1);
            mbar_init(empty_bar(s), 1);
        }
        for (int a = 0; a < 2; ++a) {
            mbar_init(tfull_bar(a), 1);
            mbar_init(tempty_bar(a), C::TEMPTY_COUNT);
        }
        mbar_init(drain_bar, 1);
        for (int b = 0; b < C::GU_CHUNKS; ++b) {
            mbar_init(gu_full(b), 1);
            mbar_init(gu_empty(b), C::EPI_WARPS);
        }
        *abort_flag = 0;
        fence_mbar_init();
        prefetch_tmap(&P.ta);
        prefetch_tmap(&P.tb0);
        prefetch_tmap(&P.tb1);
    }
    if (warp == 1) {
        tmem_alloc<PAIR>(smem_u32(tmem_slot), TMEM_COLS);
        tmem_relinquish<PAIR>();
    }
    tc_fence_before();
    if constexpr (PAIR)
        cluster_sync_all();  // the peer's barriers are initialised before anyone signals them
    else
        __syncthreads();
    tc_fence_after();
    const uint32_t tmem_base = *tmem_slot;
    pdl_wait();

    const int rounds = (P.num_tiles + num_clusters - 1) / num_clusters;
    const int num_kb = P.num_kb;

    if (warp == 0) {
        if (lane == 0) {
            // ---------------- TMA producer (both CTAs of a pair)
            pdl_launch_dependents();
            uint32_t it = 0;
            bool ok = true;
            for (int r = 0; ok && r < rounds; ++r) {
                const int tile = serpentine_tile(r, cluster_id, num_clusters);
                if (tile >= P.num_tiles) continue;
                int mb, nb;
                tile_coords(tile, P.tiles_m, P.tiles_n, P.group_m, P.group_n, mb, nb);
                const int a_row = mb * C::TILE_M + static_cast<int>(rank) * ROWS_A;
                const int col0 = nb * C::TILE_COLS;
                const CUtensorMap *tb = PAIR && rank ? &P.tb1 : &P.tb0;
                for (int kb = 0; kb < num_kb; ++kb, ++it) {
                    const int s = static_cast<int>(it % C::STAGES);
                    if (!wait_bounded(empty_bar(s), ((it / C::STAGES) & 1u) ^ 1u, abort_flag)) {
                        ok = false;
                        break;
                    }
                    const uint32_t sa = base + s * C::STAGE_BYTES, sb = sa + C::A_BYTES;
                    const uint32_t fb = PAIR ? mapa_shared(full_bar(s), 0) : full_bar(s);
                    if (rank == 0) mbar_arrive_expect_tx(full_bar(s), C::TX_BYTES);
                    tma_load_2d<PAIR>(sa, &P.ta, fb, kb * BK, a_row);
                    if constexpr (MODE == FWD) {  // K-major: 128 rows of W8 x 128 bytes of k
                        tma_load_2d<PAIR>(sb, tb, fb, kb * BK, col0);
                        if constexpr (!PAIR) tma_load_2d<PAIR>(sb + 128 * BK, &P.tb1, fb, kb * BK, col0);
                    } else {  // MN-major: 128 k-rows of Wd8 x 128 columns
                        const int at = col0 + static_cast<int>(rank) * C::ROWS_B;
                        tma_load_2d<PAIR>(sb, tb, fb, at, kb * BK);
                        if constexpr (!PAIR) tma_load_2d<PAIR>(sb + BK * 128, tb, fb, at + 128, kb * BK);
                    }
                }
            }
            if (!ok && rank == 0) {
                // let the loads already issued land before the CTA goes away
                for (uint32_t j = 1; j <= static_cast<uint32_t>(C::STAGES) && j <= it; ++j) {
                    const uint32_t at = it - j;
                    volatile int never = 0;
                    wait_bounded(full_bar(static_cast<int>(at % C::STAGES)), (at / C::STAGES) & 1u, &never);
                }
            }
        }
    } else if (warp == 1) {
        if (lane == 0 && rank == 0) {
            // ---------------- MMA issuer
            uint32_t it = 0;
            int lt = 0;
            bool ok = true;
            for (int r = 0; ok && r < rounds; ++r) {
                if (serpentine_tile(r, cluster_id, num_clusters) >= P.num_tiles) continue;
                const int acc = lt & 1;
                const uint32_t aph = (static_cast<uint32_t>(lt) >> 1) & 1u;
                ++lt;
                if (!wait_bounded(tempty_bar(acc), aph ^ 1u, abort_flag)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                const uint32_t d_tmem = tmem_base + static_cast<uint32_t>(acc * TILE_N);
                for (int kb = 0; kb < num_kb; ++kb, ++it) {
                    const int s = static_cast<int>(it % C::STAGES);
                    if (!wait_bounded(full_bar(s), (it / C::STAGES) & 1u, abort_flag)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint32_t sa = base + s * C::STAGE_BYTES, sb = sa + C::A_BYTES;
#pragma unroll
                    for (int k = 0; k < BK / UMMA_K; ++k) {
                        const uint64_t a_desc = sw128_kmajor_desc(sa + k * UMMA_K);
                        const uint64_t b_desc =
                            MODE == FWD ? sw128_kmajor_desc(sb + k * UMMA_K)
                                        : sw128_mnmajor_desc(sb + k * UMMA_K * 128, PAIR ? 1024u : BK * 128u);
                        umma_f8f6f4<PAIR>(d_tmem, a_desc, b_desc, P.idesc, (kb > 0 || k > 0) ? 1u : 0u);
                    }
                    umma_commit_all<PAIR>(empty_bar(s));
                }
                if (!ok) break;
                umma_commit_all<PAIR>(tfull_bar(acc));
            }
            if (!ok) {
                // wait for the MMAs in flight before TMEM is released
                umma_commit_local<PAIR>(drain_bar);
                volatile int never = 0;
                wait_bounded(drain_bar, 0u, &never);
            }
        }
    } else if (MODE == DGRAD && warp == 2 + C::EPI_WARPS) {
        if (lane == 0) {
            // ---------------- dgrad: the producer of g and u for the epilogue
            uint32_t n = 0;
            bool ok = true;
            for (int r = 0; ok && r < rounds; ++r) {
                const int tile = serpentine_tile(r, cluster_id, num_clusters);
                if (tile >= P.num_tiles) continue;
                int mb, nb;
                tile_coords(tile, P.tiles_m, P.tiles_n, P.group_m, P.group_n, mb, nb);
                const int row0 = mb * C::TILE_M + static_cast<int>(rank) * ROWS_A, col0 = nb * C::TILE_COLS;
                const int live = dgrad_chunks(P, row0, col0);
                for (int c = 0; c < live; ++c, ++n) {
                    const uint32_t b = n & 1u;
                    if (!wait_bounded(gu_empty(b), ((n >> 1) & 1u) ^ 1u, abort_flag)) {
                        ok = false;
                        break;
                    }
                    const uint32_t box = base + C::GU_OFFSET + b * 2 * C::GU_BOX;
                    mbar_arrive_expect_tx(gu_full(b), 2 * C::GU_BOX);
                    tma_load_2d_cta(box, &P.tg, gu_full(b), col0 + 64 * c, row0);
                    tma_load_2d_cta(box + C::GU_BOX, &P.tu, gu_full(b), col0 + 64 * c, row0);
                }
            }
            if (!ok)  // let the loads already issued land before the CTA goes away
                for (uint32_t j = 1; j <= 2 && j <= n; ++j) {
                    volatile int never = 0;
                    wait_bounded(gu_full((n - j) & 1u), ((n - j) >> 1) & 1u, &never);
                }
        }
    } else {
        // ---------------- epilogue warps (both CTAs of a pair)
        const int q = warp & 3;  // this warp may access TMEM lanes 32q .. 32q+31
        const int half = (warp - 2) >> 2;  // dgrad: which 32 columns of a chunk
        const float scale = __fmul_rn(*P.sinv_a, *P.sinv_b);
        const float out_scale = P.out_scale != nullptr ? *P.out_scale : 1.0f;
        float am = 0.0f;
        int lt = 0;
        uint32_t used = 0;  // dgrad: chunks of g and u used
        for (int r = 0; r < rounds; ++r) {
            const int tile = serpentine_tile(r, cluster_id, num_clusters);
            if (tile >= P.num_tiles) continue;
            int mb, nb;
            tile_coords(tile, P.tiles_m, P.tiles_n, P.group_m, P.group_n, mb, nb);
            const int cta_row0 = mb * C::TILE_M + static_cast<int>(rank) * ROWS_A;
            const int row = cta_row0 + q * 32 + lane, col0 = nb * C::TILE_COLS;
            const int acc = lt & 1;
            const uint32_t aph = (static_cast<uint32_t>(lt) >> 1) & 1u;
            ++lt;
            int ok = 1;
            if (lane == 0) ok = wait_bounded(tfull_bar(acc), aph, abort_flag) ? 1 : 0;
            ok = __shfl_sync(0xffffffffu, ok, 0);
            if (!ok) break;
            tc_fence_after();
            const uint32_t acc_addr =
                tmem_base + static_cast<uint32_t>(acc * TILE_N) + (static_cast<uint32_t>(q * 32) << 16);
            if constexpr (MODE == FWD) {
                am = fmaxf(am, forward_tile<ACT, H_FP8>(P, acc_addr, row, col0, scale, out_scale));
            } else {
                const int live = dgrad_chunks(P, cta_row0, col0);
#pragma unroll 1
                for (int c = 0; c < live; ++c, ++used) {
                    const uint32_t b = used & 1u;
                    const bool landed = wait_bounded(gu_full(b), (used >> 1) & 1u, abort_flag);
                    ok = __all_sync(0xffffffffu, landed);
                    if (!ok) break;
                    const uint32_t box = base + C::GU_OFFSET + b * 2 * C::GU_BOX;
                    const int at = 64 * c + 32 * half;
                    am = fmaxf(am, dgrad_columns<ACT>(P, acc_addr + static_cast<uint32_t>(at), box, box + C::GU_BOX,
                                                      q * 32 + lane, 4 * half, row, col0 + at, scale, out_scale));
                    __syncwarp();  // every lane has used its g and u
                    if (lane == 0) mbar_arrive(gu_empty(b));
                }
                if (!ok) break;
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
                if constexpr (PAIR)
                    mbar_arrive_cluster(mapa_shared(tempty_bar(acc), 0));  // the MMA issuer's barrier
                else
                    mbar_arrive(tempty_bar(acc));
            }
        }
        if (P.out_amax != nullptr) {
            am = warp_max(am);
            if (lane == 0) atomicMax(reinterpret_cast<int *>(P.out_amax), __float_as_int(am));
        }
    }

    __syncwarp();
    tc_fence_before();
    if constexpr (PAIR)
        cluster_sync_all();  // no CTA leaves while its peer may still touch its shared memory
    else
        __syncthreads();
    tc_fence_after();
    if (warp == 1) tmem_dealloc<PAIR>(tmem_base, TMEM_COLS);
}

// ------------------------------------------------- the gate's backward pass

// dg = dh u act'(g), du = dh act(g) from a stored dh, as E5M2 codes. Bound by
// HBM: dh, g and u read (2 or 4 bytes and 4), the codes written (2). Pieces of 8
// columns, so that every access of a warp is one contiguous run, and two pieces
// per thread and step, both loaded before either is used: 8192 x 14336 in 141 us
// from bf16, 0.98 of the copy rate (pieces of 16 columns, whose loads leave
// gaps: 210 us; 8 or 16 blocks per SM: 150, 64: 147; 64-bit divisions for a
// thread's first place: 146).
constexpr int kGateThreads = 256;
constexpr int64_t kGateBlocksPerSm = 32;

template <bool BF16>
struct GatePiece {
    uint4 g, u, d[BF16 ? 1 : 2];
    __device__ __forceinline__ void load(const void *dh, const uint16_t *gu, int64_t row, int64_t col, int64_t cols) {
        g = __ldcs(reinterpret_cast<const uint4 *>(gu + row * 2 * cols + col));
        u = __ldcs(reinterpret_cast<const uint4 *>(gu + row * 2 * cols + cols + col));
        if constexpr (BF16) {
            d[0] = __ldcs(reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(dh) + row * cols + col));
        } else {
            const uint4 *p = reinterpret_cast<const uint4 *>(static_cast<const float *>(dh) + row * cols + col);
            d[0] = __ldcs(p);
            d[1] = __ldcs(p + 1);
        }
    }
    // Elements 4 h .. 4 h + 3 of dh.
    __device__ __forceinline__ void gradient(int h, uint64_t (&x)[2]) const {
        if constexpr (BF16) {
            const uint32_t w0 = h ? d[0].z : d[0].x, w1 = h ? d[0].w : d[0].y;
            x[0] = f2_from_bits(w0 << 16, w0 & 0xFFFF0000u);
            x[1] = f2_from_bits(w1 << 16, w1 & 0xFFFF0000u);
        } else {
            x[0] = f2_from_bits(d[h].x, d[h].y);
            x[1] = f2_from_bits(d[h].z, d[h].w);
        }
    }
};

template <int ACT, bool BF16>
__global__ void __launch_bounds__(kGateThreads)
gate_bwd_kernel(const void *dh, const uint16_t *gu, int64_t rows, int64_t cols, const float *scale_p, uint8_t *dgu8,
                float *amax) {
    pdl_wait();
    pdl_launch_dependents();
    const uint64_t scale = f2_same(*scale_p);
    float am = 0.0f;
    // this thread's pieces are `stride` apart; its place advances without a division
    const int64_t per_row = cols >> 3;
    const int64_t stride = static_cast<int64_t>(gridDim.x) * kGateThreads;
    // (the grid's threads and a row's pieces both fit 32 bits)
    const uint32_t first = blockIdx.x * kGateThreads + threadIdx.x, width = static_cast<uint32_t>(per_row);
    const int64_t step_rows = static_cast<uint32_t>(stride) / width, step = stride - step_rows * per_row;
    int64_t row = first / width, piece = first - static_cast<uint32_t>(row) * width;
    auto advance = [&] {
        row += step_rows;
        piece += step;
        if (piece >= per_row) {
            piece -= per_row;
            ++row;
        }
    };
    while (row < rows) {
        GatePiece<BF16> x[2];
        int64_t r[2], c[2];
        bool there[2];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            r[k] = row;
            c[k] = piece << 3;
            there[k] = row < rows;
            if (there[k]) x[k].load(dh, gu, r[k], c[k], cols);
            advance();
        }
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            if (!there[k]) break;
            const uint32_t g[2][2] = {{x[k].g.x, x[k].g.y}, {x[k].g.z, x[k].g.w}};
            const uint32_t u[2][2] = {{x[k].u.x, x[k].u.y}, {x[k].u.z, x[k].u.w}};
            uint32_t qg[2], qu[2];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                uint64_t d[2];
                x[k].gradient(h, d);
                gate_grad_codes<ACT>(d, g[h], u[h], scale, qg[h], qu[h], am);
            }
            uint8_t *out = dgu8 + r[k] * 2 * cols + c[k];
            *reinterpret_cast<uint2 *>(out) = make_uint2(qg[0], qg[1]);
            *reinterpret_cast<uint2 *>(out + cols) = make_uint2(qu[0], qu[1]);
        }
    }
    if (amax != nullptr) block_amax_atomic(am, amax);
}

// The outputs of an empty contraction.
__global__ void zero_bytes_kernel(uint8_t *p, int64_t n) {
    pdl_wait();
    pdl_launch_dependents();
    const int64_t stride = static_cast<int64_t>(gridDim.x) * blockDim.x;
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x; i < (n >> 4); i += stride)
        reinterpret_cast<uint4 *>(p)[i] = make_uint4(0u, 0u, 0u, 0u);
}

int zero_bytes(void *p, int64_t n, cudaStream_t s, const DeviceInfo &dev) {  // n: a multiple of 16
    int64_t blocks = ((n >> 4) + 255) / 256;
    if (blocks > dev.num_sms * 8) blocks = dev.num_sms * 8;
    if (blocks < 1) return FP8MP_OK;
    const cudaError_t e = launch_kernel(zero_bytes_kernel, dim3(static_cast<unsigned>(blocks)), dim3(256), 0, s,
                                        static_cast<uint8_t *>(p), n);
    if (e != cudaSuccess) return fail(FP8MP_ERR_LAUNCH, "gated: fill launch failed: %s", cudaGetErrorString(e));
    return FP8MP_OK;
}

// ------------------------------------------------------------- host side

std::mutex g_prepare_mutex;

// Sets the kernel's shared memory once per device, and asks how many pairs fit.
template <bool PAIR, int MODE, int ACT, bool H_FP8>
int prepare(const DeviceInfo &dev, int *max_pairs) {
    using C = Cfg<PAIR, MODE>;
    static std::atomic<int> pairs[64];  // 0: not prepared; else resident pairs + 1
    std::atomic<int> &mine = pairs[dev.device & 63];
    int n = mine.load(std::memory_order_acquire);
    if (n == 0) {
        std::lock_guard<std::mutex> lock(g_prepare_mutex);
        const auto kernel = gated_kernel<PAIR, MODE, ACT, H_FP8>;
        const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM_ALLOC);
        if (e != cudaSuccess) return fail(FP8MP_ERR_LAUNCH, "gated: smem attribute failed: %s", cudaGetErrorString(e));
        int fit = dev.num_sms / 2;
        if (PAIR) {
            cudaLaunchConfig_t cfg = {};
            cudaLaunchAttribute attr[1];
            cfg.gridDim = dim3(static_cast<unsigned>(dev.num_sms & ~1));
            cfg.blockDim = dim3(C::THREADS);
            cfg.dynamicSmemBytes = C::SMEM_ALLOC;
            attr[0].id = cudaLaunchAttributeClusterDimension;
            attr[0].val.clusterDim.x = 2;
            attr[0].val.clusterDim.y = 1;
            attr[0].val.clusterDim.z = 1;
            cfg.attrs = attr;
            cfg.numAttrs = 1;
            int got = 0;
            if (cudaOccupancyMaxActiveClusters(&got, kernel, &cfg) == cudaSuccess && got >= 1) fit = got;
        }
        n = fit + 1;
        mine.store(n, std::memory_order_release);
    }
    *max_pairs = n - 1;
    return FP8MP_OK;
}

template <bool PAIR, int MODE, int ACT, bool H_FP8>
int launch(const GatedParams &P, cudaStream_t s, const DeviceInfo &dev) {
    int max_pairs = 0;
    const int rc = prepare<PAIR, MODE, ACT, H_FP8>(dev, &max_pairs);
    if (rc) return rc;
    const int most = PAIR ? max_pairs : dev.num_sms;
    const int clusters = P.num_tiles < most ? P.num_tiles : most;
    const cudaError_t e = launch_kernel_cluster(gated_kernel<PAIR, MODE, ACT, H_FP8>,
                                                dim3(static_cast<unsigned>(PAIR ? 2 * clusters : clusters)),
                                                dim3(Cfg<PAIR, MODE>::THREADS), Cfg<PAIR, MODE>::SMEM_ALLOC, s, PAIR ? 2u : 1u, P);
    if (e != cudaSuccess) return fail(FP8MP_ERR_LAUNCH, "gated: launch failed: %s", cudaGetErrorString(e));
    return FP8MP_OK;
}

// Pairs of SMs on 256-row tiles, or single SMs on 128-row tiles? By the rounds
// of tiles that either takes and what a round costs, fitted to six layers from
// 512 -> 16384 to 8192 -> 4096 with 65 to 4096 tokens, in us. Forward: 0.285 per
// k-block (at least 3.2, the epilogue) and 0.6 once for a pair, 0.36 (2.8) for a
// single, whose operands are half as much again per product. (4096 -> 14336, 128
// tokens: 27.9 with pairs, 25.0 with singles; 256: 28.4, 33.7; 2048 -> 5632, 384
// tokens: 15.0, 10.6.) Dgrad, where a single has three stages only: two thirds.
// (4096 x 14336, 128 tokens: 20.2, 24.3; 384: 31.7, 41.9.) The choice is within 5 %
// of the better one nearly everywhere. FP8MP_GEMM_ENGINE=pair|single overrides it.
bool use_pairs(Mode mode, int64_t rows, int64_t col_tiles, int64_t kc, const DeviceInfo &dev) {
    const char *force = std::getenv("FP8MP_GEMM_ENGINE");
    if (force != nullptr && std::strcmp(force, "pair") == 0) return true;
    if (force != nullptr && std::strcmp(force, "single") == 0) return false;
    const int64_t pairs = dev.num_sms / 2, singles = dev.num_sms;
    const double pair_rounds = static_cast<double>(((rows + 255) / 256 * col_tiles + pairs - 1) / pairs);
    const double single_rounds = static_cast<double>(((rows + 127) / 128 * col_tiles + singles - 1) / singles);
    if (mode == DGRAD) return pair_rounds <= 1.5 * single_rounds;
    const double kb = static_cast<double>((kc + BK - 1) / BK);
    return pair_rounds * std::max(0.285 * kb, 3.2) + 0.6 < single_rounds * std::max(0.36 * kb, 2.8);
}

// bf16 [outer x inner], rows `pitch` bytes apart, in boxes of 128 rows x 64.
int make_bf16_tmap(CUtensorMap *map, const void *ptr, uint64_t inner, uint64_t outer, uint64_t pitch) {
    auto enc = tensor_map_encoder();
    if (enc == nullptr) return fail(FP8MP_ERR_LAUNCH, "cuTensorMapEncodeTiled is not available");
    const cuuint64_t dims[2] = {inner, outer};
    const cuuint64_t strides[1] = {pitch};
    const cuuint32_t box[2] = {64, 128};
    const cuuint32_t estr[2] = {1, 1};
    const CUresult r = enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void *>(ptr), dims, strides, box, estr,
                           CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                           CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r != CUDA_SUCCESS) return fail(FP8MP_ERR_LAUNCH, "cuTensorMapEncodeTiled failed (%d)", static_cast<int>(r));
    return FP8MP_OK;
}

int set_tiles(GatedParams &P, bool pair, int64_t rows, int64_t cols, int64_t kc, int tile_cols, int64_t rows_b) {
    const int tile_m = pair ? 256 : 128;
    const int64_t tm = (rows + tile_m - 1) / tile_m, tn = (cols + tile_cols - 1) / tile_cols;
    if (tm * tn > 0x7FFFFFFF) return fail(FP8MP_ERR_INVALID, "gated: too many tiles");
    P.rows = static_cast<int>(rows);
    P.cols = static_cast<int>(cols);
    P.num_kb = static_cast<int>((kc + BK - 1) / BK);
    P.tiles_m = static_cast<int>(tm);
    P.tiles_n = static_cast<int>(tn);
    P.num_tiles = static_cast<int>(tm * tn);
    P.group_m = raster_group(kc, tile_m);
    P.group_n = raster_columns(rows, rows_b, kc, P.tiles_m, P.tiles_n, P.group_m);
    return FP8MP_OK;
}

}  // namespace

int launch_gated_fwd(const uint8_t *x8, const uint8_t *w8, int64_t M, int64_t F, int64_t K, int act,
                     const float *sinv_x, const float *sinv_w, const float *h_scale, void *h, float *h_amax,
                     uint16_t *gu, cudaStream_t s, const DeviceInfo &dev) {
    const int h_size = h_scale != nullptr ? 1 : 2;
    if (K == 0) {
        const int rc = zero_bytes(h, M * F * h_size, s, dev);
        return rc || gu == nullptr ? rc : zero_bytes(gu, M * F * 4, s, dev);
    }
    if (M <= kFewGatedTokens)
        return launch_few_gated(x8, w8, M, F, K, act, sinv_x, sinv_w, h_scale, h, h_amax, gu, s, dev);
    const bool pair = use_pairs(FWD, M, (F + 127) / 128, K, dev);
    GatedParams P;
    std::memset(&P, 0, sizeof P);
    int rc = set_tiles(P, pair, M, F, K, 128, 2 * F);
    if (rc) return rc;
    P.idesc = make_idesc(FP8MP_E4M3, FP8MP_E4M3, pair ? 256 : 128, TILE_N, 0, 0);
    P.sinv_a = sinv_x;
    P.sinv_b = sinv_w;
    P.out_scale = h_scale;
    P.out_amax = h_amax;
    P.gu = gu;
    P.out = h;
    P.wide = ((reinterpret_cast<uintptr_t>(gu) | (h_size == 2 ? reinterpret_cast<uintptr_t>(h) : 0)) & 31u) == 0;
    const uint64_t m = static_cast<uint64_t>(M), f = static_cast<uint64_t>(F), k = static_cast<uint64_t>(K);
    rc = make_operand_tmap(&P.ta, x8, k, m, ROWS_A);
    if (!rc) rc = make_operand_tmap(&P.tb0, w8, k, f, 128);
    if (!rc) rc = make_operand_tmap(&P.tb1, w8 + F * K, k, f, 128);
    if (rc) return rc;
#define FP8MP_LAUNCH(PAIR_, ACT_) \
    (h_size == 1 ? launch<PAIR_, FWD, ACT_, true>(P, s, dev) : launch<PAIR_, FWD, ACT_, false>(P, s, dev))
    if (act == FP8MP_SILU) return pair ? FP8MP_LAUNCH(true, FP8MP_SILU) : FP8MP_LAUNCH(false, FP8MP_SILU);
    return pair ? FP8MP_LAUNCH(true, FP8MP_GELU_TANH) : FP8MP_LAUNCH(false, FP8MP_GELU_TANH);
#undef FP8MP_LAUNCH
}

int launch_gated_dgrad(const uint8_t *dy8, const uint8_t *wd8, const uint16_t *gu, int64_t M, int64_t F, int64_t N,
                       int act, int dy_fmt, const float *sinv_dy, const float *sinv_wd, const float *dgu_scale,
                       uint8_t *dgu8, float *dgu_amax, cudaStream_t s, const DeviceInfo &dev) {
    if (N == 0) return zero_bytes(dgu8, M * F * 2, s, dev);
    const bool pair = use_pairs(DGRAD, M, (F + 255) / 256, N, dev);
    GatedParams P;
    std::memset(&P, 0, sizeof P);
    int rc = set_tiles(P, pair, M, F, N, 256, F);
    if (rc) return rc;
    P.idesc = make_idesc(dy_fmt, FP8MP_E4M3, pair ? 256 : 128, TILE_N, 0, 1);
    P.sinv_a = sinv_dy;
    P.sinv_b = sinv_wd;
    P.out_scale = dgu_scale;
    P.out_amax = dgu_amax;
    const uint64_t m = static_cast<uint64_t>(M), f = static_cast<uint64_t>(F), n = static_cast<uint64_t>(N);
    rc = make_operand_tmap(&P.ta, dy8, n, m, ROWS_A);
    if (!rc) rc = make_operand_tmap(&P.tb0, wd8, f, n, BK);
    P.tb1 = P.tb0;
    if (!rc) rc = make_bf16_tmap(&P.tg, gu, f, m, 4 * f);
    if (!rc) rc = make_bf16_tmap(&P.tu, gu + F, f, m, 4 * f);
    P.out = dgu8;
    P.wide = F % 32 == 0 && (reinterpret_cast<uintptr_t>(dgu8) & 31u) == 0;
    if (rc) return rc;
    if (act == FP8MP_SILU)
        return pair ? launch<true, DGRAD, FP8MP_SILU, true>(P, s, dev)
                    : launch<false, DGRAD, FP8MP_SILU, true>(P, s, dev);
    return pair ? launch<true, DGRAD, FP8MP_GELU_TANH, true>(P, s, dev)
                : launch<false, DGRAD, FP8MP_GELU_TANH, true>(P, s, dev);
}

int launch_gate_bwd(const void *dh, int dh_dtype, const uint16_t *gu, int64_t M, int64_t F, int act,
                    const float *dgu_scale, uint8_t *dgu8, float *dgu_amax, cudaStream_t s, const DeviceInfo &dev) {
    int64_t blocks = (M * (F >> 3) + kGateThreads - 1) / kGateThreads;
    // a thread starts slowly: two pieces each, once the SMs have their share (1237 x
    // 2736 from bf16: 5.5 us, 6.0 with one; 100 x 2064: 2.1, 1.8)
    if (blocks > 4 * dev.num_sms) blocks = (blocks + 1) / 2;
    if (blocks > dev.num_sms * kGateBlocksPerSm) blocks = dev.num_sms * kGateBlocksPerSm;
    const dim3 grid(static_cast<unsigned>(blocks)), block(kGateThreads);
    cudaError_t e;
    if (act == FP8MP_SILU)
        e = dh_dtype == FP8MP_BF16
                ? launch_kernel(gate_bwd_kernel<FP8MP_SILU, true>, grid, block, 0, s, dh, gu, M, F, dgu_scale, dgu8,
                                dgu_amax)
                : launch_kernel(gate_bwd_kernel<FP8MP_SILU, false>, grid, block, 0, s, dh, gu, M, F, dgu_scale, dgu8,
                                dgu_amax);
    else
        e = dh_dtype == FP8MP_BF16
                ? launch_kernel(gate_bwd_kernel<FP8MP_GELU_TANH, true>, grid, block, 0, s, dh, gu, M, F, dgu_scale,
                                dgu8, dgu_amax)
                : launch_kernel(gate_bwd_kernel<FP8MP_GELU_TANH, false>, grid, block, 0, s, dh, gu, M, F, dgu_scale,
                                dgu8, dgu_amax);
    if (e != cudaSuccess) return fail(FP8MP_ERR_LAUNCH, "gated: launch failed: %s", cudaGetErrorString(e));
    return FP8MP_OK;
}

int read_and_clear_gated_timeout_flag(unsigned int *value) {
    unsigned int v = 0, zero = 0;
    cudaError_t e = cudaMemcpyFromSymbol(&v, g_gated_timeout_flag, sizeof v);
    if (e == cudaSuccess && v != 0) e = cudaMemcpyToSymbol(g_gated_timeout_flag, &zero, sizeof zero);
    if (e != cudaSuccess) return fail(FP8MP_ERR_LAUNCH, "reading the timeout flag failed: %s", cudaGetErrorString(e));
    *value = v;
    return FP8MP_OK;
}

}  // namespace fp8mp
