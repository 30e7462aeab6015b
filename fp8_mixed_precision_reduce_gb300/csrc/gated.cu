// gated.cu -- the gated feed-forward block on the FP8 tensor cores:
//   forward   g = X8 Wg^T s, u = X8 Wu^T s, h = act(g) u in one launch;
//   dgrad     dh = dY8 Wd8 s, dg = dh u act'(g), du = dh act(g) in one launch;
//   gate      dg and du from a high-precision dh (an HBM-bound pass).
//
// The GEMM side is the persistent tcgen05 pipeline of gemm.cu: one CTA per SM
// (or a cluster of two on 256-row tiles), warp 0 the TMA producer, warp 1 the
// MMA issuer, warps 2-5 the epilogue, two TMEM accumulators so that a tile's
// epilogue runs beside the next tile's MMAs. What differs is what a tile is
// and what its epilogue does:
//
//   forward: the 256 accumulator columns are 128 gate columns and the same 128
//     up columns (a pair's even CTA stages the gate rows of W8, its odd CTA
//     the up rows; one CTA alone both), so g and u of one element meet in one
//     thread and h never leaves the SM in more than its 8 (or 16) bits. The
//     pre-activations go out as bf16 only when the backward pass wants them.
//   dgrad: 256 columns of dh; the epilogue fetches the tile's g and u (bf16) by
//     TMA, one 64-column chunk ahead, and writes the E5M2 codes of dg and du.
//     dh itself is never stored: against a GEMM that writes it in bf16 and a
//     pass that reads it back that is 4 bytes per element less traffic.
//
// Both are bound by the tensor cores at training sizes (an epilogue of a few
// dozen instructions per element hides behind a contraction of 4096), and by
// their output traffic at short contractions.
#include <atomic>
#include <cstdlib>
#include <cstring>
#include <mutex>

#include "fp8mp_gate.cuh"
#include "fp8mp_mma.cuh"

namespace fp8mp {

__device__ unsigned int g_gated_timeout_flag = 0;

namespace {

constexpr int NUM_EPI_WARPS = 4;
constexpr int NUM_THREADS = 64 + 32 * NUM_EPI_WARPS;
constexpr uint32_t TMEM_COLS = 2 * TILE_N;
constexpr int BOX_BYTES = 32 * 128;  // one staging box: 32 rows of 128 bytes

enum Mode { FWD = 0, DGRAD = 1 };

// Shared memory of a CTA: the operand ring, each epilogue warp's staging
// boxes, the barriers. Forward: one box each for g, u and h per warp. Dgrad:
// two sets of g and u boxes to load into, and one set (two for a pair, whose
// stages are smaller) of half boxes for the codes of dg and du.
template <bool PAIR, int MODE>
struct Cfg {
    static constexpr int TILE_M = PAIR ? 256 : 128;
    static constexpr int TILE_COLS = MODE == FWD ? 128 : 256;  // columns of h (dh) per tile
    static constexpr int ROWS_B = PAIR ? 128 : 256;
    static constexpr int STAGES = MODE == FWD ? (PAIR ? 5 : 3) : (PAIR ? 4 : 3);
    static constexpr int OUT_SETS = MODE == FWD ? 1 : (PAIR ? 2 : 1);
    static constexpr int A_BYTES = ROWS_A * BK;
    static constexpr int STAGE_BYTES = A_BYTES + ROWS_B * BK;
    static constexpr int TX_BYTES = PAIR ? 2 * STAGE_BYTES : STAGE_BYTES;
    static constexpr int EPI_OFFSET = STAGES * STAGE_BYTES;
    static constexpr int WARP_BYTES = MODE == FWD ? 3 * BOX_BYTES : 4 * BOX_BYTES + OUT_SETS * BOX_BYTES;
    static constexpr int BAR_OFFSET = EPI_OFFSET + NUM_EPI_WARPS * WARP_BYTES;
    static constexpr int NUM_BARS = 2 * STAGES + 5 + (MODE == DGRAD ? 2 * NUM_EPI_WARPS : 0);
    static constexpr int SLOT_OFFSET = BAR_OFFSET + NUM_BARS * 8;
    static constexpr int FLAG_OFFSET = SLOT_OFFSET + 8;
    static constexpr int SMEM_ALLOC = FLAG_OFFSET + 8 + 1024;
    static constexpr uint32_t TEMPTY_COUNT = PAIR ? 2 * NUM_EPI_WARPS : NUM_EPI_WARPS;
    static_assert(STAGE_BYTES % 1024 == 0 && WARP_BYTES % 1024 == 0, "swizzle atoms need 1 KB alignment");
    static_assert(SMEM_ALLOC <= 232448, "shared memory budget");
};

struct GatedParams {
    CUtensorMap ta;        // A: the rows (tokens), K-major
    CUtensorMap tb0, tb1;  // forward: the gate and the up rows of W8; dgrad: Wd8 (both)
    CUtensorMap tg, tu;    // the halves of the pre-activations (forward: written, dgrad: read)
    CUtensorMap to0, to1;  // forward: h; dgrad: the codes of dg and of du
    int rows, cols, num_kb;
    int tiles_m, tiles_n, num_tiles, group_m, group_n;
    uint32_t idesc;
    int save_gu;
    const float *sinv_a, *sinv_b;
    const float *out_scale;
    float *out_amax;
};

__device__ __forceinline__ bool wait_bounded(uint32_t bar, uint32_t parity, volatile int *abort_flag) {
    return fp8mp::wait_bounded(bar, parity, abort_flag, &g_gated_timeout_flag);
}
__device__ __forceinline__ void bulk_wait_read_all() { asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory"); }
__device__ __forceinline__ uint4 ld_shared_v4(uint32_t addr) {
    uint4 v;
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "r"(addr)
                 : "memory");
    return v;
}
// Address of 16-byte chunk `j` of row `r` in a staging box of 128-byte rows
// under the 128-byte swizzle, and of one of 64-byte rows under the 64-byte one.
__device__ __forceinline__ uint32_t box_chunk(uint32_t box, int r, int j) {
    return box + static_cast<uint32_t>(r * 128 + ((j ^ (r & 7)) << 4));
}
__device__ __forceinline__ uint32_t half_box_chunk(uint32_t box, int r, int j) {
    return box + static_cast<uint32_t>(r * 64 + ((j ^ ((r >> 1) & 3)) << 4));
}

// A tile's epilogue in the forward pass, by one warp: 32 rows, 32 columns of
// g and u at a time. Columns past F and rows past M hold zeros (the operands'
// zero fill), whose h is 0: they need no mask in the amax.
template <bool PAIR, int ACT, bool H_FP8>
__device__ __forceinline__ float forward_tile(const GatedParams &P, uint32_t acc, uint32_t boxes, int lane, int row0,
                                              int col0, float scale, float h_scale) {
    const uint32_t box_g = boxes, box_u = boxes + BOX_BYTES, box_h = boxes + 2 * BOX_BYTES;
    float am = 0.0f;
#pragma unroll 1
    for (int c = 0; c < 128; c += 32) {
        uint32_t rg[32], ru[32];
        tmem_ld32(acc + static_cast<uint32_t>(c), rg);
        tmem_ld32(acc + static_cast<uint32_t>(128 + c), ru);
        if (row0 >= P.rows || col0 + c >= P.cols) continue;  // nothing of this warp's chunk exists
        if ((c & 32) == 0) {  // the boxes' last stores must have been read
            if (lane == 0) bulk_wait_read_all();
            __syncwarp();
        }
        uint32_t hq[8];
#pragma unroll
        for (int o = 0; o < 4; ++o) {  // 8 columns each
            float g[8], u[8], h[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                g[j] = __fmul_rn(__uint_as_float(rg[8 * o + j]), scale);
                u[j] = __fmul_rn(__uint_as_float(ru[8 * o + j]), scale);
                h[j] = gate_act<ACT>(g[j]) * u[j];
                am = fmaxf(am, fabsf(h[j]));
            }
            const int chunk = ((c & 32) >> 3) + o;
            if (P.save_gu) {
                st_shared_v4(box_chunk(box_g, lane, chunk), pack_bf16x2(g[0], g[1]), pack_bf16x2(g[2], g[3]),
                             pack_bf16x2(g[4], g[5]), pack_bf16x2(g[6], g[7]));
                st_shared_v4(box_chunk(box_u, lane, chunk), pack_bf16x2(u[0], u[1]), pack_bf16x2(u[2], u[3]),
                             pack_bf16x2(u[4], u[5]), pack_bf16x2(u[6], u[7]));
            }
            if constexpr (H_FP8) {
#pragma unroll
                for (int j = 0; j < 2; ++j)
                    hq[2 * o + j] =
                        cvt_quad<FP8MP_E4M3>(__fmul_rn(h[4 * j], h_scale), __fmul_rn(h[4 * j + 1], h_scale),
                                             __fmul_rn(h[4 * j + 2], h_scale), __fmul_rn(h[4 * j + 3], h_scale));
            } else {
                st_shared_v4(box_chunk(box_h, lane, chunk), pack_bf16x2(h[0], h[1]), pack_bf16x2(h[2], h[3]),
                             pack_bf16x2(h[4], h[5]), pack_bf16x2(h[6], h[7]));
            }
        }
        if constexpr (H_FP8) {
            st_shared_v4(box_chunk(box_h, lane, c >> 4), hq[0], hq[1], hq[2], hq[3]);
            st_shared_v4(box_chunk(box_h, lane, (c >> 4) + 1), hq[4], hq[5], hq[6], hq[7]);
        }
        // a box is full after its last 32 columns, or at the last column block
        const bool last = c == 96 || col0 + c + 32 >= P.cols;
        if ((c & 32) || last) {
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
                const int at = col0 + (c & ~32);
                if (P.save_gu) {
                    tma_store_2d(&P.tg, box_g, at, row0);
                    tma_store_2d(&P.tu, box_u, at, row0);
                }
                if constexpr (!H_FP8)
                    tma_store_2d(&P.to0, box_h, at, row0);
                else if (last)
                    tma_store_2d(&P.to0, box_h, col0, row0);
                bulk_commit_group();
            }
        }
    }
    return am;
}

// The loads of a dgrad tile's g and u boxes for its chunk c (64 columns), by lane 0.
__device__ __forceinline__ void load_gu(const GatedParams &P, uint32_t boxes, uint32_t bar, int col, int row0) {
    mbar_arrive_expect_tx(bar, 2 * BOX_BYTES);
    tma_load_2d_cta(boxes, &P.tg, bar, col, row0);
    tma_load_2d_cta(boxes + BOX_BYTES, &P.tu, bar, col, row0);
}

template <bool PAIR, int MODE, int ACT, bool H_FP8>
__global__ void __launch_bounds__(NUM_THREADS, 1) gated_kernel(const __grid_constant__ GatedParams P) {
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
    auto gu_bar = [&](int w, int b) { return bar0 + 8u * (2 * C::STAGES + 5 + 2 * w + b); };  // dgrad
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
        if constexpr (MODE == DGRAD)
            for (int w = 0; w < NUM_EPI_WARPS; ++w)
                for (int b = 0; b < 2; ++b) mbar_init(gu_bar(w, b), 1);
        *abort_flag = 0;
        fence_mbar_init();
        prefetch_tmap(&P.ta);
        prefetch_tmap(&P.tb0);
        prefetch_tmap(&P.tb1);
        prefetch_tmap(&P.to0);
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
    } else {
        // ---------------- epilogue warps (both CTAs of a pair)
        const int q = warp & 3;  // this warp may access TMEM lanes 32q .. 32q+31
        const uint32_t boxes = base + C::EPI_OFFSET + static_cast<uint32_t>((warp - 2) * C::WARP_BYTES);
        const float scale = __fmul_rn(__ldg(P.sinv_a), __ldg(P.sinv_b));
        const float out_scale = P.out_scale != nullptr ? __ldg(P.out_scale) : 1.0f;
        float am = 0.0f;
        int lt = 0;
        uint32_t loaded = 0, stored = 0;  // dgrad: chunks fetched, sets of code boxes stored
        for (int r = 0; r < rounds; ++r) {
            const int tile = serpentine_tile(r, cluster_id, num_clusters);
            if (tile >= P.num_tiles) continue;
            int mb, nb;
            tile_coords(tile, P.tiles_m, P.tiles_n, P.group_m, P.group_n, mb, nb);
            const int row0 = mb * C::TILE_M + static_cast<int>(rank) * ROWS_A + q * 32;
            const int col0 = nb * C::TILE_COLS;
            // chunks of 64 columns of this warp's rows that exist (dgrad)
            int live = 0;
            if constexpr (MODE == DGRAD) {
                live = row0 < P.rows ? min(4, (P.cols - col0 + 63) / 64) : 0;
                if (lane == 0 && live > 0)
                    load_gu(P, boxes + (loaded & 1u) * 2 * BOX_BYTES, gu_bar(warp - 2, loaded & 1u), col0, row0);
            }
            const int acc = lt & 1;
            const uint32_t aph = (static_cast<uint32_t>(lt) >> 1) & 1u;
            ++lt;
            int ok = 1;
            if (lane == 0) ok = wait_bounded(tfull_bar(acc), aph, abort_flag) ? 1 : 0;
            ok = __shfl_sync(0xffffffffu, ok, 0);
            if (!ok) {
                if (MODE == DGRAD && lane == 0 && live > 0) {  // the load in flight lands first
                    volatile int never = 0;
                    wait_bounded(gu_bar(warp - 2, loaded & 1u), (loaded >> 1) & 1u, &never);
                }
                break;
            }
            tc_fence_after();
            const uint32_t acc_addr =
                tmem_base + static_cast<uint32_t>(acc * TILE_N) + (static_cast<uint32_t>(q * 32) << 16);
            if constexpr (MODE == FWD) {
                am = fmaxf(am, forward_tile<PAIR, ACT, H_FP8>(P, acc_addr, boxes, lane, row0, col0, scale, out_scale));
            } else {
                bool landed = true;
#pragma unroll 1
                for (int c = 0; c < live && landed; ++c) {
                    const uint32_t b = loaded & 1u;
                    const uint32_t box_g = boxes + b * 2 * BOX_BYTES, box_u = box_g + BOX_BYTES;
                    if (lane == 0 && c + 1 < live)  // the other set: every lane is done with it
                        load_gu(P, boxes + (b ^ 1u) * 2 * BOX_BYTES, gu_bar(warp - 2, b ^ 1u), col0 + 64 * (c + 1),
                                row0);
                    landed = wait_bounded(gu_bar(warp - 2, b), (loaded >> 1) & 1u, abort_flag);
                    ++loaded;
                    landed = __all_sync(0xffffffffu, landed);
                    if (!landed) {
                        if (lane == 0 && c + 1 < live) {
                            volatile int never = 0;
                            wait_bounded(gu_bar(warp - 2, loaded & 1u), (loaded >> 1) & 1u, &never);
                        }
                        break;
                    }
                    // the code boxes this chunk writes: their last stores must have been read
                    const uint32_t out =
                        boxes + 4 * BOX_BYTES + (C::OUT_SETS == 2 ? (stored & 1u) * BOX_BYTES : 0u);
                    if (lane == 0) {
                        if (C::OUT_SETS == 2)
                            bulk_wait_read_le1();
                        else
                            bulk_wait_read_all();
                    }
                    __syncwarp();
#pragma unroll 1
                    for (int p = 0; p < 2; ++p) {  // 32 columns each
                        uint32_t rd[32];
                        tmem_ld32(acc_addr + static_cast<uint32_t>(64 * c + 32 * p), rd);
                        uint32_t qg[8], qu[8];
#pragma unroll
                        for (int o = 0; o < 4; ++o) {  // 8 columns each
                            const uint4 wg = ld_shared_v4(box_chunk(box_g, lane, 4 * p + o));
                            const uint4 wu = ld_shared_v4(box_chunk(box_u, lane, 4 * p + o));
                            const uint32_t gw[4] = {wg.x, wg.y, wg.z, wg.w}, uw[4] = {wu.x, wu.y, wu.z, wu.w};
                            float dg[8], du[8];
#pragma unroll
                            for (int j = 0; j < 8; ++j) {
                                const float g = __uint_as_float((j & 1) ? gw[j >> 1] & 0xFFFF0000u : gw[j >> 1] << 16);
                                const float u = __uint_as_float((j & 1) ? uw[j >> 1] & 0xFFFF0000u : uw[j >> 1] << 16);
                                const float dh = __fmul_rn(__uint_as_float(rd[8 * o + j]), scale);
                                float a, da;
                                gate_act_grad<ACT>(g, a, da);
                                dg[j] = dh * u * da;
                                du[j] = dh * a;
                                am = fmaxf(am, fmaxf(fabsf(dg[j]), fabsf(du[j])));
                            }
#pragma unroll
                            for (int j = 0; j < 2; ++j) {
                                qg[2 * o + j] = cvt_quad<FP8MP_E5M2>(
                                    __fmul_rn(dg[4 * j], out_scale), __fmul_rn(dg[4 * j + 1], out_scale),
                                    __fmul_rn(dg[4 * j + 2], out_scale), __fmul_rn(dg[4 * j + 3], out_scale));
                                qu[2 * o + j] = cvt_quad<FP8MP_E5M2>(
                                    __fmul_rn(du[4 * j], out_scale), __fmul_rn(du[4 * j + 1], out_scale),
                                    __fmul_rn(du[4 * j + 2], out_scale), __fmul_rn(du[4 * j + 3], out_scale));
                            }
                        }
#pragma unroll
                        for (int j = 0; j < 2; ++j) {
                            st_shared_v4(half_box_chunk(out, lane, 2 * p + j), qg[4 * j], qg[4 * j + 1], qg[4 * j + 2],
                                         qg[4 * j + 3]);
                            st_shared_v4(half_box_chunk(out + BOX_BYTES / 2, lane, 2 * p + j), qu[4 * j],
                                         qu[4 * j + 1], qu[4 * j + 2], qu[4 * j + 3]);
                        }
                    }
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) {
                        tma_store_2d(&P.to0, out, col0 + 64 * c, row0);
                        tma_store_2d(&P.to1, out + BOX_BYTES / 2, col0 + 64 * c, row0);
                        bulk_commit_group();
                    }
                    ++stored;
                }
                if (!landed) break;
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
        if (lane == 0) bulk_wait_all();  // stores done before the CTA's shared memory goes away
        __syncwarp();
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

// dg = dh u act'(g), du = dh act(g) from a stored dh, as E5M2 codes: 16
// columns per thread and step, 16-byte loads and stores. Bound by HBM: dh, g
// and u read (2 or 4 bytes and 4), the codes written (2).
constexpr int kGateThreads = 256;

template <int ACT, bool BF16>
__global__ void __launch_bounds__(kGateThreads)
gate_bwd_kernel(const void *__restrict__ dh, const uint16_t *__restrict__ gu, int64_t rows, int64_t cols,
                const float *__restrict__ scale_p, uint8_t *__restrict__ dgu8, float *__restrict__ amax) {
    pdl_wait();
    pdl_launch_dependents();
    const float scale = __ldg(scale_p);
    float am = 0.0f;
    const int64_t per_row = cols >> 4, total = rows * per_row;
    const int64_t stride = static_cast<int64_t>(gridDim.x) * kGateThreads;
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * kGateThreads + threadIdx.x; i < total; i += stride) {
        const int64_t row = i / per_row, col = (i - row * per_row) << 4;
        const uint4 *pg = reinterpret_cast<const uint4 *>(gu + row * 2 * cols + col);
        const uint4 *pu = reinterpret_cast<const uint4 *>(gu + row * 2 * cols + cols + col);
        const uint4 g4[2] = {__ldcs(pg), __ldcs(pg + 1)}, u4[2] = {__ldcs(pu), __ldcs(pu + 1)};
        float d[16];
        if constexpr (BF16) {
            const uint4 *pd = reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(dh) + row * cols + col);
            const uint4 d4[2] = {__ldcs(pd), __ldcs(pd + 1)};
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const uint32_t w[4] = {d4[h].x, d4[h].y, d4[h].z, d4[h].w};
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    d[8 * h + 2 * j] = __uint_as_float(w[j] << 16);
                    d[8 * h + 2 * j + 1] = __uint_as_float(w[j] & 0xFFFF0000u);
                }
            }
        } else {
            const float4 *pd = reinterpret_cast<const float4 *>(static_cast<const float *>(dh) + row * cols + col);
#pragma unroll
            for (int h = 0; h < 4; ++h) {
                const float4 v = __ldcs(pd + h);
                d[4 * h] = v.x, d[4 * h + 1] = v.y, d[4 * h + 2] = v.z, d[4 * h + 3] = v.w;
            }
        }
        uint32_t qg[4], qu[4];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const uint32_t gw[4] = {g4[h].x, g4[h].y, g4[h].z, g4[h].w}, uw[4] = {u4[h].x, u4[h].y, u4[h].z, u4[h].w};
            float dg[8], du[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float g = __uint_as_float((j & 1) ? gw[j >> 1] & 0xFFFF0000u : gw[j >> 1] << 16);
                const float u = __uint_as_float((j & 1) ? uw[j >> 1] & 0xFFFF0000u : uw[j >> 1] << 16);
                float a, da;
                gate_act_grad<ACT>(g, a, da);
                dg[j] = d[8 * h + j] * u * da;
                du[j] = d[8 * h + j] * a;
                am = fmaxf(am, fmaxf(fabsf(dg[j]), fabsf(du[j])));
            }
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                qg[2 * h + j] = cvt_quad<FP8MP_E5M2>(__fmul_rn(dg[4 * j], scale), __fmul_rn(dg[4 * j + 1], scale),
                                                     __fmul_rn(dg[4 * j + 2], scale), __fmul_rn(dg[4 * j + 3], scale));
                qu[2 * h + j] = cvt_quad<FP8MP_E5M2>(__fmul_rn(du[4 * j], scale), __fmul_rn(du[4 * j + 1], scale),
                                                     __fmul_rn(du[4 * j + 2], scale), __fmul_rn(du[4 * j + 3], scale));
            }
        }
        *reinterpret_cast<uint4 *>(dgu8 + row * 2 * cols + col) = make_uint4(qg[0], qg[1], qg[2], qg[3]);
        *reinterpret_cast<uint4 *>(dgu8 + row * 2 * cols + cols + col) = make_uint4(qu[0], qu[1], qu[2], qu[3]);
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
            cfg.blockDim = dim3(NUM_THREADS);
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
                                                dim3(NUM_THREADS), Cfg<PAIR, MODE>::SMEM_ALLOC, s, PAIR ? 2u : 1u, P);
    if (e != cudaSuccess) return fail(FP8MP_ERR_LAUNCH, "gated: launch failed: %s", cudaGetErrorString(e));
    return FP8MP_OK;
}

// Pairs of SMs on 256-row tiles when there are enough of them to occupy most
// SMs, as for the plain GEMM; FP8MP_GEMM_ENGINE=pair|single overrides it.
bool use_pairs(int64_t pair_tiles, const DeviceInfo &dev) {
    const char *force = std::getenv("FP8MP_GEMM_ENGINE");
    if (force != nullptr && std::strcmp(force, "pair") == 0) return true;
    if (force != nullptr && std::strcmp(force, "single") == 0) return false;
    return pair_tiles * 2 >= dev.num_sms;
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
    if (M <= kFewTokens)
        return launch_few_gated(x8, w8, M, F, K, act, sinv_x, sinv_w, h_scale, h, h_amax, gu, s, dev);
    const bool pair = use_pairs(((M + 255) / 256) * ((F + 127) / 128), dev);
    GatedParams P;
    std::memset(&P, 0, sizeof P);
    int rc = set_tiles(P, pair, M, F, K, 128, 2 * F);
    if (rc) return rc;
    P.idesc = make_idesc(FP8MP_E4M3, FP8MP_E4M3, pair ? 256 : 128, TILE_N, 0, 0);
    P.sinv_a = sinv_x;
    P.sinv_b = sinv_w;
    P.out_scale = h_scale;
    P.out_amax = h_amax;
    P.save_gu = gu != nullptr;
    const uint64_t m = static_cast<uint64_t>(M), f = static_cast<uint64_t>(F), k = static_cast<uint64_t>(K);
    rc = make_box_tmap(&P.ta, x8, 1, k, m, k, BK, ROWS_A, true);
    if (!rc) rc = make_box_tmap(&P.tb0, w8, 1, k, f, k, BK, 128, true);
    if (!rc) rc = make_box_tmap(&P.tb1, w8 + F * K, 1, k, f, k, BK, 128, true);
    if (!rc) rc = make_box_tmap(&P.to0, h, h_size, f, m, f * h_size, 128 / h_size, 32, false);
    if (!rc && gu != nullptr) rc = make_box_tmap(&P.tg, gu, 2, f, m, 4 * f, 64, 32, false);
    if (!rc && gu != nullptr) rc = make_box_tmap(&P.tu, gu + F, 2, f, m, 4 * f, 64, 32, false);
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
    const bool pair = use_pairs(((M + 255) / 256) * ((F + 255) / 256), dev);
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
    rc = make_box_tmap(&P.ta, dy8, 1, n, m, n, BK, ROWS_A, true);
    if (!rc) rc = make_box_tmap(&P.tb0, wd8, 1, f, n, f, 128, BK, true);
    P.tb1 = P.tb0;
    if (!rc) rc = make_box_tmap(&P.tg, gu, 2, f, m, 4 * f, 64, 32, true);
    if (!rc) rc = make_box_tmap(&P.tu, gu + F, 2, f, m, 4 * f, 64, 32, true);
    if (!rc) rc = make_box_tmap(&P.to0, dgu8, 1, f, m, 2 * f, 64, 32, false);
    if (!rc) rc = make_box_tmap(&P.to1, dgu8 + F, 1, f, m, 2 * f, 64, 32, false);
    if (rc) return rc;
    if (act == FP8MP_SILU)
        return pair ? launch<true, DGRAD, FP8MP_SILU, true>(P, s, dev)
                    : launch<false, DGRAD, FP8MP_SILU, true>(P, s, dev);
    return pair ? launch<true, DGRAD, FP8MP_GELU_TANH, true>(P, s, dev)
                : launch<false, DGRAD, FP8MP_GELU_TANH, true>(P, s, dev);
}

int launch_gate_bwd(const void *dh, int dh_dtype, const uint16_t *gu, int64_t M, int64_t F, int act,
                    const float *dgu_scale, uint8_t *dgu8, float *dgu_amax, cudaStream_t s, const DeviceInfo &dev) {
    int64_t blocks = (M * (F >> 4) + kGateThreads - 1) / kGateThreads;
    if (blocks > dev.num_sms * 32ll) blocks = dev.num_sms * 32ll;
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
    if (e == cudaSuccess) e = cudaMemcpyToSymbol(g_gated_timeout_flag, &zero, sizeof zero);
    if (e != cudaSuccess) return fail(FP8MP_ERR_LAUNCH, "reading the timeout flag failed: %s", cudaGetErrorString(e));
    *value = v;
    return FP8MP_OK;
}

}  // namespace fp8mp
