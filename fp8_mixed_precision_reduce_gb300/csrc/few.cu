// few.cu -- products of FP8 weights with a few tokens: the gated feed-forward
// block's first half, h = act(x Wg^T) (x Wu^T), for 1 to 64, and a plain linear,
// y = x W^T (+ b), for 1 to 128, as a model that serves runs them token by token.
//
// Every weight byte is read once and used for at most 128 products, so the
// kernel is bound by HBM. It is shaped to keep many weight loads in flight on
// all SMs rather than to keep the tensor cores busy:
//   - the weights are the MMA's M operand (128 rows per tile; gated: 64 gate
//     rows and the 64 up rows of the same outputs), the tokens its N operand
//     (16 to 128 columns, rows past the last token zero-filled), so a stage
//     is 16 KB of weights and 2-16 KB of tokens, in a ring of 72 to 90 KB: two
//     CTAs share an SM and one streams while the other starts or ends (128
//     columns, whose sums alone take 64 KB, have an SM for each CTA, 160 KB);
//   - a tile's contraction is split over the S CTAs of a cluster (split_for
//     below). Each owns an S-th of the tile's outputs; all send it their fp32
//     partial sums of those through distributed shared memory, and after one
//     cluster barrier it adds them from its own, in rank order: no workspace, no
//     atomics on the sums, and no CTA has to outlive its peers. (Reading the
//     peers' sums instead takes a second barrier, about 1 us, and 16-byte reads
//     from 32 rows at once, 2-3 us for 33 tokens.)
// One token through 4096 -> 2 x 14336: 21.2 us (17.3 at the copy rate), through
// 14336 -> 4096: 12.6 (8.7), 128 tokens 15.6; 65536 x 14336: 137 us, the copy rate.
// What is left is the start, about 2 us to the first bytes, and the end.
#include <atomic>
#include <cstring>
#include <mutex>

#include "fp8mp_gate.cuh"
#include "fp8mp_mma.cuh"

namespace fp8mp {

__device__ unsigned int g_few_timeout_flag = 0;

namespace {

constexpr int NUM_THREADS = 192;  // producer warp, MMA warp, four epilogue warps
constexpr int W_ROWS = 128;       // weight rows of a tile
constexpr uint32_t kMaxSplits = 8;  // CTAs that may share a tile's contraction (a portable cluster)

template <int NT>
struct Cfg {
    static constexpr int STAGE_BYTES = W_ROWS * BK + NT * BK;
    static constexpr int RECV_BYTES = W_ROWS * NT * 4;  // partial sums from all ranks for this CTA's outputs
    static constexpr int CTAS = NT <= 64 ? 2 : 1;  // per SM
    static constexpr int STAGES = ((CTAS == 2 ? 112 : 224) * 1024 - RECV_BYTES) / STAGE_BYTES;
    static constexpr int RECV_OFFSET = STAGES * STAGE_BYTES;
    static constexpr int BAR_OFFSET = RECV_OFFSET + RECV_BYTES;
    static constexpr int SLOT_OFFSET = BAR_OFFSET + (2 * STAGES + 2) * 8;
    static constexpr int FLAG_OFFSET = SLOT_OFFSET + 8;
    static constexpr int SMEM_ALLOC = FLAG_OFFSET + 8 + 1024;
    static constexpr uint32_t TMEM_COLS = NT < 32 ? 32 : NT;
    static_assert(CTAS * (SMEM_ALLOC + 1024) <= 233472, "an SM's shared memory");
};

struct FewParams {
    CUtensorMap tw0, tw1, tx;  // the weights (gated: gate rows, up rows) and the tokens
    int rows, outs, num_kb;    // tokens, outputs (gated: F), 128-byte k-blocks
    uint32_t idesc;
    const float *sinv_a, *sinv_b;
    // gated: h as E4M3 under *out_scale or as bf16, gu when saved; linear: y as bf16 or fp32, with a bias
    const float *out_scale;
    void *out;
    uint16_t *gu;
    const void *bias;
    int bias_bf16, out_bf16;
    float *out_amax;
};

__device__ __forceinline__ bool wait_bounded(uint32_t bar, uint32_t parity, volatile int *abort_flag) {
    return fp8mp::wait_bounded(bar, parity, abort_flag, &g_few_timeout_flag);
}

// 16 consecutive fp32 columns of this warp's 32 TMEM lanes.
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr)
        : "memory");
}

__device__ __forceinline__ void st_shared_cluster_f32(uint32_t cluster_addr, float v) {
    asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(cluster_addr), "f"(v) : "memory");
}
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }

// GATED: ACT is the activation; otherwise unused.
template <bool GATED, int ACT, int NT>
__global__ void __launch_bounds__(NUM_THREADS, Cfg<NT>::CTAS) few_kernel(const __grid_constant__ FewParams P, uint32_t splits) {
    using C = Cfg<NT>;
    extern __shared__ uint8_t smem_raw[];
    uint32_t base = smem_u32(smem_raw);
    const uint32_t pad = (1024u - (base & 1023u)) & 1023u;
    uint8_t *smem = smem_raw + pad;
    base += pad;
    const uint32_t bar0 = base + C::BAR_OFFSET;
    auto full_bar = [&](int s) { return bar0 + 8u * s; };
    auto empty_bar = [&](int s) { return bar0 + 8u * (C::STAGES + s); };
    const uint32_t done_bar = bar0 + 8u * (2 * C::STAGES), drain_bar = done_bar + 8u;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + C::SLOT_OFFSET);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(smem + C::FLAG_OFFSET);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = splits > 1 ? cluster_ctarank() : 0u;
    const int tile = static_cast<int>(blockIdx.x / splits);

    if (threadIdx.x == 0) {
        for (int s = 0; s < C::STAGES; ++s) {
            mbar_init(full_bar(s), 1);
            mbar_init(empty_bar(s), 1);
        }
        mbar_init(done_bar, 1);
        mbar_init(drain_bar, 1);
        *abort_flag = 0;
        fence_mbar_init();
        prefetch_tmap(&P.tw0);
        if (GATED) prefetch_tmap(&P.tw1);
        prefetch_tmap(&P.tx);
    }
    if (warp == 1) {
        tmem_alloc<false>(smem_u32(tmem_slot), C::TMEM_COLS);
        tmem_relinquish<false>();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    if (splits > 1) cluster_arrive();  // this CTA has started: its peers may write to it
    pdl_wait();

    // local rows (weight rows whose sums one CTA owns) of the tile: gated, the
    // gate rows and then the up rows of its outputs
    constexpr int TILE_OUTS = GATED ? 64 : W_ROWS;
    const int mine = TILE_OUTS / static_cast<int>(splits);  // 8 .. 128, a power of two
    const int local_rows = W_ROWS / static_cast<int>(splits);
    const int64_t col0 = static_cast<int64_t>(tile) * TILE_OUTS + static_cast<int64_t>(rank) * mine;
    // what the last step needs besides the sums is fetched now (33 tokens, 1552 ->
    // 6000 with a bias: 6.5 us, 7.0 if at the end)
    const float sinv_a = *P.sinv_a, sinv_b = *P.sinv_b;
    const float h_scale = GATED && P.out_scale != nullptr ? *P.out_scale : 0.0f;
    __shared__ float bias[GATED ? 1 : W_ROWS];
    if constexpr (!GATED) {
        const int o = static_cast<int>(threadIdx.x) - 64;
        if (P.bias != nullptr && o >= 0 && o < mine && col0 + o < P.outs)
            bias[o] = P.bias_bf16 ? bf16_bits_to_f32(static_cast<const uint16_t *>(P.bias)[col0 + o])
                                  : static_cast<const float *>(P.bias)[col0 + o];
    }

    // this CTA's share of the contraction (never empty: splits <= num_kb)
    const int kb0 = static_cast<int>(static_cast<int64_t>(P.num_kb) * rank / splits);
    const int kb1 = static_cast<int>(static_cast<int64_t>(P.num_kb) * (rank + 1) / splits);
    bool failed = false;
    if (warp == 0) {
        if (lane == 0) {
            pdl_launch_dependents();
            uint32_t it = 0;
            bool ok = true;
            for (int kb = kb0; kb < kb1; ++kb, ++it) {
                const int s = static_cast<int>(it % C::STAGES);
                if (!wait_bounded(empty_bar(s), ((it / C::STAGES) & 1u) ^ 1u, abort_flag)) {
                    ok = false;
                    break;
                }
                const uint32_t sw = base + s * C::STAGE_BYTES;
                mbar_arrive_expect_tx(full_bar(s), C::STAGE_BYTES);
                if constexpr (GATED) {
                    tma_load_2d<false>(sw, &P.tw0, full_bar(s), kb * BK, tile * 64);
                    tma_load_2d<false>(sw + 64 * BK, &P.tw1, full_bar(s), kb * BK, tile * 64);
                } else {
                    tma_load_2d<false>(sw, &P.tw0, full_bar(s), kb * BK, tile * W_ROWS);
                }
                tma_load_2d<false>(sw + W_ROWS * BK, &P.tx, full_bar(s), kb * BK, 0);
            }
            if (!ok) {  // let the loads already issued land before the CTA goes away
                for (uint32_t j = 1; j <= static_cast<uint32_t>(C::STAGES) && j <= it; ++j) {
                    const uint32_t at = it - j;
                    volatile int never = 0;
                    wait_bounded(full_bar(static_cast<int>(at % C::STAGES)), (at / C::STAGES) & 1u, &never);
                }
            }
        }
    } else if (warp == 1) {
        if (lane == 0) {
            bool ok = true;
            uint32_t it = 0;
            for (int kb = kb0; kb < kb1; ++kb, ++it) {
                const int s = static_cast<int>(it % C::STAGES);
                if (!wait_bounded(full_bar(s), (it / C::STAGES) & 1u, abort_flag)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                const uint32_t sw = base + s * C::STAGE_BYTES;
#pragma unroll
                for (int k = 0; k < BK / UMMA_K; ++k)
                    umma_f8f6f4<false>(tmem, sw128_kmajor_desc(sw + k * UMMA_K),
                                       sw128_kmajor_desc(sw + W_ROWS * BK + k * UMMA_K), P.idesc,
                                       (it > 0 || k > 0) ? 1u : 0u);
                umma_commit_all<false>(empty_bar(s));
            }
            umma_commit_all<false>(ok ? done_bar : drain_bar);
            if (!ok) {  // wait for the MMAs in flight before TMEM is released
                volatile int never = 0;
                wait_bounded(drain_bar, 0u, &never);
            }
        }
    } else {
        int ok = 1;
        if (lane == 0) ok = wait_bounded(done_bar, 0u, abort_flag) ? 1 : 0;
        ok = __shfl_sync(0xffffffffu, ok, 0);
        failed = !ok;
    }
    __syncwarp();
    if (splits > 1) cluster_wait();
    if (warp >= 2 && !failed) {
        tc_fence_after();
        const int q = warp & 3, row = 32 * q + lane;
        const int o = row & (TILE_OUTS - 1);
        const uint32_t owner = static_cast<uint32_t>(o / mine);
        const int lr = (row / TILE_OUTS) * mine + (o & (mine - 1));
        // received sums: [rank][token][local row]
        uint32_t dst = base + C::RECV_OFFSET + static_cast<uint32_t>((rank * NT * local_rows + lr) * 4);
        if (splits > 1) dst = mapa_shared(dst, owner);
#pragma unroll
        for (int c = 0; c < NT; c += 16) {
            if (c >= P.rows) break;
            uint32_t r[16];
            tmem_ld16(tmem + static_cast<uint32_t>(c) + (static_cast<uint32_t>(32 * q) << 16), r);
#pragma unroll
            for (int j = 0; j < 16; ++j)
                if (c + j < P.rows)
                    st_shared_cluster_f32(dst + static_cast<uint32_t>((c + j) * local_rows * 4), __uint_as_float(r[j]));
        }
    }
    __syncwarp();
    tc_fence_before();
    if (splits > 1) cluster_arrive();
    __syncthreads();  // (tensor memory has been read by every warp)
    tc_fence_after();
    if (warp == 1) tmem_dealloc<false>(tmem, C::TMEM_COLS);
    if (splits > 1) cluster_wait();

    // this CTA's outputs, four at a time, all tokens
    const float scale = __fmul_rn(sinv_a, sinv_b);
    const int quads = mine >> 2, shift = 31 - __clz(quads);
    const float *recv = reinterpret_cast<const float *>(smem + C::RECV_OFFSET);
    auto joined = [&](int lr, int m, float(&s)[4]) {  // in rank order
        const float4 first = *reinterpret_cast<const float4 *>(recv + m * local_rows + lr);
        s[0] = first.x, s[1] = first.y, s[2] = first.z, s[3] = first.w;
        for (uint32_t r = 1; r < splits; ++r) {
            const float4 x = *reinterpret_cast<const float4 *>(recv + (r * NT + m) * local_rows + lr);
            s[0] = __fadd_rn(s[0], x.x), s[1] = __fadd_rn(s[1], x.y);
            s[2] = __fadd_rn(s[2], x.z), s[3] = __fadd_rn(s[3], x.w);
        }
    };
    float am = 0.0f;
    for (int i = threadIdx.x; i < quads * P.rows; i += NUM_THREADS) {
        const int m = i >> shift, o = 4 * (i & (quads - 1));
        const int64_t col = col0 + o;
        if (col >= P.outs) continue;  // (P.outs is a multiple of 16)
        const int64_t at = static_cast<int64_t>(m) * P.outs + col;
        float a[4], y[4];
        joined(o, m, a);
        if constexpr (GATED) {
            float u[4];
            joined(mine + o, m, u);
#pragma unroll
            for (int j = 0; j < 4; j += 2) {
                const uint64_t g2 = f2_mul(f2_pack(a[j], a[j + 1]), f2_same(scale));
                const uint64_t u2 = f2_mul(f2_pack(u[j], u[j + 1]), f2_same(scale));
                f2_split(g2, a[j], a[j + 1]);
                f2_split(u2, u[j], u[j + 1]);
                f2_split(f2_mul(gate_act<ACT>(g2), u2), y[j], y[j + 1]);
                am = fmaxf(am, fmaxf(fabsf(y[j]), fabsf(y[j + 1])));
            }
            if (P.out_scale != nullptr)
                *reinterpret_cast<uint32_t *>(static_cast<uint8_t *>(P.out) + at) =
                    cvt_quad<FP8MP_E4M3>(__fmul_rn(y[0], h_scale), __fmul_rn(y[1], h_scale), __fmul_rn(y[2], h_scale),
                                         __fmul_rn(y[3], h_scale));
            else
                *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(P.out) + at) =
                    make_uint2(pack_bf16x2(y[0], y[1]), pack_bf16x2(y[2], y[3]));
            if (P.gu != nullptr) {
                uint16_t *row = P.gu + static_cast<int64_t>(m) * 2 * P.outs + col;
                *reinterpret_cast<uint2 *>(row) = make_uint2(pack_bf16x2(a[0], a[1]), pack_bf16x2(a[2], a[3]));
                *reinterpret_cast<uint2 *>(row + P.outs) = make_uint2(pack_bf16x2(u[0], u[1]), pack_bf16x2(u[2], u[3]));
            }
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                y[j] = __fmul_rn(a[j], scale);
                if (P.bias != nullptr) y[j] = __fmaf_rn(a[j], scale, bias[o + j]);
            }
            if (P.out_bf16) {
                const uint32_t lo = pack_bf16x2(y[0], y[1]), hi = pack_bf16x2(y[2], y[3]);
                *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(P.out) + at) = make_uint2(lo, hi);
                y[0] = __uint_as_float(lo << 16), y[1] = __uint_as_float(lo & 0xFFFF0000u);
                y[2] = __uint_as_float(hi << 16), y[3] = __uint_as_float(hi & 0xFFFF0000u);
            } else {
                *reinterpret_cast<float4 *>(static_cast<float *>(P.out) + at) = make_float4(y[0], y[1], y[2], y[3]);
            }
            am = fmaxf(fmaxf(am, fmaxf(fabsf(y[0]), fabsf(y[1]))), fmaxf(fabsf(y[2]), fabsf(y[3])));
        }
    }
    if (P.out_amax != nullptr) block_amax_atomic(am, P.out_amax);
}

// How many CTAs share a tile's contraction. Each costs its share of k-blocks and,
// for starting, filling its ring and joining, about as long as `kFixed` k-blocks of
// streaming take it. The split with the least (waves of clusters) x (cost of one
// CTA) is taken: more CTAs even out the last wave of a few tiles, fewer save fixed
// costs when there are many. `fit`: the clusters of 1, 2, 4 and 8 CTAs that the
// device holds at once: at one CTA per SM fewer of 8 than SMs / 8, as not every
// group of SMs is a multiple of 8 (16 tiles of 44 k-blocks, 65 tokens: 6.9 us in
// 16 clusters of 4, 11.0 in 16 of 8, of which 15 fit).
constexpr int kFixed = 8;

int split_for(int64_t tiles, int num_kb, const std::atomic<int> (&fit)[4]) {
    int best = 1;
    double least = 0.0;
    for (int i = 0, s = 1; s <= static_cast<int>(kMaxSplits) && s <= num_kb; ++i, s *= 2) {
        const int64_t at_once = fit[i].load(std::memory_order_relaxed);
        const int64_t waves = (tiles + at_once - 1) / at_once;
        const double cost = static_cast<double>(waves) * ((num_kb + s - 1) / s + kFixed);
        if (s == 1 || cost < least) {
            least = cost;
            best = s;
        }
    }
    return best;
}

std::mutex g_prepare_mutex;

// Per device: the kernel's shared memory is set, and how many clusters fit.
struct Prepared {
    std::atomic<bool> ready;
    std::atomic<int> fit[4];
};

template <bool GATED, int ACT, int NT>
int launch(const FewParams &P, int64_t tiles, cudaStream_t s, const DeviceInfo &dev) {
    using C = Cfg<NT>;
    static Prepared prepared[64];
    Prepared &mine = prepared[dev.device & 63];
    const auto kernel = few_kernel<GATED, ACT, NT>;
    if (!mine.ready.load(std::memory_order_acquire)) {
        std::lock_guard<std::mutex> lock(g_prepare_mutex);
        const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM_ALLOC);
        if (e != cudaSuccess) return fail(FP8MP_ERR_LAUNCH, "few: smem attribute failed: %s", cudaGetErrorString(e));
        for (int i = 0; i < 4; ++i) {
            int fit = C::CTAS * dev.num_sms >> i;
            if (C::CTAS == 1 && i > 0) {
                cudaLaunchConfig_t cfg = {};
                cudaLaunchAttribute attr[1];
                cfg.gridDim = dim3(static_cast<unsigned>(C::CTAS * dev.num_sms >> i << i));
                cfg.blockDim = dim3(NUM_THREADS);
                cfg.dynamicSmemBytes = C::SMEM_ALLOC;
                attr[0].id = cudaLaunchAttributeClusterDimension;
                attr[0].val.clusterDim.x = 1u << i;
                attr[0].val.clusterDim.y = 1;
                attr[0].val.clusterDim.z = 1;
                cfg.attrs = attr;
                cfg.numAttrs = 1;
                int got = 0;
                if (cudaOccupancyMaxActiveClusters(&got, kernel, &cfg) == cudaSuccess && got >= 1) fit = got;
            }
            mine.fit[i].store(fit, std::memory_order_relaxed);
        }
        mine.ready.store(true, std::memory_order_release);
    }
    const int splits = split_for(tiles, P.num_kb, mine.fit);
    const cudaError_t e = launch_kernel_cluster(kernel, dim3(static_cast<unsigned>(tiles * splits)), dim3(NUM_THREADS),
                                                C::SMEM_ALLOC, s, static_cast<unsigned>(splits), P,
                                                static_cast<uint32_t>(splits));
    if (e != cudaSuccess) return fail(FP8MP_ERR_LAUNCH, "few: launch failed: %s", cudaGetErrorString(e));
    return FP8MP_OK;
}

template <bool GATED, int ACT>
int launch_tokens(const FewParams &P, int nt, int64_t tiles, cudaStream_t s, const DeviceInfo &dev) {
    if (nt == 16) return launch<GATED, ACT, 16>(P, tiles, s, dev);
    if (nt == 32) return launch<GATED, ACT, 32>(P, tiles, s, dev);
    if constexpr (!GATED)
        if (nt == 128) return launch<GATED, ACT, 128>(P, tiles, s, dev);
    return launch<GATED, ACT, 64>(P, tiles, s, dev);
}

// The operands of a few tokens against `outs` outputs (gated: of
// w8's 2 * outs rows) over K.
int set_operands(FewParams &P, const uint8_t *x8, const uint8_t *w8, int64_t M, int64_t outs, int64_t K, bool gated,
                 int nt) {
    std::memset(&P, 0, sizeof P);
    P.rows = static_cast<int>(M);
    P.outs = static_cast<int>(outs);
    P.num_kb = static_cast<int>((K + BK - 1) / BK);
    P.idesc = make_idesc(FP8MP_E4M3, FP8MP_E4M3, W_ROWS, nt, 0, 0);
    const uint64_t m = static_cast<uint64_t>(M), n = static_cast<uint64_t>(outs), k = static_cast<uint64_t>(K);
    const uint32_t box = gated ? 64 : W_ROWS;
    int rc = make_operand_tmap(&P.tx, x8, k, m, static_cast<uint32_t>(nt));
    if (!rc) rc = make_operand_tmap(&P.tw0, w8, k, n, box);
    if (!rc && gated) rc = make_operand_tmap(&P.tw1, w8 + outs * K, k, n, box);
    return rc;
}

int token_columns(int64_t M) { return M <= 16 ? 16 : (M <= 32 ? 32 : (M <= 64 ? 64 : 128)); }

}  // namespace

int launch_few_gated(const uint8_t *x8, const uint8_t *w8, int64_t M, int64_t F, int64_t K, int act,
                     const float *sinv_x, const float *sinv_w, const float *h_scale, void *h, float *h_amax,
                     uint16_t *gu, cudaStream_t s, const DeviceInfo &dev) {
    FewParams P;
    const int nt = token_columns(M);
    const int rc = set_operands(P, x8, w8, M, F, K, true, nt);
    if (rc) return rc;
    P.sinv_a = sinv_x;
    P.sinv_b = sinv_w;
    P.out_scale = h_scale;
    P.out = h;
    P.gu = gu;
    P.out_amax = h_amax;
    const int64_t tiles = (F + 63) / 64;
    return act == FP8MP_SILU ? launch_tokens<true, FP8MP_SILU>(P, nt, tiles, s, dev)
                             : launch_tokens<true, FP8MP_GELU_TANH>(P, nt, tiles, s, dev);
}

int launch_few_linear(const uint8_t *x8, const uint8_t *w8, int64_t M, int64_t N, int64_t K, const float *sinv_x,
                      const float *sinv_w, const void *bias, int bias_dtype, void *y, int y_dtype, float *y_amax,
                      cudaStream_t s, const DeviceInfo &dev) {
    FewParams P;
    const int nt = token_columns(M);
    const int rc = set_operands(P, x8, w8, M, N, K, false, nt);
    if (rc) return rc;
    P.sinv_a = sinv_x;
    P.sinv_b = sinv_w;
    P.out = y;
    P.out_bf16 = y_dtype == FP8MP_BF16;
    P.bias = bias;
    P.bias_bf16 = bias_dtype == FP8MP_BF16;
    P.out_amax = y_amax;
    const int64_t tiles = (N + W_ROWS - 1) / W_ROWS;
    return launch_tokens<false, FP8MP_SILU>(P, nt, tiles, s, dev);
}

int read_and_clear_few_timeout_flag(unsigned int *value) {
    unsigned int v = 0, zero = 0;
    cudaError_t e = cudaMemcpyFromSymbol(&v, g_few_timeout_flag, sizeof v);
    if (e == cudaSuccess && v != 0) e = cudaMemcpyToSymbol(g_few_timeout_flag, &zero, sizeof zero);
    if (e != cudaSuccess) return fail(FP8MP_ERR_LAUNCH, "reading the timeout flag failed: %s", cudaGetErrorString(e));
    *value = v;
    return FP8MP_OK;
}

}  // namespace fp8mp
