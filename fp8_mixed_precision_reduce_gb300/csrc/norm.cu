// norm.cu -- root-mean-square norm with the residual's addition and an E4M3
// output under a delayed scale, and its gradient.
//
// Forward, for each row of K:   t = round(x + r),  rstd = 1 / sqrt(mean(t^2) + eps),
//                               y = (t rstd) w,    code = sat_rne_E4M3(y scale)
// Backward, with n = t rstd and g = dy w:
//                               dt = rstd (g - n mean(g n)) + dT,   dw = sum over rows of dy n
// A row is read once and stays in registers between its sum and its use, so both
// are bound by HBM: bf16 and E4M3 out, 7 bytes an element forward (x, r, t, the
// code), 8 backward (dy, t, dT, dt). The weight and its gradient's running sums
// stay in registers over all rows that a thread's columns see.
//
// A thread takes 16 columns of a row (32 of rows past 4096), a warp or several up to
// 512 threads share it, and rows of up to 2048 columns are taken two to eight at a
// time by a block of 256 threads. Each warp copies its own pieces of the rows to come
// into shared memory (cp.async) and reads nothing else there, so no barrier is
// needed but the one inside a row's sum, and loads are in flight while a row is
// reduced and written. 16384 x 4096, bf16: forward with residual and E4M3 out 71 us
// (6.6 TB/s), backward 82.6 (6.5), 86 and 126 with loads into registers instead.
#include <atomic>

#include "fp8mp_lm.cuh"
#include "fp8mp_pieces.cuh"

namespace fp8mp {

namespace {

constexpr int kBlock = 256;         // threads of a block whose threads take 16 columns, at most
constexpr int kWideBlock = 512;     // 32 columns
constexpr int kMaxGroups = kBlock / 32;  // rows that a block takes at a time, at most
// Blocks of kBlock threads for each SM in the forward pass, where two or three are
// resident: shares small enough to even out the tail. 16384 x 4096, bf16 with
// residual: 82.5 us with 3, 73.9 with 4, 72.7 with 8, 76.9 with 36; without
// residual 43.4, 49.2, 45.2, 56.6; 8192 x 4096 with an fp32 residual 62.8, 62.8, 58.3, 68.3.
// Wide ones, one or two of which are resident, in whole waves: 6000 x 11472 84.9 us with
// one, 78.4 with 4, 90.4 with 5.3; 12000 x 5600 84.6, 76.3, 78.2; 8000 x 16384 151.5, 142.9.
constexpr int kBlocksPerSm = 8, kWaves = 4;
// Up to so many rows (or rows at a time) an SM, as many blocks as are resident: a second
// wave of blocks would begin with a row's whole latency. 2000 x 4096 11.3 us, 14.8 by more
// blocks; 1000 x 8192 12.8, 19.0; 8741 x 912 11.1, 14.4; 4000 x 4096 20.2, 22.0; 6000 29.2, 28.4.
constexpr int64_t kFewUnits = 28;
constexpr int kGradSms = 152;       // the backward pass's blocks are for so many SMs; each leaves a row of sums
constexpr int kSmem = 216 * 1024;   // what the blocks on an SM may use together

struct NormArgs {
    const void *x, *r, *w;
    void *t, *y;
    float *rstd, *amax;
    const float *scale;
    int64_t M;
    int K, tpr;  // threads that share a row
    float eps;
    bool w_bf16, y_bf16;
};

struct NormGradArgs {
    const void *dy, *dtotal, *t, *w;
    const float *rstd;
    void *dr, *dx;
    float *partial;  // [gridDim.x][K] sums of dy n, or NULL
    int64_t M;
    int K, tpr;
    bool w_bf16;
};

constexpr int threads_of(int n) { return n == 2 ? kBlock : kWideBlock; }
// Blocks that an SM holds, of threads with N pieces each and `bytes` of a row.
constexpr int per_sm(int threads, int n, int bytes, int stages) {
    const int by_threads = n == 2 ? 3 * kBlock / threads : kWideBlock / threads;
    const int by_smem = kSmem / (threads * bytes * stages);
    return by_threads < 1 || by_smem < 1 ? 1 : by_threads < by_smem ? by_threads : by_smem;
}
// Rows in flight for each group of threads: three where that costs no blocks, two
// where they fit; else one, refilled piece by piece as it is used for the last time.
constexpr int stages(int bytes, int n) {
    const int threads = threads_of(n), blocks = n == 2 ? 3 : 1;
    return threads * bytes * 3 * blocks <= kSmem ? 3 : threads * bytes * 2 <= kSmem ? 2 : 1;
}

// A warp's copies of one array's pieces: N of a row for each lane, 32 pieces one
// after another. A lane copies 16-byte units 32 lanes apart, so it reads what other
// lanes copied: the warp meets between the copies' arrival and their use, and
// between their use and the next copies.
template <bool BF16, int N>
struct Slot {
    static constexpr int UNITS = BF16 ? 1 : 2, BYTES = N * UNITS * 16;
    int64_t next;         // address of the lane's first unit of the next row to fetch
    int64_t step;         // to the one after it
    int units, gap;       // of the row from there on; from piece v to piece v + 1
    uint32_t to, from;    // where the lane's first unit goes, and where its first piece lies, in the first stage

    // `ring`: of this array, in the first stage; row: the first one, rows: between a block's rows.
    // x: the array, or NULL where each fetch names its own.
    __device__ __forceinline__ Slot(uint32_t ring, const void *x, int64_t row, int64_t rows, int pieces, int tid, int tpr) {
        const int lane = threadIdx.x & 31, first = (tid - lane) * UNITS + lane;
        next = reinterpret_cast<int64_t>(x) + (row * pieces * UNITS + first) * 16;
        step = rows * pieces * (UNITS * 16);
        units = pieces * UNITS - first;
        gap = tpr * UNITS;
        to = ring + (threadIdx.x - lane) * (UNITS * 16) + lane * 16;
        from = ring + threadIdx.x * (UNITS * 16);
    }
    __device__ __forceinline__ void fetch(uint32_t stage, int v, const void *x = nullptr) const {
#pragma unroll
        for (int j = 0; j < UNITS; ++j)
            if (v * gap + j * 32 < units)
                cp_async_16(to + stage + v * blockDim.x * (UNITS * 16) + j * 512,
                            static_cast<const uint8_t *>(x) + next + (v * gap + j * 32) * 16);
    }
    __device__ __forceinline__ Piece<BF16> read(uint32_t stage, int v) const {
        Piece<BF16> r;
#pragma unroll
        for (int j = 0; j < UNITS; ++j)
            asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                         : "=r"(r.w[4 * j]), "=r"(r.w[4 * j + 1]), "=r"(r.w[4 * j + 2]), "=r"(r.w[4 * j + 3])
                         : "r"(from + stage + v * blockDim.x * (UNITS * 16) + j * 16)
                         : "memory");
        return r;
    }
};

// 1 / sqrt(v) to an ulp: the hardware's approximation and a step of Newton's, where
// nothing in it leaves the normal numbers.
__device__ __forceinline__ float inverse_root(float v) {
    if (v > 0x1p-100f && v < 0x1p100f) {
        float r;
        asm("rsqrt.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
        return fmaf(r * 0.5f, fmaf(-v * r, r, 1.0f), r);
    }
    return __frcp_rn(__fsqrt_rn(v));
}

constexpr int kMaxWarps = kWideBlock / 32;

// The sum over the tpr threads of group g. `red` (zeros behind the group's warps)
// alternates between two halves from row to row: a thread writes one again only when
// all have left the barrier of the row between, and with it their reads. The warps'
// sums are joined by shuffles, or added up by every thread, which costs latency or
// instructions: forward without residual, 16384 x 4096, 40.4 us and 44.3; backward 89.2
// and 82.6.
template <bool SHUFFLE>
__device__ __forceinline__ float row_sum(float v, float (&red)[kMaxWarps], int g, int tpr, int tid) {
    v = warp_sum(v);
    if (tpr == 32) return v;
    const int lane = tid & 31, warps = tpr >> 5;
    if (lane == 0) red[tid >> 5] = v;
    asm volatile("bar.sync %0, %1;" ::"r"(g + 1), "r"(tpr) : "memory");
    if constexpr (SHUFFLE) return warp_sum(lane < warps ? red[lane] : 0.0f);
    float4 s = *reinterpret_cast<const float4 *>(red);
    for (int w = 4; w < warps; w += 4) {
        const float4 more = *reinterpret_cast<const float4 *>(red + w);
        s.x += more.x;
        s.y += more.y;
        s.z += more.z;
        s.w += more.w;
    }
    return (s.x + s.y) + (s.z + s.w);
}
__device__ __forceinline__ void clear(float (&red)[2][kMaxGroups][kMaxWarps]) {
    for (int i = threadIdx.x; i < 2 * kMaxGroups * kMaxWarps; i += blockDim.x) (&red[0][0][0])[i] = 0.0f;
    __syncthreads();
}

template <int N>
__device__ __forceinline__ void load_weight(uint64_t (&w)[N][4], const void *p, bool bf16, int tid, int tpr, int pieces) {
#pragma unroll
    for (int v = 0; v < N; ++v) {
        const int i = tid + v * tpr;
#pragma unroll
        for (int j = 0; j < 4; ++j) w[v][j] = 0ull;
        if (i >= pieces) continue;
        if (bf16) {
            const Piece<true> q = load_piece<true>(p, i);
#pragma unroll
            for (int j = 0; j < 4; ++j) w[v][j] = q.pair(j);
        } else {
            const Piece<false> q = load_piece<false>(p, i);
#pragma unroll
            for (int j = 0; j < 4; ++j) w[v][j] = q.pair(j);
        }
    }
}

// RES: 0 no residual, 1 bf16, 2 fp32. N pieces of a row for each thread.
template <bool XBF, int RES, int N>
struct Fwd {
    using SX = Slot<XBF, N>;
    using SR = Slot<RES == 1, N>;
    static constexpr int BYTES = SX::BYTES + (RES ? SR::BYTES : 0), S = stages(BYTES, N);
};

template <bool XBF, int RES, int N>
__global__ void __launch_bounds__(threads_of(N), (per_sm(threads_of(N), N, Fwd<XBF, RES, N>::BYTES, Fwd<XBF, RES, N>::S)))
    norm_fwd_kernel(const NormArgs a) {
    using F = Fwd<XBF, RES, N>;
    using SX = typename F::SX;
    using SR = typename F::SR;
    constexpr bool RBF = RES == 1, SHARED = !XBF || RES == 2;
    constexpr int BYTES = F::BYTES, S = F::S;
    extern __shared__ uint4 ring[];
    __shared__ __align__(16) float red[2][kMaxGroups][kMaxWarps];
    clear(red);
    pdl_wait();
    pdl_launch_dependents();
    const int tpr = a.tpr, g = threadIdx.x / tpr, tid = threadIdx.x - g * tpr, groups = blockDim.x / tpr;
    const int pieces = a.K / kPiece;
    const int64_t step = static_cast<int64_t>(gridDim.x) * groups;
    const uint32_t stage_bytes = blockDim.x * BYTES;
    int64_t m = static_cast<int64_t>(blockIdx.x) * groups + g, to_fetch = m;
    SX sx(smem_u32(ring), a.x, m, step, pieces, tid, tpr);
    SR sr(smem_u32(ring) + blockDim.x * SX::BYTES, a.r, m, step, pieces, tid, tpr);
    const auto fetch_row = [&](uint32_t stage) {
        if (to_fetch < a.M) {
#pragma unroll
            for (int v = 0; v < N; ++v) {
                sx.fetch(stage, v);
                if constexpr (RES != 0) sr.fetch(stage, v);
            }
        }
        to_fetch += step;
        sx.next += sx.step;
        if constexpr (RES != 0) sr.next += sr.step;
        cp_async_commit();
    };
    for (int s = 0; s < (S > 1 ? S - 1 : 1); ++s) fetch_row(s * stage_bytes);
    uint64_t w[N][4];
    load_weight<N>(w, a.w, a.w_bf16, tid, tpr, pieces);
    const float inv_k = __frcp_rn(static_cast<float>(a.K));
    const uint64_t scale = f2_same(a.scale != nullptr ? __ldg(a.scale) : 1.0f);
    float am = 0.0f;
    for (int s = 0, turn = 0; m < a.M; m += step, turn ^= 1) {
        if constexpr (S > 1) {
            if constexpr (SHARED) __syncwarp();
            fetch_row((s == 0 ? S - 1 : s - 1) * stage_bytes);
        }
        cp_async_wait<S - 1>();
        if constexpr (SHARED) __syncwarp();
        const uint32_t now = s * stage_bytes;
        s = s == S - 1 ? 0 : s + 1;
        const int64_t row = m * pieces;
        uint64_t t[N][4], sum = 0ull;
#pragma unroll
        for (int v = 0; v < N; ++v) {
            const int i = tid + v * tpr;
            if (i < pieces) {
                const Piece<XBF> x = sx.read(now, v);
#pragma unroll
                for (int j = 0; j < 4; ++j) t[v][j] = x.pair(j);
                if constexpr (RES != 0) {
                    const Piece<RBF> r = sr.read(now, v);
#pragma unroll
                    for (int j = 0; j < 4; ++j) t[v][j] = f2_add(t[v][j], r.pair(j));
                    const Piece<RBF> q = round_piece<RBF>(t[v]);
                    store_piece<RBF>(a.t, row + i, q);
#pragma unroll
                    for (int j = 0; j < 4; ++j) t[v][j] = q.pair(j);
                }
#pragma unroll
                for (int j = 0; j < 4; ++j) sum = f2_fma(t[v][j], t[v][j], sum);
            }
        }
        if constexpr (S == 1) {
            __syncwarp();
            fetch_row(0);
        }
        float s0, s1;
        f2_split(sum, s0, s1);
        const float total = row_sum<true>(s0 + s1, red[turn][g], g, tpr, tid);
        const float rstd = inverse_root(fmaf(total, inv_k, a.eps));
        if (tid == 0) a.rstd[m] = rstd;
        const uint64_t r2 = f2_same(rstd);
#pragma unroll
        for (int v = 0; v < N; ++v) {
            const int i = tid + v * tpr;
            if (i < pieces) {
                uint64_t y[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    y[j] = f2_mul(f2_mul(t[v][j], r2), w[v][j]);
                    float y0, y1;
                    f2_split(y[j], y0, y1);
                    am = fmaxf(am, fmaxf(fabsf(y0), fabsf(y1)));
                }
                if (a.scale != nullptr) {
                    uint32_t q[2];
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        float f0, f1, f2, f3;
                        f2_split(f2_mul(y[2 * j], scale), f0, f1);
                        f2_split(f2_mul(y[2 * j + 1], scale), f2, f3);
                        q[j] = cvt_quad_probed<FP8MP_E4M3>(f0, f1, f2, f3);
                    }
                    reinterpret_cast<uint2 *>(a.y)[row + i] = make_uint2(q[0], q[1]);
                } else {
                    store_rounded(a.y, row + i, y, a.y_bf16);
                }
            }
        }
    }
    if (a.amax != nullptr) block_amax_atomic(am, a.amax);
}

template <bool XBF, bool RBF, int N>
struct Bwd {
    using SX = Slot<XBF, N>;
    using SR = Slot<RBF, N>;
    static constexpr int BYTES = SX::BYTES + 2 * SR::BYTES, S = stages(BYTES, N);
};

template <bool XBF, bool RBF, int N>
__global__ void __launch_bounds__(threads_of(N), (per_sm(threads_of(N), N, Bwd<XBF, RBF, N>::BYTES, Bwd<XBF, RBF, N>::S)))
    norm_bwd_kernel(const NormGradArgs a) {
    using B = Bwd<XBF, RBF, N>;
    using SX = typename B::SX;
    using SR = typename B::SR;
    constexpr bool SHARED = !XBF || !RBF;
    constexpr int BYTES = B::BYTES, S = B::S;
    extern __shared__ uint4 ring[];
    __shared__ __align__(16) float red[2][kMaxGroups][kMaxWarps];
    clear(red);
    pdl_wait();
    pdl_launch_dependents();
    const int tpr = a.tpr, g = threadIdx.x / tpr, tid = threadIdx.x - g * tpr, groups = blockDim.x / tpr;
    const int pieces = a.K / kPiece;
    const int64_t step = static_cast<int64_t>(gridDim.x) * groups;
    const uint32_t stage_bytes = blockDim.x * BYTES;
    int64_t m = static_cast<int64_t>(blockIdx.x) * groups + g, to_fetch = m;
    // Arrays of one type share a Slot, their pieces lying one behind another: it is its
    // registers that are short (16384 x 4096 bf16 82.6 us, 85.8 with a Slot each).
    constexpr bool SAME = XBF == RBF;
    const uint32_t t_ring = SAME ? blockDim.x * SX::BYTES : 0u, dt_ring = t_ring + blockDim.x * SR::BYTES;
    SX sdy(smem_u32(ring), nullptr, m, step, pieces, tid, tpr);
    SR other(smem_u32(ring) + blockDim.x * SX::BYTES, nullptr, m, step, pieces, tid, tpr);
    const auto st = [&]() -> const SR & {
        if constexpr (SAME) return sdy;
        else return other;
    };
    const auto fetch = [&](uint32_t stage, int v) {
        if (to_fetch >= a.M) return;
        sdy.fetch(stage, v, a.dy);
        st().fetch(stage + t_ring, v, a.t);
        if (a.dtotal != nullptr) st().fetch(stage + dt_ring, v, a.dtotal);
    };
    const auto fetched = [&] {
        to_fetch += step;
        sdy.next += sdy.step;
        if constexpr (!SAME) other.next += other.step;
        cp_async_commit();
    };
    const auto fetch_row = [&](uint32_t stage) {
#pragma unroll
        for (int v = 0; v < N; ++v) fetch(stage, v);
        fetched();
    };
    for (int s = 0; s < (S > 1 ? S - 1 : 1); ++s) fetch_row(s * stage_bytes);
    const float inv_k = __frcp_rn(static_cast<float>(a.K));
    uint64_t w[N][4], dw[N][4];
    load_weight<N>(w, a.w, a.w_bf16, tid, tpr, pieces);
#pragma unroll
    for (int v = 0; v < N; ++v)
#pragma unroll
        for (int j = 0; j < 4; ++j) dw[v][j] = 0ull;
    float next_rstd = m < a.M ? __ldg(a.rstd + m) : 0.0f;
    for (int s = 0, turn = 0; m < a.M; m += step, turn ^= 1) {
        if constexpr (S > 1) {
            if constexpr (SHARED) __syncwarp();
            fetch_row((s == 0 ? S - 1 : s - 1) * stage_bytes);
        }
        const uint64_t r2 = f2_same(next_rstd);
        if (m + step < a.M) next_rstd = __ldg(a.rstd + m + step);
        cp_async_wait<S - 1>();
        if constexpr (SHARED) __syncwarp();
        const uint32_t now = s * stage_bytes;
        s = s == S - 1 ? 0 : s + 1;
        const int64_t row = m * pieces;
        uint64_t sum = 0ull;
#pragma unroll
        for (int v = 0; v < N; ++v) {
            if (tid + v * tpr < pieces) {
                const Piece<XBF> dy = sdy.read(now, v);
                const Piece<RBF> t = st().read(now + t_ring, v);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const uint64_t n = f2_mul(t.pair(j), r2), d = dy.pair(j);
                    dw[v][j] = f2_fma(d, n, dw[v][j]);
                    sum = f2_fma(f2_mul(d, w[v][j]), n, sum);
                }
            }
        }
        float s0, s1;
        f2_split(sum, s0, s1);
        const float c = row_sum<false>(s0 + s1, red[turn][g], g, tpr, tid) * inv_k;
        const uint64_t neg_c = f2_same(-c);
#pragma unroll
        for (int v = 0; v < N; ++v) {
            const int i = tid + v * tpr;
            if (i < pieces) {
                const Piece<XBF> dy = sdy.read(now, v);
                const Piece<RBF> t = st().read(now + t_ring, v);
                uint64_t d[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) d[j] = f2_fma(f2_mul(t.pair(j), r2), neg_c, f2_mul(dy.pair(j), w[v][j]));
                if (a.dtotal != nullptr) {
                    const Piece<RBF> dt = st().read(now + dt_ring, v);
#pragma unroll
                    for (int j = 0; j < 4; ++j) d[j] = f2_fma(d[j], r2, dt.pair(j));
                } else {
#pragma unroll
                    for (int j = 0; j < 4; ++j) d[j] = f2_mul(d[j], r2);
                }
                store_piece<RBF>(a.dr, row + i, round_piece<RBF>(d));
                if (a.dx != nullptr) store_piece<XBF>(a.dx, row + i, round_piece<XBF>(d));
            }
            if constexpr (S == 1) {
                __syncwarp();
                fetch(0, v);
            }
        }
        if constexpr (S == 1) fetched();
    }
    if (a.partial == nullptr) return;
    float *out = a.partial + static_cast<int64_t>(blockIdx.x) * a.K;
    if (groups > 1) {  // the groups' sums one after another, in the ring's memory
        float *join = reinterpret_cast<float *>(ring);
        cp_async_wait<0>();
        __syncthreads();
        for (int i = threadIdx.x; i < a.K; i += blockDim.x) join[i] = 0.0f;
        for (int k = 0; k < groups; ++k) {
            __syncthreads();
            if (g != k) continue;
#pragma unroll
            for (int v = 0; v < N; ++v) {
                const int i = tid + v * tpr;
                if (i < pieces) {
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        float lo, hi;
                        f2_split(dw[v][j], lo, hi);
                        join[i * kPiece + 2 * j] += lo;
                        join[i * kPiece + 2 * j + 1] += hi;
                    }
                }
            }
        }
        __syncthreads();
        for (int i = threadIdx.x; i < a.K; i += blockDim.x) out[i] = join[i];
    } else {
#pragma unroll
        for (int v = 0; v < N; ++v) {
            const int i = tid + v * tpr;
            if (i < pieces) store_piece<false>(out, i, round_piece<false>(dw[v]));
        }
    }
}

// dw[k] = the sum of the blocks' sums: a block takes 32 columns, 128 threads of
// four columns each a share of the rows, then their sums in order of the share.
constexpr int kSumThreads = 1024, kSumShares = kSumThreads / 8;

__global__ void __launch_bounds__(kSumThreads) norm_dw_kernel(const float *partial, int rows, int K, void *dw, bool bf16) {
    __shared__ float part[kSumShares][32 + 1];
    pdl_wait();
    pdl_launch_dependents();
    const int lane = threadIdx.x & 7, share = threadIdx.x >> 3;
    const int col = blockIdx.x * 32 + lane * 4;
    float4 s = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    if (col < K) {
        for (int r = share; r < rows; r += kSumShares) {
            const float4 v = __ldcg(reinterpret_cast<const float4 *>(partial + static_cast<int64_t>(r) * K + col));
            s.x += v.x;
            s.y += v.y;
            s.z += v.z;
            s.w += v.w;
        }
    }
    part[share][lane * 4] = s.x;
    part[share][lane * 4 + 1] = s.y;
    part[share][lane * 4 + 2] = s.z;
    part[share][lane * 4 + 3] = s.w;
    __syncthreads();
    // warp c of the 32: the shares of column c
    const int c = threadIdx.x >> 5, l = threadIdx.x & 31;
    float v = 0.0f;
#pragma unroll
    for (int r = 0; r < kSumShares / 32; ++r) v += part[l + 32 * r][c];
    v = warp_sum(v);
    const int k = blockIdx.x * 32 + c;
    if (l == 0 && k < K) {
        if (bf16) reinterpret_cast<__nv_bfloat16 *>(dw)[k] = __float2bfloat16_rn(v);
        else reinterpret_cast<float *>(dw)[k] = v;
    }
}

// Pieces of a row for each thread, threads that share it, rows that a block takes
// at a time.
struct Shape {
    int pieces, tpr, groups;
    int threads() const { return tpr * groups; }
};
Shape shape_of(int64_t K) {
    const int n = K <= 2 * kPiece * kBlock ? 2 : 4;
    const int64_t threads = (K / kPiece + n - 1) / n;
    const int tpr = static_cast<int>((threads + 31) / 32 * 32);
    return {n, tpr, tpr < kBlock ? kBlock / tpr : 1};
}

// Launches a kernel of `blocks` blocks, allowed once their shared memory.
template <typename A>
cudaError_t launch_rows(void (*kernel)(A), std::atomic<bool> (&ready)[64], int64_t blocks, const Shape &shape, int smem,
                        cudaStream_t s, int device, const A &a) {
    const cudaError_t e = allow_smem(kernel, kSmem, ready, device);
    if (e != cudaSuccess) return e;
    return launch_kernel(kernel, dim3(static_cast<unsigned>(blocks)), dim3(shape.threads()), smem, s, a);
}

int64_t least(int64_t a, int64_t b) { return a < b ? a : b; }

template <bool XBF, int RES, int N>
cudaError_t fwd(NormArgs a, const Shape &shape, cudaStream_t s, const DeviceInfo &dev) {
    using F = Fwd<XBF, RES, N>;
    static std::atomic<bool> ready[64];
    a.tpr = shape.tpr;
    constexpr int kResident = per_sm(threads_of(N), N, F::BYTES, F::S) * threads_of(N);  // threads
    const int64_t units = (a.M + shape.groups - 1) / shape.groups, sms = dev.num_sms;
    const int64_t resident = sms * (kResident / shape.threads());
    const int64_t most = units <= kFewUnits * sms ? resident : N == 2 ? sms * kBlocksPerSm * kBlock / shape.threads() : kWaves * resident;
    return launch_rows(norm_fwd_kernel<XBF, RES, N>, ready, least(units, most), shape,
                       F::BYTES * F::S * shape.threads(), s, dev.device, a);
}
template <bool XBF, int RES>
cudaError_t fwd(const NormArgs &a, cudaStream_t s, const DeviceInfo &dev) {
    const Shape shape = shape_of(a.K);
    return shape.pieces == 2 ? fwd<XBF, RES, 2>(a, shape, s, dev) : fwd<XBF, RES, 4>(a, shape, s, dev);
}

// Blocks of the backward pass, which fix the order of dw's sum: what an SM holds of them,
// since each leaves a row of sums, and one that starts when another ends begins with a row's
// whole latency. Of kBlock threads that is three, or two by their rows in shared memory with
// a stream in fp32. bf16 dy, by two and by three: fp32 stream 500 x 4096 10.6 and 12.8 us, 1237 x
// 2736 13.4, 15.6, 3000 x 2736 23.9, 25.8, 60000 x 256 40.6, 43.4, 8192 x 4096 91.1, 91.8, 12000 x
// 1760 57.1, 55.9; bf16 stream 500 x 4096 10.3, 9.8, 2400 x 2736 17.7, 16.7, 8192 x 4096 55.3, 45.5.
// fp32 dy, fp32 stream: 8192 x 4096 84.3, 91.2; bf16 stream 1237 x 2736 15.2, 14.4, 8192 x 4096 83.3,
// 76.6. In whole blocks: 3.4 of 224 threads in place of three, 16000 x 3584 98.7 us, not 71.5.
constexpr int grad_per_sm(bool fp32_stream) { return fp32_stream ? 2 : 3; }
int64_t grad_blocks(int64_t M, int64_t K, bool fp32_stream) {
    const Shape shape = shape_of(K);
    const int64_t units = (M + shape.groups - 1) / shape.groups;
    return least(units, kGradSms * ((shape.pieces == 2 ? grad_per_sm(fp32_stream) * kBlock : kWideBlock) / shape.threads()));
}

template <bool XBF, bool RBF, int N>
cudaError_t bwd(NormGradArgs a, const Shape &shape, cudaStream_t s, const DeviceInfo &dev) {
    using B = Bwd<XBF, RBF, N>;
    static_assert(N != 2 || per_sm(kBlock, N, B::BYTES, B::S) == grad_per_sm(!RBF), "the blocks that are resident");
    static std::atomic<bool> ready[64];
    a.tpr = shape.tpr;
    return launch_rows(norm_bwd_kernel<XBF, RBF, N>, ready, grad_blocks(a.M, a.K, !RBF), shape,
                       B::BYTES * B::S * shape.threads(), s, dev.device, a);
}
template <bool XBF, bool RBF>
cudaError_t bwd(const NormGradArgs &a, void *dw, bool dw_bf16, cudaStream_t s, const DeviceInfo &dev) {
    const Shape shape = shape_of(a.K);
    cudaError_t e = cudaSuccess;
    if (a.M > 0) e = shape.pieces == 2 ? bwd<XBF, RBF, 2>(a, shape, s, dev) : bwd<XBF, RBF, 4>(a, shape, s, dev);
    if (e == cudaSuccess && dw != nullptr)
        e = launch_kernel(norm_dw_kernel, dim3(static_cast<unsigned>((a.K + 31) / 32)), dim3(kSumThreads), 0, s,
                          static_cast<const float *>(a.partial), static_cast<int>(grad_blocks(a.M, a.K, !RBF)), a.K, dw,
                          dw_bf16);
    return e;
}

}  // namespace

int64_t rmsnorm_workspace_bytes(int64_t M, int64_t K) {
    return grad_blocks(M, K, false) * K * 4;  // (the larger)
}

int launch_rmsnorm_fwd(const void *x, int x_dtype, const void *r, void *t, int r_dtype, int64_t M, int64_t K,
                       const void *w, int w_dtype, float eps, const float *y_scale, void *y, int y_dtype,
                       float *y_amax, float *rstd, cudaStream_t s, const DeviceInfo &dev) {
    const NormArgs a = {x, r, w, t, y, rstd, y_amax, y_scale, M, static_cast<int>(K), 0, eps,
                        w_dtype == FP8MP_BF16, y_dtype == FP8MP_BF16};
    const bool xb = x_dtype == FP8MP_BF16, rb = r_dtype == FP8MP_BF16;
    cudaError_t e;
    if (r == nullptr) e = xb ? fwd<true, 0>(a, s, dev) : fwd<false, 0>(a, s, dev);
    else if (rb) e = xb ? fwd<true, 1>(a, s, dev) : fwd<false, 1>(a, s, dev);
    else e = xb ? fwd<true, 2>(a, s, dev) : fwd<false, 2>(a, s, dev);
    if (e != cudaSuccess) return fail(FP8MP_ERR_LAUNCH, "rmsnorm: launch failed: %s", cudaGetErrorString(e));
    return FP8MP_OK;
}

int launch_rmsnorm_bwd(const void *dy, int dy_dtype, const void *dtotal, const void *t, int t_dtype, const float *rstd,
                       int64_t M, int64_t K, const void *w, int w_dtype, void *dr, void *dx, void *dw, int dw_dtype,
                       void *workspace, cudaStream_t s, const DeviceInfo &dev) {
    const NormGradArgs a = {dy, dtotal, t, w, rstd, dr, dx, dw != nullptr ? static_cast<float *>(workspace) : nullptr,
                            M, static_cast<int>(K), 0, w_dtype == FP8MP_BF16};
    const bool xb = dy_dtype == FP8MP_BF16, rb = t_dtype == FP8MP_BF16;
    const bool wb = dw_dtype == FP8MP_BF16;
    cudaError_t e;
    if (rb) e = xb ? bwd<true, true>(a, dw, wb, s, dev) : bwd<false, true>(a, dw, wb, s, dev);
    else e = xb ? bwd<true, false>(a, dw, wb, s, dev) : bwd<false, false>(a, dw, wb, s, dev);
    if (e != cudaSuccess) return fail(FP8MP_ERR_LAUNCH, "rmsnorm: launch failed: %s", cudaGetErrorString(e));
    return FP8MP_OK;
}

}  // namespace fp8mp
