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
// Rows of up to kWarpRow columns belong to one warp each, which needs no barrier;
// longer ones to a block whose threads hold 16 columns each (32 from 8192 on, so
// that a block has at most 512 threads).
#include "fp8mp_pieces.cuh"

namespace fp8mp {

namespace {

constexpr int kWarpRow = 1024;      // columns up to which a warp takes a row
constexpr int kWarpRowsPerBlock = 8;
constexpr int kMaxThreads = 512;    // of a block that takes a row
constexpr int kGradBlocks = 456;    // most blocks of the backward pass, each of which leaves a row of sums

struct NormArgs {
    const void *x, *r, *w;
    void *t, *y;
    float *rstd, *amax;
    const float *scale;
    int64_t M;
    int K;
    float eps;
    bool w_bf16, y_bf16;
};

struct NormGradArgs {
    const void *dy, *dtotal, *t, *w;
    const float *rstd;
    void *dr, *dx;
    float *partial;  // [gridDim.x][K] sums of dy n, or NULL
    int64_t M;
    int K;
    bool w_bf16;
};

// The sum over the threads that share a row. `red` alternates between two halves
// from row to row: a thread writes one again only when all have left the barrier
// of the row between, and with it their reads.
template <bool WARP>
__device__ __forceinline__ float row_sum(float v, float *red) {
    v = warp_sum(v);
    if constexpr (WARP) return v;
    const int lane = threadIdx.x & 31, warps = blockDim.x >> 5;
    if (lane == 0) red[threadIdx.x >> 5] = v;
    __syncthreads();
    return warp_sum(lane < warps ? red[lane] : 0.0f);
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
template <bool XBF, int RES, int N, bool WARP>
__global__ void __launch_bounds__(WARP ? 32 * kWarpRowsPerBlock : kMaxThreads) norm_fwd_kernel(const NormArgs a) {
    __shared__ float red[2][32];
    pdl_wait();
    pdl_launch_dependents();
    constexpr bool RBF = RES == 1;
    const int tpr = WARP ? 32 : static_cast<int>(blockDim.x), tid = WARP ? threadIdx.x & 31 : threadIdx.x;
    const int64_t rows = WARP ? kWarpRowsPerBlock : 1;
    const int pieces = a.K / kPiece;
    uint64_t w[N][4];
    load_weight<N>(w, a.w, a.w_bf16, tid, tpr, pieces);
    const uint64_t scale = f2_same(a.scale != nullptr ? __ldg(a.scale) : 1.0f);
    float am = 0.0f;
    int turn = 0;
    for (int64_t m = blockIdx.x * rows + (WARP ? threadIdx.x >> 5 : 0); m < a.M; m += gridDim.x * rows, turn ^= 1) {
        const int64_t row = m * pieces;
        Piece<XBF> xs[N];
        Piece<RBF> rs[RES ? N : 1];
#pragma unroll
        for (int v = 0; v < N; ++v) {
            const int i = tid + v * tpr;
            if (i < pieces) {
                xs[v] = load_piece<XBF>(a.x, row + i);
                if constexpr (RES != 0) rs[v] = load_piece<RBF>(a.r, row + i);
            }
        }
        uint64_t t[N][4], sum = 0ull;
#pragma unroll
        for (int v = 0; v < N; ++v) {
            const int i = tid + v * tpr;
            if (i < pieces) {
#pragma unroll
                for (int j = 0; j < 4; ++j) t[v][j] = xs[v].pair(j);
                if constexpr (RES != 0) {
#pragma unroll
                    for (int j = 0; j < 4; ++j) t[v][j] = f2_add(t[v][j], rs[v].pair(j));
                    const Piece<RBF> q = round_piece<RBF>(t[v]);
                    store_piece<RBF>(a.t, row + i, q);
#pragma unroll
                    for (int j = 0; j < 4; ++j) t[v][j] = q.pair(j);
                }
#pragma unroll
                for (int j = 0; j < 4; ++j) sum = f2_fma(t[v][j], t[v][j], sum);
            }
        }
        float s0, s1;
        f2_split(sum, s0, s1);
        const float total = row_sum<WARP>(s0 + s1, red[turn]);
        const float rstd = __frcp_rn(__fsqrt_rn(__fdiv_rn(total, static_cast<float>(a.K)) + a.eps));
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

template <bool XBF, bool RBF, int N, bool WARP>
__global__ void __launch_bounds__(WARP ? 32 * kWarpRowsPerBlock : kMaxThreads) norm_bwd_kernel(const NormGradArgs a) {
    __shared__ float red[2][32];
    __shared__ float join[WARP ? kWarpRow : 1];
    pdl_wait();
    pdl_launch_dependents();
    const int tpr = WARP ? 32 : static_cast<int>(blockDim.x), tid = WARP ? threadIdx.x & 31 : threadIdx.x;
    const int64_t rows = WARP ? kWarpRowsPerBlock : 1;
    const int pieces = a.K / kPiece;
    const float inv_k = __frcp_rn(static_cast<float>(a.K));
    uint64_t w[N][4], dw[N][4];
    load_weight<N>(w, a.w, a.w_bf16, tid, tpr, pieces);
#pragma unroll
    for (int v = 0; v < N; ++v)
#pragma unroll
        for (int j = 0; j < 4; ++j) dw[v][j] = 0ull;
    int turn = 0;
    for (int64_t m = blockIdx.x * rows + (WARP ? threadIdx.x >> 5 : 0); m < a.M; m += gridDim.x * rows, turn ^= 1) {
        const int64_t row = m * pieces;
        const float rstd = __ldg(a.rstd + m);
        Piece<XBF> dy[N];
        Piece<RBF> t[N], dt[N];
#pragma unroll
        for (int v = 0; v < N; ++v) {
            const int i = tid + v * tpr;
            if (i < pieces) {
                dy[v] = load_piece<XBF>(a.dy, row + i);
                t[v] = load_piece<RBF>(a.t, row + i);
                if (a.dtotal != nullptr) dt[v] = load_piece<RBF>(a.dtotal, row + i);
            }
        }
        const uint64_t r2 = f2_same(rstd);
        uint64_t sum = 0ull;
#pragma unroll
        for (int v = 0; v < N; ++v) {
            const int i = tid + v * tpr;
            if (i < pieces) {
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const uint64_t n = f2_mul(t[v].pair(j), r2), d = dy[v].pair(j);
                    dw[v][j] = f2_fma(d, n, dw[v][j]);
                    sum = f2_fma(f2_mul(d, w[v][j]), n, sum);
                }
            }
        }
        float s0, s1;
        f2_split(sum, s0, s1);
        const float c = row_sum<WARP>(s0 + s1, red[turn]) * inv_k;
        const uint64_t neg_c = f2_same(-c);
#pragma unroll
        for (int v = 0; v < N; ++v) {
            const int i = tid + v * tpr;
            if (i < pieces) {
                uint64_t d[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const uint64_t n = f2_mul(t[v].pair(j), r2);
                    const uint64_t g = f2_fma(n, neg_c, f2_mul(dy[v].pair(j), w[v][j]));
                    d[j] = a.dtotal != nullptr ? f2_fma(g, r2, dt[v].pair(j)) : f2_mul(g, r2);
                }
                store_piece<RBF>(a.dr, row + i, round_piece<RBF>(d));
                if (a.dx != nullptr) store_piece<XBF>(a.dx, row + i, round_piece<XBF>(d));
            }
        }
    }
    if (a.partial == nullptr) return;
    float *out = a.partial + static_cast<int64_t>(blockIdx.x) * a.K;
    if constexpr (WARP) {  // the warps' sums one after another
        for (int i = threadIdx.x; i < a.K; i += blockDim.x) join[i] = 0.0f;
        for (int k = 0; k < kWarpRowsPerBlock; ++k) {
            __syncthreads();
            if (static_cast<int>(threadIdx.x >> 5) != k) continue;
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

// Threads of a block, and pieces of a row for each (4 for a warp).
struct Shape {
    int threads, pieces;
    bool warp;
};
Shape shape_of(int64_t K) {
    if (K <= kWarpRow) return {32 * kWarpRowsPerBlock, 4, true};
    const int n = K <= 2 * kPiece * kMaxThreads ? 2 : 4;
    const int64_t threads = (K / kPiece + n - 1) / n;
    return {static_cast<int>((threads + 31) / 32 * 32), n, false};
}
int64_t rows_of(const Shape &s) { return s.warp ? kWarpRowsPerBlock : 1; }

template <bool XBF, int RES>
cudaError_t fwd(const NormArgs &a, cudaStream_t s, const DeviceInfo &dev) {
    const Shape shape = shape_of(a.K);
    const int64_t need = (a.M + rows_of(shape) - 1) / rows_of(shape);
    const int64_t most = static_cast<int64_t>(dev.num_sms) * (1536 / shape.threads);
    const dim3 grid(static_cast<unsigned>(need < most ? need : most)), block(shape.threads);
    if (shape.warp) return launch_kernel(norm_fwd_kernel<XBF, RES, 4, true>, grid, block, 0, s, a);
    if (shape.pieces == 2) return launch_kernel(norm_fwd_kernel<XBF, RES, 2, false>, grid, block, 0, s, a);
    return launch_kernel(norm_fwd_kernel<XBF, RES, 4, false>, grid, block, 0, s, a);
}

int64_t grad_blocks(int64_t M, int64_t K) {
    const int64_t rows = rows_of(shape_of(K)), need = (M + rows - 1) / rows;
    return need < kGradBlocks ? need : kGradBlocks;
}

template <bool XBF, bool RBF>
cudaError_t bwd(const NormGradArgs &a, cudaStream_t s) {
    const Shape shape = shape_of(a.K);
    const dim3 grid(static_cast<unsigned>(grad_blocks(a.M, a.K))), block(shape.threads);
    if (shape.warp) return launch_kernel(norm_bwd_kernel<XBF, RBF, 4, true>, grid, block, 0, s, a);
    if (shape.pieces == 2) return launch_kernel(norm_bwd_kernel<XBF, RBF, 2, false>, grid, block, 0, s, a);
    return launch_kernel(norm_bwd_kernel<XBF, RBF, 4, false>, grid, block, 0, s, a);
}

}  // namespace

int64_t rmsnorm_workspace_bytes(int64_t M, int64_t K) { return grad_blocks(M, K) * K * 4; }

int launch_rmsnorm_fwd(const void *x, int x_dtype, const void *r, void *t, int r_dtype, int64_t M, int64_t K,
                       const void *w, int w_dtype, float eps, const float *y_scale, void *y, int y_dtype,
                       float *y_amax, float *rstd, cudaStream_t s, const DeviceInfo &dev) {
    const NormArgs a = {x, r, w, t, y, rstd, y_amax, y_scale, M, static_cast<int>(K), eps,
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
                       void *workspace, cudaStream_t s) {
    const NormGradArgs a = {dy, dtotal, t, w, rstd, dr, dx, dw != nullptr ? static_cast<float *>(workspace) : nullptr,
                            M, static_cast<int>(K), w_dtype == FP8MP_BF16};
    const bool xb = dy_dtype == FP8MP_BF16, rb = t_dtype == FP8MP_BF16;
    cudaError_t e = cudaSuccess;
    if (M > 0) {
        if (rb) e = xb ? bwd<true, true>(a, s) : bwd<false, true>(a, s);
        else e = xb ? bwd<true, false>(a, s) : bwd<false, false>(a, s);
    }
    if (e == cudaSuccess && dw != nullptr)
        e = launch_kernel(norm_dw_kernel, dim3(static_cast<unsigned>((K + 31) / 32)), dim3(kSumThreads), 0, s,
                          static_cast<const float *>(workspace), static_cast<int>(M > 0 ? grad_blocks(M, K) : 0),
                          static_cast<int>(K), dw, dw_dtype == FP8MP_BF16);
    if (e != cudaSuccess) return fail(FP8MP_ERR_LAUNCH, "rmsnorm: launch failed: %s", cudaGetErrorString(e));
    return FP8MP_OK;
}

}  // namespace fp8mp
