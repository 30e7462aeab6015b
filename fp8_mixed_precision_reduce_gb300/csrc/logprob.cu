// logprob.cu -- log probabilities of given tokens over a vocabulary, with the
// entropy and the most probable tokens, and the gradient of the logits.
//
// With m = max_v x_v and S = sum_v exp(x_v - m), of a row of logits x:
//   log p_v = (x_v - m) - log S,     H = log S - (sum_v exp(x_v - m) (x_v - m)) / S
//   dx_v = a (1[v = t] - p_v) - b p_v (log p_v + H)
// for the gradients a of log p_t and b of H. (log S)'s m and log S are kept apart:
// their sum would round away what a row of large logits needs, such as one whose
// allowed tokens all hold the type's lowest value.
//
// Forward: one pass with the running maximum and sums of a softmax, in registers,
// joined over the threads and, when there are few rows, over the up to 8 CTAs of a
// cluster that share a row, through the first one's shared memory; many short rows are
// taken by a warp each. Bound by HBM (the logits, once): 8192 x 128000 in bf16 286 us,
// 7.3 TB/s; with the entropy 295 us, where instruction issue begins to. Seven rows of
// that length, with their 20 best tokens, 6.4 us: latency of the loads, of the
// selection's barriers and of the cluster's.
//
// The k most probable tokens come out of the same pass. Each thread keeps the
// largest logit of its share of the row; with tau the k-th largest of those or a bit
// less, every one of the k largest logits is at least tau, and only the shares whose
// largest is can hold one: k to 1.5 k of 256, which are read again (from L2) by all
// threads. What they hold from tau on is ranked by counting. Where more than fits is at tau or
// above (equal logits, nearly all masked), a bisection on the value finds the k-th
// largest, and its equals are taken from the lowest index on.
//
// Backward: elementwise, 3 bytes an element with bf16 logits and E5M2 codes, bound by
// HBM: 8192 x 128000 471 us, 6.7 TB/s.
#include <cfloat>
#include <cstring>
#include <type_traits>

#include "fp8mp_async.cuh"
#include "fp8mp_lm.cuh"
#include "fp8mp_pieces.cuh"

namespace fp8mp {

namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;
// CTAs of the forward pass on an SM, and 16-byte loads that a thread of it has in
// flight. 8192 x 128000, bf16: 288 us, 295 with 5 and 4, 322 with 2 of 512 threads and 4.
constexpr int kPerSm = 4;
constexpr int kUnroll = 8;
constexpr int kMaxSplits = 8;   // CTAs that may share a row (a portable cluster)
constexpr int kMaxTop = FP8MP_MAX_TOP;
constexpr int kCandidates = 1024;
constexpr float kLog2e = 1.44269504f, kLn2 = 0.693147181f;
constexpr float kLog2eRest = 1.92596303e-8f;  // log2(e) - kLog2e

struct LogpArgs {
    const uint8_t *x;
    const int64_t *target;
    float *logprob, *entropy, *top;
    float2 *stats;
    int64_t *ids;
    int64_t V, ld;
    int splits, k;
};

__device__ __forceinline__ float exp2_approx(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// The larger of two; NaN if either is.
__device__ __forceinline__ float max_nan(float a, float b) {
    float y;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(b));
    return y;
}

// A row of logits: up to EP - 1 elements before the first 16-byte boundary, the
// pieces from there on, and the rest.
template <bool BF16>
struct Row {
    static constexpr int ES = BF16 ? 2 : 4, EP = 16 / ES;
    const uint8_t *base;
    int64_t pieces;
    int head, tail;
    __device__ __forceinline__ Row(const uint8_t *p, int64_t n) : base(p) {
        const int off = static_cast<int>(((16u - (reinterpret_cast<uintptr_t>(p) & 15u)) & 15u) / ES);
        head = static_cast<int64_t>(off) < n ? off : static_cast<int>(n);
        pieces = (n - head) / EP;
        tail = static_cast<int>(n - head - pieces * EP);
    }
    __device__ __forceinline__ const uint4 *body() const { return reinterpret_cast<const uint4 *>(base + head * ES); }
    __device__ __forceinline__ float at(int64_t i) const {
        if constexpr (BF16) return bf16_bits_to_f32(reinterpret_cast<const uint16_t *>(base)[i]);
        else return reinterpret_cast<const float *>(base)[i];
    }
    __device__ __forceinline__ int64_t tail_at() const { return head + pieces * EP; }
};

template <bool BF16>
__device__ __forceinline__ float element(const uint4 &q, int j) {
    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
    if constexpr (BF16) return __uint_as_float(j & 1 ? w[j >> 1] & 0xFFFF0000u : w[j >> 1] << 16);
    else return __uint_as_float(w[j]);
}

// The largest of a piece, NaN left out.
template <bool BF16>
__device__ __forceinline__ float piece_max(const uint4 &q) {
    if constexpr (BF16) {
        __nv_bfloat162 a, b, c, d;
        memcpy(&a, &q.x, 4);
        memcpy(&b, &q.y, 4);
        memcpy(&c, &q.z, 4);
        memcpy(&d, &q.w, 4);
        const __nv_bfloat162 m = __hmax2(__hmax2(a, b), __hmax2(c, d));
        return fmaxf(__low2float(m), __high2float(m));
    } else {
        return fmaxf(fmaxf(__uint_as_float(q.x), __uint_as_float(q.y)), fmaxf(__uint_as_float(q.z), __uint_as_float(q.w)));
    }
}

// Order of the logits as whole numbers: NaN lowest, -0 and +0 the same.
__device__ __forceinline__ uint32_t order_of(float x) {
    if (x != x) return 0u;
    const uint32_t b = __float_as_uint(x + 0.0f);
    return b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float value_of(uint32_t key) {
    return key == 0u ? __uint_as_float(0x7FC00000u) : __uint_as_float(key & 0x80000000u ? key & 0x7FFFFFFFu : ~key);
}
// Larger logits first, then lower indices; 0 is none.
__device__ __forceinline__ uint64_t candidate(uint32_t key, int64_t index) {
    return static_cast<uint64_t>(key) << 32 | (0xFFFFFFFFu - static_cast<uint32_t>(index));
}

// Running maximum m (of what is not NaN, at least -FLT_MAX, so that x - m is a
// number or -Inf for every x below +Inf), s = sum of 2^z, and t = sum of 2^z z,
// with z = (x - m) log2(e).
template <bool ENT>
struct Running {
    float m = -FLT_MAX;
    uint64_t s[2] = {0ull, 0ull}, t[2] = {0ull, 0ull};

    __device__ __forceinline__ void raise(float to) {
        if (!(to > m)) return;
        const float d = (m - to) * kLog2e, f = exp2_approx(d);
        const uint64_t f2 = f2_same(f), d2 = f2_same(f > 0.0f ? d : 0.0f);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            if constexpr (ENT) t[i] = f2_mul(f2_fma(s[i], d2, t[i]), f2);
            s[i] = f2_mul(s[i], f2);
        }
        m = to;
    }
    __device__ __forceinline__ void add(uint64_t x, uint64_t neg_m, int i) {
        uint64_t z = f2_mul(f2_add(x, neg_m), f2_same(kLog2e));
        float z0, z1;
        f2_split(z, z0, z1);
        const uint64_t e = f2_pack(exp2_approx(z0), exp2_approx(z1));
        s[i] = f2_add(s[i], e);
        if constexpr (ENT) t[i] = f2_fma(e, f2_pack(max_nan(z0, -512.0f), max_nan(z1, -512.0f)), t[i]);
    }
    __device__ __forceinline__ void total(float &S, float &T) const {
        float a, b;
        f2_split(f2_add(s[0], s[1]), a, b);
        S = a + b;
        f2_split(f2_add(t[0], t[1]), a, b);
        T = a + b;
    }
};

// (m, S, T) of two parts of a row.
__device__ __forceinline__ void join_parts(float &m, float &S, float &T, float m1, float S1, float T1) {
    const float to = fmaxf(m, m1), d0 = (m - to) * kLog2e, d1 = (m1 - to) * kLog2e;
    const float f0 = exp2_approx(d0), f1 = exp2_approx(d1);
    T = (f0 > 0.0f ? f0 * (T + d0 * S) : 0.0f) + (f1 > 0.0f ? f1 * (T1 + d1 * S1) : 0.0f);
    S = f0 * S + f1 * S1;
    m = to;
}

struct TopShared {
    uint64_t found[kCandidates];
    uint64_t best[kMaxTop];
    uint64_t merged[kMaxSplits * kMaxTop];  // the first CTA's: all the CTAs' best
    uint16_t shares[kThreads];
    uint32_t warp_count[kWarps], warp_min[kWarps];
    uint32_t n_found, n_shares;
};

struct Nothing {};

// A CTA's part of a row.
template <bool BF16>
struct Slice {
    Row<BF16> row;
    int64_t p0, p1;   // its pieces
    int head, tail;   // elements of the row's head and tail that are its own

    // Element `i` of the head (0 to 7) and of the tail (8 to 15), or -1: none.
    __device__ __forceinline__ int64_t edge(int i) const {
        return i < 8 ? (i < head ? i : -1) : i - 8 < tail ? row.tail_at() + i - 8 : -1;
    }
    __device__ __forceinline__ int64_t elements() const { return head + tail + (p1 - p0) * Row<BF16>::EP; }
    // The elements of a thread's share: f(index, logit).
    template <typename F>
    __device__ __forceinline__ void share(F f) const {
        const int t = threadIdx.x;
        for (int64_t p = p0 + t; p < p1; p += kThreads) {
            const uint4 q = __ldg(row.body() + p);
#pragma unroll
            for (int j = 0; j < Row<BF16>::EP; ++j) f(row.head + p * Row<BF16>::EP + j, element<BF16>(q, j));
        }
        if (t < head) f(t, row.at(t));
        if (t >= 32 && t - 32 < tail) f(row.tail_at() + t - 32, row.at(row.tail_at() + t - 32));
    }
};

// Sum over the block of each thread's count; every thread calls it.
__device__ __forceinline__ uint32_t block_count(uint32_t c, TopShared &sh) {
    c = __reduce_add_sync(0xffffffffu, c);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) sh.warp_count[threadIdx.x >> 5] = c;
    __syncthreads();
    uint32_t n = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) n += sh.warp_count[w];
    return n;
}

// sh.best = the `want` (at most the slice's elements) best candidates of the slice,
// best first. `largest`: the largest logit of this thread's pieces (NaN left out).
// `meanwhile` runs before the shares are read again.
template <bool BF16, typename F>
__device__ __forceinline__ void best_of_slice(const Slice<BF16> &sl, float largest, uint32_t want, TopShared &sh, F meanwhile) {
    const int tid = threadIdx.x, lane = tid & 31;
    const uint32_t mine = sl.p0 + tid < sl.p1 ? order_of(largest) : 0u;
    if (tid == 0) sh.n_found = sh.n_shares = 0u;
    // tau: the want-th largest of the shares' largest or one of the next few, by bisection
    // between their extremes, five or six barriers mostly
    const uint32_t most = __reduce_max_sync(0xffffffffu, mine), fewest = __reduce_min_sync(0xffffffffu, mine);
    if (lane == 0) {
        sh.warp_count[tid >> 5] = most;
        sh.warp_min[tid >> 5] = fewest;
    }
    __syncthreads();
    uint32_t tau = 0xFFFFFFFFu, above = 0u;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
        above = max(above, sh.warp_count[w]);
        tau = min(tau, sh.warp_min[w]);
    }
    if (want == 1u) tau = above;
    else ++above;
    const auto bisect = [&](uint32_t enough, int steps) {
        for (uint32_t have = kThreads; steps > 0 && above - tau > 1u && have > enough; --steps) {
            const uint32_t mid = tau + (above - tau) / 2u, c = static_cast<uint32_t>(__syncthreads_count(mine >= mid));
            if (c >= want) {
                tau = mid;
                have = c;
            } else {
                above = mid;
            }
        }
    };
    bisect(want + want / 2u, 16);
    if (mine >= tau) sh.shares[atomicAdd(&sh.n_shares, 1u)] = static_cast<uint16_t>(tid);
    __syncthreads();
    const auto keep = [&](int64_t index, float x) {
        const uint32_t key = order_of(x);
        if (key < tau) return;
        const uint32_t at = atomicAdd(&sh.n_found, 1u);
        if (at < kCandidates) sh.found[at] = candidate(key, index);
    };
    // their pieces, dealt to all threads, and the elements off the 16-byte boundaries. One
    // piece in flight is enough: what a share's strided pieces cost is their sectors' traffic
    // beside the other CTAs' rows (two or four in flight: as fast or slower).
    const uint32_t each = static_cast<uint32_t>((sl.p1 - sl.p0 + kThreads - 1) / kThreads), all_pieces = each * sh.n_shares;
    meanwhile();
    const int64_t off_at = tid < 16 ? sl.edge(tid) : -1;
    const float off = off_at >= 0 ? sl.row.at(off_at) : 0.0f;
    const float least = value_of(tau);
    for (uint32_t i = tid; i < all_pieces; i += kThreads) {
        const uint32_t share = i / each;
        const int64_t p = sl.p0 + sh.shares[share] + static_cast<int64_t>(i - share * each) * kThreads;
        if (p >= sl.p1) continue;
        const uint4 q = __ldg(sl.row.body() + p);
        if (piece_max<BF16>(q) < least) continue;
        uint32_t may = 0;
#pragma unroll
        for (int j = 0; j < Row<BF16>::EP; ++j) may |= static_cast<uint32_t>(!(element<BF16>(q, j) < least)) << j;
        for (; may != 0u; may &= may - 1u) {
            const int j = __ffs(may) - 1, w = BF16 ? j >> 1 : j;
            const uint32_t v = w < 2 ? (w == 0 ? q.x : q.y) : w == 2 ? q.z : q.w;
            keep(sl.row.head + p * Row<BF16>::EP + j, __uint_as_float(!BF16 ? v : j & 1 ? v & 0xFFFF0000u : v << 16));
        }
    }
    if (off_at >= 0) keep(off_at, off);
    __syncthreads();
    uint32_t n = sh.n_found;
    if (n > kCandidates || n < want) {
        // the want-th largest logit itself, by bisection, starting from what is
        // most likely: that tau, to its last bit, is it, over and over
        bisect(0u, 32);
        uint32_t lo = tau, hi = 0xFFFFFFFFu, c = 0;
        sl.share([&](int64_t, float x) { c += order_of(x) >= lo; });
        if (block_count(c, sh) < want) lo = 0u;  // (shares of NaN alone: their largest is not there)
        for (uint32_t mid = lo + 1u; hi - lo > 1u; mid = lo + (hi - lo) / 2u) {
            c = 0;
            sl.share([&](int64_t, float x) { c += order_of(x) >= mid; });
            if (block_count(c, sh) >= want) lo = mid;
            else hi = mid;
        }
        // those above it, fewer than `want`, then its equals from the lowest index on
        if (tid == 0) sh.n_found = 0u;
        __syncthreads();
        sl.share([&](int64_t index, float x) {
            const uint32_t key = order_of(x);
            if (key > lo) sh.found[atomicAdd(&sh.n_found, 1u)] = candidate(key, index);
        });
        __syncthreads();
        uint32_t have = sh.n_found;
        const int64_t body = sl.row.head;
        // step -1: the head; a piece for each thread at a time; then the tail
        const int64_t steps = (sl.p1 - sl.p0 + kThreads - 1) / kThreads;
        for (int64_t step = -1; step <= steps && have < want; ++step) {
            int64_t first = 0;
            uint32_t equal = 0;  // bit j: element first + j is one
            if (step < 0) {
                first = tid;
                if (tid < sl.head) equal = order_of(sl.row.at(first)) == lo;
            } else if (step == steps) {
                first = sl.row.tail_at() + tid;
                if (tid < sl.tail) equal = order_of(sl.row.at(first)) == lo;
            } else {
                const int64_t p = sl.p0 + step * kThreads + tid;
                first = body + p * Row<BF16>::EP;
                if (p < sl.p1) {
                    const uint4 q = __ldg(sl.row.body() + p);
#pragma unroll
                    for (int j = 0; j < Row<BF16>::EP; ++j)
                        equal |= static_cast<uint32_t>(order_of(element<BF16>(q, j)) == lo) << j;
                }
            }
            // exclusive prefix of the counts
            const uint32_t own = __popc(equal);
            uint32_t upto = own;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const uint32_t v = __shfl_up_sync(0xffffffffu, upto, o);
                if (lane >= o) upto += v;
            }
            __syncthreads();
            if (lane == 31) sh.warp_count[tid >> 5] = upto;
            __syncthreads();
            uint32_t at = have + upto - own, all = 0;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                const uint32_t v = sh.warp_count[w];
                if (w < (tid >> 5)) at += v;
                all += v;
            }
            while (equal != 0u && at < want) {
                sh.found[at++] = candidate(lo, first + __ffs(equal) - 1);
                equal &= equal - 1u;
            }
            have += all;
        }
        __syncthreads();
        n = want;
    }
    for (uint32_t i = tid; i < n; i += kThreads) {
        const uint64_t c = sh.found[i];
        uint32_t rank = 0;
        for (uint32_t j = 0; j < n; ++j) rank += sh.found[j] > c;
        if (rank < want) sh.best[rank] = c;
    }
    __syncthreads();
}

// kUnroll pieces, 16-byte loads first: those of [p, end) that lie `step` apart.
template <bool BF16, bool ENT>
__device__ __forceinline__ float add_pieces(Running<ENT> &run, const uint4 *body, int64_t p, int64_t end, int step) {
    const uint32_t none = BF16 ? 0xFF80FF80u : 0xFF800000u;  // -Inf
    uint4 q[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u)
        q[u] = p + u * step < end ? __ldg(body + p + u * step) : make_uint4(none, none, none, none);
    float top = piece_max<BF16>(q[0]);
#pragma unroll
    for (int u = 1; u < kUnroll; ++u) top = fmaxf(top, piece_max<BF16>(q[u]));
    run.raise(top);
    const uint64_t neg_m = f2_same(-run.m);
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
        const uint32_t w[4] = {q[u].x, q[u].y, q[u].z, q[u].w};
        if constexpr (BF16) {
#pragma unroll
            for (int j = 0; j < 4; ++j) run.add(f2_from_bits(w[j] << 16, w[j] & 0xFFFF0000u), neg_m, j & 1);
        } else {
            run.add(f2_from_bits(w[0], w[1]), neg_m, 0);
            run.add(f2_from_bits(w[2], w[3]), neg_m, 1);
        }
    }
    return top;
}
template <bool ENT>
__device__ __forceinline__ void add_one(Running<ENT> &run, float x) {
    run.raise(x);
    run.add(f2_from_bits(__float_as_uint(x), 0xFF800000u), f2_same(-run.m), 0);
}
// (m, S, T) of the warp's parts.
__device__ __forceinline__ void join_warp(float &m, float &S, float &T) {
    const float to = value_of(__reduce_max_sync(0xffffffffu, order_of(m))), d = (m - to) * kLog2e, f = exp2_approx(d);
    T = f > 0.0f ? f * (T + d * S) : 0.0f;
    S *= f;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        S += __shfl_xor_sync(0xffffffffu, S, o);
        T += __shfl_xor_sync(0xffffffffu, T, o);
    }
    m = to;
}

// log p of a logit, from the row's (m, log S). S is 0 where every logit is -Inf.
__device__ __forceinline__ float log_p(float x, float m, float log_s) {
    const float d = x - m, inf = __uint_as_float(0x7F800000u);
    return d == -inf && log_s == log_s ? -inf : d - log_s;
}
template <bool ENT>
__device__ __forceinline__ void write_row(const LogpArgs &a, int64_t m_row, int64_t target, float x_target, float m, float S,
                                          float T, float log_s) {
    a.stats[m_row] = make_float2(S == 0.0f ? -__uint_as_float(0x7F800000u) : m, log_s);
    if (a.logprob != nullptr) a.logprob[m_row] = target >= 0 && target < a.V ? log_p(x_target, m, log_s) : 0.0f;
    if (ENT) a.entropy[m_row] = S == 0.0f ? 0.0f : log_s - kLn2 * T / S;
}

// Short rows, without the most probable tokens: one for each warp, no barrier.
template <bool BF16, bool ENT>
__global__ void __launch_bounds__(kThreads, kPerSm) logp_rows_kernel(const LogpArgs a, int64_t M) {
    pdl_wait();
    pdl_launch_dependents();
    const int lane = threadIdx.x & 31;
    const int64_t m_row = static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
    if (m_row >= M) return;
    const Row<BF16> row(a.x + m_row * a.ld * Row<BF16>::ES, a.V);
    Running<ENT> run;
    for (int64_t p = lane; p < row.pieces; p += 32 * kUnroll) add_pieces<BF16>(run, row.body(), p, row.pieces, 32);
    const int64_t target = lane == 0 && a.logprob != nullptr ? a.target[m_row] : -1;
    if (lane < row.head) add_one(run, row.at(lane));
    if (lane < row.tail) add_one(run, row.at(row.tail_at() + lane));
    const float x_target = target >= 0 && target < a.V ? row.at(target) : 0.0f;
    float m = run.m, S, T;
    run.total(S, T);
    join_warp(m, S, T);
    if (lane == 0) write_row<ENT>(a, m_row, target, x_target, m, S, T, logf(S));
}

__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }
__device__ __forceinline__ void st_cluster_f32(uint32_t addr, float v) {
    asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(addr), "f"(v) : "memory");
}
__device__ __forceinline__ void st_cluster_u64(uint32_t addr, uint64_t v) {
    asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(addr), "l"(v) : "memory");
}

template <bool BF16, bool ENT, bool TOP>
__global__ void __launch_bounds__(kThreads, kPerSm) logp_fwd_kernel(const LogpArgs a) {
    __shared__ float warp_part[kWarps][3];
    __shared__ float cta_part[kMaxSplits][3];  // the first CTA's: all the CTAs' (m, S, T)
    __shared__ std::conditional_t<TOP, TopShared, Nothing> sh;
    using R = Row<BF16>;
    const uint32_t splits = static_cast<uint32_t>(a.splits);
    if (splits > 1) cluster_arrive();  // this CTA has started: its peers may write to it
    pdl_wait();
    pdl_launch_dependents();
    const int tid = threadIdx.x, lane = tid & 31;
    const uint32_t rank = splits > 1 ? cluster_ctarank() : 0u;
    const int64_t m_row = blockIdx.x / splits;
    const R row(a.x + m_row * a.ld * R::ES, a.V);
    const Slice<BF16> sl = {row, row.pieces * rank / splits, row.pieces * (rank + 1) / splits,
                            rank == 0 ? row.head : 0, rank == splits - 1 ? row.tail : 0};

    Running<ENT> run;
    float largest = __uint_as_float(0xFF800000u);  // -Inf
    for (int64_t p = sl.p0 + tid; p < sl.p1; p += kThreads * kUnroll) {
        const float top = add_pieces<BF16>(run, row.body(), p, sl.p1, kThreads);
        if (TOP) largest = fmaxf(largest, top);
    }
    float m = run.m, S, T;
    run.total(S, T);
    // Warp 0 joins the warps' parts (lanes 0 to 7) and the elements off the 16-byte
    // boundaries (8 to 23); these and the target's logit are on their way meanwhile.
    int64_t target = -1;
    float off = __uint_as_float(0xFF800000u), x_target = 0.0f;
    if (tid < 32) {
        const int64_t at = lane >= kWarps && lane < kWarps + 16 ? sl.edge(lane - kWarps) : -1;
        if (at >= 0) off = row.at(at);
        if (lane == 0 && rank == 0 && a.logprob != nullptr) target = a.target[m_row];
    }
    join_warp(m, S, T);
    if (lane == 0) {
        warp_part[tid >> 5][0] = m;
        warp_part[tid >> 5][1] = S;
        warp_part[tid >> 5][2] = T;
    }
    __syncthreads();
    if (tid < 32) {
        if (!TOP && target >= 0 && target < a.V) x_target = row.at(target);
        Running<ENT> one;
        add_one(one, off);
        m = one.m;
        one.total(S, T);
        if (lane < kWarps) {
            m = warp_part[lane][0];
            S = warp_part[lane][1];
            T = warp_part[lane][2];
        }
        join_warp(m, S, T);
    }
    const uint32_t k = TOP ? static_cast<uint32_t>(a.k) : 0u;
    if constexpr (TOP) {
        const int64_t n = sl.elements();
        const uint32_t want = n < static_cast<int64_t>(k) ? static_cast<uint32_t>(n) : k;
        const auto aim = [&] {
            if (target >= 0 && target < a.V) x_target = row.at(target);
        };
        if (want > 0) best_of_slice<BF16>(sl, largest, want, sh, aim);
        else aim();
        if (tid >= static_cast<int>(want) && tid < static_cast<int>(k)) sh.best[tid] = 0ull;
        __syncthreads();
    }
    if (splits > 1) {
        cluster_wait();  // all have started
        if (tid == 0) {
            const uint32_t to = mapa_shared(smem_u32(cta_part[rank]), 0u);
            st_cluster_f32(to, m);
            st_cluster_f32(to + 4, S);
            st_cluster_f32(to + 8, T);
        }
        if constexpr (TOP)
            if (tid < static_cast<int>(k)) st_cluster_u64(mapa_shared(smem_u32(&sh.merged[rank * k + tid]), 0u), sh.best[tid]);
        __syncwarp();
        cluster_arrive();
        cluster_wait();
        if (rank != 0) return;
        if (tid < 32) {
            m = -FLT_MAX;
            S = T = 0.0f;
            for (uint32_t r = 0; r < splits; ++r) join_parts(m, S, T, cta_part[r][0], cta_part[r][1], cta_part[r][2]);
        }
        if constexpr (TOP) {  // the best of the CTAs' best
            const uint32_t n = splits * k;
            for (uint32_t i = tid; i < n; i += kThreads) {
                const uint64_t c = sh.merged[i];
                uint32_t place = 0;
                for (uint32_t j = 0; j < n; ++j) place += sh.merged[j] > c;
                if (place < k && c != 0ull) sh.best[place] = c;
            }
            __syncthreads();
        }
    }
    if (tid >= 32) return;
    const float log_s = logf(S);
    if (lane == 0) write_row<ENT>(a, m_row, target, x_target, m, S, T, log_s);
    if constexpr (TOP) {
        for (uint32_t i = lane; i < k; i += 32) {
            const uint64_t c = sh.best[i];
            a.top[m_row * k + i] = log_p(value_of(static_cast<uint32_t>(c >> 32)), m, log_s);
            a.ids[m_row * k + i] = 0xFFFFFFFFu - static_cast<uint32_t>(c);
        }
    }
}

// ---------------------------------------------------------------- gradient

constexpr int kGradThreads = 256, kGradUnroll = 4;
constexpr int kGradPerSm = 5;  // CTAs: 8192 x 128000 to codes 471 us, 501 with 4, 489 with 6 (spills)
constexpr int kGradRound = kGradThreads * kGradUnroll;  // pieces of a row that a CTA has in flight

struct LogpGradArgs {
    const uint8_t *x;
    const int64_t *target;
    const float2 *stats;
    const float *da, *db, *entropy, *scale;
    float *amax;
    uint8_t *out;
    int64_t M, V, ld;
    int splits;  // CTAs that share a row
};

__host__ __device__ inline int64_t least(int64_t a, int64_t b) { return a < b ? a : b; }

// What a row's elements share: dx = p (c0 + c1 z), with z = log2 p.
struct RowGrad {
    float m, l2;       // p = 2^((x - m) log2(e) - l2), times what c0 and c1 hold
    float c0, c1, a;   // a: added at the target
    int64_t target;
};

template <bool ENT>
__device__ __forceinline__ float grad_of(float x, const RowGrad &g) {
    float z = fmaf(x - g.m, kLog2e, -g.l2);
    if constexpr (ENT) {
        z = max_nan(z, -512.0f);
        return exp2_approx(z) * fmaf(g.c1, z, g.c0);
    }
    return exp2_approx(z) * g.c0;
}

// WARP: short rows, one for each warp.
template <bool BF16, bool CODES, bool ENT, bool WARP>
__global__ void __launch_bounds__(kGradThreads, WARP ? 4 : kGradPerSm) logp_bwd_kernel(const LogpGradArgs a) {
    using R = Row<BF16>;
    constexpr int ES = R::ES, EP = R::EP, THREADS = WARP ? 32 : kGradThreads, ROUND = THREADS * kGradUnroll;
    pdl_wait();
    pdl_launch_dependents();
    const int tid = WARP ? threadIdx.x & 31 : threadIdx.x;
    const int64_t at = WARP ? static_cast<int64_t>(blockIdx.x) * (kGradThreads / 32) + (threadIdx.x >> 5) : blockIdx.x / a.splits;
    const bool mine = !WARP || at < a.M;  // (a warp without a row takes part in the last barrier)
    const int64_t m_row = mine ? at : 0;
    const int part = WARP ? 0 : static_cast<int>(blockIdx.x % a.splits), splits = WARP ? 1 : a.splits;
    const R row(a.x + m_row * a.ld * ES, a.ld);  // the columns from V on included: theirs is 0
    uint8_t *out = a.out + m_row * a.ld * (CODES ? 1 : ES);
    // whole rounds for each CTA, the row's last one but for the rest
    const int64_t rounds = (row.pieces + ROUND - 1) / ROUND;
    const int64_t p0 = rounds * part / splits * ROUND, p1 = mine ? least(rounds * (part + 1) / splits * ROUND, row.pieces) : 0;
    const uint4 *body = row.body();
    // the first logits are on their way before what the row's elements share
    uint4 q[kGradUnroll];
    const auto fetch = [&](int64_t p) {
#pragma unroll
        for (int u = 0; u < kGradUnroll; ++u)
            if (p + u * THREADS < p1) q[u] = __ldcs(body + p + u * THREADS);
    };
    fetch(p0 + tid);
    RowGrad g;
    const float2 st = a.stats[m_row];
    g.target = a.target[m_row];
    g.a = a.da[m_row];
    const float b = ENT ? a.db[m_row] : 0.0f;
    if (!(g.target >= 0 && g.target < a.V)) {
        g.target = -1;
        g.a = 0.0f;
    }
    // log2 S in two parts; the second, below an ulp of the first, goes into c
    g.m = st.x;
    g.l2 = st.y * kLog2e;
    const float rest = fmaf(st.y, kLog2e, -g.l2) + st.y * kLog2eRest, c = 1.0f - rest * kLn2;
    g.c0 = -c * (ENT ? fmaf(b, a.entropy[m_row], g.a) : g.a);
    g.c1 = -c * b * kLn2;
    // no token has a probability (log S is -Inf), or nothing asks for a gradient
    const bool zero = st.y == -__uint_as_float(0x7F800000u) || (g.a == 0.0f && b == 0.0f);
    const float scale = CODES ? __ldg(a.scale) : 1.0f;
    float am = 0.0f;
    for (int64_t p = p0 + tid; p < p1; p += THREADS * kGradUnroll) {
        if (p != p0 + tid && !zero) fetch(p);
#pragma unroll
        for (int u = 0; u < kGradUnroll; ++u) {
            const int64_t i = p + u * THREADS;
            if (i >= p1) break;
            const int64_t first = row.head + i * EP;
            float y[EP];
#pragma unroll
            for (int j = 0; j < EP; ++j) y[j] = zero ? 0.0f : grad_of<ENT>(element<BF16>(q[u], j), g);
            if (!zero && static_cast<uint64_t>(g.target - first) < EP) {
#pragma unroll
                for (int j = 0; j < EP; ++j)
                    if (first + j == g.target) y[j] += g.a;
            }
            if (first + EP > a.V) {
#pragma unroll
                for (int j = 0; j < EP; ++j)
                    if (first + j >= a.V) y[j] = 0.0f;
            }
#pragma unroll
            for (int j = 0; j < EP; ++j) am = fmaxf(am, fabsf(y[j]));
            if constexpr (CODES) {
                uint32_t c4[EP / 4];
#pragma unroll
                for (int j = 0; j < EP / 4; ++j)
                    c4[j] = cvt_quad_probed<FP8MP_E5M2>(y[4 * j] * scale, y[4 * j + 1] * scale, y[4 * j + 2] * scale,
                                                        y[4 * j + 3] * scale);
                if constexpr (BF16) reinterpret_cast<uint2 *>(out)[i] = make_uint2(c4[0], c4[1]);
                else reinterpret_cast<uint32_t *>(out)[i] = c4[0];
            } else if constexpr (BF16) {
                reinterpret_cast<uint4 *>(out + row.head * ES)[i] = make_uint4(
                    bf16_pair(y[0], y[1]), bf16_pair(y[2], y[3]), bf16_pair(y[4], y[5]), bf16_pair(y[6], y[7]));
            } else {
                reinterpret_cast<float4 *>(out + row.head * ES)[i] = make_float4(y[0], y[1], y[2], y[3]);
            }
        }
    }
    if constexpr (!CODES) {  // (codes need rows of whole pieces)
        // lanes 0 to 6 the head's, 8 to 14 the tail's
        const bool h = mine && part == 0 && tid < row.head, t = mine && part == splits - 1 && tid >= 8 && tid - 8 < row.tail;
        if (h || t) {
            const int64_t i = h ? tid : row.tail_at() + tid - 8;
            float y = zero || i >= a.V ? 0.0f : grad_of<ENT>(row.at(i), g);
            if (!zero && i == g.target) y += g.a;
            am = fmaxf(am, fabsf(y));
            if constexpr (BF16) reinterpret_cast<__nv_bfloat16 *>(out)[i] = __float2bfloat16_rn(y);
            else reinterpret_cast<float *>(out)[i] = y;
        }
    }
    if (a.amax != nullptr) block_amax_atomic(am, a.amax);
}

// CTAs that share a row of `bytes`. Clusters start later the more of them an SM gets, so
// M s^2 is bounded, and each CTA has three quarters of a round of loads at least, twice
// that where an SM has several. bf16, V 128000, by 1, 2, 4 and 8 CTAs a row: 8 rows 6.7, 4.4,
// 3.1, 2.5 us; 64 rows with their 20 best 16.3, 11.5, 9.5, 11.0; 256 with 5 18.4, 17.7, 21.8, 30;
// V 32000, 128 rows 3.8, 3.7, 4.7, 8.2; 333 rows of 50001 in fp32 14.4, 17.2, 17.8, 20.6.
int splits_for(int64_t M, int64_t bytes, int num_sms) {
    const int64_t part = kThreads * kUnroll * 16 / 4 * 3;
    int s = 1;
    while (s < kMaxSplits && M * (2 * s) * (2 * s) <= 8ll * num_sms &&
           bytes >= 2 * s * (M * 2 * s > num_sms ? 2 * part : part))
        s *= 2;
    return s;
}

// CTAs that share a row of `pieces` in the backward pass. A CTA costs an SM 0.2 us, and
// the last one's rounds, 1.3 us each, are not hidden. To codes, by 1, 2, 4 CTAs a row: 512 x
// 32000 13.9, 11.7, 12.1 us; 2048 x 32000 35.5, 35.7, 39.9; 256 x 128000 28.3, 25.3, 20.9.
int grad_splits_for(int64_t M, int64_t pieces, int num_sms) {
    const int64_t rounds = (pieces + kGradRound - 1) / kGradRound;
    int best = 1;
    int64_t least = 0;
    for (int s = 1; s <= 64 && s <= rounds; ++s) {
        const int64_t cost = M * s + 6ll * num_sms * ((rounds + s - 1) / s);
        if (s == 1 || cost < least) {
            least = cost;
            best = s;
        }
    }
    return best;
}

// Whether a warp takes a row: one round of its loads, or up to eight when there are rows
// for two blocks in every place of the device. 16384 rows of 500, bf16: 10.9 us, 63.8 by
// blocks; 8192 of 8000: 21.9 and 45.4; 700 of 8000, where a block is done first, 6.2 by blocks.
template <bool BF16>
bool short_rows(int64_t M, int64_t V, int num_sms) {
    const int64_t round = 32 * kUnroll * Row<BF16>::EP;
    return V <= round || (V <= 8 * round && M >= 2ll * num_sms * kPerSm);
}

template <bool BF16, bool ENT>
cudaError_t fwd(const LogpArgs &a, int64_t M, cudaStream_t s, int num_sms) {
    const dim3 grid(static_cast<unsigned>(M * a.splits)), block(kThreads);
    const unsigned c = static_cast<unsigned>(a.splits);
    if (a.k > 0) return launch_kernel_cluster(logp_fwd_kernel<BF16, ENT, true>, grid, block, 0, s, c, a);
    if (short_rows<BF16>(M, a.V, num_sms))
        return launch_kernel(logp_rows_kernel<BF16, ENT>, dim3(static_cast<unsigned>((M + kWarps - 1) / kWarps)), block, 0, s, a, M);
    return launch_kernel_cluster(logp_fwd_kernel<BF16, ENT, false>, grid, block, 0, s, c, a);
}

template <bool BF16, bool CODES, bool ENT>
cudaError_t bwd(const LogpGradArgs &a, cudaStream_t s, int num_sms) {
    const dim3 block(kGradThreads);
    // A warp takes up to two rounds (16384 rows of 512, codes: 9.8 us, 39.1 by blocks), up to
    // four when there is a row for every warp (8192 rows of 4000: 21.9, 29.1; 1024: 7.0, 5.3).
    const int64_t round = 32 * kGradUnroll * Row<BF16>::EP;
    if (a.ld <= 2 * round || (a.ld <= 4 * round && a.M >= 4ll * num_sms * (kGradThreads / 32))) {
        const dim3 grid(static_cast<unsigned>((a.M + kGradThreads / 32 - 1) / (kGradThreads / 32)));
        return launch_kernel(logp_bwd_kernel<BF16, CODES, ENT, true>, grid, block, 0, s, a);
    }
    return launch_kernel(logp_bwd_kernel<BF16, CODES, ENT, false>, dim3(static_cast<unsigned>(a.M * a.splits)), block, 0, s, a);
}
template <bool BF16, bool CODES>
cudaError_t bwd(const LogpGradArgs &a, cudaStream_t s, int num_sms) {
    return a.db != nullptr ? bwd<BF16, CODES, true>(a, s, num_sms) : bwd<BF16, CODES, false>(a, s, num_sms);
}

}  // namespace

int launch_logprobs_fwd(const void *x, int x_dtype, int64_t M, int64_t V, int64_t ld, const int64_t *target,
                        float *logprob, float *stats, float *entropy, float *top, int64_t *ids, int k, cudaStream_t s,
                        const DeviceInfo &dev) {
    LogpArgs a = {static_cast<const uint8_t *>(x), target, logprob, entropy, top, reinterpret_cast<float2 *>(stats), ids,
                  V, ld, 1, k};
    a.splits = splits_for(M, V * (x_dtype == FP8MP_BF16 ? 2 : 4), dev.num_sms);
    const bool b = x_dtype == FP8MP_BF16;
    cudaError_t e;
    if (entropy != nullptr) e = b ? fwd<true, true>(a, M, s, dev.num_sms) : fwd<false, true>(a, M, s, dev.num_sms);
    else e = b ? fwd<true, false>(a, M, s, dev.num_sms) : fwd<false, false>(a, M, s, dev.num_sms);
    if (e != cudaSuccess) return fail(FP8MP_ERR_LAUNCH, "logprobs: launch failed: %s", cudaGetErrorString(e));
    return FP8MP_OK;
}

int launch_logprobs_bwd(const void *x, int x_dtype, int64_t M, int64_t V, int64_t ld, const int64_t *target,
                        const float *stats, const float *dlogprob, const float *entropy, const float *dentropy,
                        const float *scale, void *dlogits, float *amax, cudaStream_t s, const DeviceInfo &dev) {
    LogpGradArgs a = {static_cast<const uint8_t *>(x), target, reinterpret_cast<const float2 *>(stats), dlogprob, dentropy,
                      entropy, scale, amax, static_cast<uint8_t *>(dlogits), M, V, ld, 1};
    a.splits = grad_splits_for(M, ld / (x_dtype == FP8MP_BF16 ? 8 : 4), dev.num_sms);
    const bool b = x_dtype == FP8MP_BF16;
    cudaError_t e;
    if (scale != nullptr) e = b ? bwd<true, true>(a, s, dev.num_sms) : bwd<false, true>(a, s, dev.num_sms);
    else e = b ? bwd<true, false>(a, s, dev.num_sms) : bwd<false, false>(a, s, dev.num_sms);
    if (e != cudaSuccess) return fail(FP8MP_ERR_LAUNCH, "logprobs: launch failed: %s", cudaGetErrorString(e));
    return FP8MP_OK;
}

}  // namespace fp8mp
