// adamw.cu -- the global gradient norm and one AdamW step over many tensors
// at once, with the moments in fp32 or in 8-bit codes under block scales.
//
// Both kernels walk the tensors' elements in units of 256 (one warp, eight
// consecutive elements per lane), eight units to a chunk, one chunk per block
// at a time. The tensors' descriptors travel as kernel parameters with the
// prefix sums of their chunk counts, so a call needs no table in device
// memory and can be captured in a graph; a call with more tensors than one
// launch's parameters hold is split into several launches.
//
// Both are bound by HBM: the norm reads the gradients once (2 or 4 B per
// parameter); the step reads gradient, master and moments and writes master,
// moments and the weight copy (bf16 gradient, E4M3 copy: 27 B per parameter
// with fp32 moments, 15.06 B with 8-bit ones).
#include <cstring>

#include "fp8mp_f32x2.cuh"
#include "fp8mp_internal.cuh"

namespace fp8mp {

namespace {

constexpr int kThreads = 256;
constexpr int kUnit = 256;                            // elements of a unit: one warp, one scale of the 8-bit moments
constexpr int kChunk = kUnit * (kThreads / 32);       // elements of a chunk
constexpr int kNormChunk = 8192;                      // elements of a chunk of the norm
constexpr int kNormBlocksPerSm = 8;
constexpr int kMaxNormBlocks = 4096;
// Blocks per SM of a step's grid (4 are resident): shares small enough to even
// out the tail, large enough to pay for their start. 243 M parameters, 32-bit
// moments: 1079 us with 4, 1069 with 8, 1046 with 16, 999 with 32, 1079 with 64
// (993 with 3 blocks resident, for their registers); 8-bit: 700 us with 4, 679
// with 8, 669 with 16, 686 with 32.
constexpr int kStepBlocksPerSm32 = 32, kStepBlocksPerSm8 = 16;

// The workspace: the arrival counter, then the running sum over launches,
// both zero between calls, then the blocks' partial sums.
struct Workspace {
    unsigned int arrivals;
    unsigned int pad;
    double sum;
    float partial[kMaxNormBlocks];
};

// The tensor that chunk c belongs to: the last one with first[t] <= c (one without
// chunks shares its `first` with the next). A walk over them instead loads a
// constant for each: the step of 61 small tensors 9.4 us, 8.3 so.
__device__ __forceinline__ int tensor_of(const int32_t *first, int count, int c) {
    int t = 0, end = count;
    while (end - t > 1) {
        const int mid = (t + end) >> 1;
        if (first[mid] <= c) t = mid;
        else end = mid;
    }
    return t;
}

// ------------------------------------------------------------------- norm

struct NormTensor {
    const void *grad;
    int64_t n;
    int32_t bf16;
};
template <int CAP>
struct NormBatch {
    NormTensor t[CAP];
    int32_t first[CAP + 1];  // chunks before tensor i
    int32_t count;
};

__device__ __forceinline__ float sum_squares(const float (&f)[8]) {
    const float a = __fmaf_rn(f[0], f[0], __fmul_rn(f[1], f[1])), b = __fmaf_rn(f[2], f[2], __fmul_rn(f[3], f[3]));
    const float c = __fmaf_rn(f[4], f[4], __fmul_rn(f[5], f[5])), d = __fmaf_rn(f[6], f[6], __fmul_rn(f[7], f[7]));
    return __fadd_rn(__fadd_rn(a, b), __fadd_rn(c, d));
}

__device__ __forceinline__ void unpack_bf16(const uint4 &d, float (&f)[8]) {
    const uint32_t w[4] = {d.x, d.y, d.z, d.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        f[2 * j] = __uint_as_float(w[j] << 16);
        f[2 * j + 1] = __uint_as_float(w[j] & 0xFFFF0000u);
    }
}

__device__ __forceinline__ float block_sum(float v, float *red) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v = __fadd_rn(v, __shfl_xor_sync(0xffffffffu, v, o));
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
    __syncthreads();
    float s = 0.0f;
    if (threadIdx.x == 0)
        for (int w = 0; w < kThreads / 32; ++w) s = __fadd_rn(s, red[w]);
    return s;
}

// The sum of squares over the batch's tensors: each thread adds its vectors'
// squares in fp32 (eight at a time, pairwise), a block its threads', the last
// block to arrive the blocks' sums in double and in block order, so the result
// does not depend on which block that is. Inf and NaN need no test of their
// own: either makes the sum Inf or NaN. A thread's or a block's squares may leave
// fp32 together, so a sum of 2^128 or more is Inf wherever they lie, and counts as
// an overflow of the step too. Bound by HBM: 243 M
// bf16 gradients in 72.6 us, 0.99 of the copy rate.
template <int CAP>
__global__ void __launch_bounds__(kThreads)
grad_norm_kernel(const __grid_constant__ NormBatch<CAP> batch, Workspace *ws, float *norm, int32_t *found_inf,
                 int finish) {
    pdl_wait();
    pdl_launch_dependents();
    __shared__ float red[kThreads / 32];
    __shared__ int last;
    float acc = 0.0f;
    int t = -1;
    const int chunks = batch.first[batch.count];
    for (int c = blockIdx.x; c < chunks; c += gridDim.x) {
        if (t < 0 || c >= batch.first[t + 1]) t = tensor_of(batch.first, batch.count, c);
        const NormTensor &T = batch.t[t];
        const int64_t base = static_cast<int64_t>(c - batch.first[t]) * kNormChunk;
        const int64_t left = T.n - base;
        const int n = left < kNormChunk ? static_cast<int>(left) : kNormChunk;
        // whole vectors of 16 bytes, all loaded before the first is used, then the
        // few elements after a tensor's last
        if (T.bf16) {
            const uint16_t *g = static_cast<const uint16_t *>(T.grad) + base;
            uint4 d[4];
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const int i = u * kThreads + threadIdx.x;
                d[u] = 8 * i + 8 <= n ? __ldcs(reinterpret_cast<const uint4 *>(g) + i) : make_uint4(0u, 0u, 0u, 0u);
            }
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                float f[8];
                unpack_bf16(d[u], f);
                acc = __fadd_rn(acc, sum_squares(f));
            }
            const int rest = (n & ~7) + threadIdx.x;
            if (rest < n) {
                const float f = bf16_bits_to_f32(g[rest]);
                acc = __fmaf_rn(f, f, acc);
            }
        } else {
            const float *g = static_cast<const float *>(T.grad) + base;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                float4 d[4];
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    const int i = (4 * h + u) * kThreads + threadIdx.x;
                    d[u] = 4 * i + 4 <= n ? __ldcs(reinterpret_cast<const float4 *>(g) + i)
                                          : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                }
#pragma unroll
                for (int u = 0; u < 4; u += 2) {
                    const float f[8] = {d[u].x,     d[u].y,     d[u].z,     d[u].w,
                                        d[u + 1].x, d[u + 1].y, d[u + 1].z, d[u + 1].w};
                    acc = __fadd_rn(acc, sum_squares(f));
                }
            }
            const int rest = (n & ~3) + threadIdx.x;
            if (rest < n) acc = __fmaf_rn(g[rest], g[rest], acc);
        }
    }
    const float s = block_sum(acc, red);
    if (threadIdx.x == 0) {
        ws->partial[blockIdx.x] = s;
        __threadfence();
        last = atomicAdd(&ws->arrivals, 1u) == gridDim.x - 1;
    }
    __syncthreads();
    if (!last) return;
    __threadfence();
    // thread i adds the partial sums i, i + 256, ...; then a fixed tree
    __shared__ double dred[kThreads];
    double d = 0.0;
    for (unsigned i = threadIdx.x; i < gridDim.x; i += kThreads) d += static_cast<double>(__ldcg(&ws->partial[i]));
    dred[threadIdx.x] = d;
    __syncthreads();
    for (int o = kThreads / 2; o > 0; o >>= 1) {
        if (threadIdx.x < static_cast<unsigned>(o)) dred[threadIdx.x] += dred[threadIdx.x + o];
        __syncthreads();
    }
    if (threadIdx.x == 0) {
        const double total = ws->sum + dred[0];
        ws->arrivals = 0u;
        ws->sum = finish ? 0.0 : total;
        if (finish) {
            // past fp32 whichever way the squares are shared out; NaN stays NaN
            *norm = total >= 0x1p128 ? INFINITY : static_cast<float>(sqrt(total));
            *found_inf = total < 0x1p128 ? 0 : 1;
        }
    }
}

// ------------------------------------------------------------------- step

struct StepTensor {
    const void *grad;
    float *w;
    void *m, *v;
    float *sm, *sv;
    void *copy;
    const float *copy_scale;
    float *copy_amax;
    int64_t n;
    float decay;
    uint32_t ordinal;
    int8_t grad_bf16;
    int8_t copy_kind;  // 0 none, 1 bf16, 2 E4M3
    int8_t codes;      // 8-bit moments
};
template <int CAP>
struct StepBatch {
    StepTensor t[CAP];
    int32_t first[CAP + 1];
    int32_t count;
};
struct StepArgs {
    float *loss_scale;
    int32_t *growth;
    const int32_t *found_inf;
    float *beta_pows;
    uint32_t *seed;
    const float *grad_norm;
    float max_norm, lr, b1, b2, eps, backoff, growth_factor;
    int32_t interval;
    int32_t finish;
    Workspace *ws;
};

struct Scalars {
    float coef, b1, c1, b2, c2, step, root, eps, lr;
};

// What every element of the step shares. The clip takes the gradients' norm
// as measured, under the loss scale.
__device__ __forceinline__ Scalars make_scalars(const StepArgs &a) {
    Scalars s;
    const float inv_s = __fdiv_rn(1.0f, *a.loss_scale);
    s.coef = inv_s;
    if (a.grad_norm != nullptr) {
        const float clip = __fdiv_rn(a.max_norm, __fadd_rn(__fmul_rn(*a.grad_norm, inv_s), 1e-6f));
        if (clip < 1.0f) s.coef = __fmul_rn(inv_s, clip);
    }
    s.b1 = a.b1;
    s.b2 = a.b2;
    s.c1 = __fsub_rn(1.0f, a.b1);
    s.c2 = __fsub_rn(1.0f, a.b2);
    s.step = __fdiv_rn(a.lr, __fsub_rn(1.0f, __fmul_rn(a.beta_pows[0], a.b1)));
    s.root = __fdiv_rn(1.0f, __fsqrt_rn(__fsub_rn(1.0f, __fmul_rn(a.beta_pows[1], a.b2))));
    s.eps = a.eps;
    s.lr = a.lr;
    return s;
}

__device__ __forceinline__ float sqrt_fast(float x) {
    float r;
    asm("sqrt.approx.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

// The moments' recurrences, every operation rounded once (no contraction:
// the 8-bit codes are a function of these bits).
__device__ __forceinline__ void moments(const Scalars &s, float g, float &m, float &v) {
    const float u = __fmul_rn(g, s.coef);
    m = __fadd_rn(__fmul_rn(m, s.b1), __fmul_rn(u, s.c1));
    v = __fadd_rn(__fmul_rn(v, s.b2), __fmul_rn(__fmul_rn(u, u), s.c2));
}
// The weight: w (1 - lr decay) - (lr / (1 - b1^t)) m / (sqrt(v / (1 - b2^t)) + eps).
// The square root and the quotient are the hardware's approximations (2 ulp):
// their error is 2^-22 of a step, far below half an ulp of w.
__device__ __forceinline__ float updated(const Scalars &s, float shrink, float w, float m, float v) {
    const float den = __fmaf_rn(sqrt_fast(v), s.root, s.eps);
    return __fmaf_rn(-s.step, __fdividef(m, den), __fmul_rn(w, shrink));
}

// The counter hash of the stochastic rounding: xor-shifts and odd multiplies.
__device__ __forceinline__ uint32_t mix32(uint32_t x) {
    x = (x ^ (x >> 16)) * 0x7FEB352Du;
    x = (x ^ (x >> 15)) * 0x846CA68Bu;
    return x ^ (x >> 16);
}

__device__ __forceinline__ float square(float c) { return __fmul_rn(c, c); }
__device__ __forceinline__ float fourth(float c) { return square(square(c)); }

// y on the grid of 0, 1, 2^p, ..., TOP^p: the largest code c with c^p <= y (the
// approximate root is corrected, so the code does not depend on its error),
// one more with probability (y - c^p) / ((c + 1)^p - c^p), r being uniform.
template <bool FOURTH>
__device__ __forceinline__ float quantize(float y, float r) {
    constexpr float TOP = FOURTH ? 255.0f : 127.0f;
    float root = sqrt_fast(y);
    if constexpr (FOURTH) root = sqrt_fast(root);
    float c = fminf(floorf(root), TOP);
    auto power = [](float x) { return FOURTH ? fourth(x) : square(x); };
    if (power(__fadd_rn(c, 1.0f)) <= y) c = __fadd_rn(c, 1.0f);
    if (power(c) > y) c = __fsub_rn(c, 1.0f);
    c = fminf(c, TOP);
    const float lo = power(c);
    const bool up = __fmul_rn(r, __fsub_rn(power(__fadd_rn(c, 1.0f)), lo)) < __fsub_rn(y, lo);
    return up ? fminf(__fadd_rn(c, 1.0f), TOP) : c;
}

constexpr float kLevelsM = 16129.0f;       // 127^2
constexpr float kLevelsV = 4228250624.0f;  // 255^4, rounded to fp32

// The codes of one element's moments, in the last bytes: im and iv are the
// levels over the block's largest moments (0 for a block of zeros), `counter`
// the element's place in the random stream.
__device__ __forceinline__ void quantize_both(float m, float v, float im, float iv, uint32_t counter, uint32_t &cm,
                                              uint32_t &cv) {
    const uint32_t h = mix32(counter);
    const float rm = __fmul_rn(static_cast<float>(h & 0xFFFFu), 0x1p-16f);
    const float rv = __fmul_rn(static_cast<float>(h >> 16), 0x1p-16f);
    const float qm = quantize<false>(__fmul_rn(fabsf(m), im), rm);
    float qv = quantize<true>(__fmul_rn(v, iv), rv);
    if (v > 0.0f && iv > 0.0f) qv = fmaxf(qv, 1.0f);  // v stays above 0 where it was: m / sqrt(v) stays bounded
    cm = static_cast<uint32_t>(static_cast<int>(m < 0.0f ? -qm : qm)) & 0xFFu;
    cv = static_cast<uint32_t>(qv);
}

// One unit of 8 elements per lane: cnt of them exist (8 but at a tensor's end).
__device__ __forceinline__ void load8(const float *p, int cnt, float (&x)[8]) {
    if (cnt == 8) {
        const float4 a = __ldcs(reinterpret_cast<const float4 *>(p)), b = __ldcs(reinterpret_cast<const float4 *>(p) + 1);
        x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w, x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) x[j] = j < cnt ? p[j] : 0.0f;
    }
}
__device__ __forceinline__ void store8(float *p, int cnt, const float (&x)[8]) {
    if (cnt == 8) {
        __stcs(reinterpret_cast<float4 *>(p), make_float4(x[0], x[1], x[2], x[3]));
        __stcs(reinterpret_cast<float4 *>(p) + 1, make_float4(x[4], x[5], x[6], x[7]));
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (j < cnt) p[j] = x[j];
    }
}
__device__ __forceinline__ uint2 load_bytes(const uint8_t *p, int cnt) {
    if (cnt == 8) return __ldcs(reinterpret_cast<const uint2 *>(p));
    uint32_t w[2] = {0u, 0u};
#pragma unroll
    for (int j = 0; j < 8; ++j)
        if (j < cnt) w[j >> 2] |= static_cast<uint32_t>(p[j]) << (8 * (j & 3));
    return make_uint2(w[0], w[1]);
}
__device__ __forceinline__ void store_bytes(uint8_t *p, int cnt, uint2 d) {
    if (cnt == 8) {
        *reinterpret_cast<uint2 *>(p) = d;
    } else {
        const uint32_t w[2] = {d.x, d.y};
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (j < cnt) p[j] = static_cast<uint8_t>(w[j >> 2] >> (8 * (j & 3)));
    }
}
// The gradients of a whole unit. (With 8-bit moments 668 us for 243 M parameters;
// by fetch_grad and grad_values below 675, with the branches exchanged 678.)
__device__ __forceinline__ void load_grad8(const StepTensor &T, int64_t at, float (&g)[8]) {
    if (!T.grad_bf16) {
        load8(static_cast<const float *>(T.grad) + at, 8, g);
        return;
    }
    unpack_bf16(__ldcs(reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(T.grad) + at)), g);
}
// The gradients of a unit as they lie in memory, and as fp32: fetched apart, so
// that the other loads are under way before the first of them is waited for.
struct GradBits {
    uint4 a, b;
};
__device__ __forceinline__ GradBits fetch_grad(const StepTensor &T, int64_t at, int cnt) {
    GradBits x;
    x.a = x.b = make_uint4(0u, 0u, 0u, 0u);
    if (cnt == 8) {
        if (T.grad_bf16) {
            x.a = __ldcs(reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(T.grad) + at));
        } else {
            const uint4 *p = reinterpret_cast<const uint4 *>(static_cast<const float *>(T.grad) + at);
            x.a = __ldcs(p);
            x.b = __ldcs(p + 1);
        }
        return x;
    }
    uint32_t w[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) w[j] = 0u;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        if (j >= cnt) continue;
        if (T.grad_bf16)
            w[j >> 1] |= static_cast<uint32_t>(static_cast<const uint16_t *>(T.grad)[at + j]) << (16 * (j & 1));
        else
            w[j] = __float_as_uint(static_cast<const float *>(T.grad)[at + j]);
    }
    x.a = make_uint4(w[0], w[1], w[2], w[3]);
    x.b = make_uint4(w[4], w[5], w[6], w[7]);
    return x;
}
__device__ __forceinline__ void grad_values(const StepTensor &T, const GradBits &x, float (&g)[8]) {
    if (T.grad_bf16) {
        unpack_bf16(x.a, g);
    } else {
        const uint32_t w[8] = {x.a.x, x.a.y, x.a.z, x.a.w, x.b.x, x.b.y, x.b.z, x.b.w};
#pragma unroll
        for (int j = 0; j < 8; ++j) g[j] = __uint_as_float(w[j]);
    }
}
__device__ __forceinline__ void store_copy(const StepTensor &T, int64_t at, int cnt, const float (&w)[8]) {
    if (T.copy_kind == 2) {
        const float sw = *T.copy_scale;
        const uint2 q = make_uint2(cvt_quad_probed<FP8MP_E4M3>(__fmul_rn(w[0], sw), __fmul_rn(w[1], sw), __fmul_rn(w[2], sw),
                                                 __fmul_rn(w[3], sw)),
                                   cvt_quad_probed<FP8MP_E4M3>(__fmul_rn(w[4], sw), __fmul_rn(w[5], sw), __fmul_rn(w[6], sw),
                                                 __fmul_rn(w[7], sw)));
        store_bytes(static_cast<uint8_t *>(T.copy) + at, cnt, q);
    } else if (T.copy_kind == 1) {
        __nv_bfloat16 *p = static_cast<__nv_bfloat16 *>(T.copy) + at;
        if (cnt == 8) {
            uint32_t q[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const __nv_bfloat162 h = __floats2bfloat162_rn(w[2 * j], w[2 * j + 1]);
                q[j] = *reinterpret_cast<const uint32_t *>(&h);
            }
            *reinterpret_cast<uint4 *>(p) = make_uint4(q[0], q[1], q[2], q[3]);
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (j < cnt) p[j] = __float2bfloat16_rn(w[j]);
        }
    }
}

// A whole unit with 8-bit moments. Per parameter it moves 15 bytes, which
// leaves about 80 instructions at the memory's rate, and as many are needed: the
// step is bound by their issue (about 78 per parameter at 2.85 per cycle and SM:
// 243 M parameters in 669 us, 0.81 of the copy rate). The loads are plain ones,
// from L2 where the Ahead below has brought their lines (700 us without it).
// Asynchronous copies into shared memory, a unit ahead per thread or by a warp
// of its own, cost as many instructions as they gained: 718-731 us. So the
// arithmetic is done
// two lanes at a time where it can be, and the codes are made without
// conversions:
//   - a byte joins the exponent of 2^23 (a byte permute) and loses it again (an
//     add): the code as fp32; a 16-bit random number joins that of 128, whose
//     last place is 2^-16;
//   - fma.rz(root, 1 - 2^-21, 2^23) is 2^23 + c with c the code sought or one
//     below: the roots are good to 2^-22. Its last byte is the code. One below,
//     the remainder e = y - c^p reaches the cell's width d and the code always
//     steps up to the one sought; should it step once more, r (the next cell's
//     width) < e - d, then r d < e - d too (e, d and e - d are exact): a lane
//     that meets that does its eight again with quantize(). So the codes are
//     those of the definition, and where they have to be exact does not depend on
//     the root's error. (Testing e >= d alone sent nearly every warp that way
//     when the gradients are small: all moments then decay alike and y stays next
//     to c^p.)
__device__ __forceinline__ float sqrt_ftz(float x) {
    float r;
    asm("sqrt.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
__device__ __forceinline__ float rcp_ftz(float x) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
// Largest of the warp's values >= 0 (whose bits order as they do).
__device__ __forceinline__ float warp_max_bits(float x) {
    return __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(x)));
}
// 0xFF or 0 in the last two bytes for the signs of a and b.
__device__ __forceinline__ uint32_t sign_bytes(float a, float b) {
    uint32_t r;
    asm("prmt.b32 %0, %1, %2, 0xBBFB;" : "=r"(r) : "r"(__float_as_uint(a)), "r"(__float_as_uint(b)));
    return r;
}
// The last bytes of t's lanes, one more where s < e, in the last two bytes of the
// result; `again` collects in its first bit whether s < e - d anywhere (or nearly:
// s - e < -d (1 - 2^-20) is what it tests). Signs of differences stand for the
// comparisons.
__device__ __forceinline__ uint32_t stepped(uint64_t t, uint64_t s, uint64_t d, uint64_t e, uint32_t &again) {
    float t0, t1, z0, z1, x0, x1;
    f2_split(t, t0, t1);
    const uint64_t z = f2_fma(e, f2_same(-1.0f), s);
    f2_split(z, z0, z1);
    f2_split(f2_fma(d, f2_same(1.0f - 0x1p-20f), z), x0, x1);
    again |= __float_as_uint(x0) | __float_as_uint(x1);
    return __byte_perm(__float_as_uint(t0) + (__float_as_uint(z0) >> 31),
                       __float_as_uint(t1) + (__float_as_uint(z1) >> 31), 0x0040u);
}
// Byte `sel` of x, as 2^23 + byte.
__device__ __forceinline__ uint32_t byte_on_2_23(uint32_t x, uint32_t sel) {
    return __byte_perm(x, 0x4B000000u, 0x7650u | sel);
}
__device__ __forceinline__ void unit_8_bits(const StepTensor &T, int64_t at, int64_t unit, const Scalars &s,
                                            float shrink, uint32_t key, float &am) {
    const int lane = threadIdx.x & 31;
    float g[8], w[8];
    load_grad8(T, at, g);
    load8(T.w + at, 8, w);
    const uint2 cm = load_bytes(static_cast<const uint8_t *>(T.m) + at, 8);
    const uint2 cv = load_bytes(static_cast<const uint8_t *>(T.v) + at, 8);
    const uint64_t sm = f2_same(T.sm[unit]), sv = f2_same(T.sv[unit]);
    uint64_t m2[4], v2[4];
    float mmax = 0.0f, vmax = 0.0f;
#pragma unroll
    for (int p = 0; p < 4; ++p) {
        const uint32_t bm = (p < 2 ? cm.x : cm.y) ^ 0x80808080u, bv = p < 2 ? cv.x : cv.y;
        const uint32_t b0 = (2 * p) & 3, b1 = b0 + 1;
        // codes as fp32: a signed one is a byte 128 higher
        const uint64_t fm = f2_add(f2_from_bits(byte_on_2_23(bm, b0), byte_on_2_23(bm, b1)), f2_same(-8388736.0f));
        const uint64_t fv = f2_add(f2_from_bits(byte_on_2_23(bv, b0), byte_on_2_23(bv, b1)), f2_same(-8388608.0f));
        float f0, f1;
        f2_split(fm, f0, f1);
        const uint64_t sq = f2_mul(fv, fv);
        uint64_t m = f2_mul(f2_pack(__fmul_rn(f0, fabsf(f0)), __fmul_rn(f1, fabsf(f1))), sm);
        uint64_t v = f2_mul(f2_mul(sq, sq), sv);
        const uint64_t u = f2_mul(f2_pack(g[2 * p], g[2 * p + 1]), f2_same(s.coef));
        m = f2_add(f2_mul_apart(m, f2_same(s.b1)), f2_mul_apart(u, f2_same(s.c1)));
        v = f2_add(f2_mul_apart(v, f2_same(s.b2)), f2_mul_apart(f2_mul(u, u), f2_same(s.c2)));
        m2[p] = m;
        v2[p] = v;
        float m0, m1, v0, v1, d0, d1;
        f2_split(m, m0, m1);
        f2_split(v, v0, v1);
        f2_split(f2_fma(f2_pack(sqrt_ftz(v0), sqrt_ftz(v1)), f2_same(s.root), f2_same(s.eps)), d0, d1);
        const uint64_t q = f2_mul(m, f2_pack(rcp_ftz(d0), rcp_ftz(d1)));
        f2_split(f2_fma(f2_same(-s.step), q, f2_mul(f2_pack(w[2 * p], w[2 * p + 1]), f2_same(shrink))), w[2 * p],
                 w[2 * p + 1]);
        mmax = fmaxf(mmax, fmaxf(fabsf(m0), fabsf(m1)));
        vmax = fmaxf(vmax, fmaxf(v0, v1));
        am = fmaxf(am, fmaxf(fabsf(w[2 * p]), fabsf(w[2 * p + 1])));
    }
    store8(T.w + at, 8, w);
    store_copy(T, at, 8, w);
    mmax = warp_max_bits(mmax);
    vmax = warp_max_bits(vmax);
    mmax = mmax >= 0x1p-100f ? mmax : 0.0f;
    vmax = vmax >= 0x1p-90f ? vmax : 0.0f;
    // the block's four quotients in one division: lanes 0 and 1 the levels over
    // the maxima, lanes 2 and 3 the steps
    const float top = lane & 1 ? vmax : mmax, levels = lane & 1 ? kLevelsV : kLevelsM;
    float ratio = __fdiv_rn(lane & 2 ? top : levels, lane & 2 ? levels : top);
    if (lane < 2 && top == 0.0f) ratio = 0.0f;
    const float im = __shfl_sync(0xffffffffu, ratio, 0), iv = __shfl_sync(0xffffffffu, ratio, 1);
    if ((lane & ~1) == 2) (lane == 2 ? T.sm : T.sv)[unit] = ratio;
    const uint32_t base = key + static_cast<uint32_t>(at) +
                          static_cast<uint32_t>(static_cast<uint64_t>(at) >> 32) * 0x85EBCA77u;
    const uint64_t below = f2_same(1.0f - 0x1p-21f), one = f2_same(1.0f), minus = f2_same(-1.0f);
    const uint64_t on = f2_same(8388608.0f), off = f2_same(-8388608.0f);
    uint32_t om[4], ov[4];  // the codes of elements 2p and 2p + 1, in the last two bytes
    uint32_t again = 0u;    // its first bit: a step up that has to be looked at
#pragma unroll
    for (int p = 0; p < 4; ++p) {
        const uint32_t h0 = mix32(base + 2 * p), h1 = mix32(base + 2 * p + 1);
        const uint64_t rm = f2_add(f2_from_bits(__byte_perm(h0, 0x43000000u, 0x7610u),
                                                __byte_perm(h1, 0x43000000u, 0x7610u)), f2_same(-128.0f));
        const uint64_t rv = f2_add(f2_from_bits(__byte_perm(h0, 0x43000000u, 0x7632u),
                                                __byte_perm(h1, 0x43000000u, 0x7632u)), f2_same(-128.0f));
        float m0, m1, y0, y1;
        f2_split(m2[p], m0, m1);
        {  // |m|: (c + 1)^2 - c^2 = 2 c + 1
            const uint64_t y = f2_mul(f2_pack(fabsf(m0), fabsf(m1)), f2_same(im));
            f2_split(y, y0, y1);
            const uint64_t t = f2_fma_rz(f2_pack(sqrt_ftz(y0), sqrt_ftz(y1)), below, on);
            const uint64_t c = f2_add(t, off), d = f2_fma(c, f2_same(2.0f), one);
            const uint64_t e = f2_fma(f2_mul_apart(c, c), minus, y);
            om[p] = stepped(t, f2_mul_apart(rm, d), d, e, again);
        }
        {
            const uint64_t y = f2_mul(v2[p], f2_same(iv));
            f2_split(y, y0, y1);
            const uint64_t t = f2_fma_rz(f2_pack(sqrt_ftz(sqrt_ftz(y0)), sqrt_ftz(sqrt_ftz(y1))), below, on);
            const uint64_t c = f2_add(t, off), up = f2_add(c, one);
            const uint64_t q = f2_mul(c, c), lo = f2_mul_apart(q, q), q1 = f2_mul(up, up);
            const uint64_t d = f2_fma(lo, minus, f2_mul_apart(q1, q1));
            const uint64_t e = f2_fma(lo, minus, y);
            ov[p] = stepped(t, f2_mul_apart(rv, d), d, e, again);
        }
    }
    uint32_t wm[2], wv[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        // the signs of four elements, one byte each, and |c| negated where they are set
        float a0, a1, a2, a3;
        f2_split(m2[2 * h], a0, a1);
        f2_split(m2[2 * h + 1], a2, a3);
        const uint32_t neg = __byte_perm(sign_bytes(a0, a1), sign_bytes(a2, a3), 0x5410u);
        const uint32_t x = __byte_perm(om[2 * h], om[2 * h + 1], 0x5410u) ^ neg;
        wm[h] = ((x & 0x7F7F7F7Fu) + (neg & 0x01010101u)) ^ (x & 0x80808080u);
        wv[h] = __byte_perm(ov[2 * h], ov[2 * h + 1], 0x5410u);
    }
    // (x - 1) & ~x has a byte's last bit set where the first zero byte is
    const uint32_t zero = (((wv[0] - 0x01010101u) & ~wv[0]) | ((wv[1] - 0x01010101u) & ~wv[1])) & 0x80808080u;
    if (zero != 0u && iv > 0.0f) {  // the code 0 is for v = 0 alone
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            float v[2];
            f2_split(v2[j >> 1], v[0], v[1]);
            if (v[j & 1] > 0.0f && ((wv[j >> 2] >> (8 * (j & 3))) & 0xFFu) == 0u) wv[j >> 2] |= 1u << (8 * (j & 3));
        }
    }
    if (again >> 31) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            wm[h] = wv[h] = 0u;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                float m[2], v[2];
                f2_split(m2[2 * h + (j >> 1)], m[0], m[1]);
                f2_split(v2[2 * h + (j >> 1)], v[0], v[1]);
                uint32_t qm, qv;
                quantize_both(m[j & 1], v[j & 1], im, iv, base + 4 * h + j, qm, qv);
                wm[h] |= qm << (8 * j);
                wv[h] |= qv << (8 * j);
            }
        }
    }
    store_bytes(static_cast<uint8_t *>(T.m) + at, 8, make_uint2(wm[0], wm[1]));
    store_bytes(static_cast<uint8_t *>(T.v) + at, 8, make_uint2(wv[0], wv[1]));
}

// Brings a warp's next unit of a tensor from DRAM to L2 while it computes this
// one: 22 lanes ask for one 128-byte line each of gradients (lanes 0-3, or 0-7 in
// fp32), weights (8-15), codes of m (16, 17), of v (18, 19) and the two scales.
// Each lane keeps its array and the step per element from tensor to tensor;
// worked out again for each unit that cost what it gained (701 us). The last
// chunk of a tensor, which may end inside a unit, is not asked for.
struct Ahead {
    const char *base;
    int shift;  // log2 of the bytes per element; 6: one in 64, a scale; -1: none
    __device__ __forceinline__ void start(const StepTensor &T, bool any) {
        const int lane = threadIdx.x & 31;
        shift = -1;
        base = nullptr;
        if (!any || !T.codes) return;  // (many small tensors: no unit to look ahead to)
        if (lane < 8) {
            shift = T.grad_bf16 ? (lane < 4 ? 1 : -1) : 2;
            base = static_cast<const char *>(T.grad) + 128 * lane;
        } else if (lane < 16) {
            shift = 2;
            base = reinterpret_cast<const char *>(T.w) + 128 * (lane - 8);
        } else if (lane >= 20 && lane < 22) {
            shift = 6;
            base = reinterpret_cast<const char *>(lane == 20 ? T.sm : T.sv);
        } else if (lane < 20) {
            shift = 0;
            base = static_cast<const char *>(lane < 18 ? T.m : T.v) + 128 * (lane & 1);
        }
    }
    __device__ __forceinline__ void fetch(int64_t first) const {
        if (shift >= 0) asm volatile("prefetch.global.L2 [%0];" ::"l"(base + (shift == 6 ? first >> 6 : first << shift)));
    }
};

// A skipped step: the copies of the weights as they are, since their scales may
// have changed since the last ones.
template <int CAP>
__device__ __noinline__ void copies_alone(const StepBatch<CAP> &batch) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int chunks = batch.first[batch.count];
    for (int c = blockIdx.x; c < chunks; c += gridDim.x) {
        const int t = tensor_of(batch.first, batch.count, c);
        const StepTensor &T = batch.t[t];
        const int64_t at = static_cast<int64_t>(c - batch.first[t]) * kChunk + warp * kUnit + 8 * lane;
        const int64_t left = T.n - at;
        const int cnt = left >= 8 ? 8 : (left > 0 ? static_cast<int>(left) : 0);
        if (T.copy_kind == 0) continue;
        float w[8], am = 0.0f;
        load8(T.w + at, cnt, w);
        store_copy(T, at, cnt, w);
#pragma unroll
        for (int j = 0; j < 8; ++j) am = fmaxf(am, j < cnt ? fabsf(w[j]) : 0.0f);
        am = warp_max(am);
        if (lane == 0 && T.copy_amax != nullptr)
            atomicMax(reinterpret_cast<int *>(T.copy_amax), __float_as_int(am));
    }
}

// The kinds of a call's moments: all in fp32, all in 8 bits, or both. A call with
// both runs in one launch too, each warp by its tensor's kind (61 small tensors
// of both kinds, walking to a chunk's tensor: 9.4 us, 11.8 in a launch for each
// kind), a little slower for large ones (243 M parameters: 677 us with 8-bit
// moments, 669 in their own kernel; 1069 with fp32 ones, 993). With fp32 moments
// alone the step is bound by HBM: 993 us, 0.97 of the copy rate. The warp's 256
// elements of a unit are one block of the 8-bit moments, so a block's largest
// moment is a warp reduction and nothing leaves the warp.
enum Kind { kMoments32, kMoments8, kMomentsBoth };
template <int KIND, int CAP>
__global__ void __launch_bounds__(kThreads, KIND == kMoments32 ? 3 : 4)
adamw_kernel(const __grid_constant__ StepBatch<CAP> batch, const StepArgs a) {
    pdl_wait();
    pdl_launch_dependents();
    const int found = *reinterpret_cast<const volatile int32_t *>(a.found_inf) != 0;
    const Scalars s = make_scalars(a);  // (loaded beside the flag)
    if (!found) {
        const uint32_t seed = KIND == kMoments32 ? 0u : *a.seed;
        const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
        const int chunks = batch.first[batch.count];
        int t = -1;
        float am = 0.0f, shrink = 0.0f;
        uint32_t key = 0;
        Ahead ahead;
        for (int c = blockIdx.x; c < chunks; c += gridDim.x) {
            if (t < 0 || c >= batch.first[t + 1]) {
                if (t >= 0 && batch.t[t].copy_amax != nullptr) {
                    am = warp_max(am);
                    if (lane == 0) atomicMax(reinterpret_cast<int *>(batch.t[t].copy_amax), __float_as_int(am));
                }
                am = 0.0f;
                t = tensor_of(batch.first, batch.count, c);
                shrink = __fsub_rn(1.0f, __fmul_rn(s.lr, batch.t[t].decay));
                key = mix32(seed + (batch.t[t].ordinal + 1u) * 0x9E3779B9u);
                if constexpr (KIND != kMoments32)
                    ahead.start(batch.t[t], c + static_cast<int>(gridDim.x) < batch.first[t + 1] - 1);
            }
            const StepTensor &T = batch.t[t];
            const int64_t unit = static_cast<int64_t>(c - batch.first[t]) * (kThreads / 32) + warp;
            const int64_t at = unit * kUnit + 8 * lane;
            if (unit * kUnit >= T.n) continue;  // the whole warp: past the tensor's end
            const bool codes = KIND == kMoments8 || (KIND == kMomentsBoth && T.codes);
            if (codes && unit * kUnit + kUnit <= T.n) {
                if (c + static_cast<int>(gridDim.x) < batch.first[t + 1] - 1)
                    ahead.fetch(unit * kUnit + static_cast<int64_t>(gridDim.x) * kChunk);
                unit_8_bits(T, at, unit, s, shrink, key, am);
                continue;
            }
            const int64_t left = T.n - at;
            const int cnt = left >= 8 ? 8 : (left > 0 ? static_cast<int>(left) : 0);
            float g[8], w[8], m[8], v[8];
            const GradBits grad = fetch_grad(T, at, cnt);
            load8(T.w + at, cnt, w);
            if (codes) {
                grad_values(T, grad, g);
                const uint2 cm = load_bytes(static_cast<const uint8_t *>(T.m) + at, cnt);
                const uint2 cv = load_bytes(static_cast<const uint8_t *>(T.v) + at, cnt);
                const float sm = T.sm[unit], sv = T.sv[unit];
                const uint32_t bm[2] = {cm.x, cm.y}, bv[2] = {cv.x, cv.y};
                float mmax = 0.0f, vmax = 0.0f;
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const float fm = static_cast<float>(static_cast<int8_t>(bm[j >> 2] >> (8 * (j & 3))));
                    const float fv = static_cast<float>((bv[j >> 2] >> (8 * (j & 3))) & 0xFFu);
                    m[j] = __fmul_rn(__fmul_rn(fm, fabsf(fm)), sm);
                    v[j] = __fmul_rn(fourth(fv), sv);
                    moments(s, g[j], m[j], v[j]);
                    w[j] = updated(s, shrink, w[j], m[j], v[j]);
                    mmax = fmaxf(mmax, fabsf(m[j]));
                    vmax = fmaxf(vmax, v[j]);
                    am = fmaxf(am, j < cnt ? fabsf(w[j]) : 0.0f);
                }
                store8(T.w + at, cnt, w);
                store_copy(T, at, cnt, w);
                mmax = warp_max(mmax);
                vmax = warp_max(vmax);
                // a block that small is zero: its scale's reciprocal would not be finite
                mmax = mmax >= 0x1p-100f ? mmax : 0.0f;
                vmax = vmax >= 0x1p-90f ? vmax : 0.0f;
                const float im = mmax > 0.0f ? __fdiv_rn(kLevelsM, mmax) : 0.0f;
                const float iv = vmax > 0.0f ? __fdiv_rn(kLevelsV, vmax) : 0.0f;
                uint32_t om[2] = {0u, 0u}, ov[2] = {0u, 0u};
                const uint32_t base = key + static_cast<uint32_t>(at) +
                                      static_cast<uint32_t>(static_cast<uint64_t>(at) >> 32) * 0x85EBCA77u;
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    uint32_t qm, qv;
                    quantize_both(m[j], v[j], im, iv, base + j, qm, qv);
                    om[j >> 2] |= qm << (8 * (j & 3));
                    ov[j >> 2] |= qv << (8 * (j & 3));
                }
                store_bytes(static_cast<uint8_t *>(T.m) + at, cnt, make_uint2(om[0], om[1]));
                store_bytes(static_cast<uint8_t *>(T.v) + at, cnt, make_uint2(ov[0], ov[1]));
                if (lane == 0) {
                    T.sm[unit] = __fdiv_rn(mmax, kLevelsM);
                    T.sv[unit] = __fdiv_rn(vmax, kLevelsV);
                }
            } else {
                load8(static_cast<const float *>(T.m) + at, cnt, m);
                load8(static_cast<const float *>(T.v) + at, cnt, v);
                grad_values(T, grad, g);
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    moments(s, g[j], m[j], v[j]);
                    w[j] = updated(s, shrink, w[j], m[j], v[j]);
                    am = fmaxf(am, j < cnt ? fabsf(w[j]) : 0.0f);
                }
                store8(static_cast<float *>(T.m) + at, cnt, m);
                store8(static_cast<float *>(T.v) + at, cnt, v);
                store8(T.w + at, cnt, w);
                store_copy(T, at, cnt, w);
            }
        }
        if (t >= 0 && batch.t[t].copy_amax != nullptr) {
            am = warp_max(am);
            if (lane == 0) atomicMax(reinterpret_cast<int *>(batch.t[t].copy_amax), __float_as_int(am));
        }
    } else {
        copies_alone(batch);
    }
    if (!a.finish) return;
    // the last block of the call's last launch: every element has read the
    // scalars, so they may change
    __syncthreads();
    if (threadIdx.x == 0) {
        __threadfence();
        if (atomicAdd(&a.ws->arrivals, 1u) == gridDim.x - 1) {
            __threadfence();
            a.ws->arrivals = 0u;
            if (found) {
                *a.loss_scale = __fmul_rn(*a.loss_scale, a.backoff);
                *a.growth = 0;
            } else {
                int32_t gr = *a.growth + 1;
                if (gr >= a.interval) {
                    *a.loss_scale = __fmul_rn(*a.loss_scale, a.growth_factor);
                    gr = 0;
                }
                *a.growth = gr;
                a.beta_pows[0] = __fmul_rn(a.beta_pows[0], a.b1);
                a.beta_pows[1] = __fmul_rn(a.beta_pows[1], a.b2);
                if (a.seed != nullptr) *a.seed += 1u;
            }
        }
    }
}

// Tensors of one launch: as many as its parameters (at most 32,764 bytes)
// hold, or few where few are left, for a launch with more parameters costs more.
constexpr int kNormCapLarge = 1000, kNormCapSmall = 64;
constexpr int kStepCapLarge = 280, kStepCapSmall = 64;
static_assert(sizeof(NormBatch<kNormCapLarge>) + 64 <= 32764, "kernel parameters");
static_assert(sizeof(StepBatch<kStepCapLarge>) + sizeof(StepArgs) <= 32764, "kernel parameters");

template <int CAP>
cudaError_t launch_norm_batch(const fp8mp_adamw_tensor *t, int32_t n, Workspace *ws, float *norm, int32_t *found,
                              int finish, cudaStream_t s, const DeviceInfo &dev) {
    NormBatch<CAP> b;
    b.count = 0;
    int64_t chunks = 0;
    b.first[0] = 0;
    for (int32_t i = 0; i < n; ++i) {
        if (t[i].n == 0) continue;
        b.t[b.count] = NormTensor{t[i].grad, t[i].n, t[i].grad_dtype == FP8MP_BF16};
        chunks += (t[i].n + kNormChunk - 1) / kNormChunk;
        b.first[++b.count] = static_cast<int32_t>(chunks);
    }
    int64_t blocks = static_cast<int64_t>(dev.num_sms) * kNormBlocksPerSm;
    if (blocks > kMaxNormBlocks) blocks = kMaxNormBlocks;
    if (blocks > chunks) blocks = chunks < 1 ? 1 : chunks;
    return launch_kernel(grad_norm_kernel<CAP>, dim3(static_cast<unsigned>(blocks)), dim3(kThreads), 0, s, b, ws, norm,
                         found, finish);
}

template <int KIND, int CAP>
cudaError_t launch_step_batch(const fp8mp_adamw_tensor *t, const int32_t *which, int32_t n, const StepArgs &a,
                              cudaStream_t s, const DeviceInfo &dev) {
    StepBatch<CAP> b;
    b.count = n;
    int64_t chunks = 0;
    b.first[0] = 0;
    for (int32_t i = 0; i < n; ++i) {
        const fp8mp_adamw_tensor &T = t[which[i]];
        b.t[i] = StepTensor{T.grad, T.master, T.exp_avg, T.exp_avg_sq, T.exp_avg_scale, T.exp_avg_sq_scale, T.copy,
                            T.copy_scale, T.copy_amax, T.n, T.weight_decay, static_cast<uint32_t>(which[i]),
                            static_cast<int8_t>(T.grad_dtype == FP8MP_BF16),
                            static_cast<int8_t>(T.copy == nullptr ? 0 : (T.copy_scale == nullptr ? 1 : 2)),
                            static_cast<int8_t>(T.state_bits == 8)};
        chunks += (T.n + kChunk - 1) / kChunk;
        b.first[i + 1] = static_cast<int32_t>(chunks);
    }
    int64_t blocks = static_cast<int64_t>(dev.num_sms) * (KIND == kMoments32 ? kStepBlocksPerSm32 : kStepBlocksPerSm8);
    if (blocks > chunks) blocks = chunks < 1 ? 1 : chunks;
    return launch_kernel(adamw_kernel<KIND, CAP>, dim3(static_cast<unsigned>(blocks)), dim3(kThreads), 0, s, b, a);
}

template <int KIND>
cudaError_t launch_step(const fp8mp_adamw_tensor *t, const int32_t *which, int32_t n, const StepArgs &a,
                        cudaStream_t s, const DeviceInfo &dev) {
    return n <= kStepCapSmall ? launch_step_batch<KIND, kStepCapSmall>(t, which, n, a, s, dev)
                              : launch_step_batch<KIND, kStepCapLarge>(t, which, n, a, s, dev);
}

}  // namespace

int64_t adamw_workspace_bytes() { return (static_cast<int64_t>(sizeof(Workspace)) + 15) & ~static_cast<int64_t>(15); }

int64_t adamw_max_elements() { return static_cast<int64_t>(kChunk) << 30; }

int launch_grad_norm(const fp8mp_adamw_tensor *t, int32_t n, float *norm, int32_t *found_inf, void *workspace,
                     cudaStream_t s, const DeviceInfo &dev) {
    Workspace *ws = static_cast<Workspace *>(workspace);
    int32_t at = 0;
    do {
        const int32_t cnt = n - at < kNormCapLarge ? n - at : kNormCapLarge;
        const int finish = at + cnt == n;
        const cudaError_t e =
            cnt <= kNormCapSmall
                ? launch_norm_batch<kNormCapSmall>(t + at, cnt, ws, norm, found_inf, finish, s, dev)
                : launch_norm_batch<kNormCapLarge>(t + at, cnt, ws, norm, found_inf, finish, s, dev);
        if (e != cudaSuccess)
            return fail(FP8MP_ERR_LAUNCH, "mp_grad_norm: launch failed: %s", cudaGetErrorString(e));
        at += cnt;
    } while (at < n);
    return FP8MP_OK;
}

int launch_adamw_step(const fp8mp_adamw_tensor *t, int32_t n, const AdamwArgs &args, cudaStream_t s,
                      const DeviceInfo &dev) {
    StepArgs a = {args.loss_scale, args.growth, args.found_inf, args.beta_pows, args.seed, args.grad_norm,
                  args.max_norm, args.lr, args.b1, args.b2, args.eps, args.backoff, args.growth_factor, args.interval,
                  0, static_cast<Workspace *>(args.workspace)};
    bool codes = false, wide = false;
    for (int32_t i = 0; i < n; ++i)
        if (t[i].n > 0) (t[i].state_bits == 8 ? codes : wide) = true;
    const auto launch = !codes ? launch_step<kMoments32> : (wide ? launch_step<kMomentsBoth> : launch_step<kMoments8>);
    int32_t at = 0;
    do {  // (a step of nothing still counts: one launch at least)
        int32_t which[kStepCapLarge], cnt = 0;
        for (; at < n && cnt < kStepCapLarge; ++at)
            if (t[at].n > 0) which[cnt++] = at;
        while (at < n && t[at].n == 0) ++at;
        a.finish = at == n;
        const cudaError_t e = launch(t, which, cnt, a, s, dev);
        if (e != cudaSuccess)
            return fail(FP8MP_ERR_LAUNCH, "mp_adamw_step: launch failed: %s", cudaGetErrorString(e));
    } while (at < n);
    return FP8MP_OK;
}

}  // namespace fp8mp
