// embed.cu -- rows of an embedding table, scaled, and the table's gradient.
//
// Forward: out[m] = table[id_m] (scale sinv), a gather bound by HBM: the rows that
// the tokens name and the output, once each.
//
// Backward: dtable[v] = scale (sum over the m with id_m = v of dy[m]), for every v: the
// whole table is written, zeros mostly, which is what bounds it. The tokens are sorted
// first, by (id, position), so that each row's sum has one order and no atomics:
//   1. sort: a stable radix sort of 9 bits a pass by one cluster of 8 CTAs. A warp
//      owns a run of consecutive positions and a histogram of its own; counts are
//      joined over the warps in shared memory and over the CTAs through distributed
//      shared memory. It also marks the ids that occur in a bitmap.
//   2. sum: the sorted tokens in chunks of equal length, whatever their ids, so that
//      an id that half of the batch holds is no one's long tail: a thread adds eight
//      columns over a chunk in fp32 and writes a row where its id's run lies within the
//      chunk, else a partial sum. The rows of ids that do not occur are zeroed.
//   3. join: the partial sums of each run over several chunks, in their order.
// Ids outside 0 .. V - 1 sort last and have no row.
#include "fp8mp_async.cuh"
#include "fp8mp_pieces.cuh"

namespace fp8mp {

namespace {

constexpr int kThreads = 256;
constexpr int kSortCtas = 8, kSortThreads = 512, kSortWarps = kSortThreads / 32;
constexpr int kDigitBits = 9, kBins = 1 << kDigitBits;
constexpr int kBatch = 8;           // keys that a lane has in flight
constexpr int kMinChunk = 16;       // tokens of a chunk, at least
constexpr int kMaxChunks = 1024;
constexpr int kZeroRows = 8;        // rows that a block zeroes at a time
static_assert(kBins == kSortThreads, "a thread for each bin");

// ----------------------------------------------------------------- forward

struct EmbedArgs {
    const int64_t *ids;
    const uint8_t *table;
    const float *sinv;
    void *out;
    int64_t M, V;
    int units;  // of 16 columns
    float scale;
    bool out_bf16;
};

__device__ __forceinline__ void e4m3_pairs(uint32_t codes, uint64_t &lo, uint64_t &hi) {
    uint32_t h0, h1;
    asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
        : "=r"(h0), "=r"(h1)
        : "r"(codes));
    const auto wide = [](uint32_t h) {
        float a, b;
        asm("{\n\t.reg .b16 x, y;\n\tmov.b32 {x, y}, %2;\n\tcvt.f32.f16 %0, x;\n\tcvt.f32.f16 %1, y;\n\t}"
            : "=f"(a), "=f"(b)
            : "r"(h));
        return f2_pack(a, b);
    };
    lo = wide(h0);
    hi = wide(h1);
}

// TABLE: 0 E4M3, 1 bf16, 2 fp32. A thread moves 16 columns of a row.
template <int TABLE>
__global__ void __launch_bounds__(kThreads) embed_fwd_kernel(const EmbedArgs a) {
    pdl_wait();
    pdl_launch_dependents();
    const float factor = TABLE == 0 ? __ldg(a.sinv) * a.scale : a.scale;
    const uint64_t f2 = f2_same(factor);
    const int64_t items = a.M * a.units, step = static_cast<int64_t>(gridDim.x) * kThreads;
    for (int64_t it = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x; it < items; it += step) {
        const int64_t m = it / a.units;
        const int64_t unit = it - m * a.units;
        const int64_t id = __ldg(a.ids + m);
        uint64_t v[2][4] = {};
        if (id >= 0 && id < a.V) {
            const int64_t at = id * a.units + unit;
            if constexpr (TABLE == 0) {
                const uint4 q = __ldg(reinterpret_cast<const uint4 *>(a.table) + at);
                e4m3_pairs(q.x, v[0][0], v[0][1]);
                e4m3_pairs(q.y, v[0][2], v[0][3]);
                e4m3_pairs(q.z, v[1][0], v[1][1]);
                e4m3_pairs(q.w, v[1][2], v[1][3]);
            } else {
                const Piece<TABLE == 1> p = load_piece<TABLE == 1>(a.table, 2 * at), r = load_piece<TABLE == 1>(a.table, 2 * at + 1);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    v[0][j] = p.pair(j);
                    v[1][j] = r.pair(j);
                }
            }
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int j = 0; j < 4; ++j) v[h][j] = f2_mul(v[h][j], f2);
        }
        store_rounded(a.out, 2 * it, v[0], a.out_bf16);
        store_rounded(a.out, 2 * it + 1, v[1], a.out_bf16);
    }
}

// -------------------------------------------------------------------- sort

struct SortArgs {
    const int64_t *ids;
    uint32_t *key[2], *pos[2];
    uint32_t *bitmap;
    int64_t M, V;
    int passes;
};

__device__ __forceinline__ uint32_t ld_cluster_u32(uint32_t addr) {
    uint32_t v;
    asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
    return v;
}

// Sorted keys and positions end up in key[passes & 1], pos[passes & 1].
__global__ void __launch_bounds__(kSortThreads, 1) embed_sort_kernel(const SortArgs a) {
    __shared__ uint32_t hist[kSortWarps][kBins];  // a warp's counts, then where its next key of a bin goes
    __shared__ uint32_t total[kBins];             // the CTA's counts
    __shared__ uint32_t scan[kSortWarps];
    pdl_wait();
    pdl_launch_dependents();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const uint32_t rank = cluster_ctarank();
    const uint32_t none = static_cast<uint32_t>(a.V);
    // a warp's run of positions
    const int64_t run = ((a.M + kSortCtas * kSortWarps - 1) / (kSortCtas * kSortWarps) + 31) / 32 * 32;
    const int64_t first = (rank * kSortWarps + warp) * run;
    const int64_t last = first + run < a.M ? first + run : a.M;
    const int64_t words = (a.V + 31) / 32;
    for (int64_t i = rank * kSortThreads + tid; i < words; i += kSortCtas * kSortThreads) a.bitmap[i] = 0u;
    for (int pass = 0; pass < a.passes; ++pass) {
        const int shift = pass * kDigitBits;
        const uint32_t *key_in = a.key[pass & 1], *pos_in = a.pos[pass & 1];
        uint32_t *key_out = a.key[~pass & 1], *pos_out = a.pos[~pass & 1];
        const auto key_at = [&](int64_t i) {
            if (pass > 0) return __ldcg(key_in + i);
            const int64_t id = __ldg(a.ids + i);
            return id >= 0 && id < a.V ? static_cast<uint32_t>(id) : none;
        };
        for (int w = 0; w < kSortWarps; ++w) hist[w][tid] = 0u;
        __syncthreads();
        for (int64_t i = first; i < last; i += 32 * kBatch) {
            uint32_t k[kBatch];
#pragma unroll
            for (int j = 0; j < kBatch; ++j)
                if (i + j * 32 + lane < last) k[j] = key_at(i + j * 32 + lane);
#pragma unroll
            for (int j = 0; j < kBatch; ++j)
                if (i + j * 32 + lane < last) atomicAdd(&hist[warp][k[j] >> shift & (kBins - 1)], 1u);
        }
        __syncthreads();
        uint32_t sum = 0;
        for (int w = 0; w < kSortWarps; ++w) {
            const uint32_t c = hist[w][tid];
            hist[w][tid] = sum;
            sum += c;
        }
        total[tid] = sum;
        cluster_sync_all();
        uint32_t before = 0, all = 0;
#pragma unroll
        for (uint32_t r = 0; r < kSortCtas; ++r) {
            const uint32_t c = ld_cluster_u32(mapa_shared(smem_u32(&total[tid]), r));
            if (r < rank) before += c;
            all += c;
        }
        uint32_t upto = all;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const uint32_t v = __shfl_up_sync(0xffffffffu, upto, o);
            if (lane >= o) upto += v;
        }
        if (lane == 31) scan[warp] = upto;
        __syncthreads();
        uint32_t base = before + upto - all;
        for (int w = 0; w < warp; ++w) base += scan[w];
        for (int w = 0; w < kSortWarps; ++w) hist[w][tid] += base;
        __syncthreads();
        for (int64_t i = first; i < last; i += 32 * kBatch) {
            uint32_t k[kBatch], p[kBatch];
#pragma unroll
            for (int j = 0; j < kBatch; ++j) {
                const int64_t at = i + j * 32 + lane;
                if (at < last) {
                    k[j] = key_at(at);
                    p[j] = pass > 0 ? __ldcg(pos_in + at) : static_cast<uint32_t>(at);
                }
            }
#pragma unroll
            for (int j = 0; j < kBatch; ++j) {
                const bool in = i + j * 32 + lane < last;
                const uint32_t digit = in ? k[j] >> shift & (kBins - 1) : kBins;
                const uint32_t peers = __match_any_sync(0xffffffffu, digit);
                uint32_t to = 0;
                if (in) to = hist[warp][digit] + __popc(peers & ((1u << lane) - 1u));
                __syncwarp();
                if (in && lane == __ffs(peers) - 1) hist[warp][digit] += __popc(peers);
                __syncwarp();
                if (in) {
                    key_out[to] = k[j];
                    pos_out[to] = p[j];
                    if (pass == 0 && k[j] < none) atomicOr(a.bitmap + (k[j] >> 5), 1u << (k[j] & 31));
                }
            }
        }
        cluster_sync_all();  // the arrays are whole, and everyone has read `total`
    }
}

// --------------------------------------------------------------------- sum

struct SumArgs {
    const void *dy;
    const uint32_t *key, *pos, *bitmap;
    void *out;
    float *partial;  // [chunks][2][K]: of a run from before the chunk, of a run past its end
    int64_t M, V;
    int64_t chunk;
    int chunks, pieces;
    float scale;
    bool out_bf16;
};

__device__ __forceinline__ void write_row(const SumArgs &a, uint32_t v, int piece, const uint64_t (&sum)[4]) {
    uint64_t r[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) r[j] = f2_mul(sum[j], f2_same(a.scale));
    store_rounded(a.out, static_cast<int64_t>(v) * a.pieces + piece, r, a.out_bf16);
}

template <bool BF16>
__global__ void __launch_bounds__(kThreads) embed_sum_kernel(const SumArgs a) {
    pdl_wait();
    pdl_launch_dependents();
    const uint32_t none = static_cast<uint32_t>(a.V);
    const int64_t items = static_cast<int64_t>(a.chunks) * a.pieces, step = static_cast<int64_t>(gridDim.x) * kThreads;
    for (int64_t it = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x; it < items; it += step) {
        const int c = static_cast<int>(it / a.pieces), piece = static_cast<int>(it - static_cast<int64_t>(c) * a.pieces);
        const int64_t i0 = c * a.chunk, i1 = i0 + a.chunk < a.M ? i0 + a.chunk : a.M;
        uint32_t now = __ldg(a.key + i0);
        bool whole = i0 == 0 || __ldg(a.key + i0 - 1) != now;  // the run starts in this chunk
        uint64_t sum[4] = {0ull, 0ull, 0ull, 0ull};
        constexpr int kAhead = 4;
        for (int64_t i = i0; i < i1 && now != none; i += kAhead) {
            uint32_t key[kAhead];
            Piece<BF16> d[kAhead];
#pragma unroll
            for (int j = 0; j < kAhead; ++j) {
                key[j] = i + j < i1 ? __ldg(a.key + i + j) : none;
                if (key[j] != none) d[j] = load_piece<BF16>(a.dy, static_cast<int64_t>(__ldg(a.pos + i + j)) * a.pieces + piece);
            }
#pragma unroll
            for (int j = 0; j < kAhead; ++j) {
                if (i + j >= i1) break;
                if (key[j] != now) {
                    if (whole) write_row(a, now, piece, sum);
                    else store_piece<false>(a.partial, 2ll * c * a.pieces + piece, round_piece<false>(sum));
                    now = key[j];
                    whole = true;
#pragma unroll
                    for (int q = 0; q < 4; ++q) sum[q] = 0ull;
                }
                if (now == none) break;
#pragma unroll
                for (int q = 0; q < 4; ++q) sum[q] = f2_add(sum[q], d[j].pair(q));
            }
        }
        if (now != none) {
            const bool ends = i1 == a.M || __ldg(a.key + i1) != now;
            if (whole && ends) write_row(a, now, piece, sum);
            else store_piece<false>(a.partial, (2ll * c + (whole ? 1 : 0)) * a.pieces + piece, round_piece<false>(sum));
        }
    }
    // the rows of ids that do not occur
    const int across = a.pieces < kThreads ? a.pieces : kThreads, down = kThreads / across;
    const int r0 = threadIdx.x / across, p0 = threadIdx.x - r0 * across;
    if (r0 >= down) return;
    const uint64_t zero[4] = {0ull, 0ull, 0ull, 0ull};
    const int64_t groups = (a.V + kZeroRows - 1) / kZeroRows;
    for (int64_t g = blockIdx.x; g < groups; g += gridDim.x) {
        const uint32_t bits = __ldg(a.bitmap + g * kZeroRows / 32) >> (g * kZeroRows & 31);
        for (int r = r0; r < kZeroRows; r += down) {
            const int64_t v = g * kZeroRows + r;
            if (v >= a.V || bits >> r & 1u) continue;
            for (int p = p0; p < a.pieces; p += across) store_rounded(a.out, v * a.pieces + p, zero, a.out_bf16);
        }
    }
}

// -------------------------------------------------------------------- join

__global__ void __launch_bounds__(kThreads) embed_join_kernel(const SumArgs a) {
    pdl_wait();
    pdl_launch_dependents();
    const uint32_t none = static_cast<uint32_t>(a.V);
    const int64_t it = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x;
    if (it >= static_cast<int64_t>(a.chunks) * a.pieces) return;
    const int c = static_cast<int>(it / a.pieces), piece = static_cast<int>(it - static_cast<int64_t>(c) * a.pieces);
    // the run that the chunk ends in, if it starts in it and goes on
    const int64_t end = (c + 1) * a.chunk;
    if (end >= a.M) return;
    const uint32_t v = __ldg(a.key + end - 1);
    if (v == none || __ldg(a.key + end) != v) return;
    const int64_t begin = c * a.chunk;
    if (__ldg(a.key + begin) == v && begin > 0 && __ldg(a.key + begin - 1) == v) return;
    uint64_t sum[4] = {0ull, 0ull, 0ull, 0ull};
    int64_t row = 2ll * c + 1;
    for (int next = c + 1;; ++next) {
        const float4 *p = reinterpret_cast<const float4 *>(a.partial) + 2 * (row * a.pieces + piece);
        const float4 x = __ldcg(p), y = __ldcg(p + 1);
        sum[0] = f2_add(sum[0], f2_pack(x.x, x.y));
        sum[1] = f2_add(sum[1], f2_pack(x.z, x.w));
        sum[2] = f2_add(sum[2], f2_pack(y.x, y.y));
        sum[3] = f2_add(sum[3], f2_pack(y.z, y.w));
        if (next >= a.chunks || __ldg(a.key + next * a.chunk) != v) break;
        row = 2ll * next;
    }
    write_row(a, v, piece, sum);
}

// The workspace: keys and positions, each twice; the bitmap; the partial sums.
struct Layout {
    int64_t chunk, chunks, bitmap, partial, bytes;
};
int64_t round16(int64_t n) { return (n + 15) / 16 * 16; }
Layout layout_of(int64_t M, int64_t V, int64_t K) {
    Layout l;
    l.chunk = (M + kMaxChunks - 1) / kMaxChunks;
    if (l.chunk < kMinChunk) l.chunk = kMinChunk;
    l.chunks = (M + l.chunk - 1) / l.chunk;
    l.bitmap = 4 * round16(4 * M);
    l.partial = l.bitmap + round16((V + 31) / 32 * 4);
    l.bytes = l.partial + 2 * l.chunks * K * 4;
    return l;
}

}  // namespace

int64_t embedding_workspace_bytes(int64_t M, int64_t V, int64_t K) { return layout_of(M, V, K).bytes; }

int launch_embedding_fwd(const int64_t *ids, int64_t M, const void *table, int table_kind, int64_t V, int64_t K,
                         const float *sinv, float scale, void *out, int out_dtype, cudaStream_t s, const DeviceInfo &dev) {
    const EmbedArgs a = {ids, static_cast<const uint8_t *>(table), sinv, out, M, V, static_cast<int>(K / 16), scale,
                         out_dtype == FP8MP_BF16};
    const int64_t need = (M * a.units + kThreads - 1) / kThreads, most = 32ll * dev.num_sms;
    const dim3 grid(static_cast<unsigned>(need < most ? need : most)), block(kThreads);
    cudaError_t e;
    if (table_kind == 0) e = launch_kernel(embed_fwd_kernel<0>, grid, block, 0, s, a);
    else if (table_kind == 1) e = launch_kernel(embed_fwd_kernel<1>, grid, block, 0, s, a);
    else e = launch_kernel(embed_fwd_kernel<2>, grid, block, 0, s, a);
    if (e != cudaSuccess) return fail(FP8MP_ERR_LAUNCH, "embedding: launch failed: %s", cudaGetErrorString(e));
    return FP8MP_OK;
}

int launch_embedding_bwd(const int64_t *ids, int64_t M, const void *dy, int dy_dtype, int64_t V, int64_t K, float scale,
                         void *dtable, int out_dtype, void *workspace, cudaStream_t s, const DeviceInfo &dev) {
    const Layout l = layout_of(M, V, K);
    uint8_t *ws = static_cast<uint8_t *>(workspace);
    SortArgs so = {};
    so.ids = ids;
    const int64_t each = round16(4 * M);
    for (int i = 0; i < 2; ++i) {
        so.key[i] = reinterpret_cast<uint32_t *>(ws + i * each);
        so.pos[i] = reinterpret_cast<uint32_t *>(ws + (2 + i) * each);
    }
    so.bitmap = reinterpret_cast<uint32_t *>(ws + l.bitmap);
    so.M = M;
    so.V = V;
    so.passes = 1;  // keys are 0 .. V
    while (V >> (so.passes * kDigitBits) != 0) ++so.passes;
    cudaError_t e = launch_kernel_cluster(embed_sort_kernel, dim3(kSortCtas), dim3(kSortThreads), 0, s, kSortCtas, so);
    SumArgs a = {};
    a.dy = dy;
    a.key = so.key[so.passes & 1];
    a.pos = so.pos[so.passes & 1];
    a.bitmap = so.bitmap;
    a.out = dtable;
    a.partial = reinterpret_cast<float *>(ws + l.partial);
    a.M = M;
    a.V = V;
    a.chunk = l.chunk;
    a.chunks = static_cast<int>(l.chunks);
    a.pieces = static_cast<int>(K / kPiece);
    a.scale = scale;
    a.out_bf16 = out_dtype == FP8MP_BF16;
    const int64_t items = l.chunks * a.pieces, groups = (V + kZeroRows - 1) / kZeroRows;
    const int64_t blocks = (items + kThreads - 1) / kThreads, need = blocks > groups ? blocks : groups, most = 4ll * dev.num_sms;
    const dim3 grid(static_cast<unsigned>(need < most ? need : most)), block(kThreads);
    if (e == cudaSuccess)
        e = dy_dtype == FP8MP_BF16 ? launch_kernel(embed_sum_kernel<true>, grid, block, 0, s, a)
                                   : launch_kernel(embed_sum_kernel<false>, grid, block, 0, s, a);
    if (e == cudaSuccess && l.chunks > 1)
        e = launch_kernel(embed_join_kernel, dim3(static_cast<unsigned>(blocks)), block, 0, s, a);
    if (e != cudaSuccess) return fail(FP8MP_ERR_LAUNCH, "embedding: launch failed: %s", cudaGetErrorString(e));
    return FP8MP_OK;
}

}  // namespace fp8mp
