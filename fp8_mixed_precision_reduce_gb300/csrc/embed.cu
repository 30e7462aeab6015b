// embed.cu -- rows of an embedding table, scaled, and the table's gradient.
//
// Forward: out[m] = table[id_m] (scale sinv), a gather bound by HBM: the rows that
// the tokens name and the output, once each. 16384 tokens of 4096 columns from an E4M3
// table to bf16: 28 us, the output alone 21 at the rate that stores reach (6.5 TB/s).
//
// Backward: dtable[v] = scale (sum over the m with id_m = v of dy[m]), for every v: the
// whole table is written, zeros mostly, which is what bounds it. The tokens are sorted
// first, by (id, position), so that each row's sum has one order and no atomics:
//   1. sort. Up to 4096 tokens: every block counts, for its share of the tokens, the
//      smaller keys and the equal ones before it (4096^2 comparisons are 1.5 us of the
//      device). More: a stable radix sort, in which a warp owns a run of consecutive
//      positions and a histogram of its own; up to 32768 by a cluster of 8 CTAs, whose
//      counts and words of id and position go through distributed shared memory (16384
//      tokens and 50000 x 768: 42.5 us in all); more, or with ids too large for that, by
//      a cluster through global memory.
//   2. zero: every block looks through the ids for those among its rows and zeroes the
//      others. It runs beside the counting, or a sort in shared memory (one through global
//      memory takes 4 times as long beside it, and does not).
//   3. sum: the sorted tokens in chunks of equal length, whatever their ids, so that
//      an id that half of the batch holds is no one's long tail: a thread adds eight
//      columns over a chunk in fp32 and writes a row where its id's run lies within the
//      chunk, else a partial sum.
//   4. join: the partial sums of each run over several chunks, in their order.
// Ids outside 0 .. V - 1 sort last and have no row.
// Few tokens and short rows (128 and 1024 columns at most) take one launch instead, which
// finds equal ids by votes: it saves two launches and, where one id is nearly all of them,
// loses some of it to that row's sum. fp32, 77 tokens, 1000 x 272: 3.8 us, 7.3 in steps, one
// id throughout 8.2 and 8.9; 128 tokens, 8000 x 1024: 9.7 and 11.9, one id 18.4 and 15.2.
// 16384 tokens, 128000 x 4096 in bf16: 194 us, of which the zeros 152 (6.5 TB/s) and the
// sum 29. Where the sort goes through global memory: 65536 tokens, 50000 x 768 95 us; 32768 tokens,
// 151936 x 2048 152 (128000 x 2048, whose ids still fit beside the position, 129).
#include <atomic>

#include "fp8mp_async.cuh"
#include "fp8mp_lm.cuh"
#include "fp8mp_pieces.cuh"

namespace fp8mp {

namespace {

constexpr int kThreads = 256;
constexpr int kSortCtas = 8, kSortThreads = 512, kSortWarps = kSortThreads / 32;
constexpr int kZeroThreads = 512, kZeroBatch = 8;
constexpr int kDigitBits = 9, kBins = 1 << kDigitBits;
constexpr int kBatch = 8;           // keys that a lane has in flight
constexpr int kFewMost = 128, kFewPieces = 128;  // tokens, and pieces of a row, whose gradient takes one launch
constexpr int kMinChunk = 4;        // tokens of a chunk, at least
constexpr int64_t kSumItems = 1024 * 152;  // chunks times pieces of a row, about, where the chunks are longer
constexpr int64_t kWindow = 32 * 4096;  // rows whose marks a block of the zeroing holds at a time
static_assert(kBins == kSortThreads, "a thread for each bin");

// ----------------------------------------------------------------- forward

struct EmbedArgs {
    const int64_t *ids;
    const uint8_t *table;
    const float *sinv;
    void *out;
    int64_t M, V;
    int units;  // 16-byte units of an output row
    float scale;
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

// TABLE: 0 E4M3, 1 bf16, 2 fp32. A thread writes 16 bytes (8 bf16 or 4 fp32 columns, so that
// a warp's store covers whole lines) of each of kRows rows at a time, whose ids and then
// whose columns are in flight together; blockDim.x threads or fewer take a row.
constexpr int kRows = 4;

template <int BYTES>
__device__ __forceinline__ void load_words(uint32_t (&w)[BYTES / 4], const uint8_t *p) {
    if constexpr (BYTES == 4) {
        w[0] = __ldg(reinterpret_cast<const uint32_t *>(p));
    } else if constexpr (BYTES == 8) {
        const uint2 v = __ldg(reinterpret_cast<const uint2 *>(p));
        w[0] = v.x;
        w[1] = v.y;
    } else {
#pragma unroll
        for (int j = 0; j < BYTES / 16; ++j) {
            const uint4 v = __ldg(reinterpret_cast<const uint4 *>(p) + j);
            w[4 * j] = v.x;
            w[4 * j + 1] = v.y;
            w[4 * j + 2] = v.z;
            w[4 * j + 3] = v.w;
        }
    }
}

template <int TABLE, bool OBF>
__global__ void __launch_bounds__(kThreads) embed_fwd_kernel(const EmbedArgs a) {
    constexpr int COLS = OBF ? 8 : 4, BYTES = COLS * (TABLE == 0 ? 1 : TABLE == 1 ? 2 : 4);
    pdl_wait();
    pdl_launch_dependents();
    const float factor = TABLE == 0 ? __ldg(a.sinv) * a.scale : a.scale;
    const int across = a.units < kThreads ? a.units : kThreads, down = kThreads / across;
    const int r0 = threadIdx.x / across, p0 = threadIdx.x - r0 * across;
    if (r0 >= down) return;
    const int64_t m0 = static_cast<int64_t>(blockIdx.x) * (down * kRows) + r0;
    int64_t id[kRows];  // -1: no row
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
        id[r] = m0 + r * down < a.M ? __ldg(a.ids + m0 + r * down) : -1;
        if (id[r] >= a.V) id[r] = -1;
    }
    for (int p = p0; p < a.units; p += across) {
        uint32_t q[kRows][BYTES / 4];
#pragma unroll
        for (int r = 0; r < kRows; ++r)
            if (id[r] >= 0) load_words<BYTES>(q[r], a.table + (id[r] * a.units + p) * BYTES);
#pragma unroll
        for (int r = 0; r < kRows; ++r) {
            if (m0 + r * down >= a.M) break;
            uint32_t o[4] = {0u, 0u, 0u, 0u};
            if (id[r] >= 0) {
                uint64_t v[COLS / 2];
#pragma unroll
                for (int j = 0; j < COLS / 2; ++j) {
                    if constexpr (TABLE == 0) {
                        if ((j & 1) == 0) e4m3_pairs(q[r][j / 2], v[j], v[j + 1]);
                    } else if constexpr (TABLE == 1) {
                        v[j] = f2_from_bits(q[r][j] << 16, q[r][j] & 0xFFFF0000u);
                    } else {
                        v[j] = f2_from_bits(q[r][2 * j], q[r][2 * j + 1]);
                    }
                }
#pragma unroll
                for (int j = 0; j < COLS / 2; ++j) {
                    float lo, hi;
                    f2_split(f2_mul(v[j], f2_same(factor)), lo, hi);
                    if constexpr (OBF) {
                        o[j] = bf16_pair(lo, hi);
                    } else {
                        o[2 * j] = __float_as_uint(lo);
                        o[2 * j + 1] = __float_as_uint(hi);
                    }
                }
            }
            reinterpret_cast<uint4 *>(a.out)[(m0 + r * down) * a.units + p] = make_uint4(o[0], o[1], o[2], o[3]);
        }
    }
}

// -------------------------------------------------------------------- sort

struct SortArgs {
    const int64_t *ids;
    uint32_t *key[2], *pos[2];
    int64_t M, V;
    int passes;
};

struct ZeroArgs {
    const int64_t *ids;
    uint4 *table;  // the gradient
    int64_t M, V;
    int row;       // 16-byte units of a row of it
};

// Block `part` of `parts`, of THREADS threads, zeroes the rows of its share of the table
// but for those whose ids occur: it marks them in shared memory, kWindow rows at a time.
// `tokens(f)`: f of each id, from one thread. The first ZEROS threads zero, while the
// others run `beside`, once.
template <int THREADS, int ZEROS, typename F, typename G>
__device__ __forceinline__ void zero_rows(const ZeroArgs &a, uint32_t *marks, int64_t part, int64_t parts, F tokens, G beside) {
    const int across = a.row < ZEROS ? a.row : ZEROS, down = ZEROS / across;
    const int r0 = threadIdx.x / across, p0 = threadIdx.x - r0 * across;
    const int64_t begin = a.V * part / parts, end = a.V * (part + 1) / parts;
    for (int64_t v0 = begin; v0 < end || v0 == begin; v0 += kWindow) {
        const uint32_t rows = static_cast<uint32_t>(end - v0 < kWindow ? end - v0 : kWindow);
        __syncthreads();
        for (uint32_t i = threadIdx.x; i < (rows + 31) / 32; i += THREADS) marks[i] = 0u;
        __syncthreads();
        tokens([&](int64_t id) {
            const uint64_t at = static_cast<uint64_t>(id) - static_cast<uint64_t>(v0);
            if (at < rows) atomicOr(&marks[at >> 5], 1u << (at & 31));
        });
        __syncthreads();
        if (ZEROS < THREADS && threadIdx.x >= ZEROS) {
            if (v0 == begin) beside();
            continue;
        }
        for (uint32_t r = r0; r < rows && r0 < down; r += down) {
            if (marks[r >> 5] >> (r & 31) & 1u) continue;
            uint4 *row = a.table + (v0 + r) * a.row;
            for (int p = p0; p < a.row; p += across) row[p] = make_uint4(0, 0, 0, 0);
        }
    }
}
template <int THREADS>
__device__ __forceinline__ void zero_rows(const ZeroArgs &a, uint32_t *marks, int64_t part, int64_t parts) {
    const auto tokens = [&](auto f) {
        for (int64_t i = threadIdx.x; i < a.M; i += THREADS * kZeroBatch) {
            int64_t id[kZeroBatch];
#pragma unroll
            for (int j = 0; j < kZeroBatch; ++j) id[j] = i + j * THREADS < a.M ? __ldg(a.ids + i + j * THREADS) : -1;
#pragma unroll
            for (int j = 0; j < kZeroBatch; ++j) f(id[j]);
        }
    };
    zero_rows<THREADS, THREADS>(a, marks, part, parts, tokens, [] {});
}

// EARLY: it runs beside the kernel before it, whose arrays it does not touch and which
// lets it start when whatever came before is complete; it waits for it at its end.
template <bool EARLY>
__global__ void __launch_bounds__(kZeroThreads, 2) embed_zero_kernel(const ZeroArgs a) {
    __shared__ uint32_t marks[kWindow / 32];
    if constexpr (!EARLY) {
        pdl_wait();
        pdl_launch_dependents();
    }
    zero_rows<kZeroThreads>(a, marks, blockIdx.x, gridDim.x);
    if constexpr (EARLY) {
        pdl_wait();
        pdl_launch_dependents();
    }
}

__device__ __forceinline__ uint32_t ld_cluster_u32(uint32_t addr) {
    uint32_t v;
    asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
    return v;
}

// The lanes whose digit is this one's: a vote for each bit. (__match_any_sync is slow where
// many lanes differ.)
template <int BITS>
__device__ __forceinline__ uint32_t lanes_with(uint32_t digit, bool in) {
    uint32_t peers = __ballot_sync(0xffffffffu, in);
#pragma unroll
    for (int b = 0; b < BITS; ++b) {
        const uint32_t ones = __ballot_sync(0xffffffffu, (digit & (1u << b)) != 0u);
        peers &= ones ^ ((digit >> b & 1u) - 1u);
    }
    return peers;
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
    for (int pass = 0; pass < a.passes; ++pass) {
        const int shift = pass * kDigitBits;
        const bool odd = pass & 1;  // (no index into the parameters: they would be copied to the stack)
        const uint32_t *key_in = odd ? a.key[1] : a.key[0], *pos_in = odd ? a.pos[1] : a.pos[0];
        uint32_t *key_out = odd ? a.key[0] : a.key[1], *pos_out = odd ? a.pos[0] : a.pos[1];
        const auto key_at = [&](int64_t i) {
            if (pass > 0) return __ldcg(key_in + i);
            const int64_t id = __ldg(a.ids + i);
            return id >= 0 && id < a.V ? static_cast<uint32_t>(id) : none;
        };
        for (int w = 0; w < kSortWarps; ++w) hist[w][tid] = 0u;
        __syncthreads();
        uint32_t k[kBatch], p[kBatch];
        const auto load = [&](int64_t i) {
#pragma unroll
            for (int j = 0; j < kBatch; ++j) {
                const int64_t at = i + j * 32 + lane;
                if (at >= last) continue;
                k[j] = key_at(at);
                p[j] = pass > 0 ? __ldcg(pos_in + at) : static_cast<uint32_t>(at);
            }
        };
        for (int64_t i = first; i < last; i += 32 * kBatch) {
            load(i);
#pragma unroll
            for (int j = 0; j < kBatch; ++j)
                if (i + j * 32 + lane < last) atomicAdd(&hist[warp][k[j] >> shift & (kBins - 1)], 1u);
        }
        __syncthreads();
        uint32_t count[kSortWarps], sum = 0;
#pragma unroll
        for (int w = 0; w < kSortWarps; ++w) count[w] = hist[w][tid];
#pragma unroll
        for (int w = 0; w < kSortWarps; ++w) sum += count[w];
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
#pragma unroll
        for (int w = 0; w < kSortWarps; ++w) {
            hist[w][tid] = base;
            base += count[w];
        }
        __syncthreads();
        for (int64_t i = first; i < last; i += 32 * kBatch) {
            if (run > 32 * kBatch) load(i);  // (else they are still there)
#pragma unroll
            for (int j = 0; j < kBatch; ++j) {
                const bool in = i + j * 32 + lane < last;
                const uint32_t digit = in ? k[j] >> shift & (kBins - 1) : 0u, peers = lanes_with<kDigitBits>(digit, in);
                uint32_t to = 0;
                if (in) to = hist[warp][digit] + __popc(peers & ((1u << lane) - 1u));
                __syncwarp();
                if (in && lane == __ffs(peers) - 1) hist[warp][digit] += __popc(peers);
                __syncwarp();
                if (in) {
                    key_out[to] = k[j];
                    pos_out[to] = p[j];
                }
            }
        }
        cluster_sync_all();  // the arrays are whole, and everyone has read `total`
    }
}

// Up to kRankMost tokens: half of every block zeroes its rows, and the other half finds
// where its share of the tokens goes, two for a warp at a time, by counting the keys before
// them. bf16, 4096 tokens: 5000 x 64 13.8 us (16.5 and 15.2 with 8 and 24 warps of 32 that
// count), 32000 x 2048 35.5 (34.8, 39.5); 3361 in fp32, 2952 x 1120 19.3, by a radix sort in
// one block 22.9.
constexpr int kRankThreads = 1024, kRankZeros = 512, kRankWarps = (kRankThreads - kRankZeros) / 32;
constexpr int kRankMost = 4096;

__global__ void __launch_bounds__(kRankThreads, 1) embed_rank_kernel(const SortArgs a, const ZeroArgs z) {
    constexpr int kEach = kRankMost / kRankThreads;
    __shared__ uint32_t marks[kWindow / 32];
    __shared__ __align__(16) uint32_t key[kRankMost];
    pdl_wait();
    pdl_launch_dependents();
    const int M = static_cast<int>(a.M), lane = threadIdx.x & 31, fours = (M + 3) / 4;
    int64_t id[kEach];
#pragma unroll
    for (int j = 0; j < kEach; ++j) {
        const int i = threadIdx.x + j * kRankThreads;
        id[j] = i < M ? __ldg(a.ids + i) : -1;
    }
#pragma unroll
    for (int j = 0; j < kEach; ++j) {
        const int i = threadIdx.x + j * kRankThreads;
        if (i < 4 * fours) key[i] = i >= M ? 0xFFFFFFFFu : static_cast<uint32_t>(id[j] >= 0 && id[j] < a.V ? id[j] : a.V);
    }
    const auto tokens = [&](auto f) {
#pragma unroll
        for (int j = 0; j < kEach; ++j) f(id[j]);
    };
    const auto rank = [&] {
        const int last = static_cast<int>(a.M * (blockIdx.x + 1) / gridDim.x);
        const int warp = (threadIdx.x - kRankZeros) >> 5;
        for (int i = static_cast<int>(a.M * blockIdx.x / gridDim.x) + 2 * warp; i < last; i += 2 * kRankWarps) {
            // smaller keys, and of its own those of earlier positions: all but its own four's
            const int at[2] = {i, i + 1 < last ? i + 1 : i};
            const uint32_t mine[2] = {key[at[0]], key[at[1]]};
            uint32_t n[2] = {0u, 0u};
#pragma unroll 4
            for (int c = lane; c < fours; c += 32) {
                const uint4 q = reinterpret_cast<const uint4 *>(key)[c];
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    const uint32_t below = mine[u] + (4 * c + 3 < at[u] ? 1u : 0u);
                    n[u] += (q.x < below) + (q.y < below) + (q.z < below) + (q.w < below);
                }
            }
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                if (lane < (at[u] & 3)) n[u] += key[(at[u] & ~3) + lane] == mine[u];
                n[u] = __reduce_add_sync(0xffffffffu, n[u]);
                if (lane == 0) {
                    a.key[0][n[u]] = mine[u];
                    a.pos[0][n[u]] = static_cast<uint32_t>(at[u]);
                }
            }
        }
    };
    zero_rows<kRankThreads, kRankZeros>(z, marks, blockIdx.x, gridDim.x, tokens, rank);
}

// More tokens: a radix sort by a cluster of words of (key, position), the key above `low`
// bits of position. A CTA holds consecutive words in registers, and they change places
// through distributed shared memory.
constexpr int kWideEach = 8;
constexpr int kWideMost = kSortCtas * kSortThreads * kWideEach;
constexpr int kWideSmem = (kSortThreads * kWideEach + (kSortWarps + 1) * kBins) * 4;

__device__ __forceinline__ void st_cluster_u32(uint32_t addr, uint32_t v) {
    asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}

__global__ void __launch_bounds__(kSortThreads, 1) embed_sort_wide_kernel(const SortArgs a, int low, int digit_bits) {
    extern __shared__ uint32_t sorted[];  // the CTA's words, a histogram for each warp, the CTA's counts
    __shared__ uint32_t scan[kSortWarps];
    pdl_wait();
    pdl_launch_dependents();
    uint32_t *hist = sorted + kSortThreads * kWideEach, *total = hist + kSortWarps * kBins;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const uint32_t rank = cluster_ctarank();
    const int M = static_cast<int>(a.M), rounds = (M + kSortCtas * kSortThreads - 1) / (kSortCtas * kSortThreads);
    const int each = kSortThreads * rounds;                                 // words of a CTA
    const int mine0 = warp * rounds * 32 + lane, first = static_cast<int>(rank) * each + mine0;  // a warp's: consecutive
    const uint32_t bins = 1u << digit_bits, mask = bins - 1u;
    uint32_t w[kWideEach];
#pragma unroll
    for (int j = 0; j < kWideEach; ++j) {
        const int i = first + j * 32;
        if (j >= rounds || i >= M) continue;
        const int64_t id = __ldg(a.ids + i);
        w[j] = static_cast<uint32_t>(id >= 0 && id < a.V ? id : a.V) << low | static_cast<uint32_t>(i);
    }
    uint32_t *mine = hist + warp * kBins;
    for (int pass = 0; pass < a.passes; ++pass) {
        const int shift = low + pass * digit_bits;
        for (uint32_t i = lane; i < kBins; i += 32) mine[i] = 0u;
        __syncwarp();
#pragma unroll
        for (int j = 0; j < kWideEach; ++j)
            if (j < rounds && first + j * 32 < M) atomicAdd(&mine[w[j] >> shift & mask], 1u);
        __syncthreads();
        // a thread for each bin
        uint32_t count[kSortWarps], sum = 0;
#pragma unroll
        for (int k = 0; k < kSortWarps; ++k) count[k] = hist[k * kBins + tid];
#pragma unroll
        for (int k = 0; k < kSortWarps; ++k) sum += count[k];
        total[tid] = sum;
        cluster_sync_all();  // (every CTA has its words in registers, too)
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
        uint32_t base = before + upto - all + __reduce_add_sync(0xffffffffu, lane < warp ? scan[lane] : 0u);
#pragma unroll
        for (int k = 0; k < kSortWarps; ++k) {
            hist[k * kBins + tid] = base;
            base += count[k];
        }
        __syncthreads();
#pragma unroll
        for (int j = 0; j < kWideEach; ++j) {
            if (j >= rounds) break;
            const bool in = first + j * 32 < M;
            const uint32_t digit = in ? w[j] >> shift & mask : 0u, peers = lanes_with<kDigitBits>(digit, in);
            uint32_t to = 0;
            if (in) to = mine[digit] + __popc(peers & ((1u << lane) - 1u));
            __syncwarp();
            if (in && lane == __ffs(peers) - 1) mine[digit] += __popc(peers);
            __syncwarp();
            if (in) {
                const uint32_t cta = to / static_cast<uint32_t>(each);
                st_cluster_u32(mapa_shared(smem_u32(&sorted[to - cta * each]), cta), w[j]);
            }
        }
        cluster_sync_all();
        if (pass + 1 < a.passes) {
#pragma unroll
            for (int j = 0; j < kWideEach; ++j)
                if (j < rounds && first + j * 32 < M) w[j] = sorted[mine0 + j * 32];
        }
    }
    for (int i = tid; i < each && static_cast<int>(rank) * each + i < M; i += kSortThreads) {
        const uint32_t v = sorted[i];
        a.key[0][rank * each + i] = v >> low;
        a.pos[0][rank * each + i] = v & ((1u << low) - 1u);
    }
}

// --------------------------------------------------------------------- sum

struct SumArgs {
    const void *dy;
    const uint32_t *key, *pos;
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
__global__ void __launch_bounds__(kThreads, BF16 ? 4 : 3) embed_sum_kernel(const SumArgs a) {
    pdl_wait();
    pdl_launch_dependents();
    const uint32_t none = static_cast<uint32_t>(a.V);
    const int64_t it = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x;
    if (it < static_cast<int64_t>(a.chunks) * a.pieces) {
        const int c = static_cast<int>(it / a.pieces), piece = static_cast<int>(it - static_cast<int64_t>(c) * a.pieces);
        const int64_t i0 = c * a.chunk, i1 = i0 + a.chunk < a.M ? i0 + a.chunk : a.M;
        uint32_t now = __ldg(a.key + i0);
        bool whole = i0 == 0 || __ldg(a.key + i0 - 1) != now;  // the run starts in this chunk
        uint64_t sum[4] = {0ull, 0ull, 0ull, 0ull};
        // fp32: 32768 tokens, 1000 x 2048 70.8 us, 76.6 with 4, which do not fit the registers. bf16: four,
        // with 68 bytes of them spilled, 193.4 us for 16384 tokens, 128000 x 4096 and 49.2 for 32768,
        // 1000 x 2048; two, none spilled, 194.4 and 50.2; four in three blocks an SM, none spilled, 200.9 and 55.3.
        constexpr int kAhead = BF16 ? 4 : 2;
        uint32_t next_key[kAhead], next_pos[kAhead];  // a batch ahead of the rows that they name
        const auto look = [&](int64_t i) {
#pragma unroll
            for (int j = 0; j < kAhead; ++j) {
                next_key[j] = i + j < i1 ? __ldg(a.key + i + j) : none;
                next_pos[j] = i + j < i1 ? __ldg(a.pos + i + j) : 0u;
            }
        };
        look(i0);
        for (int64_t i = i0; i < i1 && now != none; i += kAhead) {
            uint32_t key[kAhead];
            Piece<BF16> d[kAhead];
#pragma unroll
            for (int j = 0; j < kAhead; ++j) {
                key[j] = next_key[j];
                if (key[j] != none) d[j] = load_piece<BF16>(a.dy, static_cast<int64_t>(next_pos[j]) * a.pieces + piece);
            }
            look(i + kAhead);
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
    const int64_t begin = c * a.chunk, end = begin + a.chunk;
    if (end >= a.M) return;
    const uint32_t v = __ldg(a.key + end - 1), after = __ldg(a.key + end), start = __ldg(a.key + begin),
                   before = begin > 0 ? __ldg(a.key + begin - 1) : none;
    if (v == none || after != v || (start == v && before == v)) return;
    const float4 *partial = reinterpret_cast<const float4 *>(a.partial) + 2 * piece;
    const auto part = [&](int64_t row, int h) { return __ldcg(partial + row * a.pieces * 2 + h); };
    float4 x = part(2ll * c + 1, 0), y = part(2ll * c + 1, 1);
    uint64_t sum[4] = {f2_pack(x.x, x.y), f2_pack(x.z, x.w), f2_pack(y.x, y.y), f2_pack(y.z, y.w)};
    // the chunks that begin with it, some at a time so that their loads overlap
    constexpr int kAhead = 8;
    for (int next = c + 1; next < a.chunks; next += kAhead) {
        bool more[kAhead];
        float4 p[kAhead][2];
#pragma unroll
        for (int j = 0; j < kAhead; ++j) {
            more[j] = next + j < a.chunks && __ldg(a.key + (next + j) * a.chunk) == v;
            if (next + j < a.chunks) {
                p[j][0] = part(2ll * (next + j), 0);
                p[j][1] = part(2ll * (next + j), 1);
            }
        }
#pragma unroll
        for (int j = 0; j < kAhead; ++j) {
            if (!more[j]) break;
            sum[0] = f2_add(sum[0], f2_pack(p[j][0].x, p[j][0].y));
            sum[1] = f2_add(sum[1], f2_pack(p[j][0].z, p[j][0].w));
            sum[2] = f2_add(sum[2], f2_pack(p[j][1].x, p[j][1].y));
            sum[3] = f2_add(sum[3], f2_pack(p[j][1].z, p[j][1].w));
        }
        if (!more[kAhead - 1]) break;
    }
    write_row(a, v, piece, sum);
}

// ---------------------------------------------------------------- few tokens

// Zeros and sums in one launch: every block finds the tokens of its rows by votes. A
// fourth of the block adds a row's tokens of 32 positions each, and the first one their
// sums, in the positions' order.
template <bool BF16>
__global__ void __launch_bounds__(kZeroThreads, 2) embed_few_kernel(const ZeroArgs z, const SumArgs a) {
    constexpr int kWords = kFewMost / 32, kEach = kZeroThreads / kWords, kAhead = BF16 ? 8 : 4;
    __shared__ __align__(16) uint32_t marks[kWindow / 32];  // then the parts' sums, [2][kZeroThreads] of 16 bytes
    __shared__ int64_t id[kFewMost];
    __shared__ uint32_t with[kFewMost][kWords];  // the tokens whose id a first one's is
    __shared__ uint32_t first[kFewMost], n_first;
    static_assert(kZeroThreads * 32 <= sizeof(marks) && kFewPieces == kEach, "a thread for each piece of a row");
    pdl_wait();
    pdl_launch_dependents();
    const int tid = threadIdx.x, lane = tid & 31, M = static_cast<int>(a.M);
    const int64_t v0 = a.V * blockIdx.x / gridDim.x, v1 = a.V * (blockIdx.x + 1) / gridDim.x;
    if (tid < kFewMost) id[tid] = tid < M ? __ldg(z.ids + tid) : -1;
    if (tid == 0) n_first = 0u;
    zero_rows<kZeroThreads>(z, marks, blockIdx.x, gridDim.x);
    __syncthreads();
    for (int i = tid >> 5; i < M; i += kZeroThreads / 32) {
        const int64_t v = id[i];
        if (v < v0 || v >= v1) continue;
        uint32_t mine = 0u, earlier = 0u;
#pragma unroll
        for (int j = 0; j < kWords; ++j) {
            const uint32_t m = __ballot_sync(0xffffffffu, id[j * 32 + lane] == v);
            if (lane == j) mine = m;
            earlier |= j * 32 + 32 <= i ? m : j * 32 <= i ? m & ((1u << (i & 31)) - 1u) : 0u;
        }
        if (earlier != 0u) continue;
        if (lane < kWords) with[i][lane] = mine;
        if (lane == 0) first[atomicAdd(&n_first, 1u)] = static_cast<uint32_t>(i);
    }
    __syncthreads();
    const int word = tid / kEach, at = tid % kEach, rows = kEach / a.pieces, r = at / a.pieces, piece = at - r * a.pieces;
    float4 *part = reinterpret_cast<float4 *>(marks);
    for (uint32_t n0 = 0; n0 < n_first; n0 += rows) {
        const bool in = r < rows && n0 + r < n_first;
        const uint32_t i = in ? first[n0 + r] : 0u;
        uint64_t sum[4] = {0ull, 0ull, 0ull, 0ull};
        for (uint32_t m = in ? with[i][word] : 0u; m != 0u;) {
            Piece<BF16> d[kAhead];
            bool is[kAhead];
#pragma unroll
            for (int u = 0; u < kAhead; ++u) {
                is[u] = m != 0u;
                if (is[u]) d[u] = load_piece<BF16>(a.dy, static_cast<int64_t>(word * 32 + __ffs(m) - 1) * a.pieces + piece);
                m &= m - 1u;
            }
#pragma unroll
            for (int u = 0; u < kAhead; ++u) {
                if (!is[u]) break;
#pragma unroll
                for (int q = 0; q < 4; ++q) sum[q] = f2_add(sum[q], d[u].pair(q));
            }
        }
        if (word > 0) {
            const Piece<false> s = round_piece<false>(sum);
            part[tid] = make_float4(__uint_as_float(s.w[0]), __uint_as_float(s.w[1]), __uint_as_float(s.w[2]), __uint_as_float(s.w[3]));
            part[kZeroThreads + tid] = make_float4(__uint_as_float(s.w[4]), __uint_as_float(s.w[5]), __uint_as_float(s.w[6]), __uint_as_float(s.w[7]));
        }
        __syncthreads();
        if (word == 0 && in) {
#pragma unroll
            for (int j = 1; j < kWords; ++j) {
                if (with[i][j] == 0u) continue;
                const float4 x = part[j * kEach + at], y = part[kZeroThreads + j * kEach + at];
                sum[0] = f2_add(sum[0], f2_pack(x.x, x.y));
                sum[1] = f2_add(sum[1], f2_pack(x.z, x.w));
                sum[2] = f2_add(sum[2], f2_pack(y.x, y.y));
                sum[3] = f2_add(sum[3], f2_pack(y.z, y.w));
            }
            write_row(a, static_cast<uint32_t>(id[i]), piece, sum);
        }
        __syncthreads();
    }
}

template <bool BF16>
cudaError_t few(const ZeroArgs &z, const SumArgs &a, cudaStream_t s, const DeviceInfo &dev) {
    const int64_t want = z.V * z.row / 512 + 1, most = 2ll * dev.num_sms;  // of at least 8 KB
    return launch_kernel(embed_few_kernel<BF16>, dim3(static_cast<unsigned>(want < most ? want : most)), dim3(kZeroThreads), 0, s, z, a);
}

// The tokens sorted and the rows without one zeroed.
cudaError_t sort_and_zero(SortArgs so, const ZeroArgs &z, int key_bits, int low, cudaStream_t s, const DeviceInfo &dev) {
    const bool rank = so.M <= kRankMost, wide = !rank && so.M <= kWideMost && key_bits + low <= 32;
    so.passes = (key_bits + kDigitBits - 1) / kDigitBits;
    const int digit_bits = (key_bits + so.passes - 1) / so.passes;
    // blocks of at least 32 KB, one or two to an SM, but where the sort runs
    const int64_t want = z.V * z.row / 2048 + 1, sms = dev.num_sms;
    if (rank) {  // (and of at most two tokens for each warp that ranks)
        const int64_t for_tokens = so.M / (2 * kRankWarps) + 1, blocks = want > for_tokens ? want : for_tokens;
        return launch_kernel(embed_rank_kernel, dim3(static_cast<unsigned>(blocks < sms ? blocks : sms)), dim3(kRankThreads), 0, s, so, z);
    }
    const int64_t most = wide ? 2 * sms - kSortCtas : 2 * sms;
    const unsigned blocks = static_cast<unsigned>(want < most ? want : most);
    cudaError_t e;
    if (wide) {
        static std::atomic<bool> ready[64];
        e = allow_smem(embed_sort_wide_kernel, kWideSmem, ready, dev.device);
        if (e == cudaSuccess)
            e = launch_kernel_cluster(embed_sort_wide_kernel, dim3(kSortCtas), dim3(kSortThreads), kWideSmem, s, kSortCtas, so,
                                      low, digit_bits);
    } else {
        e = launch_kernel_cluster(embed_sort_kernel, dim3(kSortCtas), dim3(kSortThreads), 0, s, kSortCtas, so);
    }
    if (e != cudaSuccess) return e;
    return launch_kernel(wide ? embed_zero_kernel<true> : embed_zero_kernel<false>, dim3(blocks), dim3(kZeroThreads), 0, s, z);
}

// The workspace: keys and positions, each twice; the partial sums.
struct Layout {
    int64_t chunk, chunks, partial, bytes;
};
int64_t round16(int64_t n) { return (n + 15) / 16 * 16; }
Layout layout_of(int64_t M, int64_t K) {
    Layout l;
    l.chunk = (M * (K / kPiece) + kSumItems - 1) / kSumItems;
    int64_t shortest = kMinChunk;  // about sqrt(M / 64): the sum walks a chunk, the join the chunks of a run
    while (shortest * shortest * 64 < M) shortest *= 2;
    if (l.chunk < shortest) l.chunk = shortest;
    l.chunks = (M + l.chunk - 1) / l.chunk;
    l.partial = 4 * round16(4 * M);
    l.bytes = l.partial + 2 * l.chunks * K * 4;
    return l;
}

}  // namespace

int64_t embedding_workspace_bytes(int64_t M, int64_t K) { return layout_of(M, K).bytes; }

int launch_embedding_fwd(const int64_t *ids, int64_t M, const void *table, int table_kind, int64_t V, int64_t K,
                         const float *sinv, float scale, void *out, int out_dtype, cudaStream_t s, const DeviceInfo &dev) {
    const bool bf16 = out_dtype == FP8MP_BF16;
    const EmbedArgs a = {ids, static_cast<const uint8_t *>(table), sinv, out, M, V, static_cast<int>(K / (bf16 ? 8 : 4)), scale};
    const int64_t rows = (a.units < kThreads ? kThreads / a.units : 1) * kRows;  // of a block
    const dim3 grid(static_cast<unsigned>((M + rows - 1) / rows)), block(kThreads);
    cudaError_t e;
    if (table_kind == 0)
        e = launch_kernel(bf16 ? embed_fwd_kernel<0, true> : embed_fwd_kernel<0, false>, grid, block, 0, s, a);
    else if (table_kind == 1)
        e = launch_kernel(bf16 ? embed_fwd_kernel<1, true> : embed_fwd_kernel<1, false>, grid, block, 0, s, a);
    else
        e = launch_kernel(bf16 ? embed_fwd_kernel<2, true> : embed_fwd_kernel<2, false>, grid, block, 0, s, a);
    if (e != cudaSuccess) return fail(FP8MP_ERR_LAUNCH, "embedding: launch failed: %s", cudaGetErrorString(e));
    return FP8MP_OK;
}

int launch_embedding_bwd(const int64_t *ids, int64_t M, const void *dy, int dy_dtype, int64_t V, int64_t K, float scale,
                         void *dtable, int out_dtype, void *workspace, cudaStream_t s, const DeviceInfo &dev) {
    const Layout l = layout_of(M, K);
    uint8_t *ws = static_cast<uint8_t *>(workspace);
    SortArgs so = {};
    so.ids = ids;
    const int64_t each = round16(4 * M);
    for (int i = 0; i < 2; ++i) {
        so.key[i] = reinterpret_cast<uint32_t *>(ws + i * each);
        so.pos[i] = reinterpret_cast<uint32_t *>(ws + (2 + i) * each);
    }
    so.M = M;
    so.V = V;
    int key_bits = 1, low = 1;  // keys are 0 .. V, positions 0 .. M - 1
    while (V >> key_bits != 0) ++key_bits;
    while ((M - 1) >> low > 0) ++low;
    const ZeroArgs z = {ids, static_cast<uint4 *>(dtable), M, V, static_cast<int>(K * (out_dtype == FP8MP_BF16 ? 2 : 4) / 16)};
    SumArgs a = {};
    a.dy = dy;
    // (a sort through global memory leaves them in the arrays of the other turn after an odd number of passes)
    const bool words = M <= kRankMost || (M <= kWideMost && key_bits + low <= 32);
    const int turn = words ? 0 : (key_bits + kDigitBits - 1) / kDigitBits & 1;
    a.key = so.key[turn];
    a.pos = so.pos[turn];
    a.out = dtable;
    a.partial = reinterpret_cast<float *>(ws + l.partial);
    a.M = M;
    a.V = V;
    a.chunk = l.chunk;
    a.chunks = static_cast<int>(l.chunks);
    a.pieces = static_cast<int>(K / kPiece);
    a.scale = scale;
    a.out_bf16 = out_dtype == FP8MP_BF16;
    cudaError_t e;
    if (M <= kFewMost && a.pieces <= kFewPieces) {
        e = dy_dtype == FP8MP_BF16 ? few<true>(z, a, s, dev) : few<false>(z, a, s, dev);
        if (e != cudaSuccess) return fail(FP8MP_ERR_LAUNCH, "embedding: launch failed: %s", cudaGetErrorString(e));
        return FP8MP_OK;
    }
    e = sort_and_zero(so, z, key_bits, low, s, dev);
    const int64_t items = l.chunks * a.pieces, blocks = (items + kThreads - 1) / kThreads;
    const dim3 grid(static_cast<unsigned>(blocks)), block(kThreads);
    if (e == cudaSuccess && items > 0)
        e = dy_dtype == FP8MP_BF16 ? launch_kernel(embed_sum_kernel<true>, grid, block, 0, s, a)
                                   : launch_kernel(embed_sum_kernel<false>, grid, block, 0, s, a);
    if (e == cudaSuccess && l.chunks > 1)
        e = launch_kernel(embed_join_kernel, dim3(static_cast<unsigned>(blocks)), block, 0, s, a);
    if (e != cudaSuccess) return fail(FP8MP_ERR_LAUNCH, "embedding: launch failed: %s", cudaGetErrorString(e));
    return FP8MP_OK;
}

}  // namespace fp8mp
