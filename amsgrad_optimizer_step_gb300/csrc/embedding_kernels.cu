// The embedding lookup with scaling and its gradient by sorted tokens.
//
// Gradient of row v: scale * sum over the tokens t with id v of dout[t].  The tokens
// are sorted by id (stable: ascending t within an id), so that each id's rows are one
// run of the sorted order, and the sorted order is cut into units of kSumUnit tokens,
// each added by one CTA in order: the work of a unit does not depend on how the ids
// are distributed.  A run inside one unit is finished there; a run that several units
// share leaves FP32 partial sums, which the join adds in unit order.
//
// Sort: each CTA sorts a chunk of kSortChunk tokens in shared memory (least significant
// digit first, 4 bits a pass); a token's place in the whole order is then its place in
// its chunk plus, for every other chunk, the number of its ids that come before (ties:
// earlier chunks come before), found by binary search.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "internal.h"
#include "model_device.cuh"
#include "model_internal.h"

namespace fa {
namespace {

FA_BOUNDS_COUNTER(g_embedding_oob)

constexpr int kLookupThreads = 256;
constexpr int kLookupGroups = 4;  // 16-byte groups a lane has in flight
constexpr int kSortThreads = 1024;
constexpr int kSortItems = kSortChunk / kSortThreads;
constexpr int kDigits = 16;
constexpr int kSumThreads = 128;
constexpr int kMergeThreads = 256;

// Elements a thread handles at once: 16 bytes of the narrower type when both sides are
// aligned for it, else one.
template <int AT, int BT, bool VEC>
constexpr int kGroup =
    VEC ? (Elem<AT>::kVec > Elem<BT>::kVec ? Elem<AT>::kVec : Elem<BT>::kVec) : 1;

// ---- lookup --------------------------------------------------------------------

// 2^lanes_log2 lanes take a token's stretch (blockIdx.y) of kLookupGroups groups each: a row's
// loads are in flight together once its id is there.
template <int TT, int OT, int IT, bool VEC>
__global__ void __launch_bounds__(kLookupThreads)
lookup_kernel(LookupArgs a, int groups, int lanes_log2) {
    constexpr int N = kGroup<TT, OT, VEC>;
    using TE = typename Elem<TT>::T;
    using OE = typename Elem<OT>::T;
    const int64_t thread = static_cast<int64_t>(blockIdx.x) * kLookupThreads + threadIdx.x;
    const int64_t t = thread >> lanes_log2;
    if (t >= a.tokens) return;
    const int lanes = 1 << lanes_log2;
    const int g0 = (blockIdx.y * kLookupGroups << lanes_log2) + (threadIdx.x & (lanes - 1));
    const int64_t id = load_id<IT>(a.ids, t);
    const bool known = id >= 0 && id < a.vocab;
    const TE *row = static_cast<const TE *>(a.table) + (known ? id : 0) * a.table_ld;
    OE *out = static_cast<OE *>(a.out) + t * a.out_ld;
    float x[kLookupGroups][N];
#pragma unroll
    for (int k = 0; k < kLookupGroups; ++k) {
        const int g = g0 + k * lanes;
        if (known && g < groups && fa_in_bounds(static_cast<int64_t>(g) * N, N, a.dim))
            read_n<TT, N>(row + static_cast<int64_t>(g) * N, x[k]);
    }
#pragma unroll
    for (int k = 0; k < kLookupGroups; ++k) {
        const int g = g0 + k * lanes;
        if (g >= groups || !fa_in_bounds(static_cast<int64_t>(g) * N, N, a.dim)) break;
#pragma unroll
        for (int j = 0; j < N; ++j) x[k][j] = known ? x[k][j] * a.scale : 0.f;
        store_n<OT, N>(out + static_cast<int64_t>(g) * N, x[k]);
    }
}

// ---- sort ----------------------------------------------------------------------

struct SortArgs {
    const void *ids;
    int64_t tokens, vocab, padding_idx;
    uint32_t *keys, *pos;    // this chunk's sorted ids and token indices
    int bits;                // of the largest key: vocab, which marks a token without an id
};

// Shared memory of a chunk: keys, local indices, digit counters.
constexpr int kSortSmem = kSortChunk * 4 + kSortChunk * 2 + kDigits * kSortThreads * 2 + 32 * 4;

template <int IT>
__global__ void __launch_bounds__(kSortThreads) sort_chunk_kernel(SortArgs a) {
    fa_allow_dependents();
    extern __shared__ uint4 smem[];
    uint32_t *keys = reinterpret_cast<uint32_t *>(smem);
    uint16_t *local = reinterpret_cast<uint16_t *>(keys + kSortChunk);
    uint16_t *count = local + kSortChunk;  // [digit][thread]
    uint32_t *warp_total = reinterpret_cast<uint32_t *>(count + kDigits * kSortThreads);
    const int t = threadIdx.x, lane = t & 31, warp = t / 32;
    const int64_t base = static_cast<int64_t>(blockIdx.x) * kSortChunk;
    const int64_t left = a.tokens - base;
    const int n = left < kSortChunk ? static_cast<int>(left) : kSortChunk;

    for (int i = t; i < kSortChunk; i += kSortThreads) {
        uint32_t key = 0xffffffffu;  // past the end: after everything
        if (i < n && fa_in_bounds(base + i, 1, a.tokens)) {
            const int64_t id = load_id<IT>(a.ids, base + i);
            key = id >= 0 && id < a.vocab && id != a.padding_idx ? static_cast<uint32_t>(id)
                                                                 : static_cast<uint32_t>(a.vocab);
        }
        keys[i] = key;
        local[i] = static_cast<uint16_t>(i);
    }
    __syncthreads();
    // a short chunk's filler has every bit set and came last: it stays last
    for (int shift = 0; shift < a.bits; shift += 4) {
        uint32_t k[kSortItems];
        uint16_t v[kSortItems], rank[kSortItems];
#pragma unroll
        for (int j = 0; j < kSortItems; ++j) {
            k[j] = keys[t * kSortItems + j];
            v[j] = local[t * kSortItems + j];
        }
#pragma unroll
        for (int d = 0; d < kDigits; ++d) count[d * kSortThreads + t] = 0;
#pragma unroll
        for (int j = 0; j < kSortItems; ++j) {
            uint16_t *c = &count[((k[j] >> shift) & (kDigits - 1)) * kSortThreads + t];
            rank[j] = *c;
            *c = static_cast<uint16_t>(rank[j] + 1);
        }
        __syncthreads();
        // exclusive prefix over (digit, thread): kDigits consecutive counters a thread
        uint16_t *mine = count + t * kDigits;
        uint32_t sum = 0;
        uint16_t c[kDigits];
#pragma unroll
        for (int d = 0; d < kDigits; ++d) {
            c[d] = mine[d];
            sum += c[d];
        }
        uint32_t incl = sum;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const uint32_t up = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += up;
        }
        if (lane == 31) warp_total[warp] = incl;
        __syncthreads();
        uint32_t run = incl - sum;
        for (int w = 0; w < warp; ++w) run += warp_total[w];
#pragma unroll
        for (int d = 0; d < kDigits; ++d) {
            mine[d] = static_cast<uint16_t>(run);
            run += c[d];
        }
        __syncthreads();
#pragma unroll
        for (int j = 0; j < kSortItems; ++j) {
            const int at = count[((k[j] >> shift) & (kDigits - 1)) * kSortThreads + t] + rank[j];
            keys[at] = k[j];
            local[at] = v[j];
        }
        __syncthreads();
    }
    for (int i = t; i < n; i += kSortThreads) {
        if (!fa_in_bounds(base + i, 1, a.tokens)) continue;
        a.keys[base + i] = keys[i];
        a.pos[base + i] = static_cast<uint32_t>(base + local[i]);
    }
}

// First index in keys[0, n) whose key is >= key (strict: > key).
__device__ __forceinline__ int64_t bound(const uint32_t *keys, int64_t n, uint32_t key,
                                         bool strict) {
    int64_t lo = 0, len = n;
    while (len > 0) {
        const int64_t half = len >> 1;
        const uint32_t k = __ldg(keys + lo + half);
        const bool right = strict ? k <= key : k < key;
        lo = right ? lo + half + 1 : lo;
        len = right ? len - half - 1 : half;
    }
    return lo;
}

// Places every chunk's sorted tokens in the order of all.
__global__ void __launch_bounds__(kMergeThreads)
merge_chunks_kernel(const uint32_t *keys, const uint32_t *pos, uint32_t *out_keys,
                    uint32_t *out_pos, int64_t tokens, int64_t chunks) {
    fa_grid_dependency_wait();
    fa_allow_dependents();
    const int64_t i = static_cast<int64_t>(blockIdx.x) * kMergeThreads + threadIdx.x;
    if (i >= tokens) return;
    const uint32_t key = keys[i];
    const int64_t mine = i / kSortChunk;
    int64_t at = i - mine * kSortChunk;
    for (int64_t c = 0; c < chunks; ++c) {
        if (c == mine) continue;
        const int64_t base = c * kSortChunk;
        const int64_t n = tokens - base < kSortChunk ? tokens - base : kSortChunk;
        at += bound(keys + base, n, key, c < mine);
    }
    if (!fa_in_bounds(at, 1, tokens)) return;
    out_keys[at] = key;
    out_pos[at] = pos[i];
}

// ---- sums ----------------------------------------------------------------------

struct SumArgs {
    EmbeddingGradArgs g;
    const uint32_t *keys, *pos;  // sorted
    float *partial;              // [units][2][dim]
    int64_t units;               // CTAs that add
    int64_t zero_rows;           // rows of dtable a zeroing CTA covers (0: none)
};

// Adds ``sum * scale`` to (or writes it over) elements [c, c + N) of table row v.
template <int TT, int N>
__device__ __forceinline__ void finish_row(const EmbeddingGradArgs &g, int64_t v, int64_t c,
                                           const float *sum) {
    using TE = typename Elem<TT>::T;
    if (!fa_in_bounds(v, 1, g.vocab) || !fa_in_bounds(c, N, g.dim)) return;
    TE *row = static_cast<TE *>(g.dtable) + v * g.table_ld + c;
    float y[N];
    if (g.accumulate) {
        load_n<TT, N>(row, y);
#pragma unroll
        for (int j = 0; j < N; ++j) y[j] = fmaf(sum[j], g.scale, y[j]);
    } else {
#pragma unroll
        for (int j = 0; j < N; ++j) y[j] = sum[j] * g.scale;
    }
    store_n<TT, N>(row, y);
}

// CTA (u, slab): unit u's tokens, columns of slab.  A run that began before the unit
// leaves its sum in partial[u][0], one that goes on after it in partial[u][1] (a run
// that does both, in [0]).  CTAs past the units zero the table rows of absent ids.
template <int DT, int TT, bool VEC>
__global__ void __launch_bounds__(kSumThreads) sum_units_kernel(SumArgs a) {
    constexpr int N = kGroup<DT, TT, VEC>;
    using DE = typename Elem<DT>::T;
    const EmbeddingGradArgs &g = a.g;
    fa_grid_dependency_wait();
    fa_allow_dependents();
    const int64_t c = (static_cast<int64_t>(blockIdx.y) * kSumThreads + threadIdx.x) * N;
    const int64_t u = blockIdx.x;
    __shared__ uint32_t key[kSumUnit + 2];  // with the neighbours on both sides
    __shared__ uint32_t pos[kSumUnit];
    if (u >= a.units) {
        __shared__ bool absent[kSumThreads];
        const int64_t v0 = (u - a.units) * a.zero_rows;
        const int64_t rows = g.vocab - v0 < a.zero_rows ? g.vocab - v0 : a.zero_rows;
        if (threadIdx.x < rows) {
            const uint32_t v = static_cast<uint32_t>(v0 + threadIdx.x);
            const int64_t at = bound(a.keys, g.tokens, v, false);
            absent[threadIdx.x] = at >= g.tokens || a.keys[at] != v;
        }
        __syncthreads();
        if (c >= g.dim) return;
        float zero[N];
#pragma unroll
        for (int j = 0; j < N; ++j) zero[j] = 0.f;
        for (int64_t r = 0; r < rows; ++r)
            if (absent[r] && fa_in_bounds(v0 + r, 1, g.vocab) && fa_in_bounds(c, N, g.dim))
                store_n<TT, N>(static_cast<typename Elem<TT>::T *>(g.dtable) +
                                   (v0 + r) * g.table_ld + c, zero);
        return;
    }
    const int64_t first = u * kSumUnit;
    const int n = g.tokens - first < kSumUnit ? static_cast<int>(g.tokens - first) : kSumUnit;
    for (int i = threadIdx.x; i < n + 2; i += kSumThreads) {
        const int64_t at = first + i - 1;
        key[i] = at >= 0 && at < g.tokens ? a.keys[at] : 0xffffffffu;
    }
    if (threadIdx.x < n) pos[threadIdx.x] = a.pos[first + threadIdx.x];
    __syncthreads();
    if (c >= g.dim) return;
    const DE *dout = static_cast<const DE *>(g.dout) + c;
    float sum[N];
#pragma unroll
    for (int j = 0; j < N; ++j) sum[j] = 0.f;
    bool began_before = key[0] == key[1];
    constexpr int kAhead = 8;  // rows in flight
    for (int i0 = 0; i0 < n; i0 += kAhead) {
        float x[kAhead][N];
#pragma unroll
        for (int k = 0; k < kAhead; ++k)
            if (i0 + k < n && key[i0 + k + 1] < g.vocab && fa_in_bounds(c, N, g.dim) &&
                fa_in_bounds(pos[i0 + k], 1, g.tokens))
                load_n<DT, N>(dout + static_cast<int64_t>(pos[i0 + k]) * g.dout_ld, x[k]);
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
            const int i = i0 + k;
            if (i >= n || key[i + 1] >= g.vocab) break;  // the tokens without an id come last
#pragma unroll
            for (int j = 0; j < N; ++j) sum[j] += x[k][j];
            if (i + 1 < n && key[i + 2] == key[i + 1]) continue;
            // the run's last token here
            const bool goes_on = key[i + 2] == key[i + 1];
            if (began_before || goes_on) {
                float *p = a.partial + (2 * u + (began_before ? 0 : 1)) * g.dim + c;
#pragma unroll
                for (int j = 0; j < N; ++j) p[j] = sum[j];
            } else {
                finish_row<TT, N>(g, key[i + 1], c, sum);
            }
            began_before = false;
#pragma unroll
            for (int j = 0; j < N; ++j) sum[j] = 0.f;
        }
    }
}

// CTA (u, slab): the run that unit u began and did not end, if there is one: its partial
// sums in unit order.
template <int TT, bool VEC, int DT>
__global__ void __launch_bounds__(kSumThreads) join_units_kernel(SumArgs a) {
    constexpr int N = kGroup<DT, TT, VEC>;
    const EmbeddingGradArgs &g = a.g;
    fa_grid_dependency_wait();
    fa_allow_dependents();
    const int64_t u = blockIdx.x;
    const int64_t first = u * kSumUnit, last = first + kSumUnit - 1;
    if (last + 1 >= g.tokens) return;  // the last unit: nothing goes on
    const uint32_t key = a.keys[last];
    if (key >= g.vocab || a.keys[last + 1] != key) return;
    if (first > 0 && a.keys[first] == key && a.keys[first - 1] == key) return;  // began before u
    const int64_t c = (static_cast<int64_t>(blockIdx.y) * kSumThreads + threadIdx.x) * N;
    if (c >= g.dim) return;
    const int64_t end = last + 1 + bound(a.keys + last + 1, g.tokens - last - 1, key, true);
    const int64_t last_unit = (end - 1) / kSumUnit;
    float sum[N];
    const float *p = a.partial + (2 * u + 1) * g.dim + c;
#pragma unroll
    for (int j = 0; j < N; ++j) sum[j] = p[j];
    for (int64_t w = u + 1; w <= last_unit; ++w) {
        const float *q = a.partial + 2 * w * g.dim + c;
        if (!fa_in_bounds(w, 1, a.units)) return;
#pragma unroll
        for (int j = 0; j < N; ++j) sum[j] += q[j];
    }
    finish_row<TT, N>(g, key, c, sum);
}

int64_t round_up(int64_t x, int64_t to) { return (x + to - 1) / to * to; }

bool aligned16(const void *p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; }

// Whether rows of both matrices can be taken N = kGroup<..., true> elements at a time.
bool vector_rows(const void *a, int64_t a_ld, fa_dtype at, const void *b, int64_t b_ld,
                 fa_dtype bt, int64_t dim) {
    const int n = at == FA_F32 && bt == FA_F32 ? 4 : 8;
    return aligned16(a) && aligned16(b) && a_ld % n == 0 && b_ld % n == 0 && dim % n == 0;
}

}  // namespace

cudaError_t embedding_bounds_violations(unsigned long long *count, bool clear) {
#if FA_BOUNDS_CHECK
    cudaError_t err = cudaMemcpyFromSymbol(count, g_embedding_oob, sizeof(*count));
    if (err != cudaSuccess || !clear) return err;
    const unsigned long long zero = 0;
    return cudaMemcpyToSymbol(g_embedding_oob, &zero, sizeof(zero));
#else
    (void)clear;
    *count = 0;
    return cudaSuccess;
#endif
}

cudaError_t launch_embedding_lookup(const LookupArgs &a, fa_itype idt, fa_dtype tdt, fa_dtype odt,
                                    cudaStream_t stream) {
    const bool vec = vector_rows(a.table, a.table_ld, tdt, a.out, a.out_ld, odt, a.dim);
    return for_dtype(tdt, [&](auto td) {
        return for_dtype(odt, [&](auto od) {
            return for_itype(idt, [&](auto id) {
                const auto go = [&](auto v) {
                    constexpr bool VEC = decltype(v)::value;
                    const int64_t groups = a.dim / kGroup<td(), od(), VEC>;
                    int lanes_log2 = 0;
                    while (lanes_log2 < 5 && (int64_t(kLookupGroups) << lanes_log2) < groups)
                        ++lanes_log2;
                    const int64_t ctas = ((a.tokens << lanes_log2) + kLookupThreads - 1) /
                                         kLookupThreads;
                    const int64_t stretch = int64_t(kLookupGroups) << lanes_log2;
                    const int64_t stretches = (groups + stretch - 1) / stretch;
                    if (ctas > kMaxGridX || stretches > 65535) return cudaErrorInvalidConfiguration;
                    lookup_kernel<td(), od(), id(), VEC>
                        <<<dim3(static_cast<unsigned>(ctas), static_cast<unsigned>(stretches)),
                           kLookupThreads, 0, stream>>>(a, static_cast<int>(groups), lanes_log2);
                    return cudaGetLastError();
                };
                return vec ? go(std::true_type{}) : go(std::false_type{});
            });
        });
    });
}

EmbeddingScratch embedding_scratch_layout(int64_t tokens, int64_t dim) {
    EmbeddingScratch s;
    s.chunks = (tokens + kSortChunk - 1) / kSortChunk;
    s.units = (tokens + kSumUnit - 1) / kSumUnit;
    s.sorted_words = round_up(tokens, 4);
    s.bytes = 4 * (s.sorted_words * (s.chunks > 1 ? 4 : 2) + s.units * 2 * round_up(dim, 4));
    return s;
}

cudaError_t launch_embedding_gradient(const EmbeddingGradArgs &g, fa_itype idt, fa_dtype ddt,
                                      fa_dtype tdt, cudaStream_t stream) {
    const EmbeddingScratch s = embedding_scratch_layout(g.tokens, g.dim);
    uint32_t *keys = static_cast<uint32_t *>(g.scratch), *pos = keys + s.sorted_words;
    uint32_t *chunk_keys = keys, *chunk_pos = pos;
    uint32_t *end = pos + s.sorted_words;
    if (s.chunks > 1) {
        chunk_keys = end;
        chunk_pos = chunk_keys + s.sorted_words;
        end = chunk_pos + s.sorted_words;
    }
    cudaError_t err = cudaSuccess;
    if (g.tokens > 0) {
        SortArgs sa;
        sa.ids = g.ids;
        sa.tokens = g.tokens;
        sa.vocab = g.vocab;
        sa.padding_idx = g.padding_idx;
        sa.keys = chunk_keys;
        sa.pos = chunk_pos;
        sa.bits = 1;
        while (g.vocab >> sa.bits) ++sa.bits;  // vocab itself is a key
        err = for_itype(idt, [&](auto it) {
            auto kernel = sort_chunk_kernel<it()>;
            cudaError_t e = cudaFuncSetAttribute(
                kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSortSmem);
            if (e != cudaSuccess) return e;
            kernel<<<static_cast<unsigned>(s.chunks), kSortThreads, kSortSmem, stream>>>(sa);
            return cudaGetLastError();
        });
        if (err != cudaSuccess) return err;
        if (s.chunks > 1) {
            err = launch_dependent(merge_chunks_kernel,
                                   dim3(static_cast<unsigned>((g.tokens + kMergeThreads - 1) /
                                                              kMergeThreads)),
                                   dim3(kMergeThreads), 0, stream,
                                   static_cast<const uint32_t *>(chunk_keys),
                                   static_cast<const uint32_t *>(chunk_pos), keys, pos, g.tokens,
                                   s.chunks);
            if (err != cudaSuccess) return err;
        }
    }
    SumArgs a;
    a.g = g;
    a.keys = keys;
    a.pos = pos;
    a.partial = reinterpret_cast<float *>(end);
    a.units = s.units;
    a.zero_rows = g.accumulate ? 0 : 64;
    const int64_t zero_ctas = g.accumulate ? 0 : (g.vocab + a.zero_rows - 1) / a.zero_rows;
    const bool vec = vector_rows(g.dout, g.dout_ld, ddt, g.dtable, g.table_ld, tdt, g.dim);
    return for_dtype(ddt, [&](auto dd) {
        return for_dtype(tdt, [&](auto td) {
            const auto go = [&](auto v) {
                constexpr bool VEC = decltype(v)::value;
                constexpr int N = kGroup<dd(), td(), VEC>;
                const unsigned slabs = static_cast<unsigned>(
                    (g.dim / N + (g.dim % N ? 1 : 0) + kSumThreads - 1) / kSumThreads);
                cudaError_t e = launch_dependent(
                    sum_units_kernel<dd(), td(), VEC>,
                    dim3(static_cast<unsigned>(a.units + zero_ctas), slabs), dim3(kSumThreads), 0,
                    stream, a);
                if (e != cudaSuccess || a.units < 2) return e;
                return launch_dependent(join_units_kernel<td(), VEC, dd()>,
                                        dim3(static_cast<unsigned>(a.units - 1), slabs),
                                        dim3(kSumThreads), 0, stream, a);
            };
            return vec ? go(std::true_type{}) : go(std::false_type{});
        });
    });
}

}  // namespace fa
