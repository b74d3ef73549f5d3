// The embedding lookup with scaling and its gradient by sorted tokens.
//
// Gradient of row v: scale * sum over the tokens t with id v of dout[t].  The tokens
// are sorted by id (stable: ascending t within an id), so that each id's rows are one
// run of the sorted order, and the sorted order is cut into units of kSumUnit tokens,
// each added by one CTA in order: the work of a unit does not depend on how the ids
// are distributed.  A run inside one unit is finished there; a run that several units
// share leaves FP32 partial sums, which the join adds in unit order.
//
// Sort: a cluster of up to eight CTAs sorts up to kSortChunk tokens in its shared memory,
// least significant digit first: each warp ranks its tokens by digit, the CTAs exchange
// their digit counts, and every token goes to its place in the cluster, in whichever
// CTA's memory that is.  A chunk's ids are sorted in two or three such passes with no
// global memory between them.  With several chunks, a token's place in the whole order is
// its place in its chunk plus, for every other chunk, the number of its ids that come
// before (ties: earlier chunks come before), found by binary search.
#include <cooperative_groups.h>
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
namespace cg = cooperative_groups;

constexpr int kSortThreads = 1024;
constexpr int kSortWarps = kSortThreads / 32;
constexpr int kSortItems = kSortSlots / kSortThreads;
constexpr int kMostDigits = 512;  // values of a digit: up to nine bits
constexpr int kSumThreads = 256;
constexpr int kMergeThreads = 256;
constexpr int kJoinWarps = 8;

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
    uint32_t *keys, *pos;     // the chunks' sorted ids and token indices
    int passes, digit_bits;   // passes * digit_bits bits hold vocab, the key of a token without an id
};

// Shared memory of a sorting CTA.
struct SortSmem {
    uint32_t key[kSortSlots];
    uint16_t place[kSortSlots];                // the token's index in the chunk
    uint16_t count[kSortWarps][kMostDigits];   // each warp's tokens by digit, then those before it
    uint32_t total[kMostDigits];               // the CTA's tokens by digit
    uint32_t base[kMostDigits];                // where the CTA's first of a digit goes
    uint32_t warp_total[kSortWarps];
};

template <int IT>
__global__ void __launch_bounds__(kSortThreads) sort_chunk_kernel(SortArgs a, unsigned ctas) {
    fa_allow_dependents();
    extern __shared__ uint4 raw[];
    SortSmem &s = *reinterpret_cast<SortSmem *>(raw);
    cg::cluster_group cluster = cg::this_cluster();
    const int t = threadIdx.x, lane = t & 31, warp = t / 32;
    const unsigned rank = blockIdx.x % ctas;
    const int64_t chunk = static_cast<int64_t>(blockIdx.x / ctas) * kSortChunk;
    const int64_t left = a.tokens - chunk;
    const int n = left < kSortChunk ? static_cast<int>(left) : kSortChunk;
    const int digits = 1 << a.digit_bits;
    // a thread's items are 32 apart: a warp's are consecutive, taken in rounds
    const int first = warp * 32 * kSortItems + lane;

    uint32_t key[kSortItems];
    uint16_t place[kSortItems];
#pragma unroll
    for (int j = 0; j < kSortItems; ++j) {
        const int i = static_cast<int>(rank) * kSortSlots + first + 32 * j;
        key[j] = 0xffffffffu;  // past the end: came last, and stays last
        place[j] = static_cast<uint16_t>(i);
        if (i < n && fa_in_bounds(chunk + i, 1, a.tokens)) {
            const int64_t id = load_id<IT>(a.ids, chunk + i);
            key[j] = id >= 0 && id < a.vocab && id != a.padding_idx ? static_cast<uint32_t>(id)
                                                                    : static_cast<uint32_t>(a.vocab);
        }
    }
    for (int pass = 0; pass < a.passes; ++pass) {
        const int shift = pass * a.digit_bits;
        for (int d = lane; d < digits; d += 32) s.count[warp][d] = 0;
        __syncwarp();
        uint16_t before[kSortItems];  // tokens of the digit before this one in the warp
#pragma unroll
        for (int j = 0; j < kSortItems; ++j) {
            const uint32_t d = (key[j] >> shift) & (digits - 1);
            const unsigned same = __match_any_sync(0xffffffffu, d);
            const int ahead = __popc(same & ((1u << lane) - 1));
            const uint16_t c = s.count[warp][d];
            __syncwarp();
            if (ahead == 0) s.count[warp][d] = static_cast<uint16_t>(c + __popc(same));
            __syncwarp();
            before[j] = static_cast<uint16_t>(c + ahead);
        }
        __syncthreads();
        uint32_t mine = 0;
        if (t < digits) {  // thread d: the warps' counts of digit d
            uint16_t c[kSortWarps];
#pragma unroll
            for (int w = 0; w < kSortWarps; ++w) c[w] = s.count[w][t];
#pragma unroll
            for (int w = 0; w < kSortWarps; ++w) {
                s.count[w][t] = static_cast<uint16_t>(mine);
                mine += c[w];
            }
            s.total[t] = mine;
        }
        cluster.sync();
        uint32_t all = 0, earlier = 0;  // tokens of digit d in the cluster, and in earlier CTAs
        if (t < digits)
            for (unsigned r = 0; r < ctas; ++r) {
                const uint32_t c = *cluster.map_shared_rank(&s.total[t], r);
                all += c;
                if (r < rank) earlier += c;
            }
        // tokens of smaller digits: a prefix sum over the threads
        uint32_t upto = all;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const uint32_t x = __shfl_up_sync(0xffffffffu, upto, o);
            if (lane >= o) upto += x;
        }
        if (lane == 31) s.warp_total[warp] = upto;
        __syncthreads();
        if (t < digits) {
            for (int w = 0; w < warp; ++w) upto += s.warp_total[w];
            s.base[t] = upto - all + earlier;
        }
        __syncthreads();
#pragma unroll
        for (int j = 0; j < kSortItems; ++j) {
            const uint32_t d = (key[j] >> shift) & (digits - 1);
            const uint32_t at = s.base[d] + s.count[warp][d] + before[j];  // < ctas * kSortSlots
            if (!fa_in_bounds(at, 1, static_cast<int64_t>(ctas) * kSortSlots)) continue;
            const unsigned r = at / kSortSlots, slot = at % kSortSlots;
            *cluster.map_shared_rank(&s.key[slot], r) = key[j];
            *cluster.map_shared_rank(&s.place[slot], r) = place[j];
        }
        cluster.sync();
#pragma unroll
        for (int j = 0; j < kSortItems; ++j) {
            key[j] = s.key[first + 32 * j];
            place[j] = s.place[first + 32 * j];
        }
    }
#pragma unroll
    for (int j = 0; j < kSortItems; ++j) {
        const int i = static_cast<int>(rank) * kSortSlots + first + 32 * j;
        if (i >= n || !fa_in_bounds(chunk + i, 1, a.tokens)) continue;
        a.keys[chunk + i] = key[j];
        a.pos[chunk + i] = static_cast<uint32_t>(chunk + place[j]);
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
    int64_t zero_ctas;           // CTAs that zero the rows of absent ids, kZeroRows each
};
constexpr int kZeroRows = 32;

// Writes ``sum * scale`` to (or adds it to) elements [c, c + N) of table row v.
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

// N FP32 partial sums, 16 bytes at a time where N fills them (rows of dim floats are
// 16-byte aligned then).
template <int N>
__device__ __forceinline__ void store_partial(float *p, const float *x) {
    if constexpr (N % 4 == 0) {
#pragma unroll
        for (int j = 0; j < N; j += 4)
            *reinterpret_cast<float4 *>(p + j) = make_float4(x[j], x[j + 1], x[j + 2], x[j + 3]);
    } else {
#pragma unroll
        for (int j = 0; j < N; ++j) p[j] = x[j];
    }
}
template <int N>
__device__ __forceinline__ void load_partial(const float *p, float *x) {
    if constexpr (N % 4 == 0) {
#pragma unroll
        for (int j = 0; j < N; j += 4) {
            const float4 f = *reinterpret_cast<const float4 *>(p + j);
            x[j] = f.x;
            x[j + 1] = f.y;
            x[j + 2] = f.z;
            x[j + 3] = f.w;
        }
    } else {
#pragma unroll
        for (int j = 0; j < N; ++j) x[j] = p[j];
    }
}

// The rows [v0, v0 + kZeroRows) of ids that no token has.
template <int TT, int N>
__device__ __forceinline__ void zero_absent(const SumArgs &a, int64_t v0, int64_t c) {
    const EmbeddingGradArgs &g = a.g;
    __shared__ bool absent[kZeroRows];
    if (threadIdx.x < kZeroRows) {
        const int64_t v = v0 + threadIdx.x;
        bool none = false;
        if (v < g.vocab) {
            const int64_t at = bound(a.keys, g.tokens, static_cast<uint32_t>(v), false);
            none = at >= g.tokens || a.keys[at] != v;
        }
        absent[threadIdx.x] = none;
    }
    __syncthreads();
    if (c >= g.dim || !fa_in_bounds(c, N, g.dim)) return;
    float zero[N];
#pragma unroll
    for (int j = 0; j < N; ++j) zero[j] = 0.f;
    for (int r = 0; r < kZeroRows; ++r)
        if (absent[r] && fa_in_bounds(v0 + r, 1, g.vocab))
            store_n<TT, N>(
                static_cast<typename Elem<TT>::T *>(g.dtable) + (v0 + r) * g.table_ld + c, zero);
}

// CTA (u, slab): unit u's tokens, columns of slab.  A run that began before the unit
// leaves its sum in partial[u][0], one that goes on after it in partial[u][1] (a run
// that does both, in [0]).  The zeroing CTAs lie between the adding ones, so that their
// searches wait beside loads.
template <int DT, int TT, bool VEC>
__global__ void __launch_bounds__(kSumThreads, 4) sum_units_kernel(SumArgs a) {
    constexpr int N = kGroup<DT, TT, VEC>;
    constexpr int kAhead = 8;  // rows in flight
    using DE = typename Elem<DT>::T;
    const EmbeddingGradArgs &g = a.g;
    fa_grid_dependency_wait();
    fa_allow_dependents();
    const int64_t c = (static_cast<int64_t>(blockIdx.y) * blockDim.x + threadIdx.x) * N;
    const int64_t both = 2 * min(a.units, a.zero_ctas);
    int64_t u = blockIdx.x;
    if (u < both ? (u & 1) : a.zero_ctas > a.units) {
        zero_absent<TT, N>(a, (u < both ? u / 2 : u - a.units) * kZeroRows, c);
        return;
    }
    u = u < both ? u / 2 : u - a.zero_ctas;
    __shared__ uint32_t key[kSumUnit];
    __shared__ uint32_t pos[kSumUnit];
    __shared__ uint32_t ends, bounds;  // bit i: token i is its run's last here; began before, goes on
    const int64_t first = u * kSumUnit;
    if (threadIdx.x < 32) {
        const int lane = threadIdx.x;
        const int64_t at = first + lane;
        const uint32_t none = 0xffffffffu;  // no id has it: ids are below 2^31
        const uint32_t k = at < g.tokens ? a.keys[at] : none;
        pos[lane] = at < g.tokens ? a.pos[at] : 0u;
        key[lane] = k < g.vocab ? k : none;
        uint32_t next = __shfl_down_sync(0xffffffffu, k, 1);
        if (lane == 31) next = at + 1 < g.tokens ? a.keys[at + 1] : none;
        const uint32_t e = __ballot_sync(0xffffffffu, next != k || lane == 31);
        if (lane == 0) {
            ends = e;
            bounds = first > 0 && a.keys[first - 1] == k ? 1u : 0u;
        }
        __syncwarp();
        if (lane == 31 && next == k) bounds |= 2u;
    }
    __syncthreads();
    if (c >= g.dim) return;
    const DE *dout = static_cast<const DE *>(g.dout) + c;
    const uint32_t last = ends;
    bool began_before = bounds & 1u;
    const bool goes_on = bounds & 2u;
    float sum[N];
#pragma unroll
    for (int j = 0; j < N; ++j) sum[j] = 0.f;
#pragma unroll 1
    for (int i0 = 0; i0 < kSumUnit; i0 += kAhead) {
        Raw<DT, N> rows[kAhead];
#pragma unroll
        for (int k = 0; k < kAhead; ++k)
            if (key[i0 + k] != 0xffffffffu && fa_in_bounds(c, N, g.dim) &&
                fa_in_bounds(pos[i0 + k], 1, g.tokens))
                rows[k].load(dout + static_cast<int64_t>(pos[i0 + k]) * g.dout_ld);
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
            const int i = i0 + k;
            const uint32_t v = key[i];
            if (v == 0xffffffffu) return;  // tokens without an id come last
            float x[N];
            rows[k].widen(x);
#pragma unroll
            for (int j = 0; j < N; ++j) sum[j] += x[j];
            if (!(last >> i & 1u)) continue;
            const bool on = i == kSumUnit - 1 && goes_on;
            if (began_before || on)
                store_partial<N>(a.partial + (2 * u + (began_before ? 0 : 1)) * g.dim + c, sum);
            else
                finish_row<TT, N>(g, v, c, sum);
            began_before = false;
#pragma unroll
            for (int j = 0; j < N; ++j) sum[j] = 0.f;
        }
    }
}

// Runs that several units share.  A warp looks after one unit, for the columns of slab: if
// the unit began a run that goes on, it adds the run's partial sums in unit order.  Runs of
// more than kLong units are taken by the CTA's warps together, each a stretch of them, and
// the stretches' sums are added in order.
constexpr int kLong = 16;
template <int DT, int TT, bool VEC>
__global__ void __launch_bounds__(kJoinWarps * 32) join_units_kernel(SumArgs a) {
    constexpr int N = kGroup<DT, TT, VEC>;
    const EmbeddingGradArgs &g = a.g;
    __shared__ int64_t last_unit[kJoinWarps];  // of the run that the warp's unit began (0: none)
    __shared__ float stretch[kJoinWarps][32 * N];
    const int warp = threadIdx.x / 32, lane = threadIdx.x & 31;
    const int64_t u0 = static_cast<int64_t>(blockIdx.x) * kJoinWarps;
    const int64_t c = (static_cast<int64_t>(blockIdx.y) * 32 + lane) * N;
    fa_grid_dependency_wait();
    fa_allow_dependents();
    int64_t end = 0;
    {
        const int64_t u = u0 + warp, first = u * kSumUnit, last = first + kSumUnit - 1;
        if (last + 1 < g.tokens) {
            const uint32_t key = a.keys[last];
            if (key < g.vocab && a.keys[last + 1] == key &&
                !(first > 0 && a.keys[first] == key && a.keys[first - 1] == key)) {
                // the run's end: steps of growing length, then a search within the last
                int64_t lo = last + 1, step = kSumUnit;
                while (lo + step < g.tokens && a.keys[lo + step] == key) {
                    lo += step;
                    step *= 2;
                }
                const int64_t room = min(step, g.tokens - lo);
                end = (lo + bound(a.keys + lo, room, key, true) - 1) / kSumUnit;
            }
        }
        if (lane == 0) last_unit[warp] = end;
    }
    __syncthreads();
    const bool here = c < g.dim;
    // partials of units [w0, w1], added onto sum in order
    const auto add = [&](float *sum, int64_t w0, int64_t w1) {
#pragma unroll 8
        for (int64_t w = w0; w <= w1; ++w) {
            float x[N];
            if (!fa_in_bounds(w, 1, a.units)) break;
            load_partial<N>(a.partial + 2 * w * g.dim + c, x);
#pragma unroll
            for (int j = 0; j < N; ++j) sum[j] += x[j];
        }
    };
    const int64_t mine = u0 + warp;
    if (end && end - mine <= kLong && here) {
        float sum[N];
        load_partial<N>(a.partial + (2 * mine + 1) * g.dim + c, sum);
        add(sum, mine + 1, end);
        finish_row<TT, N>(g, a.keys[(mine + 1) * kSumUnit], c, sum);
    }
    for (int k = 0; k < kJoinWarps; ++k) {
        const int64_t u = u0 + k, units = last_unit[k] - u;
        if (!last_unit[k] || units <= kLong) continue;  // the same for the whole CTA
        const int64_t each = (units + kJoinWarps - 1) / kJoinWarps;
        float sum[N];
#pragma unroll
        for (int j = 0; j < N; ++j) sum[j] = 0.f;
        if (here) {
            if (warp == 0) load_partial<N>(a.partial + (2 * u + 1) * g.dim + c, sum);
            add(sum, u + 1 + warp * each, min(u + (warp + 1) * each, last_unit[k]));
        }
#pragma unroll
        for (int j = 0; j < N; ++j) stretch[warp][j * 32 + lane] = sum[j];
        __syncthreads();
        if (warp == 0 && here) {
            for (int w = 1; w < kJoinWarps; ++w)
#pragma unroll
                for (int j = 0; j < N; ++j) sum[j] += stretch[w][j * 32 + lane];
            finish_row<TT, N>(g, a.keys[(u + 1) * kSumUnit], c, sum);
        }
        __syncthreads();
    }
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
    if (g.tokens > 0) {
        SortArgs sa;
        sa.ids = g.ids;
        sa.tokens = g.tokens;
        sa.vocab = g.vocab;
        sa.padding_idx = g.padding_idx;
        sa.keys = chunk_keys;
        sa.pos = chunk_pos;
        int bits = 1;
        while (g.vocab >> bits) ++bits;  // vocab itself is a key
        sa.passes = (bits + 8) / 9;
        sa.digit_bits = (bits + sa.passes - 1) / sa.passes;
        const unsigned ctas =
            s.chunks > 1 ? kSortChunk / kSortSlots
                         : static_cast<unsigned>((g.tokens + kSortSlots - 1) / kSortSlots);
        cudaError_t err = for_itype(idt, [&](auto it) {
            auto kernel = sort_chunk_kernel<it()>;
            constexpr int kSmem = sizeof(SortSmem);
            cudaError_t e = cudaFuncSetAttribute(
                kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
            if (e != cudaSuccess) return e;
            return launch_clusters(kernel, dim3(static_cast<unsigned>(s.chunks) * ctas),
                                   dim3(kSortThreads), kSmem, ctas, false, stream, sa, ctas);
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
    a.zero_ctas = g.accumulate ? 0 : (g.vocab + kZeroRows - 1) / kZeroRows;
    const bool vec = vector_rows(g.dout, g.dout_ld, ddt, g.dtable, g.table_ld, tdt, g.dim);
    return for_dtype(ddt, [&](auto dd) {
        return for_dtype(tdt, [&](auto td) {
            const auto go = [&](auto v) {
                constexpr bool VEC = decltype(v)::value;
                constexpr int N = kGroup<dd(), td(), VEC>;
                const int64_t groups = (g.dim + N - 1) / N;
                const int threads = static_cast<int>(
                    groups < kSumThreads ? round_up(groups, 32) : kSumThreads);
                const int64_t slabs = (groups + threads - 1) / threads;
                cudaError_t e = launch_dependent(
                    sum_units_kernel<dd(), td(), VEC>,
                    dim3(static_cast<unsigned>(a.units + a.zero_ctas),
                         static_cast<unsigned>(slabs)),
                    dim3(threads), 0, stream, a);
                if (e != cudaSuccess || a.units < 2) return e;
                return launch_dependent(
                    join_units_kernel<dd(), td(), VEC>,
                    dim3(static_cast<unsigned>((a.units - 1 + kJoinWarps - 1) / kJoinWarps),
                         static_cast<unsigned>((groups + 31) / 32)),
                    dim3(kJoinWarps * 32), 0, stream, a);
            };
            return vec ? go(std::true_type{}) : go(std::false_type{});
        });
    });
}

}  // namespace fa
