// The embedding lookup with scaling and its gradient by sorted tokens.
//
// Gradient of row v: scale * sum over the tokens t with id v of dout[t].  The tokens
// are sorted by id (stable: ascending t within an id), so that each id's rows are one
// run of the sorted order, and the sorted order is cut into units of kSumUnit tokens,
// one CTA each.  A run of at most kSumUnit tokens is added by the unit it begins in, past
// that unit's end if need be; a longer one is cut where the units are, and their FP32
// partial sums are added in unit order by the join.  So the work of a unit is at most twice
// another's however the ids are distributed, and only long runs pay for partial sums.
//
// Sort: a cluster of up to sixteen CTAs sorts up to kSortChunk tokens in its shared memory,
// least significant digit first: each warp ranks its tokens by digit, the CTAs exchange
// their digit counts, each CTA orders its own by digit, and the runs so made go to their
// places in the cluster, in whichever CTA's memory that is (sent token by token, each to
// a place of its own, a pass took 18 us).  A chunk's ids are sorted in two or three such passes with no
// global memory between them; the rest of the GPU zeroes the table meanwhile.  With several
// chunks, a token's place in the whole order is
// its place in its chunk plus, for every other chunk, the number of its ids that come
// before (ties: earlier chunks come before), found by binary search.
#include <algorithm>

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

namespace cg = cooperative_groups;

constexpr int kLookupThreads = 256;
constexpr int kLookupGroups = 4;  // 16-byte groups a lane has in flight

constexpr int kSortThreads = 1024;
constexpr int kSortWarps = kSortThreads / 32;
constexpr int kSortItems = kSortSlots / kSortThreads;
constexpr int kMostDigitBits = 9;
constexpr int kMostDigits = 1 << kMostDigitBits;
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
// loads are in flight together once its id is there.  Rows aligned for whole groups.  The
// writes bound it, and the reads of the rows that occur: 65536 tokens of 2048 BF16 from a table
// of 131 MB take 53 us, 6.1 TB/s of both (the table's 55 MB that L2 does not hold are read once).
template <int TT, int OT, int IT>
__global__ void __launch_bounds__(kLookupThreads)
lookup_kernel(LookupArgs a, int groups, int lanes_log2) {
    constexpr int N = kGroup<TT, OT, true>;
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

// The same for rows that begin anywhere: groups begin at the output's 16-byte lines, wherever
// their elements lie in the table's; what is left of a row before and after them goes
// element by element, an element a lane (65536 rows of 2047 BF16: 78 us; 154 us with single
// elements throughout).
template <int TT, int OT, int IT>
__global__ void __launch_bounds__(kLookupThreads) lookup_any_kernel(LookupArgs a, int lanes_log2) {
    constexpr int N = kGroup<TT, OT, true>, kGroups = 2;
    using TE = typename Elem<TT>::T;
    using OE = typename Elem<OT>::T;
    const int64_t thread = static_cast<int64_t>(blockIdx.x) * kLookupThreads + threadIdx.x;
    const int64_t t = thread >> lanes_log2;
    if (t >= a.tokens) return;
    const int lanes = 1 << lanes_log2, lane = threadIdx.x & (lanes - 1);
    const int dim = static_cast<int>(a.dim);
    const int64_t id = load_id<IT>(a.ids, t);
    const bool known = id >= 0 && id < a.vocab;
    const TE *row = static_cast<const TE *>(a.table) + (known ? id : 0) * a.table_ld;
    OE *out = static_cast<OE *>(a.out) + t * a.out_ld;
    const Span table(a.table, ((a.vocab - 1) * a.table_ld + a.dim) * sizeof(TE));
    const int past = static_cast<int>(reinterpret_cast<uintptr_t>(out) & 15);
    const int head = min(dim, past ? (16 - past) / static_cast<int>(sizeof(OE)) : 0);
    const int groups = (dim - head) / N, tail = head + groups * N;
    if (blockIdx.y == 0)
        for (int i = lane; i < head + dim - tail; i += lanes) {
            const int e = i < head ? i : i - head + tail;
            if (fa_in_bounds(e, 1, dim))
                out[e] = Elem<OT>::round(known ? Elem<TT>::widen(row[e]) * a.scale : 0.f);
        }
    const int g0 = (blockIdx.y * kGroups << lanes_log2) + lane;
    RawAny<TT, N> x[kGroups];
#pragma unroll
    for (int k = 0; k < kGroups; ++k) {
        const int g = g0 + k * lanes;
        if (known && g < groups && fa_in_bounds(head + g * N, N, dim))
            x[k].load(row + head + g * N, N, table);
    }
#pragma unroll
    for (int k = 0; k < kGroups; ++k) {
        const int g = g0 + k * lanes;
        if (g >= groups || !fa_in_bounds(head + g * N, N, dim)) break;
        float y[N];
        x[k].widen(y);
#pragma unroll
        for (int j = 0; j < N; ++j) y[j] = known ? y[j] * a.scale : 0.f;
        store_n<OT, N>(out + head + g * N, y);
    }
}

// ---- sort ----------------------------------------------------------------------

// What is zeroed of the table while its gradient's tokens are sorted: rows of ``bytes`` bytes
// from p, ld bytes apart; with claims, only the rows of ids that no token has.
struct ZeroArgs {
    char *p;
    int64_t rows, bytes, ld;
    const uint32_t *claims;  // [rows], or nullptr
};

// claims[id] = a token that has the id, whichever comes last.  Entries of other ids hold
// anything: a token that does not have the id shows that the entry is none.
template <int IT>
__global__ void __launch_bounds__(256)
claim_kernel(const void *ids, uint32_t *claims, int64_t tokens, int64_t vocab, int64_t padding_idx) {
    fa_allow_dependents();
    const int64_t t = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
    if (t >= tokens) return;
    const int64_t id = load_id<IT>(ids, t);
    if (id >= 0 && id < vocab && id != padding_idx && fa_in_bounds(id, 1, vocab))
        claims[id] = static_cast<uint32_t>(t);
}

// ``bytes`` zeros from p (two-byte aligned) by ``count`` threads, of which this is ``rank``.
__device__ __forceinline__ void zero_bytes(char *p, int64_t bytes, int64_t rank, int64_t count) {
    const int64_t past = reinterpret_cast<uintptr_t>(p) & 15;
    const int64_t head = past ? min(int64_t(16) - past, bytes) : 0;
    const int64_t vecs = (bytes - head) / 16, tail = head + vecs * 16;
    if (2 * rank < head) *reinterpret_cast<uint16_t *>(p + 2 * rank) = 0;
    if (tail + 2 * rank < bytes) *reinterpret_cast<uint16_t *>(p + tail + 2 * rank) = 0;
    uint4 *q = reinterpret_cast<uint4 *>(p + head);
    for (int64_t i = rank; i < vecs; i += count)
        if (fa_in_bounds(i, 1, vecs)) __stcs(q + i, make_uint4(0u, 0u, 0u, 0u));
}

// The share of CTA ``cta`` of ``ctas``.
template <int IT>
__device__ __forceinline__ void zero_rows(const ZeroArgs &z, const void *ids, int64_t tokens,
                                          int64_t padding_idx, int64_t cta, int64_t ctas) {
    if (z.rows == 1) {
        zero_bytes(z.p, z.bytes, cta * kSortThreads + threadIdx.x, ctas * kSortThreads);
        return;
    }
    // a warp takes kRows rows at a time; lane r asks whether row r has a token
    constexpr int kRows = 4;
    const int lane = threadIdx.x & 31;
    const int64_t warps = ctas * kSortWarps, warp = cta * kSortWarps + threadIdx.x / 32;
    for (int64_t v0 = warp * kRows; v0 < z.rows; v0 += warps * kRows) {
        bool absent = lane < kRows && v0 + lane < z.rows;
        if (z.claims && absent) {
            const uint32_t t = z.claims[v0 + lane];
            absent = t >= tokens || load_id<IT>(ids, t) != v0 + lane || v0 + lane == padding_idx;
        }
        const unsigned rows = __ballot_sync(0xffffffffu, absent);
        for (int r = 0; r < kRows; ++r)
            if (rows >> r & 1u) zero_bytes(z.p + (v0 + r) * z.ld, z.bytes, lane, 32);
    }
}

// Rows that are asked into L2 while the tokens are sorted: the sums read them next.
struct PrefetchArgs {
    const char *p;
    int64_t rows, bytes, ld;
};
__device__ __forceinline__ void prefetch_rows(const PrefetchArgs &f, int64_t cta, int64_t ctas) {
    const int lane = threadIdx.x & 31;
    const int64_t warps = ctas * kSortWarps, warp = cta * kSortWarps + threadIdx.x / 32;
    for (int64_t r = warp; r < f.rows; r += warps) {
        const char *row = f.p + r * f.ld;
        for (int64_t i = lane * 128; i < f.bytes; i += 32 * 128)
            asm volatile("prefetch.global.L2 [%0];" ::"l"(row + i));
    }
}

struct SortArgs {
    const void *ids;
    int64_t tokens, vocab, padding_idx;
    uint32_t *keys, *pos;     // the chunks' sorted ids and token indices
    int passes, digit_bits;   // passes * digit_bits bits hold vocab, the key of a token without an id
    unsigned chunks, ctas;    // clusters that sort, and the CTAs of a cluster
    ZeroArgs zero;
    PrefetchArgs prefetch;
    uint32_t *long_runs;      // their number, zeroed here
};

// A token on its way: its id above its index in the chunk.
template <typename Item>
struct SortSmem {
    Item item[kSortSlots];
    Item own[kSortSlots];                      // the CTA's, by digit
    uint16_t count[kSortWarps][kMostDigits];   // each warp's tokens by digit, then their places
    uint32_t total[kMostDigits];               // the CTA's tokens by digit
    int base[kMostDigits];                     // from a place among its own to one in the chunk
    uint32_t warp_total[2][kSortWarps];
};

// The first chunks' clusters sort; the CTAs after them zero the table meanwhile.  Latency
// bounds the sort, not its 0.8 MB: barriers of the cluster, ballots, prefix sums (65536 tokens
// and 32000 ids, two digits: 18.5 us; 4096 tokens: 12.3; 333: 8.3).
template <int IT, typename Item>
__global__ void __launch_bounds__(kSortThreads) sort_chunk_kernel(SortArgs a) {
    fa_allow_dependents();
    if (blockIdx.x >= a.chunks * a.ctas) {
        const int64_t cta = blockIdx.x - a.chunks * a.ctas, ctas = gridDim.x - a.chunks * a.ctas;
        if (a.zero.rows) {
            fa_grid_dependency_wait();  // the claims
            zero_rows<IT>(a.zero, a.ids, a.tokens, a.padding_idx, cta, ctas);
        }
        prefetch_rows(a.prefetch, cta, ctas);
        return;
    }
    if (blockIdx.x == 0 && threadIdx.x == 0) *a.long_runs = 0;
    extern __shared__ uint4 raw[];
    SortSmem<Item> &s = *reinterpret_cast<SortSmem<Item> *>(raw);
    cg::cluster_group cluster = cg::this_cluster();
    const int t = threadIdx.x, lane = t & 31, warp = t / 32;
    const unsigned rank = blockIdx.x % a.ctas;
    const int64_t chunk = static_cast<int64_t>(blockIdx.x / a.ctas) * kSortChunk;
    const int64_t left = a.tokens - chunk;
    const int n = left < kSortChunk ? static_cast<int>(left) : kSortChunk;
    const int digits = 1 << a.digit_bits;
    // a thread's items are 32 apart: a warp's are consecutive, taken in rounds
    const int first = warp * 32 * kSortItems + lane;
    const auto finish = [&](int i, Item x) {  // the i-th of the sorted chunk
        if (!fa_in_bounds(chunk + i, 1, a.tokens)) return;
        a.keys[chunk + i] = static_cast<uint32_t>(x >> 16);
        a.pos[chunk + i] = static_cast<uint32_t>(chunk + static_cast<uint16_t>(x));
    };

    Item item[kSortItems];
#pragma unroll
    for (int j = 0; j < kSortItems; ++j) {
        const int i = static_cast<int>(rank) * kSortSlots + first + 32 * j;
        item[j] = 0;
        if (i < n && fa_in_bounds(chunk + i, 1, a.tokens)) {
            const int64_t id = load_id<IT>(a.ids, chunk + i);
            const bool known = id >= 0 && id < a.vocab && id != a.padding_idx;
            item[j] = static_cast<Item>(known ? id : a.vocab) << 16 | static_cast<Item>(i);
        }
    }
    // places from n on stay empty: a CTA's tokens are its first ``held``, in every pass
    const int held = min(max(n - static_cast<int>(rank) * kSortSlots, 0), kSortSlots);
    for (int pass = 0; pass < a.passes; ++pass) {
        const int shift = 16 + pass * a.digit_bits;
        const auto digit = [&](Item x) { return static_cast<int>(x >> shift) & (digits - 1); };
        for (int d = 2 * lane; d < digits; d += 64)
            *reinterpret_cast<uint32_t *>(&s.count[warp][d]) = 0u;
        __syncwarp();
        uint16_t before[kSortItems];  // tokens of the digit before this one in the warp
#pragma unroll
        for (int j = 0; j < kSortItems; ++j) {
            if (warp * 32 * kSortItems + 32 * j >= held) break;  // the whole warp
            const int d = digit(item[j]);
            const bool in = first + 32 * j < held;
            // the lanes with this digit, from a ballot of each of its bits (with match.any a
            // sort of 4096 tokens took 2 us more)
            unsigned same = __ballot_sync(0xffffffffu, in);
#pragma unroll
            for (int b = 0; b < kMostDigitBits; ++b) {
                const bool bit = d >> b & 1;
                const unsigned set = __ballot_sync(0xffffffffu, bit);
                same &= bit ? set : ~set;
            }
            const int ahead = __popc(same & ((1u << lane) - 1));
            const uint16_t c = s.count[warp][d];
            __syncwarp();
            if (in && ahead == 0) s.count[warp][d] = static_cast<uint16_t>(c + __popc(same));
            __syncwarp();
            before[j] = static_cast<uint16_t>(c + ahead);
        }
        __syncthreads();
        uint32_t mine = 0;  // thread d: the CTA's tokens of digit d
        uint16_t c[kSortWarps];
        if (t < digits) {
#pragma unroll
            for (int w = 0; w < kSortWarps; ++w) mine += c[w] = s.count[w][t];
            s.total[t] = mine;
        }
        cluster.sync();
        uint32_t all = 0, earlier = 0;  // tokens of digit d in the cluster, and in earlier CTAs
        if (t < digits)
            for (unsigned r = 0; r < a.ctas; ++r) {
                const uint32_t x = *cluster.map_shared_rank(&s.total[t], r);
                all += x;
                if (r < rank) earlier += x;
            }
        // tokens of smaller digits, in the cluster and of its own: prefix sums over the threads
        uint32_t upto = all, own_upto = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const uint32_t x = __shfl_up_sync(0xffffffffu, upto, o);
            const uint32_t y = __shfl_up_sync(0xffffffffu, own_upto, o);
            if (lane >= o) {
                upto += x;
                own_upto += y;
            }
        }
        if (lane == 31) {
            s.warp_total[0][warp] = upto;
            s.warp_total[1][warp] = own_upto;
        }
        __syncthreads();
        if (t < digits) {
            for (int w = 0; w < warp; ++w) {
                upto += s.warp_total[0][w];
                own_upto += s.warp_total[1][w];
            }
            uint32_t own = own_upto - mine;
            s.base[t] = static_cast<int>(upto - all + earlier) - static_cast<int>(own);
#pragma unroll
            for (int w = 0; w < kSortWarps; ++w) {
                s.count[w][t] = static_cast<uint16_t>(own);
                own += c[w];
            }
        }
        __syncthreads();
#pragma unroll
        for (int j = 0; j < kSortItems; ++j) {
            if (first + 32 * j >= held) continue;
            const int at = s.count[warp][digit(item[j])] + before[j];
            if (fa_in_bounds(at, 1, kSortSlots)) s.own[at] = item[j];
        }
        __syncthreads();
        const bool last = pass == a.passes - 1;
#pragma unroll
        for (int j = 0; j < kSortItems; ++j) {
            const int i = t + j * kSortThreads;
            if (i >= held) break;
            const Item x = s.own[i];
            const int at = s.base[digit(x)] + i;  // < n
            if (!fa_in_bounds(at, 1, static_cast<int64_t>(a.ctas) * kSortSlots)) continue;
            if (last)
                finish(at, x);
            else
                *cluster.map_shared_rank(&s.item[at % kSortSlots],
                                         static_cast<unsigned>(at) / kSortSlots) = x;
        }
        // the next pass's items have come; after the last, no CTA still reads another's counts
        cluster.sync();
        if (last) break;
#pragma unroll
        for (int j = 0; j < kSortItems; ++j) item[j] = s.item[first + 32 * j];
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

// A run of more than kSumUnit tokens that several units share: its first and last unit.
struct LongRun {
    uint32_t first, last, key;
};

struct SumArgs {
    EmbeddingGradArgs g;
    const uint32_t *keys, *pos;  // sorted
    uint32_t *long_runs;         // how many there are,
    LongRun *runs;               // and which, in any order
    float *partial;              // [units][2][dim]
    int64_t units;
};

// Elements [c, c + N) of table row v.
template <int TT>
__device__ __forceinline__ typename Elem<TT>::T *table_row(const EmbeddingGradArgs &g, int64_t v,
                                                           int64_t c) {
    return static_cast<typename Elem<TT>::T *>(g.dtable) + v * g.table_ld + c;
}

// Writes ``sum * scale`` to elements [c, c + N) of table row v, or with ACC adds it to what
// they were.
template <int TT, int N, bool ACC>
__device__ __forceinline__ void finish_row(const EmbeddingGradArgs &g, int64_t v, int64_t c,
                                           const float *sum, const Raw<TT, N> &before) {
    if (!fa_in_bounds(v, 1, g.vocab) || !fa_in_bounds(c, N, g.dim)) return;
    typename Elem<TT>::T *row = table_row<TT>(g, v, c);
    float y[N];
    if (ACC) {
        before.widen(y);
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

// The last token of the run of ``key`` that goes through token ``from``, by a warp: the lanes
// probe further and further ahead, then the stretch that the end is in, 31 points at a time.
__device__ __forceinline__ int64_t run_end(const uint32_t *keys, int64_t tokens, int64_t from,
                                           uint32_t key, int lane) {
    const auto same = [&](int64_t i) { return i < tokens && keys[i] == key; };
    int64_t lo = from, hi = from + (int64_t(1) << 31);  // same(lo), not same(hi)
    const unsigned far = __ballot_sync(0xffffffffu, same(from + (int64_t(1) << lane)));
    const int k = far == 0xffffffffu ? 32 : __ffs(~far) - 1;
    if (k < 32) hi = from + (int64_t(1) << k);
    if (k > 0) lo = from + (int64_t(1) << (k - 1));
    while (hi - lo > 1) {
        const int64_t step = (hi - lo + 31) / 32;
        const unsigned on = __ballot_sync(0xffffffffu, lo + (lane + 1) * step < hi &&
                                                           same(lo + (lane + 1) * step));
        const int n = __popc(on);  // the run is sorted: a prefix of the points
        hi = min(hi, lo + (n + 1) * step);
        lo += n * step;
    }
    return lo;
}

// Bound by its reads and writes: 65536 rows of 2048 BF16 with Zipf-distributed ids, summed into
// the 13100 rows that occur, take 53 us: 332 MB with the partial sums, 6.3 TB/s, with up to six
// rows' loads of a thread in flight.
// CTA (u, slab): unit u's runs, columns of slab.  A long run that began before the unit
// leaves its sum in partial[u][0], one that goes on after it in partial[u][1] (a run
// that does both, in [0]).
template <int DT, int TT, bool VEC, bool ACC>
__global__ void __launch_bounds__(kSumThreads, ACC ? 4 : 5) sum_units_kernel(SumArgs a) {
    // rows a thread has in flight, of dout and the table: more of single elements
    constexpr int kSumAhead = VEC ? (ACC ? 4 : 6) : 16;
    constexpr int N = kGroup<DT, TT, VEC>;
    constexpr uint32_t kNone = 0xffffffffu;  // no id: ids are below 2^31
    using DE = typename Elem<DT>::T;
    const EmbeddingGradArgs &g = a.g;
    fa_grid_dependency_wait();
    fa_allow_dependents();
    const int64_t c = (static_cast<int64_t>(blockIdx.y) * blockDim.x + threadIdx.x) * N;
    const int64_t u = blockIdx.x, first = u * kSumUnit;
    __shared__ uint32_t key[2 * kSumUnit], pos[2 * kSumUnit];
    __shared__ uint64_t ends;         // bit i: token i is its run's last here
    __shared__ int begin, end;        // the tokens to add
    __shared__ int head_end, tail;    // where a long head ends; the token that leaves a long run
    static_assert(kSumUnit == 32, "a warp holds a unit");
    if (threadIdx.x < 32) {
        constexpr unsigned kAll = 0xffffffffu;
        const int lane = threadIdx.x;
        const auto key_at = [&](int64_t i) {
            const uint32_t k = i >= 0 && i < g.tokens ? a.keys[i] : kNone;
            return k < g.vocab ? k : kNone;
        };
        const uint32_t prev = key_at(first - 32 + lane), own = key_at(first + lane),
                       next = key_at(first + 32 + lane);
        const uint32_t own_pos = first + lane < g.tokens ? a.pos[first + lane] : 0u;
        const uint32_t next_pos = first + 32 + lane < g.tokens ? a.pos[first + 32 + lane] : 0u;
        key[lane] = own;
        key[32 + lane] = next;
        pos[lane] = own_pos;
        pos[32 + lane] = next_pos;
        const uint32_t h = __shfl_sync(kAll, own, 0), t = __shfl_sync(kAll, own, 31);
        // tokens of the first run before, in and after the unit; of the last run in and after it
        const auto from_low = [](unsigned same) { return same == kAll ? 32 : __ffs(~same) - 1; };
        const int h_before = __clz(~__ballot_sync(kAll, prev == h));
        const int h_in = from_low(__ballot_sync(kAll, own == h));
        const int t_in = __clz(~__ballot_sync(kAll, own == t));
        const int t_after = from_low(__ballot_sync(kAll, next == t));
        const bool in = h != kNone && h_before > 0, on = t != kNone && t_after > 0;
        const bool h_long = in && h_before + h_in + (h_in == 32 ? t_after : 0) > 32;
        const bool t_long = on && (t_in == 32 ? h_before : 0) + t_in + t_after > 32;
        const int valid = __popc(__ballot_sync(kAll, own != kNone));
        const int to = on && !t_long ? 32 + t_after : valid;
        uint32_t after = __shfl_down_sync(kAll, own, 1);
        const uint32_t next0 = __shfl_sync(kAll, next, 0);
        const uint32_t after_next = __shfl_down_sync(kAll, next, 1);
        if (lane == 31) after = to > 32 ? next0 : kNone;
        const uint64_t e = __ballot_sync(kAll, own != after) |
                           static_cast<uint64_t>(
                               __ballot_sync(kAll, next != after_next || lane == 31)) << 32;
        if (lane == 0) {
            ends = e;
            begin = in && !h_long ? h_in : 0;  // a short run is the unit's before
            end = to;
            head_end = h_long ? h_in : 0;
            tail = t_long ? 31 : -1;
        }
        if (blockIdx.y == 0 && t_long && !(in && t_in == 32)) {  // begins here, and goes on
            const int64_t last = run_end(a.keys, g.tokens, first + 32, t, lane);
            if (lane == 0) {
                const uint32_t k = atomicAdd(a.long_runs, 1u);
                if (fa_in_bounds(k, 1, a.units))
                    a.runs[k] = LongRun{static_cast<uint32_t>(u),
                                        static_cast<uint32_t>(last / kSumUnit), t};
            }
        }
    }
    __syncthreads();
    if (c >= g.dim) return;
    const DE *dout = static_cast<const DE *>(g.dout) + c;
    const uint64_t last = ends;
    const int to = end;
    float sum[N];
#pragma unroll
    for (int j = 0; j < N; ++j) sum[j] = 0.f;
#pragma unroll 1
    for (int i0 = begin; i0 < to; i0 += kSumAhead) {
        Raw<DT, N> rows[kSumAhead];
        Raw<TT, N> before[ACC ? kSumAhead : 1];  // the table's rows of the runs that end here
#pragma unroll
        for (int k = 0; k < kSumAhead; ++k)
            if (i0 + k < to && fa_in_bounds(c, N, g.dim) && fa_in_bounds(pos[i0 + k], 1, g.tokens)) {
                rows[k].load(dout + static_cast<int64_t>(pos[i0 + k]) * g.dout_ld);
                if (ACC && (last >> (i0 + k) & 1u) && fa_in_bounds(key[i0 + k], 1, g.vocab))
                    before[ACC ? k : 0].load(table_row<TT>(g, key[i0 + k], c));
            }
#pragma unroll
        for (int k = 0; k < kSumAhead; ++k) {
            const int i = i0 + k;
            if (i >= to) break;
            float x[N];
            rows[k].widen(x);
#pragma unroll
            for (int j = 0; j < N; ++j) sum[j] += x[j];
            if (!(last >> i & 1u)) continue;
            if (i < head_end || i == tail)
                store_partial<N>(a.partial + (2 * u + (i < head_end ? 0 : 1)) * g.dim + c, sum);
            else
                finish_row<TT, N, ACC>(g, key[i], c, sum, before[ACC ? k : 0]);
#pragma unroll
            for (int j = 0; j < N; ++j) sum[j] = 0.f;
        }
    }
}

// The long runs: a CTA at a time adds one in columns [32 N slab, + 32 N), its warps each a
// stretch of the partial sums in unit order, then the stretches' sums in order.  The partial
// sums (10 MB for 65536 Zipf-distributed tokens of 2048) are still in L2: about 5 us, in the
// wake of the sums.
template <int DT, int TT, bool VEC, bool ACC>
__global__ void __launch_bounds__(kJoinWarps * 32) join_units_kernel(SumArgs a, uint32_t slabs) {
    constexpr int N = kGroup<DT, TT, VEC>;
    const EmbeddingGradArgs &g = a.g;
    __shared__ float stretch[kJoinWarps][32 * N];
    const int warp = threadIdx.x / 32, lane = threadIdx.x & 31;
    fa_grid_dependency_wait();
    fa_allow_dependents();
    const int64_t work = static_cast<int64_t>(*a.long_runs) * slabs;
    for (int64_t i = blockIdx.x; i < work; i += gridDim.x) {
        const int64_t k = i / slabs;
        if (!fa_in_bounds(k, 1, a.units)) break;
        const LongRun run = a.runs[k];
        const int64_t c = ((i - k * slabs) * 32 + lane) * N;
        const int64_t u = run.first, each = (run.last - u + kJoinWarps - 1) / kJoinWarps;
        const int64_t w0 = u + 1 + warp * each, w1 = min(w0 + each - 1, int64_t(run.last));
        const bool here = c < g.dim;
        float sum[N];
        Raw<TT, N> before;
        if (ACC && warp == 0 && here && fa_in_bounds(run.key, 1, g.vocab))
            before.load(table_row<TT>(g, run.key, c));
#pragma unroll
        for (int j = 0; j < N; ++j) sum[j] = 0.f;
        if (here) {
            if (warp == 0) load_partial<N>(a.partial + (2 * u + 1) * g.dim + c, sum);
#pragma unroll 8
            for (int64_t w = w0; w <= w1; ++w) {
                float x[N];
                if (!fa_in_bounds(w, 1, a.units)) break;
                load_partial<N>(a.partial + 2 * w * g.dim + c, x);
#pragma unroll
                for (int j = 0; j < N; ++j) sum[j] += x[j];
            }
        }
#pragma unroll
        for (int j = 0; j < N; ++j) stretch[warp][j * 32 + lane] = sum[j];
        __syncthreads();
        if (warp == 0 && here) {
#pragma unroll
            for (int w = 1; w < kJoinWarps; ++w)
#pragma unroll
                for (int j = 0; j < N; ++j) sum[j] += stretch[w][j * 32 + lane];
            finish_row<TT, N, ACC>(g, run.key, c, sum, before);
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
                const int64_t groups = (a.dim - 1) / kGroup<td(), od(), true> + 1;
                const int64_t in_flight = vec ? kLookupGroups : 2;
                int log2 = 0;
                while (log2 < 5 && in_flight << log2 < groups) ++log2;
                const int64_t ctas = ((a.tokens << log2) + kLookupThreads - 1) / kLookupThreads;
                const int64_t stretch = in_flight << log2;
                const int64_t stretches = (groups + stretch - 1) / stretch;
                if (ctas > kMaxGridX || stretches > 65535) return cudaErrorInvalidConfiguration;
                const dim3 grid(static_cast<unsigned>(ctas), static_cast<unsigned>(stretches));
                if (vec)
                    lookup_kernel<td(), od(), id()><<<grid, kLookupThreads, 0, stream>>>(
                        a, static_cast<int>(groups), log2);
                else
                    lookup_any_kernel<td(), od(), id()>
                        <<<grid, kLookupThreads, 0, stream>>>(a, log2);
                return cudaGetLastError();
            });
        });
    });
}

EmbeddingScratch embedding_scratch_layout(int64_t tokens, int64_t vocab, int64_t dim) {
    EmbeddingScratch s;
    s.chunks = (tokens + kSortChunk - 1) / kSortChunk;
    s.units = (tokens + kSumUnit - 1) / kSumUnit;
    s.sorted_words = round_up(tokens, 4);
    s.claim_words = round_up(vocab, 4);
    s.run_words = 4 + round_up(3 * s.units, 4);  // their number, and the runs
    s.bytes = 4 * (s.sorted_words * (s.chunks > 1 ? 4 : 2) + s.claim_words + s.run_words +
                   s.units * 2 * round_up(dim, 4));
    return s;
}

cudaError_t launch_embedding_gradient(const EmbeddingGradArgs &g, fa_itype idt, fa_dtype ddt,
                                      fa_dtype tdt, cudaStream_t stream) {
    const EmbeddingScratch s = embedding_scratch_layout(g.tokens, g.vocab, g.dim);
    uint32_t *keys = static_cast<uint32_t *>(g.scratch), *pos = keys + s.sorted_words;
    uint32_t *chunk_keys = keys, *chunk_pos = pos;
    uint32_t *end = pos + s.sorted_words;
    if (s.chunks > 1) {
        chunk_keys = end;
        chunk_pos = chunk_keys + s.sorted_words;
        end = chunk_pos + s.sorted_words;
    }
    {
        SortArgs sa;
        sa.ids = g.ids;
        sa.tokens = g.tokens;
        sa.vocab = g.vocab;
        sa.padding_idx = g.padding_idx;
        sa.keys = chunk_keys;
        sa.pos = chunk_pos;
        int bits = 1;
        while (g.vocab >> bits) ++bits;  // vocab itself is a key
        sa.passes = (bits + kMostDigitBits - 1) / kMostDigitBits;
        sa.digit_bits = (bits + sa.passes - 1) / sa.passes;
        sa.chunks = static_cast<unsigned>(s.chunks);
        sa.ctas = s.chunks > 1 ? kSortChunk / kSortSlots
                               : static_cast<unsigned>(
                                     std::max<int64_t>(1, (g.tokens + kSortSlots - 1) / kSortSlots));
        const int64_t elem = tdt == FA_F32 ? 4 : 2;
        // Rows of ids that occur are written anyway: zeroed before too, they cost a second
        // write.  Above 16 MB of them at most, that costs more than finding them (3.3 us; of
        // 65536 tokens in a table of 131 MB, it shortens the sort's stage, which zeroes,
        // from 26 us to 21).
        const bool claim =
            !g.accumulate && std::min(g.tokens, g.vocab) * g.dim * elem > (int64_t(16) << 20);
        uint32_t *claims = claim ? end : nullptr;
        const bool flat = g.table_ld == g.dim && !claim;
        sa.zero.p = static_cast<char *>(g.dtable);
        sa.zero.rows = g.accumulate ? 0 : flat ? 1 : g.vocab;
        sa.zero.bytes = (flat ? g.vocab * g.dim : g.dim) * elem;
        sa.zero.ld = g.table_ld * elem;
        sa.zero.claims = claims;
        sa.long_runs = end + s.claim_words;
        if (claim) {
            cudaError_t err = for_itype(idt, [&](auto it) {
                claim_kernel<it()><<<static_cast<unsigned>((g.tokens + 255) / 256), 256, 0, stream>>>(
                    g.ids, claims, g.tokens, g.vocab, g.padding_idx);
                return cudaGetLastError();
            });
            if (err != cudaSuccess) return err;
        }
        // The first rows are asked into L2 meanwhile (32 MB: 2 to 6 us of 90; 96 MB would push
        // out the zeros that L2 still holds), unless they are shorter than a few lines.
        const int64_t row_bytes = g.dim * (ddt == FA_F32 ? 4 : 2);
        sa.prefetch.p = static_cast<const char *>(g.dout);
        sa.prefetch.rows =
            row_bytes < 512 ? 0 : std::min(g.tokens, (int64_t(32) << 20) / row_bytes);
        sa.prefetch.bytes = row_bytes;
        sa.prefetch.ld = g.dout_ld * (ddt == FA_F32 ? 4 : 2);
        // enough CTAs to zero the table, or to ask for rows, at the memory's rate; 64 KB each
        // at least
        const int64_t beside = (g.accumulate ? 0 : g.vocab * g.dim * elem) +
                               sa.prefetch.rows * row_bytes;
        const int64_t zeroing = std::min<int64_t>(2 * kSms, beside / 65536 + !g.accumulate);
        const int64_t zero_clusters = (zeroing + sa.ctas - 1) / sa.ctas;
        const auto go = [&](auto it, auto item) {
            auto kernel = sort_chunk_kernel<it(), decltype(item)>;
            constexpr int kSmem = sizeof(SortSmem<decltype(item)>);
            cudaError_t e = cudaFuncSetAttribute(
                kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
            if (e == cudaSuccess && sa.ctas > 8)
                e = cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
            if (e != cudaSuccess) return e;
            return launch_clusters(
                kernel, dim3(static_cast<unsigned>((sa.chunks + zero_clusters) * sa.ctas)),
                dim3(kSortThreads), kSmem, sa.ctas, claim, stream, sa);
        };
        cudaError_t err = for_itype(idt, [&](auto it) {
            return g.vocab < 65536 ? go(it, uint32_t{}) : go(it, uint64_t{});
        });
        if (err != cudaSuccess || g.tokens == 0) return err;
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
    a.long_runs = end + s.claim_words;
    a.runs = reinterpret_cast<LongRun *>(a.long_runs + 4);
    a.partial = reinterpret_cast<float *>(a.long_runs + s.run_words);
    a.units = s.units;
    const bool vec = vector_rows(g.dout, g.dout_ld, ddt, g.dtable, g.table_ld, tdt, g.dim);
    return for_dtype(ddt, [&](auto dd) {
        return for_dtype(tdt, [&](auto td) {
            const auto go = [&](auto v, auto acc) {
                constexpr bool VEC = decltype(v)::value, ACC = decltype(acc)::value;
                constexpr int N = kGroup<dd(), td(), VEC>;
                const int64_t groups = (g.dim + N - 1) / N;
                const int threads = static_cast<int>(
                    groups < kSumThreads ? round_up(groups, 32) : kSumThreads);
                const int64_t slabs = (groups + threads - 1) / threads;
                cudaError_t e = launch_dependent(
                    sum_units_kernel<dd(), td(), VEC, ACC>,
                    dim3(static_cast<unsigned>(a.units), static_cast<unsigned>(slabs)),
                    dim3(threads), 0, stream, a);
                if (e != cudaSuccess || a.units < 2) return e;
                const uint32_t join_slabs = static_cast<uint32_t>((groups + 31) / 32);
                // a long run takes two units at least
                const int64_t most = std::min<int64_t>(a.units / 2 * join_slabs, 8 * kSms);
                return launch_dependent(join_units_kernel<dd(), td(), VEC, ACC>,
                                        dim3(static_cast<unsigned>(most)), dim3(kJoinWarps * 32),
                                        0, stream, a, join_slabs);
            };
            const std::true_type yes{};
            const std::false_type no{};
            if (vec) return g.accumulate ? go(yes, yes) : go(yes, no);
            return g.accumulate ? go(no, yes) : go(no, no);
        });
    });
}

}  // namespace fa
