// The embedding lookup with scaling and its gradient by sorted tokens.
//
// Gradient of row v: scale * sum over the tokens t with id v of dout[t].  The tokens
// are sorted by id (stable: ascending t within an id), so that each id's rows are one
// run of the sorted order, and the sorted order is cut into units of kSumUnit tokens,
// each added by one CTA in order: the work of a unit does not depend on how the ids
// are distributed.  A run inside one unit is finished there.  Units that share a run leave
// FP32 partial sums: of two, the one that comes second adds both; more are added in unit
// order by the join.  (Two numbers have one sum, whoever adds them: the result does not
// depend on the order in which CTAs run.)
//
// Sort: a cluster of up to sixteen CTAs sorts up to kSortChunk tokens in its shared memory,
// least significant digit first: each warp ranks its tokens by digit, the CTAs exchange
// their digit counts, each CTA orders its own by digit, and the runs so made go to their
// places in the cluster, in whichever CTA's memory that is (sent token by token, each to
// a place of its own, a pass took 18 us).  A chunk's ids are sorted in two or three such passes with no
// global memory between them; the rest of the GPU zeroes the table meanwhile, so that only
// ids that occur are written after.  With several chunks, a token's place in the whole order is
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

// Rows of the table that are zeroed while its gradient's tokens are sorted: bytes from p,
// ld bytes apart.
struct ZeroArgs {
    char *p;
    int64_t rows, bytes, ld;
};

// The share of CTA ``rank`` of ``ctas``: rows in turn, or stretches of a single row.
__device__ __forceinline__ void zero_rows(const ZeroArgs &z, int64_t rank, int64_t ctas) {
    const int64_t parts = z.rows == 1 ? ctas : 1;
    for (int64_t row = z.rows == 1 ? 0 : rank; row < z.rows; row += z.rows == 1 ? 1 : ctas) {
        char *p = z.p + row * z.ld;
        const int64_t past = reinterpret_cast<uintptr_t>(p) & 15;
        const int64_t head = past ? min(int64_t(16) - past, z.bytes) : 0;
        const int64_t vecs = (z.bytes - head) / 16, tail = head + vecs * 16;
        if (parts == 1 || rank == 0) {  // elements are two bytes at least
            for (int64_t i = 2 * threadIdx.x; i < head; i += 2 * blockDim.x)
                *reinterpret_cast<uint16_t *>(p + i) = 0;
            for (int64_t i = tail + 2 * threadIdx.x; i < z.bytes; i += 2 * blockDim.x)
                *reinterpret_cast<uint16_t *>(p + i) = 0;
        }
        uint4 *q = reinterpret_cast<uint4 *>(p + head);
        const int64_t each = (vecs + parts - 1) / parts;
        const int64_t begin = parts == 1 ? 0 : rank * each, end = min(vecs, begin + each);
        for (int64_t i = begin + threadIdx.x; i < end; i += blockDim.x)
            if (fa_in_bounds(i, 1, vecs)) q[i] = make_uint4(0u, 0u, 0u, 0u);
    }
}

struct SortArgs {
    const void *ids;
    int64_t tokens, vocab, padding_idx;
    uint32_t *keys, *pos;     // the chunks' sorted ids and token indices
    int passes, digit_bits;   // passes * digit_bits bits hold vocab, the key of a token without an id
    unsigned chunks, ctas;    // clusters that sort, and the CTAs of a cluster
    ZeroArgs zero;
    uint32_t *arrived;        // counters of the sums' kernel, zeroed here
    int64_t counters;
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

// The first chunks' clusters sort; the CTAs after them zero the table meanwhile.
template <int IT, typename Item>
__global__ void __launch_bounds__(kSortThreads) sort_chunk_kernel(SortArgs a) {
    fa_allow_dependents();
    if (blockIdx.x >= a.chunks * a.ctas) {
        zero_rows(a.zero, blockIdx.x - a.chunks * a.ctas, gridDim.x - a.chunks * a.ctas);
        return;
    }
    for (int64_t i = blockIdx.x * kSortThreads + threadIdx.x; i < a.counters;
         i += static_cast<int64_t>(a.chunks * a.ctas) * kSortThreads)
        a.arrived[i] = 0;
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
        if (i >= n || !fa_in_bounds(chunk + i, 1, a.tokens)) return;
        a.keys[chunk + i] = static_cast<uint32_t>(x >> 16);
        a.pos[chunk + i] = static_cast<uint32_t>(chunk + static_cast<uint16_t>(x));
    };

    Item item[kSortItems];
#pragma unroll
    for (int j = 0; j < kSortItems; ++j) {
        const int i = static_cast<int>(rank) * kSortSlots + first + 32 * j;
        item[j] = ~Item(0);  // past the end: came last, and stays last
        if (i < n && fa_in_bounds(chunk + i, 1, a.tokens)) {
            const int64_t id = load_id<IT>(a.ids, chunk + i);
            const bool known = id >= 0 && id < a.vocab && id != a.padding_idx;
            item[j] = static_cast<Item>(known ? id : a.vocab) << 16 | static_cast<Item>(i);
        }
    }
    for (int pass = 0; pass < a.passes; ++pass) {
        const int shift = 16 + pass * a.digit_bits;
        const auto digit = [&](Item x) { return static_cast<int>(x >> shift) & (digits - 1); };
        for (int d = 2 * lane; d < digits; d += 64)
            *reinterpret_cast<uint32_t *>(&s.count[warp][d]) = 0u;
        __syncwarp();
        uint16_t before[kSortItems];  // tokens of the digit before this one in the warp
#pragma unroll
        for (int j = 0; j < kSortItems; ++j) {
            const int d = digit(item[j]);
            const unsigned same = __match_any_sync(0xffffffffu, d);
            const int ahead = __popc(same & ((1u << lane) - 1));
            const uint16_t c = s.count[warp][d];
            __syncwarp();
            if (ahead == 0) s.count[warp][d] = static_cast<uint16_t>(c + __popc(same));
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
            const int at = s.count[warp][digit(item[j])] + before[j];
            if (fa_in_bounds(at, 1, kSortSlots)) s.own[at] = item[j];
        }
        __syncthreads();
        const bool last = pass == a.passes - 1;
#pragma unroll
        for (int j = 0; j < kSortItems; ++j) {
            const int i = t + j * kSortThreads;
            const Item x = s.own[i];
            const int at = s.base[digit(x)] + i;  // < ctas * kSortSlots
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

struct SumArgs {
    EmbeddingGradArgs g;
    const uint32_t *keys, *pos;  // sorted
    uint32_t *shared;            // [units]: runs that the join adds up
    uint32_t *arrived;           // [slabs][units]: sums of the run across the unit's end so far
    float *partial;              // [units][2][dim]
    int64_t units;
};
// shared[u]: the unit is one run that began before it and goes on after it; it begins a run
// that goes on past the next unit.
constexpr uint32_t kThrough = 1, kBegins = 2;

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
// (another CTA's: from L2)
template <int N>
__device__ __forceinline__ void load_partial(const float *p, float *x) {
    if constexpr (N % 4 == 0) {
#pragma unroll
        for (int j = 0; j < N; j += 4) {
            const float4 f = __ldcg(reinterpret_cast<const float4 *>(p + j));
            x[j] = f.x;
            x[j + 1] = f.y;
            x[j + 2] = f.z;
            x[j + 3] = f.w;
        }
    } else {
#pragma unroll
        for (int j = 0; j < N; ++j) x[j] = __ldcg(p + j);
    }
}

// CTA (u, slab): unit u's tokens, columns of slab.  A run that began before the unit
// leaves its sum in partial[u][0], one that goes on after it in partial[u][1] (a run
// that does both, in [0]).
template <int DT, int TT, bool VEC>
__global__ void __launch_bounds__(kSumThreads, 4) sum_units_kernel(SumArgs a) {
    constexpr int N = kGroup<DT, TT, VEC>;
    constexpr int kAhead = 8;  // rows in flight
    constexpr uint32_t kNone = 0xffffffffu;  // no id: ids are below 2^31
    using DE = typename Elem<DT>::T;
    const EmbeddingGradArgs &g = a.g;
    fa_grid_dependency_wait();
    fa_allow_dependents();
    const int64_t c = (static_cast<int64_t>(blockIdx.y) * blockDim.x + threadIdx.x) * N;
    const int64_t u = blockIdx.x, first = u * kSumUnit;
    __shared__ uint32_t key[kSumUnit];
    __shared__ uint32_t pos[kSumUnit];
    __shared__ uint32_t ends;       // bit i: token i is its run's last here
    __shared__ bool began, goes;    // the first run began before the unit; the last goes on
    __shared__ bool with_last, with_next;  // and is shared with that one unit only
    __shared__ bool add_last, add_next;    // whose sum came first: this CTA adds both
    if (threadIdx.x < 32) {
        const int lane = threadIdx.x;
        const auto key_at = [&](int64_t i) { return i >= 0 && i < g.tokens ? a.keys[i] : kNone; };
        const uint32_t k = key_at(first + lane);
        // lanes 0 to 3: the tokens on both sides of the units before and after this one
        const uint32_t around =
            key_at(lane == 0   ? first - 1
                   : lane == 1 ? first - kSumUnit - 1
                   : lane == 2 ? first + kSumUnit
                   : lane == 3 ? first + 2 * kSumUnit
                               : -1);
        pos[lane] = first + lane < g.tokens ? a.pos[first + lane] : 0u;
        key[lane] = k < g.vocab ? k : kNone;
        const uint32_t head = __shfl_sync(0xffffffffu, k, 0), tail = __shfl_sync(0xffffffffu, k, 31);
        const uint32_t after = __shfl_sync(0xffffffffu, around, 2);
        uint32_t next = __shfl_down_sync(0xffffffffu, k, 1);
        if (lane == 31) next = after;
        const uint32_t e = __ballot_sync(0xffffffffu, next != k || lane == 31);
        const bool in = __shfl_sync(0xffffffffu, around, 0) == head && head < g.vocab;
        const bool on = after == tail && tail < g.vocab;
        const bool one = e == 0x80000000u;  // one run: only the last token ends one
        const bool before_last = __shfl_sync(0xffffffffu, around, 1) == head;
        const bool after_next = __shfl_sync(0xffffffffu, around, 3) == tail;
        if (lane == 0) {
            ends = e;
            began = in;
            goes = on;
            with_last = in && !(one && on) && !before_last;
            with_next = on && !(one && in) && !after_next;
            if (blockIdx.y == 0)
                a.shared[u] = in && on && one ? kThrough : on && after_next ? kBegins : 0u;
        }
    }
    __syncthreads();
    const bool here = c < g.dim;
    const uint32_t last = ends;
    bool began_before = began;
    const bool goes_on = goes;
    if (here) {
        const DE *dout = static_cast<const DE *>(g.dout) + c;
        float sum[N];
#pragma unroll
        for (int j = 0; j < N; ++j) sum[j] = 0.f;
#pragma unroll 1
        for (int i0 = 0; i0 < kSumUnit && key[i0] != kNone; i0 += kAhead) {
            Raw<DT, N> rows[kAhead];
#pragma unroll
            for (int k = 0; k < kAhead; ++k)
                if (key[i0 + k] != kNone && fa_in_bounds(c, N, g.dim) &&
                    fa_in_bounds(pos[i0 + k], 1, g.tokens))
                    rows[k].load(dout + static_cast<int64_t>(pos[i0 + k]) * g.dout_ld);
#pragma unroll
            for (int k = 0; k < kAhead; ++k) {
                const int i = i0 + k;
                const uint32_t v = key[i];
                if (v == kNone) break;  // tokens without an id come last
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
    if (!with_last && !with_next) return;  // the same for the whole CTA
    // partial sums are in memory before they are counted, and the other's read after
    __threadfence();
    __syncthreads();
    if (threadIdx.x == 0) {
        uint32_t *arrived = a.arrived + blockIdx.y * a.units;
        add_last = with_last && atomicAdd(&arrived[u - 1], 1u) == 1u;
        add_next = with_next && atomicAdd(&arrived[u], 1u) == 1u;
        __threadfence();
    }
    __syncthreads();
    if (!here) return;
    const auto add_pair = [&](int64_t w, uint32_t v) {  // the run across the end of unit w
        float x[N], y[N];
        load_partial<N>(a.partial + (2 * w + 1) * g.dim + c, x);
        load_partial<N>(a.partial + 2 * (w + 1) * g.dim + c, y);
#pragma unroll
        for (int j = 0; j < N; ++j) x[j] += y[j];
        finish_row<TT, N>(g, v, c, x);
    };
    if (add_last) add_pair(u - 1, key[0]);
    if (add_next) add_pair(u, key[kSumUnit - 1]);
}

// Runs of three units and more, in columns [32 N blockIdx.y, + 32 N).  Each warp of a CTA looks
// whether one unit began such a run; the CTA's warps then add each of these runs together,
// each a stretch of its partial sums in unit order, and the stretches' sums in order.
template <int DT, int TT, bool VEC>
__global__ void __launch_bounds__(kJoinWarps * 32) join_units_kernel(SumArgs a) {
    constexpr int N = kGroup<DT, TT, VEC>;
    const EmbeddingGradArgs &g = a.g;
    __shared__ int64_t last_unit[kJoinWarps];  // of the run that the warp's unit began (0: none)
    __shared__ float stretch[kJoinWarps][32 * N];
    const int warp = threadIdx.x / 32, lane = threadIdx.x & 31;
    const int64_t u0 = static_cast<int64_t>(blockIdx.x) * kJoinWarps, mine = u0 + warp;
    const int64_t c = (static_cast<int64_t>(blockIdx.y) * 32 + lane) * N;
    fa_grid_dependency_wait();
    fa_allow_dependents();
    int64_t end = 0;
    {
        const auto through = [&](int64_t w) { return w < a.units && a.shared[w] == kThrough; };
        const bool next = through(mine + 1 + lane);  // asked for together with the unit's own
        if (mine < a.units && a.shared[mine] == kBegins) {
            end = mine + 1;
            unsigned on = __ballot_sync(0xffffffffu, next);
            while (on == 0xffffffffu) {
                end += 32;
                on = __ballot_sync(0xffffffffu, through(end + lane));
            }
            end += __ffs(~on) - 1;
        }
    }
    if (lane == 0) last_unit[warp] = end;
    __syncthreads();
    const bool here = c < g.dim;
    for (int k = 0; k < kJoinWarps; ++k) {
        if (!last_unit[k]) continue;  // the same for the whole CTA
        const int64_t u = u0 + k, each = (last_unit[k] - u + kJoinWarps - 1) / kJoinWarps;
        const int64_t w1 = min(u + (warp + 1) * each, last_unit[k]);
        float sum[N];
#pragma unroll
        for (int j = 0; j < N; ++j) sum[j] = 0.f;
        if (here) {
            if (warp == 0) load_partial<N>(a.partial + (2 * u + 1) * g.dim + c, sum);
#pragma unroll 4
            for (int64_t w = u + 1 + warp * each; w <= w1; ++w) {
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
    // slabs of the sums' kernel: a column a thread at most
    s.counters = s.units * ((dim + kSumThreads - 1) / kSumThreads);
    s.bytes = 4 * (s.sorted_words * (s.chunks > 1 ? 4 : 2) + round_up(s.units, 4) +
                   round_up(s.counters, 4) + s.units * 2 * round_up(dim, 4));
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
        sa.passes = (bits + 8) / 9;
        sa.digit_bits = (bits + sa.passes - 1) / sa.passes;
        sa.chunks = static_cast<unsigned>(s.chunks);
        sa.ctas = s.chunks > 1 ? kSortChunk / kSortSlots
                               : static_cast<unsigned>(
                                     std::max<int64_t>(1, (g.tokens + kSortSlots - 1) / kSortSlots));
        const int64_t elem = tdt == FA_F32 ? 4 : 2;
        const bool flat = g.table_ld == g.dim;
        sa.zero.p = static_cast<char *>(g.dtable);
        sa.zero.rows = flat ? 1 : g.vocab;
        sa.zero.bytes = (flat ? g.vocab * g.dim : g.dim) * elem;
        sa.zero.ld = g.table_ld * elem;
        sa.arrived = end + round_up(s.units, 4);
        sa.counters = s.counters;
        // enough CTAs to zero the table at the memory's rate, 64 KB each at least
        const int64_t zeroing =
            g.accumulate ? 0 : std::min<int64_t>(2 * 152, g.vocab * g.dim * elem / 65536 + 1);
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
                dim3(kSortThreads), kSmem, sa.ctas, false, stream, sa);
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
    a.shared = end;
    a.arrived = end + round_up(s.units, 4);
    a.partial = reinterpret_cast<float *>(a.arrived + round_up(s.counters, 4));
    a.units = s.units;
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
                    dim3(static_cast<unsigned>(a.units), static_cast<unsigned>(slabs)),
                    dim3(threads), 0, stream, a);
                if (e != cudaSuccess || a.units < 3) return e;
                return launch_dependent(
                    join_units_kernel<dd(), td(), VEC>,
                    dim3(static_cast<unsigned>((a.units - 2 + kJoinWarps - 1) / kJoinWarps),
                         static_cast<unsigned>((groups + 31) / 32)),
                    dim3(kJoinWarps * 32), 0, stream, a);
            };
            return vec ? go(std::true_type{}) : go(std::false_type{});
        });
    });
}

}  // namespace fa
