// Token log-probabilities from logits, their gradient, and the two losses built on
// them: the preference loss from paired log ratios and the clipped policy loss.
//
// Row t of the logits is a softmax over vocab ids after multiplication by scale:
//   top = max_v x_v,  s = sum_v exp(scale (x_v - top)),
//   logp = scale (x_label - top) - ln s,
//   dlogits_v = c (1[v = label] - exp(scale (x_v - top)) / s).
// exp(scale (x - top)) is 2^(k d) with d = x - top (rounded for FP32 logits, close to exact for
// 16-bit ones) and k = scale log2(e) in two FP32 parts.  With k in one part the
// log-probabilities were 2e-8 of a row's spread off, all the same way.
//
// Reads and writes of the logits bound them: one read for the log-probabilities (7296 rows of
// 32000: FP32 134 us, 7.0 TB/s; FP16 and BF16 74 us, 6.3 TB/s, with the issue slots 53 % busy: 52
// instructions on eight elements), a second read and the write for their gradient (6.7 TB/s),
// and one of each for the policy loss, which holds the row on chip between its sum and its
// gradient (16384 rows of 32000 BF16: 318 us, 6.3 TB/s).  The preference loss cannot: a
// token's coefficient needs every row of its pair.
#include <algorithm>
#include <type_traits>

#include <cooperative_groups.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "internal.h"
#include "model_device.cuh"
#include "model_internal.h"

namespace fa {
namespace {

namespace cg = cooperative_groups;

FA_BOUNDS_COUNTER(g_logprob_oob)

constexpr int kBatch = 4;  // 16-byte vectors a thread takes at a time
// A row's kernels are compiled for NT = 32, 64, 128 and 256 threads a row: a row of few
// vectors is a warp's, without barriers (65536 policy rows of 1000 BF16 logits by 256 threads
// each took 330 us, nine tenths of it in starting and joining them).  A CTA has one row, or
// kWarpRows of a warp each where there are many: an SM runs no more than 32 CTAs (the
// log-probabilities of 65536 rows of 1000 BF16: 70 us by CTAs of one warp, 33 by four).
constexpr int kMostThreads = 256;
constexpr int kWarpRows = 4;
template <int NT>
constexpr int kBlockThreads = NT == 32 ? 32 * kWarpRows : NT;

// A row cut for 16-byte accesses: head scalars up to the first boundary, then nvec
// vectors, then the scalars left over.
struct RowSpan {
    int head, nvec, tail;  // tail: the first scalar after the vectors
};
template <int DT>
__host__ __device__ __forceinline__ RowSpan row_span(const void *row, int64_t n) {
    constexpr int V = Elem<DT>::kVec;
    const int past =
        static_cast<int>((reinterpret_cast<uintptr_t>(row) & 15) / sizeof(typename Elem<DT>::T));
    RowSpan r;
    r.head = past ? V - past : 0;
    if (r.head > n) r.head = static_cast<int>(n);
    r.nvec = (static_cast<int>(n) - r.head) / V;
    r.tail = r.head + r.nvec * V;
    return r;
}

// One of the 2^log2 CTAs that take a row together, and the row.  (Powers of two: with
// divisions by a number known at run time the log-probabilities executed 6 % more.)
struct Share {
    unsigned rank, log2;
    int64_t row;

    __device__ __forceinline__ explicit Share(unsigned log2_, bool warp_rows = false)
        : rank(blockIdx.x & ((1u << log2_) - 1)), log2(log2_), row(blockIdx.x >> log2_) {
        if (warp_rows) row = row * blockDim.y + threadIdx.y;
    }
    __device__ __forceinline__ unsigned split() const { return 1u << log2; }
    __device__ __forceinline__ bool first() const { return rank == 0; }
    __device__ __forceinline__ bool last() const { return rank == split() - 1; }
};

// 2^(k (x - top)) for the elements of a row.  k_lo > 0, so that -inf stays -inf.
struct Exponent {
    float k, k_lo;
    float top;  // 0 while nothing but -inf has been seen

    __device__ __forceinline__ Exponent(const LogitsArgs &a, float top_) : k(a.k), k_lo(a.k_lo) {
        set(top_);
    }
    __device__ __forceinline__ void set(float top_) { top = top_ == -INFINITY ? 0.f : top_; }
    __device__ __forceinline__ float log2_of(float x) const {
        const float d = x - top;
        return fmaf(d, k, d * k_lo);
    }
    __device__ __forceinline__ float operator()(float x) const { return exp2_fast(log2_of(x)); }
    __device__ __forceinline__ uint64_t of_pair(float x0, float x1) const {
        const uint64_t d = add2(pair(x0, x1), pair(-top, -top));
        float lo, hi;
        unpair(fma2(d, pair(k, k), mul2(d, pair(k_lo, k_lo))), lo, hi);
        return pair(exp2_fast(lo), exp2_fast(hi));
    }
};

// exp2_fast truncates: its values are low by half a unit in the last place on average, which
// over mantissas of every size is 2^-25 / ln 2 = 4.3e-8 of a sum (measured: 3.5e-8 to 5.5e-8, rows
// of 100 to 131072 logits of each type).  v + kHalfUnit * v, rounded, is one unit above v
// where v's mantissa is above 4/3 and v elsewhere: the same 4.3e-8 on average, and 1 and 2 stay,
// so that sums of equal terms are exact.  Taken over sums of two terms (a preference loss of 3501
// counted rows of 32000 FP16: 46.7 us; of every term 47.0; not at all 45.9, and every
// log-probability 4.5e-8 too high).  What it leaves is below 1e-8, or 2.5e-8 in rows of nine logits;
// rows whose logits are multiples of 1/2 have too few arguments for an average, and up to 4.2e-8.
constexpr float kHalfUnit = 1.5f * 0x1p-25f;

// The running maximum and the sum of 2^(k (x - top)) over the elements a warp has seen: the
// maximum is the warp's, so that it rises for all lanes at once (and seldom: after the
// first vectors, once in n times for n times the elements); each lane has its own sum, in
// two interleaved parts.  Every lane of the warp calls add.
struct Softmax {
    float top = -INFINITY;
    Exponent e;
    uint64_t sum;

    __device__ __forceinline__ explicit Softmax(const LogitsArgs &a)
        : e(a, -INFINITY), sum(pair(0.f, 0.f)) {}

    __device__ __forceinline__ void raise(float best) {
        if (!__any_sync(0xffffffffu, best > top)) return;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1)
            best = fmaxf(best, __shfl_xor_sync(0xffffffffu, best, o));
        e.set(best);
        // a sum of nothing but -inf so far is 0, or NaN, and stays
        const float f = top == -INFINITY ? 1.f : exp2_exact(e.log2_of(top));
        sum = mul2(sum, pair(f, f));
        top = best;
    }
    // A scalar per lane (-inf: none).
    __device__ __forceinline__ void add1(float x) {
        raise(x);
        const float y = e(x);
        sum = add2(sum, pair(fmaf(y, kHalfUnit, y), 0.f));
    }
    template <int DT, int N>
    __device__ __forceinline__ void add(const uint4 *r) {
        constexpr int V = Elem<DT>::kVec;
        raise(Elem<DT>::template largest<N>(r));
        // these vectors' sum first: small terms beside a large one in the running sum would
        // be rounded off one by one, all the same way
        uint64_t some = pair(0.f, 0.f);
#pragma unroll
        for (int i = 0; i < N; ++i) {
            float x[V];
            Elem<DT>::unpack(r[i], x);
#pragma unroll
            for (int j = 0; j < V; j += 4) {
                const uint64_t v = add2(e.of_pair(x[j], x[j + 1]), e.of_pair(x[j + 2], x[j + 3]));
                some = add2(some, fma2(v, pair(kHalfUnit, kHalfUnit), v));
            }
        }
        sum = add2(sum, some);
    }
};

// What a row comes to: the largest logit and the sum of 2^(k (x - top)).
struct RowSum {
    float top, s;

    // The sum relative to a larger maximum, that of e.
    __device__ __forceinline__ float at(const Exponent &e) const {
        return top == -INFINITY || top == e.top ? s : s * exp2_exact(e.log2_of(top));
    }
};

// The CTAs that take a row together write to one another's shared memory: each says here,
// early, that it runs; merge_row waits for all of them.
__device__ __forceinline__ void enter_row(const Share &sh) {
    if (sh.log2 > 0) cg::this_cluster().barrier_arrive();
}

// Merges what the warps of the CTAs of a cluster hold of a row; every thread returns the
// row's.  Every warp sends its part to every CTA, so that the cluster waits once and reads only
// its own memory, and each part is rebased once, to the row's maximum (merged in each CTA first
// and then read from one another's memory, 1111 policy rows of 131072 BF16 took 110 us instead
// of 104, 1999 of 100003 FP32 411 us instead of 359).  ``part``: shared,
// [kMostSplit * warps].  After enter_row.
constexpr int kMostSplit = 8;
template <int NT>
__device__ __forceinline__ RowSum merge_row(const Softmax &acc, RowSum *part, const Share &sh) {
    constexpr int warps = NT / 32;
    const int lane = threadIdx.x & 31, warp = threadIdx.x / 32;
    const auto warp_total = [](float s) {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
        return s;
    };
    float lo, hi;
    unpair(acc.sum, lo, hi);
    RowSum row{acc.top, warp_total(lo + hi)};
    if (sh.log2 > 0) {
        cg::cluster_group cluster = cg::this_cluster();
        cluster.barrier_wait();  // the other CTAs run
        if (lane < static_cast<int>(sh.split()))
            *cluster.map_shared_rank(part + sh.rank * warps + warp, lane) = row;
        cluster.sync();
    } else if constexpr (warps > 1) {
        if (lane == 0) part[warp] = row;
        __syncthreads();
    }
    if (warps > 1 || sh.log2 > 0) {  // every warp adds the parts alike
        const int parts = warps << sh.log2;
        const RowSum none{-INFINITY, 0.f};
        const RowSum w = lane < parts ? part[lane] : none;
        const RowSum v = lane + 32 < parts ? part[lane + 32] : none;
        float top = fmaxf(w.top, v.top);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
        Exponent e = acc.e;
        e.set(top);
        row = RowSum{top, warp_total(w.at(e) + v.at(e))};
    }
    if (row.top == -INFINITY) row.s = NAN;  // no finite logit
    return row;
}

// x + y exactly, as the rounded sum and what the rounding left.
__device__ __forceinline__ Sum2 two_sum(float x, float y) {
    Sum2 s;
    s.hi = x + y;
    const float b = s.hi - x;
    s.lo = (x - (s.hi - b)) + (y - b);
    return s;
}

// ln s for a normal s >= 1, within 4e-9 of it: s = 2^e m with m from 1/sqrt 2 to sqrt 2, and
// ln m = 2 atanh r, r = (m - 1) / (m + 1), by its series (|r| < 0.172: the term left out is
// below 2^-40 of the first).
__device__ __forceinline__ Sum2 log_parts(float s) {
    const int e = (__float_as_int(s) - __float_as_int(0.70710678f)) >> 23;
    const float m = __int_as_float(__float_as_int(s) - (e << 23)), f = static_cast<float>(e);
    const float num = m - 1.f;  // exact
    const Sum2 den = two_sum(m, 1.f);
    const float r = __fdiv_rn(num, den.hi);
    const float r_lo = __fdividef(fmaf(-r, den.lo, fmaf(-r, den.hi, num)), den.hi);
    const float q = r * r;
    float p = 1.f / 15.f;  // 1/3 + q/5 + ... + q^6/15
    p = fmaf(p, q, 1.f / 13.f);
    p = fmaf(p, q, 1.f / 11.f);
    p = fmaf(p, q, 1.f / 9.f);
    p = fmaf(p, q, 1.f / 7.f);
    p = fmaf(p, q, 1.f / 5.f);
    p = fmaf(p, q, 1.f / 3.f);
    // ln 2 in two parts, the first short enough that e times it is exact
    constexpr float kLn2Hi = 0.693145751953125f, kLn2Lo = 1.4286068203094172e-06f;
    Sum2 l = two_sum(f * kLn2Hi, 2.f * r);
    l.lo += fmaf(f, kLn2Lo, 2.f * fmaf(q * r, p, r_lo));
    return two_sum(l.hi, l.lo);
}

// logp of the label from its logit and the row's statistics, with one rounding of its own (d is
// rounded before it where the logits are FP32, and s is an FP32 sum).  The scale is in two
// parts, as k is: rounded, 0.7 made the log-probabilities 1e-7 too high.
__device__ __forceinline__ float label_logp(float x, const RowSum &r, const LogitsArgs &a) {
    const float d = x - r.top;
    // outside this the parts would not be finite
    if (!(d > -1e30f) || !(r.s >= 1.f) || !(r.s < 1e30f)) return d * a.scale - logf(r.s);
    const Sum2 log_s = log_parts(r.s);
    const float p = d * a.scale, p_lo = fmaf(d, a.scale_lo, fmaf(d, a.scale, -p));
    const Sum2 y = two_sum(p, -log_s.hi);
    return y.hi + (y.lo + (p_lo - log_s.lo));
}

// A token's label; whether it is counted.  Both types by 32-bit words, so that the kernels
// are compiled once for them: a counted label's upper word is zero.
__device__ __forceinline__ bool load_label(const LogitsArgs &x, int64_t t, int64_t *label) {
    const unsigned *word = static_cast<const unsigned *>(x.labels) + (t << x.wide_labels);
    const unsigned low = word[0], high = x.wide_labels ? word[1] : 0u;
    *label = low;
    return high == 0 && low < static_cast<unsigned>(x.vocab);
}

// The part of a row's vectors that a CTA takes.
struct RowPart {
    int begin, nvec, count;

    __device__ __forceinline__ RowPart(const RowSpan &sp, const Share &sh) : nvec(sp.nvec) {
        const int each = (nvec + static_cast<int>(sh.split()) - 1) >> sh.log2;
        begin = min(nvec, each * static_cast<int>(sh.rank));
        count = min(each, nvec - begin);
    }
    __device__ __forceinline__ bool in_bounds(int i) const {
        return fa_in_bounds(begin + i, 1, nvec);
    }
};

// The scalars of a row outside its vectors: the head by the first CTA, the tail by the last.
template <typename F>
__device__ __forceinline__ void row_ends(const RowSpan &sp, int64_t n, const Share &sh, F f) {
    const int t = threadIdx.x;
    if (sh.first() && t < sp.head && fa_in_bounds(t, 1, n)) f(t);
    if (sh.last() && t < n - sp.tail && fa_in_bounds(sp.tail + t, 1, n)) f(sp.tail + t);
}

// One vector of the gradient but for the label's element: -c 2^(k (x - top)) / s.
template <int DT>
__device__ __forceinline__ uint4 gradient_vector(const uint4 &r, const Exponent &e, float w) {
    constexpr int V = Elem<DT>::kVec;
    float x[V];
    Elem<DT>::unpack(r, x);
#pragma unroll
    for (int j = 0; j < V; j += 2)
        unpair(mul2(e.of_pair(x[j], x[j + 1]), pair(w, w)), x[j], x[j + 1]);
    return Elem<DT>::pack(x);
}

// Whether this thread writes the label's element of the row: it then reads the logit before
// it writes anything, and the element, c (1 - p), last.
template <int DT, int NT>
__device__ __forceinline__ bool label_is_mine(int64_t label, const RowSpan &sp,
                                              const RowPart &part, const Share &sh) {
    const int at = static_cast<int>(label), t = threadIdx.x;
    if (at < sp.head) return sh.first() && t == at;
    if (at >= sp.tail) return sh.last() && t == at - sp.tail;
    const int i = (at - sp.head) / Elem<DT>::kVec - part.begin;
    return i >= 0 && i < part.count && i % NT == t;
}

// f(i, whole batch) for the vectors i, i + NT, ... of a thread in batches of N: whole
// ones first, without a check of each vector, then one that may be cut short.
template <int NT, int N, typename F>
__device__ __forceinline__ void for_batches(int count, F f) {
    int i0 = 0;
    for (; i0 + N * NT <= count; i0 += N * NT) f(i0, std::true_type{});
    if (i0 < count) f(i0, std::false_type{});
}

// dlogits of (a part of) one row from global memory.  The output may be the row itself:
// every element is read before it is written, by the thread that writes it.
template <int DT, int NT>
__device__ __forceinline__ void row_gradient(const void *row, void *out, int64_t n,
                                             const LogitsArgs &a, RowSum r, float c,
                                             int64_t label, const Share &sh) {
    using E = Elem<DT>;
    using T = typename E::T;
    const T *x = static_cast<const T *>(row);
    T *y = static_cast<T *>(out);
    const Exponent e(a, r.top);
    const float w = -c / r.s;
    const int tid = threadIdx.x;
    if ((reinterpret_cast<uintptr_t>(row) ^ reinterpret_cast<uintptr_t>(out)) & 15) {
        // not co-aligned: element by element
        for (int64_t i = sh.rank * NT + tid; i < n; i += sh.split() * NT)
            if (fa_in_bounds(i, 1, n))
                y[i] = E::round(fmaf(e(E::widen(x[i])), w, i == label ? c : 0.f));
        return;
    }
    const RowSpan sp = row_span<DT>(row, n);
    const RowPart part(sp, sh);
    const bool mine = label_is_mine<DT, NT>(label, sp, part, sh);
    const float label_logit = mine ? E::widen(x[label]) : 0.f;
    row_ends(sp, n, sh, [&](int i) { y[i] = E::round(e(E::widen(x[i])) * w); });
    const uint4 *q = reinterpret_cast<const uint4 *>(x + sp.head) + part.begin + tid;
    uint4 *o = reinterpret_cast<uint4 *>(y + sp.head) + part.begin + tid;
    for_batches<NT, kBatch>(part.count, [&](int i0, auto whole) {
        uint4 v[kBatch];
#pragma unroll
        for (int j = 0; j < kBatch; ++j) {
            const int i = i0 + j * NT;
            if ((decltype(whole)::value || i + tid < part.count) && part.in_bounds(i + tid)) v[j] = __ldcs(q + i);
        }
#pragma unroll
        for (int j = 0; j < kBatch; ++j) {
            const int i = i0 + j * NT;
            if ((decltype(whole)::value || i + tid < part.count) && part.in_bounds(i + tid))
                __stcs(o + i, gradient_vector<DT>(v[j], e, w));
        }
    });
    if (mine) y[label] = E::round(fmaf(e(label_logit), w, c));
}

// Zeros for (a part of) the row of a token that is not counted.
template <int DT>
__device__ __forceinline__ void row_zeros(void *out, int64_t n, const Share &sh) {
    using E = Elem<DT>;
    using T = typename E::T;
    T *y = static_cast<T *>(out);
    const RowSpan sp = row_span<DT>(out, n);
    row_ends(sp, n, sh, [&](int i) { y[i] = E::round(0.f); });
    const RowPart part(sp, sh);
    uint4 *o = reinterpret_cast<uint4 *>(y + sp.head) + part.begin;
    for (int i = threadIdx.x; i < part.count; i += blockDim.x)
        if (part.in_bounds(i)) __stcs(o + i, make_uint4(0u, 0u, 0u, 0u));
}

// The scalars of a row into its sum: warp 0 of the first CTA has the head, of the last the
// tail (both are shorter than a warp).
template <int DT>
__device__ __forceinline__ void add_ends(Softmax &acc, const void *row, const RowSpan &sp,
                                         int64_t n, const Share &sh) {
    if (threadIdx.x >= 32 || sp.nvec * Elem<DT>::kVec == n) return;
    const typename Elem<DT>::T *x = static_cast<const typename Elem<DT>::T *>(row);
    float head = -INFINITY, tail = -INFINITY;
    row_ends(sp, n, sh, [&](int i) {
        (i < sp.head ? head : tail) = Elem<DT>::widen(x[i]);
    });
    acc.add1(head);
    acc.add1(tail);
}

// -inf in every element of a vector: what a lane without one adds.
template <int DT>
__device__ __forceinline__ uint4 no_vector() {
    constexpr uint32_t w = DT == FA_F32 ? 0xff800000u : DT == FA_BF16 ? 0xff80ff80u : 0xfc00fc00u;
    return make_uint4(w, w, w, w);
}

// The softmax statistics of a row by the CTAs of a cluster, read from global memory.
template <int DT, int NT>
__device__ __forceinline__ RowSum row_softmax(const void *row, const LogitsArgs &a,
                                              const Share &sh) {
    using T = typename Elem<DT>::T;
    __shared__ RowSum parts[kMostSplit * NT / 32];
    const RowSpan sp = row_span<DT>(row, a.vocab);
    Softmax acc(a);
    add_ends<DT>(acc, row, sp, a.vocab, sh);
    const RowPart part(sp, sh);
    const int tid = threadIdx.x;
    const uint4 *q =
        reinterpret_cast<const uint4 *>(static_cast<const T *>(row) + sp.head) + part.begin + tid;
    for_batches<NT, kBatch>(part.count, [&](int i0, auto full) {
        if (!decltype(full)::value && i0 + (tid & ~31) >= part.count) return;  // whole warps
        uint4 r[kBatch];
#pragma unroll
        for (int j = 0; j < kBatch; ++j) {
            const int i = i0 + j * NT;
            r[j] = (decltype(full)::value || i + tid < part.count) && part.in_bounds(i + tid)
                       ? q[i]
                       : no_vector<DT>();
        }
        acc.add<DT, kBatch>(r);
    });
    return merge_row<NT>(acc, parts, sh);
}

template <int DT, int NT>
__global__ void __launch_bounds__(kBlockThreads<NT>, 1536 / kBlockThreads<NT>)
token_logprobs_kernel(LogitsArgs x, float *logp, float *lse, unsigned split_log2) {
    using T = typename Elem<DT>::T;
    fa_allow_dependents();
    const Share sh(split_log2, NT == 32);
    const int64_t t = sh.row;
    if (NT == 32 && t >= x.tokens) return;
    int64_t label;
    if (!load_label(x, t, &label)) {
        if (sh.first() && threadIdx.x == 0) {
            logp[t] = 0.f;
            if (lse) reinterpret_cast<float2 *>(lse)[t] = make_float2(0.f, 1.f);
        }
        return;
    }
    enter_row(sh);
    const T *row = static_cast<const T *>(x.logits) + t * x.ld;
    const bool first = sh.first() && threadIdx.x == 0;
    const float label_logit = first ? Elem<DT>::widen(row[label]) : 0.f;  // before the sum
    const RowSum r = row_softmax<DT, NT>(row, x, sh);
    if (first) {
        logp[t] = label_logp(label_logit, r, x);
        if (lse) reinterpret_cast<float2 *>(lse)[t] = make_float2(r.top, r.s);
    }
}

// One pass over the rows with no sum in it: 64 bytes of loads a thread, their gradient, and
// the stores; read and write bound it (4980 rows of 32000 BF16, a quarter of them zeros: 80 us,
// 7.0 TB/s).  Rows are taken from the last to the first: the pass that made the statistics
// left the last rows in L2.
template <int DT, int NT>
__global__ void __launch_bounds__(kBlockThreads<NT>, 1536 / kBlockThreads<NT>)
logprob_gradient_kernel(LogitGradArgs a, unsigned split_log2) {
    using T = typename Elem<DT>::T;
    const Share sh(split_log2, NT == 32);
    const int64_t t = a.x.tokens - 1 - sh.row;
    if (NT == 32 && t < 0) return;
    T *out = static_cast<T *>(a.dlogits) + t * a.dlogits_ld;
    int64_t label;
    if (!load_label(a.x, t, &label)) {
        row_zeros<DT>(out, a.x.vocab, sh);
        return;
    }
    const T *row = static_cast<const T *>(a.x.logits) + t * a.x.ld;
    const float2 l = reinterpret_cast<const float2 *>(a.lse)[t];
    const RowSum r{l.x, l.y};
    const float c = a.dlogp[t] * a.factor * (a.grad_loss ? *a.grad_loss : 1.f);
    row_gradient<DT, NT>(row, out, a.x.vocab, a.x, r, c, label, sh);
}

// ---- preference loss ------------------------------------------------------------

constexpr int kPairThreads = 512;

// Sum of one value a thread over the CTA, as FP32 pairs; every thread returns it.  ``part``:
// shared, [warps].
__device__ __forceinline__ Sum2 cta_sum2(Sum2 s, Sum2 *part) {
    s = warp_sum2(s);
    if ((threadIdx.x & 31) == 0) part[threadIdx.x / 32] = s;
    __syncthreads();
    s = Sum2();
    if ((threadIdx.x & 31) < blockDim.x / 32) s = part[threadIdx.x & 31];
    s = warp_sum2(s);
    s.hi = __shfl_sync(0xffffffffu, s.hi, 0);
    s.lo = __shfl_sync(0xffffffffu, s.lo, 0);
    return s;
}

// ln(1 + e^z) without overflow.
__device__ __forceinline__ float softplus(float z) {
    return fmaxf(z, 0.f) + log1pf(expf(-fabsf(z)));
}

// One CTA per pair: a half of it for each sequence's sum, the pair's loss and the
// coefficient of each of its tokens.  Tokens of no sequence are zeroed by the first and the
// last pair's CTA.  Up to kPairCluster pairs are one cluster, whose first CTA takes the mean
// of their losses (a launch less); more leave it to preference_mean_kernel.
constexpr unsigned kPairCluster = 8;
template <int IT>
__global__ void __launch_bounds__(kPairThreads) preference_pair_kernel(PreferenceArgs a) {
    constexpr int kHalf = kPairThreads / 2, kWarps = kHalf / 32;
    __shared__ Sum2 part[2][kWarps];
    __shared__ int counts[2][kWarps];
    __shared__ float my_loss;
    const int64_t pair = blockIdx.x;
    const int q = threadIdx.x / kHalf, tid = threadIdx.x % kHalf, lane = tid & 31;
    const auto clamped = [&](int64_t j) {
        const int64_t o = a.seq_offsets[j];
        return o < 0 ? 0 : o > a.tokens ? a.tokens : o;
    };
    const auto counted = [&](int64_t t) {
        const int64_t label = load_id<IT>(a.labels, t);
        return label >= 0 && label < a.vocab;
    };
    fa_grid_dependency_wait();
    fa_allow_dependents();
    const int64_t lo = clamped(2 * pair + q), hi = clamped(2 * pair + q + 1);
    Sum2 s;
    int n = 0;
#pragma unroll 4
    for (int64_t t = lo + tid; t < hi; t += kHalf)
        if (counted(t) && fa_in_bounds(t, 1, a.tokens)) {
            s.add(a.logp[t] - a.ref_logp[t]);
            ++n;
        }
    s = warp_sum2(s);
    n = __reduce_add_sync(0xffffffffu, n);
    if (lane == 0) {
        part[q][tid / 32] = s;
        counts[q][tid / 32] = n;
    }
    __syncthreads();
    float mean[2], per[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        s = part[h][0];
        n = counts[h][0];
#pragma unroll
        for (int w = 1; w < kWarps; ++w) {
            s.add(part[h][w]);
            n += counts[h][w];
        }
        per[h] = a.average ? 1.f / static_cast<float>(max(n, 1)) : 1.f;
        mean[h] = a.average ? s.value() / static_cast<float>(max(n, 1)) : s.value();
    }
    const float z = a.beta * (mean[0] - mean[1]);
    const float e = a.smoothing;
    // d pair_loss / dz = -(1 - e) sigmoid(-z) + e sigmoid(z)
    const float dz = e / (1.f + expf(-z)) - (1.f - e) / (1.f + expf(z));
    const float d = dz * a.beta / static_cast<float>(a.pairs);
    if (threadIdx.x == 0) {
        const float keep = (1.f - e) * softplus(-z);
        my_loss = e > 0.f ? keep + e * softplus(z) : keep;
        a.pair_loss[pair] = my_loss;
        a.rewards[2 * pair] = a.beta * mean[0];
        a.rewards[2 * pair + 1] = a.beta * mean[1];
    }
    const float c = q ? -d * per[1] : d * per[0];
#pragma unroll 4
    for (int64_t t = lo + tid; t < hi; t += kHalf)
        if (fa_in_bounds(t, 1, a.tokens)) a.dlogp[t] = counted(t) ? c : 0.f;
    if (pair == 0 && q == 0)
        for (int64_t t = tid; t < lo; t += kHalf) a.dlogp[t] = 0.f;
    if (pair == a.pairs - 1 && q == 1)
        for (int64_t t = hi + tid; t < a.tokens; t += kHalf) a.dlogp[t] = 0.f;
    if (gridDim.x > kPairCluster) return;
    cg::cluster_group cluster = cg::this_cluster();
    cluster.sync();
    if (pair == 0 && threadIdx.x == 0) {
        Sum2 total;
        for (unsigned r = 0; r < gridDim.x; ++r) total.add(*cluster.map_shared_rank(&my_loss, r));
        *a.loss = total.value() / static_cast<float>(gridDim.x);
    }
    cluster.sync();  // no CTA leaves while the first reads its loss
}

// The mean over the pairs, by one CTA (no pairs: 0, and no token has a coefficient).
__global__ void __launch_bounds__(kPairThreads) preference_mean_kernel(PreferenceArgs a) {
    __shared__ Sum2 part[kPairThreads / 32];
    fa_grid_dependency_wait();
    Sum2 s;
    for (int64_t k = threadIdx.x; k < a.pairs; k += kPairThreads) s.add(a.pair_loss[k]);
    s = cta_sum2(s, part);
    if (threadIdx.x == 0) *a.loss = a.pairs ? s.value() / static_cast<float>(a.pairs) : 0.f;
    if (a.pairs == 0)
        for (int64_t t = threadIdx.x; t < a.tokens; t += kPairThreads) a.dlogp[t] = 0.f;
}

// ---- policy loss ------------------------------------------------------------------

constexpr int kSummaryThreads = 1024;

// exp(d) - d - 1, by its series where the difference would cancel.
__device__ __forceinline__ float kl_term(float d) {
    if (fabsf(d) < 0.5f) {
        // d^2 (1/2! + d/3! + ... + d^7/9!): the next term is below 2^-24 of the first
        float p = 1.f / 362880.f;
        p = fmaf(p, d, 1.f / 40320.f);
        p = fmaf(p, d, 1.f / 5040.f);
        p = fmaf(p, d, 1.f / 720.f);
        p = fmaf(p, d, 1.f / 120.f);
        p = fmaf(p, d, 1.f / 24.f);
        p = fmaf(p, d, 1.f / 6.f);
        p = fmaf(p, d, 0.5f);
        return d * d * p;
    }
    return d == INFINITY ? d : expm1f(d) - d;  // its limit, where the label's logit is -inf
}

// A token's inputs, and what its log-probability makes of them.
struct PolicyToken {
    float old_logp, adv, ref_logp, weight;

    __device__ __forceinline__ PolicyToken(const PolicyArgs &a, int64_t t)
        : old_logp(a.old_logp[t]), adv(a.advantages[t]), ref_logp(a.ref_logp ? a.ref_logp[t] : 0.f),
          weight(a.weights ? a.weights[t] : 1.f) {}
};
// w * x for an advantage or a weight w: nothing where w is 0, beside a ratio or a loss past
// FP32's range too (0 * inf would make the loss and the token's gradient row NaN); a NaN stays.
__device__ __forceinline__ float scaled(float w, float x) {
    return w == 0.f && fabsf(x) == INFINITY ? 0.f : w * x;
}
struct PolicyTerms {
    float loss, kl, dlogp;  // dlogp: d loss / d logp
    bool clipped;
};
__device__ __forceinline__ PolicyTerms policy_terms(const PolicyArgs &a, const PolicyToken &in,
                                                    float logp) {
    const float r = expf(logp - in.old_logp);
    const float free = scaled(in.adv, r);
    const float held = fminf(fmaxf(r, a.clip_lo), a.clip_hi) * in.adv;
    PolicyTerms o;
    o.clipped = free > held;
    o.loss = o.clipped ? -held : -free;  // a NaN ratio is not clipped, and stays
    o.dlogp = o.clipped ? 0.f : -free;
    o.kl = 0.f;
    if (a.ref_logp) {
        const float d = in.ref_logp - logp;
        o.kl = kl_term(d);
        if (a.kl_coef != 0.f) {
            o.loss = fmaf(a.kl_coef, o.kl, o.loss);
            o.dlogp = fmaf(-a.kl_coef, expm1f(d), o.dlogp);
        }
    }
    return o;
}

// Counted tokens among the labels, by a warp (WARP) or the whole CTA; every thread returns
// their number.
template <bool WARP>
__device__ __forceinline__ int count_labels(const LogitsArgs &x) {
    int n = 0;
    for (int64_t t = threadIdx.x; t < x.tokens; t += blockDim.x) {
        int64_t label;
        n += load_label(x, t, &label);
    }
    n = __reduce_add_sync(0xffffffffu, n);
    if constexpr (!WARP) {
        __shared__ int total[32];
        if ((threadIdx.x & 31) == 0) total[threadIdx.x / 32] = n;
        __syncthreads();
        n = 0;
        for (int w = 0; w < static_cast<int>(blockDim.x) / 32; ++w) n += total[w];
    }
    return n;
}

// summary[3] = the number of counted tokens, for the rows' kernel.
__global__ void __launch_bounds__(kSummaryThreads) policy_count_kernel(PolicyArgs a) {
    fa_allow_dependents();
    const int n = count_labels<false>(a.x);
    if (threadIdx.x == 0) a.summary[3] = static_cast<float>(n);
}

// Where the rows' kernel has the divisor of a loss without a denominator from.
enum Divisor { kGiven, kFromKernel, kCountHere };

// One row by a cluster of 2^split_log2 CTAs.  HELD > 0: each CTA's part of the row, at most
// 4 * HELD vectors a thread, is read once and held on chip: three groups of HELD vectors
// come to shared memory asynchronously, so that the sum begins when the first has come, the
// fourth to registers (four CTAs of 64 KB rows then fit an SM instead of three: 65,536
// registers and 192 KB of shared memory).  The gradient is made from there: one read and one
// write of the logits, which bound it (16384 rows of 32000 BF16: 318 us with the sums over
// the tokens, 6.3 TB/s; the sum of one CTA and the writes of another overlap, what does not is
// the last wave).  Rows past 64 KB go to clusters (1111 rows of 131072 BF16, four CTAs each:
// 103 us, 5.4 TB/s: 7.3 waves are run as eight, and the parts wait for one another).
// HELD == 0 (rows wider than a cluster holds, or no gradient): the row is read again.
template <int DT, int NT, int HELD>
__global__ void __launch_bounds__(kBlockThreads<NT>,
                                  (HELD == 1 ? 1280 : 1024) / kBlockThreads<NT>)
policy_row_kernel(PolicyArgs a, unsigned split_log2, Divisor divisor) {
    using E = Elem<DT>;
    using T = typename E::T;
    extern __shared__ uint4 slots[];  // [3 * HELD][NT], for each row
    uint4 *slot = NT == 32 ? slots + threadIdx.y * (3 * HELD * NT) : slots;
    __shared__ RowSum parts[kMostSplit * NT / 32];
    const Share sh(split_log2, NT == 32);
    const int64_t t = sh.row, n = a.x.vocab;
    if (NT == 32 && t >= a.x.tokens) return;
    const int tid = threadIdx.x;
    T *out = a.dlogits ? static_cast<T *>(a.dlogits) + t * a.dlogits_ld : nullptr;
    // Nothing here but summary[3] comes from the counting kernel, which began after all
    // earlier work of the stream had ended: only its reader waits for it.
    fa_allow_dependents();
    int64_t label;
    if (!load_label(a.x, t, &label)) {
        if (sh.first() && tid == 0) {
            a.logp[t] = 0.f;
            a.token_loss[t] = 0.f;
            a.token_kl[t] = 0.f;
            if (a.lse) reinterpret_cast<float2 *>(a.lse)[t] = make_float2(0.f, 1.f);
            if (a.dlogp) a.dlogp[t] = 0.f;
        }
        if (out) row_zeros<DT>(out, n, sh);
        if (divisor == kFromKernel) fa_grid_dependency_wait();
        return;
    }
    enter_row(sh);
    const T *row = static_cast<const T *>(a.x.logits) + t * a.x.ld;
    const RowSpan sp = row_span<DT>(row, n);
    const RowPart part(sp, sh);  // HELD: at most 4 * HELD * NT vectors
    const uint4 *q = reinterpret_cast<const uint4 *>(row + sp.head) + part.begin + tid;
    constexpr int kGroup = HELD * NT;
    constexpr int kRegs = HELD > 0 ? HELD : 1;
    uint4 held[kRegs];
    if constexpr (HELD > 0) {
#pragma unroll
        for (int g = 0; g < 3; ++g) {
#pragma unroll
            for (int j = 0; j < HELD; ++j) {
                const int i = g * kGroup + j * NT;
                if (i + tid < part.count && part.in_bounds(i + tid))
                    copy_async16(slot + i + tid, q + i);
            }
            copy_async_commit();
        }
#pragma unroll
        for (int j = 0; j < HELD; ++j) {
            const int i = 3 * kGroup + j * NT;
            held[j] = i + tid < part.count && part.in_bounds(i + tid) ? __ldcs(q + i)
                                                                     : no_vector<DT>();
        }
    }
    // what one thread needs of the token, asked for before the sum
    const bool first = tid == 0;
    const PolicyToken in(a, first ? t : 0);
    const float label_logit = E::widen(row[label]);
    float denom = a.denominator;
    if (divisor == kCountHere) denom = static_cast<float>(count_labels<NT == 32>(a.x));

    RowSum r;
    if constexpr (HELD > 0) {
        Softmax acc(a.x);
        add_ends<DT>(acc, row, sp, n, sh);
        const auto group = [&](int g) {
            const int i0 = g * kGroup;
            if (i0 + (tid & ~31) >= part.count) return;
            const bool full = i0 + kGroup <= part.count;
            uint4 v[kRegs];
#pragma unroll
            for (int j = 0; j < HELD; ++j) {
                const int i = i0 + j * NT + tid;
                v[j] = full || i < part.count ? slot[i] : no_vector<DT>();
            }
            acc.add<DT, HELD>(v);
        };
        copy_async_wait<2>();
        group(0);
        copy_async_wait<1>();
        group(1);
        copy_async_wait<0>();
        group(2);
        if (3 * kGroup + (tid & ~31) < part.count) acc.add<DT, HELD>(held);
        r = merge_row<NT>(acc, parts, sh);
    } else {
        r = row_softmax<DT, NT>(row, a.x, sh);
    }
    float coef = 0.f;
    if (first) {
        const float logp = label_logp(label_logit, r, a.x);
        const PolicyTerms o = policy_terms(a, in, logp);
        if (sh.first()) {
            a.logp[t] = logp;
            a.token_loss[t] = o.loss;
            a.token_kl[t] = o.kl;
            if (a.lse) reinterpret_cast<float2 *>(a.lse)[t] = make_float2(r.top, r.s);
        }
        if (divisor == kFromKernel) {
            fa_grid_dependency_wait();
            denom = a.summary[3];
        }
        const float dlogp = scaled(in.weight / denom, o.dlogp);
        if (a.dlogp && sh.first()) a.dlogp[t] = dlogp;
        coef = dlogp * a.grad_factor;
    }
    if (!out) return;
    if constexpr (NT == 32) {
        coef = __shfl_sync(0xffffffffu, coef, 0);
    } else {
        __shared__ float shared_coef;
        if (first) shared_coef = coef;
        __syncthreads();
        coef = shared_coef;
    }
    if constexpr (HELD > 0) {
        if (((reinterpret_cast<uintptr_t>(row) ^ reinterpret_cast<uintptr_t>(out)) & 15) == 0) {
            const Exponent e(a.x, r.top);
            const float c = coef, w = -c / r.s;
            row_ends(sp, n, sh, [&](int i) { out[i] = E::round(e(E::widen(row[i])) * w); });
            uint4 *o = reinterpret_cast<uint4 *>(out + sp.head) + part.begin + tid;
            const auto write = [&](int i, const uint4 &v) {
                if (part.in_bounds(i + tid)) __stcs(o + i, gradient_vector<DT>(v, e, w));
            };
            if (3 * kGroup + (HELD - 1) * NT + tid < part.count) {  // all of its vectors
#pragma unroll 1
                for (int g = 0; g < 3; ++g)
#pragma unroll
                    for (int j = 0; j < HELD; ++j)
                        write(g * kGroup + j * NT, slot[g * kGroup + j * NT + tid]);
#pragma unroll
                for (int j = 0; j < HELD; ++j) write(3 * kGroup + j * NT, held[j]);
            } else {
#pragma unroll 1
                for (int i = 0; i < 3 * kGroup && i + tid < part.count; i += NT)
                    write(i, slot[i + tid]);
#pragma unroll
                for (int j = 0; j < HELD; ++j)
                    if (3 * kGroup + j * NT + tid < part.count)
                        write(3 * kGroup + j * NT, held[j]);
            }
            if (label_is_mine<DT, NT>(label, sp, part, sh))
                out[label] = E::round(fmaf(e(label_logit), w, c));
            return;
        }
    }
    row_gradient<DT, NT>(row, out, n, a.x, r, coef, label, sh);
}

// The sums over the tokens, by a cluster of CTAs: each adds its tokens, the first adds the
// CTAs' sums in order.  Bound by its own latencies: 6 us for 1111 tokens by one CTA, 8 us for
// 4096 by eight (alone, with cold caches and a CTA-wide sum after the other; all sums in one
// pass take 0.8 us off a call of 1111).
constexpr unsigned kSummaryCtas = 8;
struct PolicySums {
    Sum2 loss, kl;
    int n = 0, clipped = 0;
};
__global__ void __launch_bounds__(kSummaryThreads) policy_summary_kernel(PolicyArgs a) {
    __shared__ PolicySums parts[kSummaryThreads / 32], sums;
    const int lane = threadIdx.x & 31, warps = blockDim.x / 32;
    fa_grid_dependency_wait();
    Sum2 loss, kl;
    int n = 0, clipped = 0;
#pragma unroll 2
    for (int64_t t = blockIdx.x * blockDim.x + threadIdx.x; t < a.x.tokens;
         t += gridDim.x * blockDim.x) {
        int64_t label;
        const bool counted = load_label(a.x, t, &label);
        const PolicyToken in(a, t);  // loaded beside the label
        const float token_loss = a.token_loss[t], token_kl = a.token_kl[t], logp = a.logp[t];
        if (!counted) continue;
        loss.add(scaled(in.weight, token_loss));
        kl.add(token_kl);
        // the ratio and the clip as the rows' kernel took them
        const float r = expf(logp - in.old_logp);
        clipped += r * in.adv > fminf(fmaxf(r, a.clip_lo), a.clip_hi) * in.adv;
        ++n;
    }
    const auto by_warp = [](const PolicySums &s) {
        return PolicySums{warp_sum2(s.loss), warp_sum2(s.kl), __reduce_add_sync(0xffffffffu, s.n),
                          __reduce_add_sync(0xffffffffu, s.clipped)};
    };
    PolicySums all = by_warp(PolicySums{loss, kl, n, clipped});
    if (lane == 0) parts[threadIdx.x / 32] = all;
    __syncthreads();
    if (threadIdx.x < 32) {
        all = by_warp(lane < warps ? parts[lane] : PolicySums{});
        if (lane == 0) sums = all;
    }
    if (gridDim.x > 1) cg::this_cluster().sync();
    if (blockIdx.x == 0 && threadIdx.x == 0) {
        for (unsigned r = 1; r < gridDim.x; ++r) {
            const PolicySums *o = cg::this_cluster().map_shared_rank(&sums, r);
            all.loss.add(o->loss);
            all.kl.add(o->kl);
            all.n += o->n;
            all.clipped += o->clipped;
        }
        const float count = static_cast<float>(all.n), by = fmaxf(count, 1.f);
        a.summary[0] = all.loss.value() / (a.denominator != 0.f ? a.denominator : by);
        a.summary[1] = all.kl.value() / by;
        a.summary[2] = static_cast<float>(all.clipped) / by;
        a.summary[3] = count;
    }
    // no CTA leaves while the first reads its sums
    if (gridDim.x > 1) cg::this_cluster().sync();
}

// CTAs a row is split over (their logarithm) so that a call of few tokens covers the GPU:
// doubled while the grid is under two CTAs an SM and each still has ``least`` vectors.
unsigned split_for(int64_t tokens, int64_t nvec, int64_t least, unsigned log2) {
    while (1 << log2 < kMostSplit && (tokens << log2) < 2 * kSms && nvec >> (log2 + 1) >= least) ++log2;
    return log2;
}

// CTAs and threads for ``tokens`` rows by clusters of 2^log2 CTAs of nt threads a row: with
// more rows of a warp than an SM runs CTAs, kWarpRows to a CTA.
struct RowGrid {
    dim3 ctas, threads;
    RowGrid(int64_t tokens, int nt, unsigned log2) : threads(nt) {
        if (nt == 32 && log2 == 0 && tokens > 32 * kSms) threads.y = kWarpRows;
        ctas = dim3(static_cast<unsigned>((tokens + threads.y - 1) / threads.y << log2));
    }
};

// Calls f with the threads of a CTA that has ``nvec`` vectors of a row: sixteen vectors a
// thread, as far as the sizes go.
template <typename F>
cudaError_t for_threads(int64_t nvec, F f) {
    if (nvec <= 16 * 32) return f(std::integral_constant<int, 32>{});
    if (nvec <= 16 * 64) return f(std::integral_constant<int, 64>{});
    if (nvec <= 16 * 128) return f(std::integral_constant<int, 128>{});
    return f(std::integral_constant<int, kMostThreads>{});
}

}  // namespace

cudaError_t logprob_bounds_violations(unsigned long long *count, bool clear) {
#if FA_BOUNDS_CHECK
    cudaError_t err = cudaMemcpyFromSymbol(count, g_logprob_oob, sizeof(*count));
    if (err != cudaSuccess || !clear) return err;
    const unsigned long long zero = 0;
    return cudaMemcpyToSymbol(g_logprob_oob, &zero, sizeof(zero));
#else
    (void)clear;
    *count = 0;
    return cudaSuccess;
#endif
}

cudaError_t launch_token_logprobs(const LogitsArgs &x, fa_dtype dt, float *logp, float *lse,
                                  cudaStream_t stream) {
    return for_dtype(dt, [&](auto d) {
        const int64_t nvec = x.vocab / Elem<d()>::kVec;
        const unsigned log2 = split_for(x.tokens, nvec, kBatch * kMostThreads, 0);
        if (x.tokens << log2 > kMaxGridX) return cudaErrorInvalidConfiguration;
        // From 24 rows an SM on, twice the vectors a thread: fewer warps begin and join (3648
        // rows of 32000 FP16: 40.9 us against 41.6, BF16 39.8 against 41.8; 912 rows, no longer
        // one wave, FP16: 15.2 against 14.6; the gradient, which joins nothing, gains nothing).
        const int longer = x.tokens >= 24 * kSms;
        return for_threads(nvec >> (log2 + longer), [&](auto nt) {
            const RowGrid g(x.tokens, nt(), log2);
            return launch_clusters(token_logprobs_kernel<d(), nt()>, g.ctas, g.threads, 0,
                                   1u << log2, false, stream, x, logp, lse, log2);
        });
    });
}

cudaError_t launch_token_logprobs_gradient(const LogitGradArgs &a, fa_dtype dt,
                                           cudaStream_t stream) {
    return for_dtype(dt, [&](auto d) {
        const int64_t nvec = a.x.vocab / Elem<d()>::kVec;
        const unsigned log2 = split_for(a.x.tokens, nvec, kBatch * kMostThreads, 0);
        if (a.x.tokens << log2 > kMaxGridX) return cudaErrorInvalidConfiguration;
        return for_threads(nvec >> log2, [&](auto nt) {
            const RowGrid g(a.x.tokens, nt(), log2);
            logprob_gradient_kernel<d(), nt()><<<g.ctas, g.threads, 0, stream>>>(a, log2);
            return cudaGetLastError();
        });
    });
}

cudaError_t launch_preference(const PreferenceArgs &a, fa_itype lt, cudaStream_t stream) {
    return for_itype(lt, [&](auto i) {
        if (a.pairs > 0) {
            const bool whole = a.pairs <= kPairCluster;
            const unsigned pairs = static_cast<unsigned>(a.pairs);
            cudaError_t err =
                launch_clusters(preference_pair_kernel<i()>, dim3(pairs), dim3(kPairThreads), 0,
                                whole ? pairs : 1, true, stream, a);
            if (err != cudaSuccess || whole) return err;
        }
        return launch_dependent(preference_mean_kernel, dim3(1), dim3(kPairThreads), 0, stream, a);
    });
}

namespace {

template <int DT, int NT, int HELD>
cudaError_t launch_policy_rows(const PolicyArgs &a, unsigned log2, Divisor divisor,
                               cudaStream_t stream) {
    constexpr int kSmem = 3 * HELD * NT * 16;
    auto kernel = policy_row_kernel<DT, NT, HELD>;
    if (kSmem >= 48 * 1024) {  // with the static part, past what needs no asking
        cudaError_t err =
            cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
        if (err != cudaSuccess) return err;
    }
    const RowGrid g(a.x.tokens, NT, log2);
    return launch_clusters(kernel, g.ctas, g.threads, kSmem * g.threads.y, 1u << log2,
                           divisor == kFromKernel, stream, a, log2, divisor);
}

}  // namespace

cudaError_t launch_policy(const PolicyArgs &a, fa_dtype dt, cudaStream_t stream) {
    if (a.x.tokens > 0) {
        cudaError_t err = for_dtype(dt, [&](auto d) {
            constexpr int64_t kMost = 4 * 4 * kMostThreads;  // vectors a CTA holds
            const int64_t nvec = a.x.vocab / Elem<d()>::kVec;
            unsigned log2 = 0;
            while (1 << log2 < kMostSplit && nvec > kMost << log2) ++log2;
            const bool held = a.dlogits && nvec <= kMost << log2;
            log2 = split_for(a.x.tokens, nvec, kMostThreads, held ? log2 : 0);
            if (a.x.tokens << log2 > kMaxGridX) return cudaErrorInvalidConfiguration;
            const int64_t each = (nvec + (int64_t(1) << log2) - 1) >> log2;
            return for_threads(each, [&](auto nt) {
                // Every CTA counts the labels itself when that is a few loads a thread (a
                // launch less); else one kernel does before the rows'.
                const bool counts = (a.dlogits || a.dlogp) && a.denominator == 0.f;
                const Divisor divisor = !counts                   ? kGiven
                                        : a.x.tokens <= 8 * nt() ? kCountHere
                                                                 : kFromKernel;
                if (divisor == kFromKernel) {
                    policy_count_kernel<<<1, kSummaryThreads, 0, stream>>>(a);
                    cudaError_t e = cudaGetLastError();
                    if (e != cudaSuccess) return e;
                }
                if (!held) return launch_policy_rows<d(), nt(), 0>(a, log2, divisor, stream);
                // (rows of up to four vectors a lane of one warp)
                if (nt() == 32 && each <= 4 * 32)
                    return launch_policy_rows<d(), 32, 1>(a, log2, divisor, stream);
                return launch_policy_rows<d(), nt(), 4>(a, log2, divisor, stream);
            });
        });
        if (err != cudaSuccess) return err;
    }
    const unsigned ctas = a.x.tokens > 2 * kSummaryThreads ? kSummaryCtas : 1;
    const unsigned warps = static_cast<unsigned>(
        std::min<int64_t>(std::max<int64_t>(1, (a.x.tokens + 31) / 32), kSummaryThreads / 32));
    return launch_clusters(policy_summary_kernel, dim3(ctas), dim3(32 * warps), 0, ctas, true,
                           stream, a);
}

}  // namespace fa
