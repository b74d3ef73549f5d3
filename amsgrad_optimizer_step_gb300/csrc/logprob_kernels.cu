// Token log-probabilities from logits, their gradient, and the two losses built on
// them: the preference loss from paired log ratios and the clipped policy loss.
//
// Row t of the logits is a softmax over vocab ids after multiplication by scale:
//   top = max_v x_v,  s = sum_v exp(scale (x_v - top)),
//   logp = scale (x_label - top) - ln s,
//   dlogits_v = c (1[v = label] - exp(scale (x_v - top)) / s).
// exp(scale (x - top)) is 2^(k x - k top) with k = scale log2(e): one fused
// multiply-add whose product is exact, so that every term of a row, and its label's,
// carries the same rounding of k top; rows whose k top leaves FP32's range (masks of
// the type's lowest value) take the difference first.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "internal.h"
#include "model_device.cuh"
#include "model_internal.h"

namespace fa {
namespace {

FA_BOUNDS_COUNTER(g_logprob_oob)

constexpr int kRowThreads = 256;
constexpr int kBatch = 4;  // 16-byte vectors a thread has in flight

// A row cut for 16-byte accesses: head scalars up to the first boundary, then nvec
// vectors, then the scalars left over.
struct RowSpan {
    int64_t head, nvec, n;
};
template <int DT>
__device__ __forceinline__ RowSpan row_span(const void *row, int64_t n) {
    constexpr int V = Elem<DT>::kVec;
    const int64_t past = (reinterpret_cast<uintptr_t>(row) & 15) / sizeof(typename Elem<DT>::T);
    RowSpan r;
    r.n = n;
    r.head = past ? V - past : 0;
    if (r.head > n) r.head = n;
    r.nvec = (n - r.head) / V;
    return r;
}

// The running maximum and the sum of 2^(k (x - top)) over some of a row's elements.
struct Softmax {
    float top = -INFINITY, s = 0.f;

    // 2^(k x - k top), by one FMA where k top is finite.
    static __device__ __forceinline__ float term(float x, float top, float k, float ktop) {
        return isfinite(ktop) ? exp2_fast(fmaf(x, k, -ktop)) : exp2_fast((x - top) * k);
    }

    template <int N>
    __device__ __forceinline__ void add(const float *x, float k) {
        float best = x[0];
#pragma unroll
        for (int j = 1; j < N; ++j) best = fmaxf(best, x[j]);
        if (best > top) {
            s = s == 0.f ? 0.f : s * exp2_fast((top - best) * k);
            top = best;
        }
        if (top == -INFINITY) {  // nothing but -inf (and NaN) so far
#pragma unroll
            for (int j = 0; j < N; ++j)
                if (isnan(x[j])) s = x[j];
            return;
        }
        const float ktop = k * top;
#pragma unroll
        for (int j = 0; j < N; ++j) s += term(x[j], top, k, ktop);
    }
    __device__ __forceinline__ void merge(const Softmax &o, float k) {
        const float best = fmaxf(top, o.top);
        // a part without any finite value keeps its sum (0, or NaN)
        const float a = top == best || top == -INFINITY ? s : s * exp2_fast((top - best) * k);
        const float b = o.top == best || o.top == -INFINITY ? o.s
                                                            : o.s * exp2_fast((o.top - best) * k);
        top = best;
        s = a + b;
    }
};

// The softmax statistics of one row, by the whole CTA; every thread returns them.
template <int DT>
__device__ __forceinline__ Softmax row_softmax(const void *row, int64_t n, float k) {
    using E = Elem<DT>;
    using T = typename E::T;
    const T *x = static_cast<const T *>(row);
    const RowSpan sp = row_span<DT>(row, n);
    Softmax acc;
    const int t = threadIdx.x, nt = blockDim.x;
    if (t < sp.head && fa_in_bounds(t, 1, n)) {
        const float v = E::widen(x[t]);
        acc.add<1>(&v, k);
    }
    const uint4 *q = reinterpret_cast<const uint4 *>(x + sp.head);
    int64_t i = t;
    for (; i + (kBatch - 1) * nt < sp.nvec; i += kBatch * nt) {
        uint4 r[kBatch];
#pragma unroll
        for (int j = 0; j < kBatch; ++j) r[j] = __ldg(q + i + j * nt);
        float v[kBatch * E::kVec];
#pragma unroll
        for (int j = 0; j < kBatch; ++j) E::unpack(r[j], v + j * E::kVec);
        acc.add<kBatch * E::kVec>(v, k);
    }
    for (; i < sp.nvec; i += nt) {
        float v[E::kVec];
        E::unpack(__ldg(q + i), v);
        acc.add<E::kVec>(v, k);
    }
    const int64_t tail = sp.head + sp.nvec * E::kVec + t;
    if (tail < n && fa_in_bounds(tail, 1, n)) {
        const float v = E::widen(x[tail]);
        acc.add<1>(&v, k);
    }
    // lanes, then warps
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        Softmax other;
        other.top = __shfl_xor_sync(0xffffffffu, acc.top, o);
        other.s = __shfl_xor_sync(0xffffffffu, acc.s, o);
        acc.merge(other, k);
    }
    __shared__ Softmax part[32];
    const int warps = nt / 32;
    __syncthreads();  // part may still be read for the row before
    if ((t & 31) == 0) part[t / 32] = acc;
    __syncthreads();
    acc = part[0];
    for (int w = 1; w < warps; ++w) acc.merge(part[w], k);
    if (acc.top == -INFINITY) acc.s = NAN;  // no finite logit
    return acc;
}

// logp of the label from its logit and the row's statistics: the exponent is the one the
// sum's terms have, so that the rounding of k top cancels.
__device__ __forceinline__ float label_logp(float x, const Softmax &r, const LogitsArgs &a) {
    constexpr float kLn2 = 0.693147180559945309f;
    const float ktop = a.k * r.top;
    const float d = isfinite(ktop) ? fmaf(x, a.k, -ktop) * kLn2 : (x - r.top) * a.scale;
    return d - logf(r.s);
}

template <int IT>
__device__ __forceinline__ bool load_label(const LogitsArgs &x, int64_t t, int64_t *label) {
    *label = load_id<IT>(x.labels, t);
    return *label >= 0 && *label < x.vocab;
}

// dlogits of one row: c (1[v = label] - 2^(k (x - top)) / s), by the whole CTA.  The
// output may be the row itself: every element is read before it is written, by the
// thread that writes it.
template <int DT>
__device__ __forceinline__ void row_gradient(const void *row, void *out, int64_t n, float k,
                                             Softmax r, float c, int64_t label, int t, int nt) {
    using E = Elem<DT>;
    using T = typename E::T;
    const T *x = static_cast<const T *>(row);
    T *y = static_cast<T *>(out);
    const float ktop = k * r.top, w = -c / r.s;
    const auto one = [&](int64_t i) {
        if (!fa_in_bounds(i, 1, n)) return;
        const float p = Softmax::term(E::widen(x[i]), r.top, k, ktop) * w;
        y[i] = E::round(i == label ? p + c : p);
    };
    RowSpan sp = row_span<DT>(row, n);
    if ((reinterpret_cast<uintptr_t>(row) ^ reinterpret_cast<uintptr_t>(out)) & 15) {
        for (int64_t i = t; i < n; i += nt) one(i);  // the two are not co-aligned
        return;
    }
    if (t < sp.head) one(t);
    const uint4 *q = reinterpret_cast<const uint4 *>(x + sp.head);
    uint4 *o = reinterpret_cast<uint4 *>(y + sp.head);
    for (int64_t i = t; i < sp.nvec; i += nt) {
        float v[E::kVec];
        E::unpack(q[i], v);
#pragma unroll
        for (int j = 0; j < E::kVec; ++j) v[j] = Softmax::term(v[j], r.top, k, ktop) * w;
        const int64_t at = label - sp.head - i * E::kVec;
#pragma unroll
        for (int j = 0; j < E::kVec; ++j)
            if (at == j) v[j] += c;
        __stcs(o + i, E::pack(v));
    }
    const int64_t tail = sp.head + sp.nvec * E::kVec + t;
    if (tail < n) one(tail);
}

// Zeros for the row of a token that is not counted.
template <int DT>
__device__ __forceinline__ void row_zeros(void *out, int64_t n, int t, int nt) {
    using E = Elem<DT>;
    using T = typename E::T;
    T *y = static_cast<T *>(out);
    const RowSpan sp = row_span<DT>(out, n);
    if (t < sp.head && fa_in_bounds(t, 1, n)) y[t] = E::round(0.f);
    uint4 *o = reinterpret_cast<uint4 *>(y + sp.head);
    for (int64_t i = t; i < sp.nvec; i += nt) __stcs(o + i, make_uint4(0u, 0u, 0u, 0u));
    const int64_t tail = sp.head + sp.nvec * E::kVec + t;
    if (tail < n && fa_in_bounds(tail, 1, n)) y[tail] = E::round(0.f);
}

template <int DT, int IT>
__global__ void __launch_bounds__(kRowThreads)
token_logprobs_kernel(LogitsArgs x, float *logp, float *lse) {
    using T = typename Elem<DT>::T;
    const int64_t t = blockIdx.x;
    int64_t label;
    if (!load_label<IT>(x, t, &label)) {
        if (threadIdx.x == 0) {
            logp[t] = 0.f;
            if (lse) reinterpret_cast<float2 *>(lse)[t] = make_float2(0.f, 1.f);
        }
        return;
    }
    const T *row = static_cast<const T *>(x.logits) + t * x.ld;
    const Softmax r = row_softmax<DT>(row, x.vocab, x.k);
    if (threadIdx.x == 0) {
        logp[t] = label_logp(Elem<DT>::widen(row[label]), r, x);
        if (lse) reinterpret_cast<float2 *>(lse)[t] = make_float2(r.top, r.s);
    }
}

template <int DT, int IT>
__global__ void __launch_bounds__(kRowThreads) logprob_gradient_kernel(LogitGradArgs a) {
    using T = typename Elem<DT>::T;
    const int64_t t = blockIdx.x;
    T *out = static_cast<T *>(a.dlogits) + t * a.dlogits_ld;
    int64_t label;
    if (!load_label<IT>(a.x, t, &label)) {
        row_zeros<DT>(out, a.x.vocab, threadIdx.x, kRowThreads);
        return;
    }
    const T *row = static_cast<const T *>(a.x.logits) + t * a.x.ld;
    const float2 l = reinterpret_cast<const float2 *>(a.lse)[t];
    Softmax r;
    r.top = l.x;
    r.s = l.y;
    const float c = a.dlogp[t] * a.factor * (a.grad_loss ? *a.grad_loss : 1.f);
    row_gradient<DT>(row, out, a.x.vocab, a.x.k, r, c, label, threadIdx.x, kRowThreads);
}

// ---- preference loss ------------------------------------------------------------

constexpr int kPairThreads = 256;

// Sum of one value a thread over the CTA, as FP32 pairs; every thread returns it.
__device__ __forceinline__ Sum2 cta_sum2(Sum2 s) {
    __shared__ Sum2 part[32];
    s = warp_sum2(s);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) part[threadIdx.x / 32] = s;
    __syncthreads();
    Sum2 total = part[0];
    for (int w = 1; w < static_cast<int>(blockDim.x) / 32; ++w) total.add(part[w]);
    return total;
}

// ln(1 + e^z) without overflow.
__device__ __forceinline__ float softplus(float z) {
    return fmaxf(z, 0.f) + log1pf(expf(-fabsf(z)));
}

// One CTA per pair: both sequences' sums, the pair's loss and the coefficient of each of
// its tokens.  Tokens of no sequence are zeroed by the first and the last pair's CTA.
template <int IT>
__global__ void __launch_bounds__(kPairThreads) preference_pair_kernel(PreferenceArgs a) {
    fa_allow_dependents();
    const int64_t pair = blockIdx.x;
    const auto clamped = [&](int64_t j) {
        const int64_t o = a.seq_offsets[j];
        return o < 0 ? 0 : o > a.tokens ? a.tokens : o;
    };
    const auto counted = [&](int64_t t) {
        const int64_t label = load_id<IT>(a.labels, t);
        return label >= 0 && label < a.vocab;
    };
    int64_t lo[2], hi[2];
    float mean[2], per[2];
    for (int q = 0; q < 2; ++q) {
        lo[q] = clamped(2 * pair + q);
        hi[q] = clamped(2 * pair + q + 1);
        Sum2 s, n;
        for (int64_t t = lo[q] + threadIdx.x; t < hi[q]; t += kPairThreads)
            if (counted(t) && fa_in_bounds(t, 1, a.tokens)) {
                s.add(a.logp[t] - a.ref_logp[t]);
                n.add(1.f);
            }
        s = cta_sum2(s);
        n = cta_sum2(n);
        per[q] = a.average ? 1.f / fmaxf(n.value(), 1.f) : 1.f;
        mean[q] = a.average ? s.value() / fmaxf(n.value(), 1.f) : s.value();
    }
    const float z = a.beta * (mean[0] - mean[1]);
    const float e = a.smoothing;
    // d pair_loss / dz = -(1 - e) sigmoid(-z) + e sigmoid(z)
    const float dz = e / (1.f + expf(-z)) - (1.f - e) / (1.f + expf(z));
    const float d = dz * a.beta / static_cast<float>(a.pairs);
    if (threadIdx.x == 0) {
        const float keep = (1.f - e) * softplus(-z);
        a.pair_loss[pair] = e > 0.f ? keep + e * softplus(z) : keep;
        a.rewards[2 * pair] = a.beta * mean[0];
        a.rewards[2 * pair + 1] = a.beta * mean[1];
    }
    for (int q = 0; q < 2; ++q) {
        const float c = (q ? -d : d) * per[q];
        for (int64_t t = lo[q] + threadIdx.x; t < hi[q]; t += kPairThreads)
            if (fa_in_bounds(t, 1, a.tokens)) a.dlogp[t] = counted(t) ? c : 0.f;
    }
    if (pair == 0)
        for (int64_t t = threadIdx.x; t < lo[0]; t += kPairThreads) a.dlogp[t] = 0.f;
    if (pair == a.pairs - 1)
        for (int64_t t = hi[1] + threadIdx.x; t < a.tokens; t += kPairThreads) a.dlogp[t] = 0.f;
}

// The mean over the pairs, by one CTA (no pairs: 0, and no token has a coefficient).
__global__ void __launch_bounds__(kPairThreads) preference_mean_kernel(PreferenceArgs a) {
    fa_grid_dependency_wait();
    Sum2 s;
    for (int64_t k = threadIdx.x; k < a.pairs; k += kPairThreads) s.add(a.pair_loss[k]);
    s = cta_sum2(s);
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
    return expm1f(d) - d;
}

struct PolicyToken {
    float loss, kl, dlogp;  // dlogp: d loss / d logp
    bool clipped;
};
__device__ __forceinline__ PolicyToken policy_token(const PolicyArgs &a, int64_t t, float logp) {
    const float r = expf(logp - a.old_logp[t]), adv = a.advantages[t];
    const float free = r * adv, held = fminf(fmaxf(r, a.clip_lo), a.clip_hi) * adv;
    PolicyToken o;
    o.clipped = free > held;
    o.kl = 0.f;
    o.dlogp = free <= held ? -free : 0.f;
    // a NaN ratio stays one (fminf would drop it)
    o.loss = isnan(free) ? free : o.clipped ? -held : -free;
    if (isnan(free)) o.dlogp = free;
    if (a.ref_logp) {
        const float d = a.ref_logp[t] - logp;
        o.kl = kl_term(d);
        if (a.kl_coef != 0.f) {
            o.loss = fmaf(a.kl_coef, o.kl, o.loss);
            o.dlogp = fmaf(-a.kl_coef, expm1f(d), o.dlogp);
        }
    }
    return o;
}

// summary[3] = the number of counted tokens.
template <int IT>
__global__ void __launch_bounds__(kSummaryThreads) policy_count_kernel(PolicyArgs a) {
    fa_allow_dependents();
    int n = 0;
    for (int64_t t = threadIdx.x; t < a.x.tokens; t += kSummaryThreads) {
        int64_t label;
        n += load_label<IT>(a.x, t, &label);
    }
    __shared__ int total[kSummaryThreads / 32];
    n = __reduce_add_sync(0xffffffffu, n);
    if ((threadIdx.x & 31) == 0) total[threadIdx.x / 32] = n;
    __syncthreads();
    if (threadIdx.x == 0) {
        for (int w = 1; w < kSummaryThreads / 32; ++w) n += total[w];
        a.summary[3] = static_cast<float>(n);
    }
}

template <int DT, int IT>
__global__ void __launch_bounds__(kRowThreads) policy_row_kernel(PolicyArgs a) {
    using T = typename Elem<DT>::T;
    const int64_t t = blockIdx.x;
    T *out = a.dlogits ? static_cast<T *>(a.dlogits) + t * a.dlogits_ld : nullptr;
    fa_grid_dependency_wait();
    fa_allow_dependents();
    int64_t label;
    if (!load_label<IT>(a.x, t, &label)) {
        if (threadIdx.x == 0) {
            a.logp[t] = 0.f;
            a.token_loss[t] = 0.f;
            a.token_kl[t] = 0.f;
        }
        if (out) row_zeros<DT>(out, a.x.vocab, threadIdx.x, kRowThreads);
        return;
    }
    const T *row = static_cast<const T *>(a.x.logits) + t * a.x.ld;
    const Softmax r = row_softmax<DT>(row, a.x.vocab, a.x.k);
    __shared__ float coef;
    if (threadIdx.x == 0) {
        const float logp = label_logp(Elem<DT>::widen(row[label]), r, a.x);
        const PolicyToken o = policy_token(a, t, logp);
        a.logp[t] = logp;
        a.token_loss[t] = o.loss;
        a.token_kl[t] = o.kl;
        const float denom = a.denominator != 0.f ? a.denominator : a.summary[3];
        const float w = (a.weights ? a.weights[t] : 1.f) / denom;
        coef = o.dlogp * w * a.grad_factor;
    }
    if (!out) return;
    __syncthreads();
    row_gradient<DT>(row, out, a.x.vocab, a.x.k, r, coef, label, threadIdx.x, kRowThreads);
}

// The sums over the tokens, by one CTA.
template <int IT>
__global__ void __launch_bounds__(kSummaryThreads) policy_summary_kernel(PolicyArgs a) {
    fa_grid_dependency_wait();
    Sum2 loss, kl, clipped;
    for (int64_t t = threadIdx.x; t < a.x.tokens; t += kSummaryThreads) {
        int64_t label;
        if (!load_label<IT>(a.x, t, &label)) continue;
        loss.add(a.weights ? a.weights[t] * a.token_loss[t] : a.token_loss[t]);
        kl.add(a.token_kl[t]);
        const float r = expf(a.logp[t] - a.old_logp[t]), adv = a.advantages[t];
        if (r * adv > fminf(fmaxf(r, a.clip_lo), a.clip_hi) * adv) clipped.add(1.f);
    }
    loss = cta_sum2(loss);
    kl = cta_sum2(kl);
    clipped = cta_sum2(clipped);
    if (threadIdx.x == 0) {
        const float n = a.summary[3], by = fmaxf(n, 1.f);
        a.summary[0] = loss.value() / (a.denominator != 0.f ? a.denominator : by);
        a.summary[1] = kl.value() / by;
        a.summary[2] = clipped.value() / by;
    }
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

cudaError_t launch_token_logprobs(const LogitsArgs &x, fa_dtype dt, fa_itype lt, float *logp,
                                  float *lse, cudaStream_t stream) {
    return for_dtype(dt, [&](auto d) {
        return for_itype(lt, [&](auto i) {
            token_logprobs_kernel<d(), i()>
                <<<static_cast<unsigned>(x.tokens), kRowThreads, 0, stream>>>(x, logp, lse);
            return cudaGetLastError();
        });
    });
}

cudaError_t launch_token_logprobs_gradient(const LogitGradArgs &a, fa_dtype dt, fa_itype lt,
                                           cudaStream_t stream) {
    return for_dtype(dt, [&](auto d) {
        return for_itype(lt, [&](auto i) {
            logprob_gradient_kernel<d(), i()>
                <<<static_cast<unsigned>(a.x.tokens), kRowThreads, 0, stream>>>(a);
            return cudaGetLastError();
        });
    });
}

cudaError_t launch_preference(const PreferenceArgs &a, fa_itype lt, cudaStream_t stream) {
    return for_itype(lt, [&](auto i) {
        if (a.pairs > 0) {
            preference_pair_kernel<i()>
                <<<static_cast<unsigned>(a.pairs), kPairThreads, 0, stream>>>(a);
            cudaError_t err = cudaGetLastError();
            if (err != cudaSuccess) return err;
        }
        return launch_dependent(preference_mean_kernel, dim3(1), dim3(kPairThreads), 0, stream, a);
    });
}

cudaError_t launch_policy(const PolicyArgs &a, fa_dtype dt, fa_itype lt, cudaStream_t stream) {
    return for_itype(lt, [&](auto i) {
        policy_count_kernel<i()><<<1, kSummaryThreads, 0, stream>>>(a);
        cudaError_t err = cudaGetLastError();
        if (err != cudaSuccess) return err;
        if (a.x.tokens > 0) {
            err = for_dtype(dt, [&](auto d) {
                return launch_dependent(policy_row_kernel<d(), i()>,
                                        dim3(static_cast<unsigned>(a.x.tokens)),
                                        dim3(kRowThreads), 0, stream, a);
            });
            if (err != cudaSuccess) return err;
        }
        return launch_dependent(policy_summary_kernel<i()>, dim3(1), dim3(kSummaryThreads), 0,
                                stream, a);
    });
}

}  // namespace fa
