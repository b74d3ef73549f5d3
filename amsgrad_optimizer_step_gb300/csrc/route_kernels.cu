// The router of gated experts: choice, weights, counts and the balance loss of tokens from
// their logits, and the logits' gradient.
//
// A token's row belongs to a group of 1 to 32 lanes, up to 16 experts a lane (32 beyond 512), in
// registers.  Up to eight experts are chosen from lists: every lane sorts its keys once, keeping
// eight, and a choice is the maximum of the lists' heads, whose lane moves on to its next.  Keys are
// integers in the logits' order with the expert's number in their low bits, so that one maximum
// gives the expert, ties to the lower number: those of 16-bit logits hold the whole logit, those
// of FP32 its upper bits, and where two of the keys that matter agree in these (one token in some
// hundred) the warp chooses again by whole logits, an expert at a time, which is also how more
// than eight are chosen.  Sums over tokens stay with the lane that holds the expert, then go by
// CTA and in order.
//
// Exponentials and quotients are the hardware's, two units each in the last place beside the rounding of
// an exponential's argument, as the weights' and probabilities' bounds in the tests have it; the
// logarithm is the library's, since the hardware's error is absolute and the sum is often next to 1.
//
// 65536 tokens, 8 of 128 experts, BF16, take 21 us, of which the bytes need 3 (51 with a maximum over
// all keys for every choice), the join of the CTAs' sums 8 and the gradient 16.5; 8 of 256, FP32, 49, 8
// and 30.5.  Neither memory (10 to 34 % of its rate) nor issue slots (59 and 53 %, the gradient 53 and
// 47) bound it: with 80 registers a thread a third of the warps fit an SM, and a warp spends 26 % of its
// time waiting for memory (the gradient 42 to 53): for its logits and the chosen ones' second reading;
// 13 to 16 % for shuffles and shared memory, 15 to 18 % for the arithmetic before it.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "internal.h"

FA_BOUNDS_COUNTER(g_route_oob)

#include "block_internal.h"
#include "model_runs.cuh"

namespace fa {
namespace {

constexpr int kRouteThreads = 256;
constexpr int kRouteCtas = 3;  // on an SM: what 80 registers a thread allow
constexpr int kRouteWarps = kRouteThreads / 32;
constexpr int kGradThreads = 256;
constexpr int kListed = 8;  // keys of a lane's list, and experts chosen from lists at most
constexpr float kLog2E = 1.4426950408889634f;

// Keys in the order of the logits: larger logits have larger keys, -0 and 0 the same one, and
// every NaN the largest (an addition's NaN is 0x7fffffff, whatever went in).
__device__ __forceinline__ uint32_t whole_key(float x) {
    const uint32_t b = __float_as_uint(__fadd_rn(x, 0.f));  // -0 becomes 0
    return b ^ (static_cast<uint32_t>(static_cast<int32_t>(b) >> 31) | 0x80000000u);
}
// With the expert's number in the low BITS, ten at most: the widened 16-bit types have 13 or 16
// zeros there.
template <int BITS>
__device__ __forceinline__ uint32_t numbered_key(float x, int expert) {
    constexpr uint32_t kNumber = (1u << BITS) - 1;
    return (whole_key(x) & ~kNumber) | (kNumber - static_cast<uint32_t>(expert));
}

template <int L>
__device__ __forceinline__ float group_sum(float x) {
#pragma unroll
    for (int o = L / 2; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    return x;
}
template <int L>
__device__ __forceinline__ uint32_t group_max(uint32_t x) {
#pragma unroll
    for (int o = L / 2; o > 0; o >>= 1) x = max(x, __shfl_xor_sync(0xffffffffu, x, o));
    return x;
}

__device__ __forceinline__ void order(uint32_t &a, uint32_t &b) {
    const uint32_t hi = max(a, b);
    b = min(a, b);
    a = hi;
}
// Eight keys, the largest first (Batcher's odd-even merge network: 19 exchanges).
__device__ __forceinline__ void sort8(uint32_t *k) {
    order(k[0], k[1]), order(k[2], k[3]), order(k[4], k[5]), order(k[6], k[7]);
    order(k[0], k[2]), order(k[1], k[3]), order(k[4], k[6]), order(k[5], k[7]);
    order(k[1], k[2]), order(k[5], k[6]);
    order(k[0], k[4]), order(k[1], k[5]), order(k[2], k[6]), order(k[3], k[7]);
    order(k[2], k[4]), order(k[3], k[5]);
    order(k[1], k[2]), order(k[3], k[4]), order(k[5], k[6]);
}
// The largest eight of two such lists, in a: the larger ones of a and of b backwards rise and
// fall once, which three steps sort.
__device__ __forceinline__ void merge8(uint32_t *a, const uint32_t *b) {
#pragma unroll
    for (int j = 0; j < 8; ++j) a[j] = max(a[j], b[7 - j]);
#pragma unroll
    for (int d = 4; d > 0; d >>= 1)
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (!(j & d)) order(a[j], a[j + d]);
}

// A lane's experts: R runs of eight, L runs apart.
template <int L>
__device__ __forceinline__ int expert_of(int part, int j) {
    return ((j / kRun) * L + part) * kRun + j % kRun;
}
template <int DT, int L, int R>
__device__ __forceinline__ void load_logits(const MatrixArgs &m, int64_t row, int part, bool vec,
                                            float *x) {
#pragma unroll
    for (int r = 0; r < R; ++r) {
        const int c = (r * L + part) * kRun;
        const Raw<DT, kRun> raw =
            vec ? load_run<DT, true>(m, row, c) : load_run<DT, false>(m, row, c);
        raw.widen(x + r * kRun);
    }
    if (L * R * kRun == m.cols) return;
#pragma unroll
    for (int j = 0; j < R * kRun; ++j)
        if (expert_of<L>(part, j) >= m.cols) x[j] = -INFINITY;
}

// Calls take(i, expert) in every lane of a group for the choices i < k, by whole logits.
template <int L, int N, typename Take>
__device__ __forceinline__ void choose_whole(const float *x, int part, int experts, int k,
                                             Take take) {
    uint32_t gone = 0;  // of this lane's
    for (int i = 0; i < k; ++i) {
        uint32_t best = 0;
        int mine = 0x7fffffff;
#pragma unroll
        for (int j = 0; j < N; ++j) {
            const int e = expert_of<L>(part, j);
            const uint32_t key = e < experts && !(gone >> j & 1u) ? whole_key(x[j]) : 0u;
            if (key > best) {
                best = key;
                mine = e;
            }
        }
        const uint32_t top = group_max<L>(best);
        if (best != top) mine = 0x7fffffff;
        int e = mine;
#pragma unroll
        for (int o = L / 2; o > 0; o >>= 1) e = min(e, __shfl_xor_sync(0xffffffffu, e, o));
#pragma unroll
        for (int j = 0; j < N; ++j)
            if (expert_of<L>(part, j) == e) gone |= 1u << j;
        take(i, e);
    }
}

// What a CTA leaves of its tokens: per expert the probabilities' sum and the count, then z's sum
// and the counted tokens.
struct RouteSums {
    float *prob;   // [ctas][experts]
    int32_t *count;  // [ctas][experts]
    float *z;        // [ctas]
    int32_t *tokens;  // [ctas]
    float *dot;      // of the joining CTAs: sums of counts * mean probability
    int32_t *joined;  // how many of them are done
};
__host__ __device__ inline RouteSums route_sums(void *scratch, int64_t ctas, int64_t experts) {
    RouteSums s;
    s.prob = static_cast<float *>(scratch);
    s.count = reinterpret_cast<int32_t *>(s.prob + ctas * experts);
    s.z = reinterpret_cast<float *>(s.count + ctas * experts);
    s.tokens = reinterpret_cast<int32_t *>(s.z + ctas);
    s.dot = reinterpret_cast<float *>(s.tokens + ctas);
    s.joined = reinterpret_cast<int32_t *>(s.dot + FA_ROUTE_MAX_EXPERTS / 8);
    return s;
}

// L lanes a token, R runs of eight experts a lane.  LISTED: at most kListed are chosen.
template <int DT, int L, int R, bool LISTED>
__global__ void __launch_bounds__(kRouteThreads, R < 4 ? kRouteCtas : 2)
route_kernel(RouteArgs a, bool vec) {
    constexpr int kTokens = 32 / L, N = R * kRun;  // tokens of a warp's turn; a lane's experts
    constexpr int kBits = 31 - __builtin_clz(L * N);
    constexpr int kItems = ((LISTED ? kListed : FA_ROUTE_MAX_CHOSEN) + L - 1) / L;  // of a lane
    extern __shared__ uint32_t shared[];
    int32_t *const count = reinterpret_cast<int32_t *>(shared);  // the CTA's
    const int k = a.top_k, warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int sub = lane / L, part = lane % L;
    const int64_t tokens = a.logits.rows;
    const int experts = static_cast<int>(a.logits.cols);
    const bool sums = a.summary != nullptr;
    if (sums) {
        for (int e = threadIdx.x; e < experts; e += kRouteThreads) count[e] = 0;
        // how many CTAs have joined the sums, for the kernel that does
        if (blockIdx.x == 0 && threadIdx.x == 0)
            *route_sums(a.scratch, gridDim.x, experts).joined = 0;
        __syncthreads();
    }
    float prob[N] = {}, z = 0.f;
    int counted = 0;
    const int64_t step = static_cast<int64_t>(gridDim.x) * kRouteWarps * kTokens;
    for (int64_t t0 = (static_cast<int64_t>(blockIdx.x) * kRouteWarps + warp) * kTokens;
         t0 < tokens; t0 += step) {
        const int64_t t = t0 + sub;
        const bool on = t < tokens && (!a.counted || a.counted[t]);
        float x[N];
        if (on) {
            load_logits<DT, L, R>(a.logits, t, part, vec, x);
        } else {
#pragma unroll
            for (int j = 0; j < N; ++j) x[j] = 0.f;
        }
        int item[kItems];  // the choices part, part + L, ... of the token
        const auto take = [&](int i, int e) {
#pragma unroll
            for (int s = 0; s < kItems; ++s)
                if (i == s * L + part) item[s] = e;
        };
        bool again = !LISTED;
        if (LISTED) {
            constexpr uint32_t kNumber = (1u << kBits) - 1;
            uint32_t key[N], cut = 0;
            // (what is past the last expert is -infinity, and its number is behind all that there are)
#pragma unroll
            for (int j = 0; j < N; ++j) key[j] = numbered_key<kBits>(x[j], expert_of<L>(part, j));
#pragma unroll
            for (int r = 0; r < R; ++r) sort8(key + r * kRun);
#pragma unroll
            for (int r = 1; r < R; ++r) {
                if (DT == FA_F32 && k == kListed)  // the largest key that a list of eight leaves out
#pragma unroll
                    for (int j = 0; j < kRun; ++j) cut = max(cut, min(key[j], key[r * kRun + 7 - j]));
                merge8(key, key + r * kRun);
            }
            uint32_t before = 0xffffffffu;
            bool same = false;
#pragma unroll
            for (int i = 0; i <= kListed; ++i) {
                // (FP32 asks for one more, which the last choice has to be above)
                if (i > k || (i == k && (DT != FA_F32 || k == experts))) break;
                // a lane that gave all eight has its ninth outside its list (65536 tokens whose largest lie in
                // one of 32 runs: 43 us, 111 where such lanes were all chosen again; 3 % of any other)
                if (DT == FA_F32 && R > 1 && i == kListed) key[0] = max(key[0], cut);
                const uint32_t best = group_max<L>(key[0]);
                if (DT == FA_F32) same |= i > 0 && (best | kNumber) == (before | kNumber);
                before = best;
                if (i == k) break;
                take(i, static_cast<int>(kNumber - (best & kNumber)));
                if (key[0] == best) {  // the keys are distinct: one lane of the group
#pragma unroll
                    for (int j = 0; j < kListed - i; ++j)  // as far as later choices reach
                        key[j] = j + 1 < kListed ? key[j + 1] : 0u;
                }
            }
            if (DT == FA_F32) again = __any_sync(0xffffffffu, same && on);
        }
        if (again) choose_whole<L, N>(x, part, experts, k, take);
        // the first choice is the row's largest logit
        float ex[kItems], picked = 0.f;
#pragma unroll
        for (int s = 0; s < kItems; ++s) {
            ex[s] = 0.f;
            if (s * L + part < k && on) {
                const auto *p = static_cast<const typename Elem<DT>::T *>(a.logits.p);
                ex[s] = Elem<DT>::widen(p[t * a.logits.ld + item[s]]);
            }
        }
        const float top = __shfl_sync(0xffffffffu, ex[0], 0, L);
        float total = 0.f;
#pragma unroll
        for (int j = 0; j < N; ++j) {
            x[j] = exp2_fast((x[j] - top) * kLog2E);
            total += x[j];
        }
        total = group_sum<L>(total);
#pragma unroll
        for (int s = 0; s < kItems; ++s)
            if (s * L + part < k && on) {
                ex[s] = exp2_fast((ex[s] - top) * kLog2E);
                picked += ex[s];
                if (sums) atomicAdd(count + item[s], 1);
            }
        picked = group_sum<L>(picked);
        const float factor = __fdividef(a.weight_scale, a.renormalise ? picked : total);
#pragma unroll
        for (int s = 0; s < kItems; ++s) {
            const int i = s * L + part;
            if (i < k && t < tokens) {
                a.chosen[t * k + i] = on ? item[s] : -1;
                a.weights[t * k + i] = on ? ex[s] * factor : 0.f;
            }
        }
        if (!sums) continue;
        if (on) {
            const float inv = __fdividef(1.f, total);
#pragma unroll
            for (int j = 0; j < N; ++j) prob[j] = fmaf(x[j], inv, prob[j]);
            if (part == 0) {
                const float lse = top + logf(total);
                z = fmaf(lse, lse, z);
                ++counted;
            }
        }
        if (part == 0 && t < tokens)
            reinterpret_cast<float2 *>(a.lse)[t] = on ? make_float2(top, total)
                                                      : make_float2(0.f, 1.f);
    }
    if (!sums) return;
    fa_allow_dependents();
    // the lanes that hold the same experts: of the warp, then of the CTA
#pragma unroll
    for (int j = 0; j < N; ++j)
#pragma unroll
        for (int o = 16; o >= L; o >>= 1) prob[j] += __shfl_xor_sync(0xffffffffu, prob[j], o);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        z += __shfl_xor_sync(0xffffffffu, z, o);
        counted += __shfl_xor_sync(0xffffffffu, counted, o);
    }
    float *const sum = reinterpret_cast<float *>(count + experts);  // [warps][L * N + 1]
    int32_t *const seen = reinterpret_cast<int32_t *>(sum + kRouteWarps * (L * N + 1));
    if (lane < L)
#pragma unroll
        for (int j = 0; j < N; ++j) sum[warp * (L * N + 1) + expert_of<L>(part, j)] = prob[j];
    if (lane == 0) {
        sum[warp * (L * N + 1) + L * N] = z;
        seen[warp] = counted;
    }
    __syncthreads();
    const RouteSums out = route_sums(a.scratch, gridDim.x, experts);
    for (int e = threadIdx.x; e <= experts; e += kRouteThreads) {
        const int at = e < experts ? e : L * N;
        float s = 0.f;
        for (int w = 0; w < kRouteWarps; ++w) s += sum[w * (L * N + 1) + at];
        if (e < experts) {
            out.prob[static_cast<int64_t>(blockIdx.x) * experts + e] = s;
            out.count[static_cast<int64_t>(blockIdx.x) * experts + e] = count[e];
        } else {
            out.z[blockIdx.x] = s;
            int n = 0;
            for (int w = 0; w < kRouteWarps; ++w) n += seen[w];
            out.tokens[blockIdx.x] = n;
        }
    }
}

template <int L, int R>
size_t route_shared(const RouteArgs &a) {
    constexpr int kMost = L * R * kRun;  // experts
    static_assert(4 * (kMost + kRouteWarps * (kMost + 2)) <= 48 * 1024, "what every kernel may have");
    return a.summary ? 4 * (a.logits.cols + kRouteWarps * (L * R * kRun + 1) + kRouteWarps) : 0;
}

// Joins the CTAs' sums in order, eight experts a CTA and 128 CTAs' parts side by side; the CTA that
// comes last takes the losses.
constexpr int kSumThreads = 1024, kSumExperts = 8;
template <typename T>
__device__ __forceinline__ T warp_total(T x) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    return x;
}
__global__ void __launch_bounds__(kSumThreads) route_sums_kernel(RouteArgs a) {
    constexpr int kWarps = kSumThreads / 32, kSlices = kSumThreads / kSumExperts;
    __shared__ float prob[kWarps][kSumExperts], z_part[kWarps];
    __shared__ int32_t count[kWarps][kSumExperts], n_part[kWarps];
    fa_grid_dependency_wait();
    const int experts = static_cast<int>(a.logits.cols);
    const int ctas = static_cast<int>(a.plan.ctas);
    const RouteSums in = route_sums(a.scratch, ctas, experts);
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int e = blockIdx.x * kSumExperts + threadIdx.x % kSumExperts;
    float s = 0.f, z = 0.f;
    int32_t k = 0, n = 0;
    if (e < experts) {
#pragma unroll 4
        for (int c = threadIdx.x / kSumExperts; c < ctas; c += kSlices) {
            s += in.prob[static_cast<int64_t>(c) * experts + e];
            k += in.count[static_cast<int64_t>(c) * experts + e];
        }
    }
    for (int c = threadIdx.x; c < ctas; c += kSumThreads) {
        z += in.z[c];
        n += in.tokens[c];
    }
    z = warp_total(z);
    n = warp_total(n);
#pragma unroll
    for (int o = 16; o >= kSumExperts; o >>= 1) {
        s += __shfl_xor_sync(0xffffffffu, s, o);
        k += __shfl_xor_sync(0xffffffffu, k, o);
    }
    if (lane < kSumExperts) {
        prob[warp][lane] = s;
        count[warp][lane] = k;
    }
    if (lane == 0) {
        z_part[warp] = z;
        n_part[warp] = n;
    }
    __syncthreads();
    if (warp) return;
    z = warp_total(z_part[lane]);
    n = warp_total(n_part[lane]);
    s = 0.f;
    k = 0;
#pragma unroll
    for (int w = 0; w < kWarps; w += 32 / kSumExperts) {
        s += prob[w + lane / kSumExperts][lane % kSumExperts];
        k += count[w + lane / kSumExperts][lane % kSumExperts];
    }
#pragma unroll
    for (int o = 16; o >= kSumExperts; o >>= 1) {
        s += __shfl_xor_sync(0xffffffffu, s, o);
        k += __shfl_xor_sync(0xffffffffu, k, o);
    }
    const float counted = static_cast<float>(n);
    const float inv = n ? __fdiv_rn(1.f, counted) : 0.f;
    s *= inv;
    const bool mine = lane < kSumExperts && e < experts;
    if (mine) {
        a.mean_prob[e] = s;
        a.counts[e] = k;
    }
    float dot = warp_total(mine ? static_cast<float>(k) * s : 0.f);
    int32_t before = 0;
    if (lane == 0) {
        __stcg(in.dot + blockIdx.x, dot);
        __threadfence();
        before = atomicAdd(in.joined, 1);
        __threadfence();
    }
    if (__shfl_sync(0xffffffffu, before, 0) != static_cast<int32_t>(gridDim.x) - 1) return;
    dot = 0.f;
    for (unsigned i = lane; i < gridDim.x; i += 32) dot += __ldcg(in.dot + i);
    dot = warp_total(dot);
    if (lane) return;
    const float balance =
        dot * __fdiv_rn(static_cast<float>(experts), static_cast<float>(a.top_k)) * inv;
    // without a coefficient z adds nothing, its overflow (but not a NaN) included
    const float z_loss = a.z_coef == 0.f && isinf(z) ? 0.f : a.z_coef * (z * inv);
    a.summary[0] = a.balance_coef * balance + z_loss;
    a.summary[1] = balance;
    a.summary[2] = z * inv;
    a.summary[3] = counted;
}

// LISTED: as the forward pass (at most kListed were chosen).
template <int DT, int L, int R, bool LISTED>
__global__ void __launch_bounds__(kGradThreads) route_gradient_kernel(RouteGradArgs a, bool vec) {
    constexpr int kTokens = 32 / L, N = R * kRun, kWarps = kGradThreads / 32;
    constexpr int kItems = ((LISTED ? kListed : FA_ROUTE_MAX_CHOSEN) + L - 1) / L;  // of a lane
    __shared__ long long counted_part[kWarps];
    __shared__ __align__(16) float row[kWarps][32 * N];  // the chosen experts' part, by expert
    const RouteArgs &r = a.r;
    const int k = r.top_k, warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int sub = lane / L, part = lane % L;
    const int64_t tokens = r.logits.rows;
    const int experts = static_cast<int>(r.logits.cols);
    // the counted tokens are the counts' sum over top_k
    long long n = 0;
    for (int e = threadIdx.x; e < experts; e += kGradThreads) n += r.counts[e];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) n += __shfl_xor_sync(0xffffffffu, n, o);
    if (lane == 0) counted_part[warp] = n;
    __syncthreads();
    n = 0;
    for (int w = 0; w < kWarps; ++w) n += counted_part[w];
    const float gl = a.grad_loss && n ? *a.grad_loss : 0.f;
    const float inv = n ? __fdiv_rn(static_cast<float>(k), static_cast<float>(n)) : 0.f;
    // balance_coef * experts / n * f_e = bal * counts_e, with f_e = counts_e / (n k)
    const float bal = gl * r.balance_coef * static_cast<float>(experts) * inv *
                      (n ? __fdiv_rn(1.f, static_cast<float>(n)) : 0.f);
    const float zc = 2.f * gl * r.z_coef * inv;
    float load[N];
#pragma unroll
    for (int j = 0; j < N; ++j) {
        const int e = expert_of<L>(part, j);
        load[j] = e < experts ? bal * static_cast<float>(r.counts[e]) : 0.f;
    }
    const float inv_scale = __fdiv_rn(1.f, r.weight_scale);
    float *const mine = row[warp] + sub * L * N;
    const int64_t step = static_cast<int64_t>(gridDim.x) * kWarps * kTokens;
    for (int64_t t0 = (static_cast<int64_t>(blockIdx.x) * kWarps + warp) * kTokens; t0 < tokens;
         t0 += step) {
        const int64_t t = t0 + sub;
        const bool in = t < tokens, on = in && (!r.counted || r.counted[t]);
        float x[N], w[kItems], d[kItems];
        int e[kItems];
        float2 lse = make_float2(0.f, 1.f);
        float z_part = 0.f;
#pragma unroll
        for (int i = 0; i < kItems; ++i) {
            w[i] = d[i] = 0.f;
            e[i] = -1;
        }
        if (on) {
            load_logits<DT, L, R>(r.logits, t, part, vec, x);
            lse = reinterpret_cast<const float2 *>(r.lse)[t];
            z_part = lse.x + logf(lse.y);
            if (a.dweights) {
#pragma unroll
                for (int i = 0; i < kItems; ++i)
                    if (i * L + part < k) {
                        const int64_t at = t * k + i * L + part;
                        w[i] = r.weights[at];
                        d[i] = a.dweights[at];
                        e[i] = r.chosen[at];
                    }
            }
        } else {
#pragma unroll
            for (int j = 0; j < N; ++j) x[j] = -INFINITY;
        }
        // dweights * weights: their sum, and each at its expert
        float back = 0.f;
        if (a.dweights) {
#pragma unroll
            for (int i = 0; i < kItems; ++i) back = fmaf(d[i], w[i], back);
            back = group_sum<L>(back) * inv_scale;
#pragma unroll
            for (int j = 0; j < N; j += 4)
                *reinterpret_cast<float4 *>(mine + expert_of<L>(part, j)) =
                    make_float4(0.f, 0.f, 0.f, 0.f);
            __syncwarp();
#pragma unroll
            for (int i = 0; i < kItems; ++i)
                if (static_cast<unsigned>(e[i]) < static_cast<unsigned>(L * N))
                    mine[e[i]] = r.renormalise ? w[i] * (d[i] - back) : w[i] * d[i];
            __syncwarp();
        }
        const float s = __fdividef(1.f, lse.y);
        float mean = 0.f;
#pragma unroll
        for (int j = 0; j < N; ++j) {
            x[j] = exp2_fast((x[j] - lse.x) * kLog2E) * s;
            mean = fmaf(x[j], load[j], mean);
        }
        mean = group_sum<L>(mean);
        float same = fmaf(zc, z_part, -mean);
        // without renormalising, every expert takes from the chosen ones' weights
        if (a.dweights && !r.renormalise) same -= back * r.weight_scale;
#pragma unroll
        for (int j = 0; j < N; ++j) {
            x[j] *= load[j] + same;
            if (r.counted && !on) x[j] = 0.f;
        }
        if (a.dweights) {
#pragma unroll
            for (int j = 0; j < N; j += 4) {
                const float4 m = *reinterpret_cast<const float4 *>(mine + expert_of<L>(part, j));
                x[j] += m.x;
                x[j + 1] += m.y;
                x[j + 2] += m.z;
                x[j + 3] += m.w;
            }
        }
        __syncwarp();
        // a token past the last one has no run to write
        MatrixArgs to = a.dlogits;
        if (!in) to.cols = 0;
#pragma unroll
        for (int q = 0; q < R; ++q) {
            const int c = (q * L + part) * kRun;
            if (vec)
                store_run<DT, true>(to, t, c, x + q * kRun, 0xffffffffu, L);
            else
                store_run<DT, false>(to, t, c, x + q * kRun, 0xffffffffu, L);
        }
    }
}

// Calls f with the lanes of a token and the runs of a lane.
template <typename F>
cudaError_t for_lanes(int64_t experts, F f) {
    using std::integral_constant;
    const integral_constant<int, 1> r1{};
    const integral_constant<int, 2> r2{};
    if (experts <= 8) return f(integral_constant<int, 1>{}, r1);
    if (experts <= 16) return f(integral_constant<int, 2>{}, r1);
    if (experts <= 32) return f(integral_constant<int, 4>{}, r1);
    if (experts <= 64) return f(integral_constant<int, 8>{}, r1);
    if (experts <= 128) return f(integral_constant<int, 8>{}, r2);
    if (experts <= 256) return f(integral_constant<int, 16>{}, r2);
    if (experts <= 512) return f(integral_constant<int, 32>{}, r2);
    return f(integral_constant<int, 32>{}, integral_constant<int, 4>{});
}

// Tokens of a warp's turn.
int tokens_of(int64_t experts) {
    int tokens = 1;
    for_lanes(experts, [&](auto l, auto) {
        tokens = 32 / l();
        return cudaSuccess;
    });
    return tokens;
}

}  // namespace

FA_BOUNDS_VIOLATIONS(route_bounds_violations, g_route_oob)

// CTAs of a pass: every warp with one turn of tokens until the SMs are full.
RoutePlan route_plan(int64_t tokens, int64_t experts) {
    RoutePlan p{0, 0};
    const int64_t turn = kRouteWarps * tokens_of(experts);
    p.ctas = (tokens + turn - 1) / turn;
    if (p.ctas > kRouteCtas * kSms) p.ctas = kRouteCtas * kSms;
    p.bytes = p.ctas * (experts + 1) * 8 + 4 * (FA_ROUTE_MAX_EXPERTS / 8 + 1);
    return p;
}

cudaError_t launch_route(const RouteArgs &a, fa_dtype dt, cudaStream_t stream) {
    const bool vec = aligned_rows(a.logits, dt);
    const cudaError_t err = for_dtype(dt, [&](auto d) {
        return for_lanes(a.logits.cols, [&](auto l, auto r) {
            auto *kernel = route_kernel<d(), l(), r(), true>;
            if constexpr (l() > 1)  // (one lane: there are no more experts than a list has)
                if (a.top_k > kListed) kernel = route_kernel<d(), l(), r(), false>;
            const size_t smem = route_shared<l(), r()>(a);
            if (a.plan.ctas)
                kernel<<<static_cast<unsigned>(a.plan.ctas), kRouteThreads, smem, stream>>>(a, vec);
            return cudaGetLastError();
        });
    });
    if (err != cudaSuccess || !a.summary) return err;
    if (!a.plan.ctas) {  // no token: nothing was summed
        const size_t row = 4 * a.logits.cols;
        cudaError_t e = cudaMemsetAsync(a.counts, 0, row, stream);
        if (e == cudaSuccess) e = cudaMemsetAsync(a.mean_prob, 0, row, stream);
        return e == cudaSuccess ? cudaMemsetAsync(a.summary, 0, 16, stream) : e;
    }
    return launch_dependent(route_sums_kernel, 
                            dim3((a.logits.cols + kSumExperts - 1) / kSumExperts),
                            dim3(kSumThreads), 0, stream, a);
}

cudaError_t launch_route_gradient(const RouteGradArgs &a, fa_dtype dt, cudaStream_t stream) {
    const bool vec = aligned_rows(a.r.logits, dt) && aligned_rows(a.dlogits, dt);
    const int64_t turn = kGradThreads / 32 * tokens_of(a.r.logits.cols);
    int64_t ctas = (a.r.logits.rows + turn - 1) / turn;
    if (ctas > 3 * kSms) ctas = 3 * kSms;
    return for_dtype(dt, [&](auto d) {
        return for_lanes(a.r.logits.cols, [&](auto l, auto r) {
            auto *kernel = route_gradient_kernel<d(), l(), r(), true>;
            if constexpr (l() > 1)
                if (a.r.top_k > kListed) kernel = route_gradient_kernel<d(), l(), r(), false>;
            kernel<<<static_cast<unsigned>(ctas), kGradThreads, 0, stream>>>(a, vec);
            return cudaGetLastError();
        });
    });
}

}  // namespace fa
