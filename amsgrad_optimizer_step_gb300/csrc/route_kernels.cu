// The router of gated experts: choice, weights, counts and the balance loss of tokens from
// their logits, and the logits' gradient.
//
// A token's row belongs to a group of 1 to 32 lanes, eight experts a lane (up to 256 experts;
// 16 or 32 beyond), in registers.  The choice takes the largest key top_k times: keys are
// integers in the logits' order, and for 16-bit types carry the expert's number below them, so
// that one maximum over the group gives both the logit and the expert, ties to the lower number.
// The first key is the row's maximum, which the softmax is taken from.  Sums over tokens stay
// with the lane that holds the expert, then go by CTA and in order.
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
constexpr int kRouteWarps = kRouteThreads / 32;

// Keys in the order of the logits: larger logits have larger keys, -0 and 0 the same one, and
// every NaN the largest.  0 is below every key.
template <int DT>
struct Key;

template <>
struct Key<FA_F32> {
    static constexpr bool kNumbered = false;
    static __device__ __forceinline__ uint32_t of(float x, int) {
        const uint32_t b = __float_as_uint(x + 0.f);  // -0 becomes 0
        const uint32_t k = b & 0x80000000u ? ~b : b | 0x80000000u;
        return x != x ? 0xffffffffu : k;
    }
    static __device__ __forceinline__ float logit(uint32_t k) {
        return __uint_as_float(k & 0x80000000u ? k ^ 0x80000000u : ~k);
    }
};

// The upper 16 bits of the widened logit hold a BF16; an FP16 keeps its own bits.
template <int DT>
struct Key16 {
    static constexpr bool kNumbered = true;
    static __device__ __forceinline__ uint32_t of(float x, int expert) {
        const typename Elem<DT>::T e = Elem<DT>::round(x + 0.f);  // exact
        const uint32_t b = *reinterpret_cast<const uint16_t *>(&e);
        uint32_t k = b & 0x8000u ? ~b & 0xffffu : b | 0x8000u;
        if (x != x) k = 0xffffu;
        return k << 16 | (0xffffu - static_cast<uint32_t>(expert));
    }
    static __device__ __forceinline__ float logit(uint32_t k) {
        k >>= 16;
        const uint16_t b = static_cast<uint16_t>(k & 0x8000u ? k ^ 0x8000u : ~k);
        return Elem<DT>::widen(*reinterpret_cast<const typename Elem<DT>::T *>(&b));
    }
};
template <>
struct Key<FA_F16> : Key16<FA_F16> {};
template <>
struct Key<FA_BF16> : Key16<FA_BF16> {};

// N experts of a token, as they lie in memory; those past the end are -infinity.
template <int DT, int N>
__device__ __forceinline__ void load_logits(const MatrixArgs &m, int64_t row, int c, bool vec,
                                            float *x) {
    using T = typename Elem<DT>::T;
    const T *p = static_cast<const T *>(m.p) + row * m.ld + c;
    const int left = static_cast<int>(m.cols) - c, valid = left < 0 ? 0 : left < N ? left : N;
    if (valid && !fa_in_bounds(c, valid, m.cols)) return;
    if (vec && valid == N) {
        Raw<DT, N> r;
        r.load(p);
        r.widen(x);
    } else {
        RawAny<DT, N> r;
        r.load(p, valid, Span(m.p, ((m.rows - 1) * m.ld + m.cols) * sizeof(T)));
        r.widen(x);
    }
#pragma unroll
    for (int j = 0; j < N; ++j)
        if (j >= valid) x[j] = -INFINITY;
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

// What a CTA leaves of its tokens: per expert the probabilities' sum and the count, then z's sum
// and the counted tokens.
struct RouteSums {
    float *prob;   // [ctas][experts]
    int32_t *count;  // [ctas][experts]
    float *z;        // [ctas]
    int32_t *tokens;  // [ctas]
};
__host__ __device__ inline RouteSums route_sums(void *scratch, int64_t ctas, int64_t experts) {
    RouteSums s;
    s.prob = static_cast<float *>(scratch);
    s.count = reinterpret_cast<int32_t *>(s.prob + ctas * experts);
    s.z = reinterpret_cast<float *>(s.count + ctas * experts);
    s.tokens = reinterpret_cast<int32_t *>(s.z + ctas);
    return s;
}

// L lanes a token, N experts a lane.
template <int DT, int L, int N>
__global__ void __launch_bounds__(kRouteThreads) route_kernel(RouteArgs a, bool vec) {
    constexpr int kTokens = 32 / L;  // of a warp's turn
    extern __shared__ uint32_t shared[];
    // a warp's choices before they are written: the experts and their exponentials, then each
    // token's factor
    const int k = a.top_k, warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int sub = lane / L, part = lane % L;
    uint32_t *const my = shared + warp * kTokens * (2 * k + 1);
    int32_t *const expert = reinterpret_cast<int32_t *>(my);
    float *const weight = reinterpret_cast<float *>(my + kTokens * k);
    float *const factor = weight + kTokens * k;
    // then the CTA's counts
    int32_t *const count = reinterpret_cast<int32_t *>(shared + kRouteWarps * kTokens * (2 * k + 1));
    const int64_t tokens = a.logits.rows;
    const int experts = static_cast<int>(a.logits.cols);
    const bool sums = a.summary != nullptr;
    if (sums) {
        for (int e = threadIdx.x; e < experts; e += kRouteThreads) count[e] = 0;
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
        uint32_t key[N];
        if (on) {
            load_logits<DT, N>(a.logits, t, part * N, vec, x);
        } else {
#pragma unroll
            for (int j = 0; j < N; ++j) x[j] = 0.f;
        }
#pragma unroll
        for (int j = 0; j < N; ++j)
            key[j] = part * N + j < experts ? Key<DT>::of(x[j], part * N + j) : 0u;
        float top = 0.f, picked = 0.f;
        for (int i = 0; i < k; ++i) {
            uint32_t best = key[0];
#pragma unroll
            for (int j = 1; j < N; ++j) best = max(best, key[j]);
            const uint32_t mine = best;
            best = group_max<L>(best);
            int e = 0;
            if (Key<DT>::kNumbered) {
                e = static_cast<int>(0xffffu - (best & 0xffffu));
#pragma unroll
                for (int j = 0; j < N; ++j)
                    if (key[j] == best) key[j] = 0u;
            } else {
                // the first lane that has the key, and its first expert with it
                const unsigned have = __ballot_sync(0xffffffffu, mine == best);
                const int winner = __ffs(static_cast<int>(have >> (sub * L))) - 1;
                bool found = part != winner;
#pragma unroll
                for (int j = 0; j < N; ++j)
                    if (!found && key[j] == best) {
                        key[j] = 0u;
                        e = part * N + j;
                        found = true;
                    }
                e = __shfl_sync(0xffffffffu, e, winner, L);
            }
            const float logit = Key<DT>::logit(best);
            if (i == 0) top = logit;
            const float ex = expf(logit - top);
            picked += ex;
            if (part == 0) {
                expert[sub * k + i] = on ? e : -1;
                weight[sub * k + i] = ex;
                if (sums && on) atomicAdd(count + e, 1);
            }
        }
        float total = 0.f;
#pragma unroll
        for (int j = 0; j < N; ++j) {
            x[j] = expf(x[j] - top);
            total += x[j];
        }
        total = group_sum<L>(total);
        if (part == 0)
            factor[sub] = on ? __fdiv_rn(a.weight_scale, a.renormalise ? picked : total) : 0.f;
        if (sums && on) {
            const float inv = __fdiv_rn(1.f, total);
#pragma unroll
            for (int j = 0; j < N; ++j) prob[j] = fmaf(x[j], inv, prob[j]);
            if (part == 0) {
                const float lse = top + logf(total);
                z = fmaf(lse, lse, z);
                ++counted;
            }
        }
        if (sums && part == 0 && t < tokens)
            reinterpret_cast<float2 *>(a.lse)[t] = on ? make_float2(top, total)
                                                      : make_float2(0.f, 1.f);
        __syncwarp();
        const int n = static_cast<int>(min(static_cast<int64_t>(kTokens), tokens - t0)) * k;
        for (int i = lane; i < n; i += 32) {
            const float f = factor[a.by_k.quotient(i)];
            a.chosen[t0 * k + i] = expert[i];
            a.weights[t0 * k + i] = f == 0.f ? 0.f : weight[i] * f;
        }
        __syncwarp();
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
        for (int j = 0; j < N; ++j) sum[warp * (L * N + 1) + lane * N + j] = prob[j];
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

template <int L, int N>
size_t route_shared(const RouteArgs &a) {
    const size_t words = kRouteWarps * (32 / L) * (2 * static_cast<size_t>(a.top_k) + 1);
    return 4 * (words + (a.summary ? a.logits.cols + kRouteWarps * (L * N + 1) + kRouteWarps : 0));
}

// Joins the CTAs' sums in order and takes the losses: one CTA, a warp for 32 experts at a time
// and the CTAs' parts in turn.
__global__ void __launch_bounds__(1024) route_sums_kernel(RouteArgs a) {
    __shared__ float part[32][33];
    __shared__ int32_t parti[32][33];
    __shared__ float fp[32];
    __shared__ float z_sum;
    __shared__ int32_t n_sum;
    fa_grid_dependency_wait();
    const int experts = static_cast<int>(a.logits.cols);
    const int ctas = static_cast<int>(a.plan.ctas);
    const RouteSums in = route_sums(a.scratch, ctas, experts);
    const int x = threadIdx.x % 32, y = threadIdx.x / 32;
    if (y == 0) {
        float z = 0.f;
        int32_t n = 0;
        for (int c = x; c < ctas; c += 32) {
            z += in.z[c];
            n += in.tokens[c];
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            z += __shfl_xor_sync(0xffffffffu, z, o);
            n += __shfl_xor_sync(0xffffffffu, n, o);
        }
        if (x == 0) {
            z_sum = z;
            n_sum = n;
        }
    }
    __syncthreads();
    const float n = static_cast<float>(n_sum);
    const float inv = n_sum ? __fdiv_rn(1.f, n) : 0.f;
    float dot = 0.f;  // of counts and mean probabilities, in the first warp
    for (int e0 = 0; e0 < experts; e0 += 32) {
        const int e = e0 + x;
        float s = 0.f;
        int32_t k = 0;
        if (e < experts)
            for (int c = y; c < ctas; c += 32) {
                s += in.prob[static_cast<int64_t>(c) * experts + e];
                k += in.count[static_cast<int64_t>(c) * experts + e];
            }
        part[y][x] = s;
        parti[y][x] = k;
        __syncthreads();
        if (y == 0 && e < experts) {
            s = 0.f;
            k = 0;
#pragma unroll
            for (int i = 0; i < 32; ++i) {
                s += part[i][x];
                k += parti[i][x];
            }
            s *= inv;
            a.mean_prob[e] = s;
            a.counts[e] = k;
            dot = fmaf(static_cast<float>(k), s, dot);
        }
        __syncthreads();
    }
    if (y == 0) fp[x] = dot;
    __syncthreads();
    if (threadIdx.x == 0) {
        dot = 0.f;
        for (int i = 0; i < 32; ++i) dot += fp[i];
        const float balance =
            dot * __fdiv_rn(static_cast<float>(experts), static_cast<float>(a.top_k)) * inv;
        const float z = z_sum * inv;
        a.summary[0] = a.balance_coef * balance + a.z_coef * z;
        a.summary[1] = balance;
        a.summary[2] = z;
        a.summary[3] = n;
    }
}

template <int DT, int L, int N>
__global__ void __launch_bounds__(kRouteThreads) route_gradient_kernel(RouteGradArgs a, bool vec) {
    constexpr int kTokens = 32 / L;
    __shared__ long long counted_part[kRouteWarps];
    __shared__ float row[kRouteWarps][32 * N];  // the chosen experts' part, by expert
    const RouteArgs &r = a.r;
    const int k = r.top_k, warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int sub = lane / L, part = lane % L;
    const int64_t tokens = r.logits.rows;
    const int experts = static_cast<int>(r.logits.cols);
    // the counted tokens are the counts' sum over top_k
    long long n = 0;
    for (int e = threadIdx.x; e < experts; e += kRouteThreads) n += r.counts[e];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) n += __shfl_xor_sync(0xffffffffu, n, o);
    if (lane == 0) counted_part[warp] = n;
    __syncthreads();
    n = 0;
    for (int w = 0; w < kRouteWarps; ++w) n += counted_part[w];
    const float total = static_cast<float>(n / k);
    const float gl = a.grad_loss && n ? *a.grad_loss : 0.f;
    const float inv = n ? __fdiv_rn(1.f, total) : 0.f;
    const float bal = gl * r.balance_coef * static_cast<float>(experts) * inv;
    const float zc = 2.f * gl * r.z_coef * inv;
    float load[N];  // balance_coef * experts / n * f of this lane's experts
#pragma unroll
    for (int j = 0; j < N; ++j) {
        const int e = part * N + j;
        load[j] = e < experts && n
                      ? bal * __fdiv_rn(static_cast<float>(r.counts[e]), static_cast<float>(n))
                      : 0.f;
    }
    const float inv_scale = __fdiv_rn(1.f, r.weight_scale);
    float *const mine = row[warp] + sub * L * N;
    const int64_t step = static_cast<int64_t>(gridDim.x) * kRouteWarps * kTokens;
    for (int64_t t0 = (static_cast<int64_t>(blockIdx.x) * kRouteWarps + warp) * kTokens;
         t0 < tokens; t0 += step) {
        const int64_t t = t0 + sub;
        const bool in = t < tokens, on = in && (!r.counted || r.counted[t]);
        float x[N];
        float2 lse = make_float2(0.f, 1.f);
        if (on) {
            load_logits<DT, N>(r.logits, t, part * N, vec, x);
            lse = reinterpret_cast<const float2 *>(r.lse)[t];
        } else {
#pragma unroll
            for (int j = 0; j < N; ++j) x[j] = -INFINITY;
        }
        // dweights * weights: their sum, and each at its expert
        float back = 0.f;
        if (a.dweights) {
#pragma unroll
            for (int j = 0; j < N; ++j) mine[part * N + j] = 0.f;
            for (int i = part; i < k; i += L)
                if (on) back = fmaf(a.dweights[t * k + i], r.weights[t * k + i], back);
            back = group_sum<L>(back) * inv_scale;
            __syncwarp();
            for (int i = part; i < k; i += L)
                if (on) {
                    const float w = r.weights[t * k + i], d = a.dweights[t * k + i];
                    const int e = r.chosen[t * k + i];
                    if (static_cast<unsigned>(e) < static_cast<unsigned>(L * N))
                        mine[e] = r.renormalise ? w * (d - back) : w * d;
                }
            __syncwarp();
        }
        const float s = __fdiv_rn(1.f, lse.y);
        float mean = 0.f;
#pragma unroll
        for (int j = 0; j < N; ++j) {
            x[j] = expf(x[j] - lse.x) * s;
            mean = fmaf(x[j], load[j], mean);
        }
        mean = group_sum<L>(mean);
        float same = fmaf(zc, lse.x + logf(lse.y), -mean);
        // without renormalising, every expert takes from the chosen ones' weights
        if (a.dweights && !r.renormalise) same -= back * r.weight_scale;
#pragma unroll
        for (int j = 0; j < N; ++j) {
            x[j] *= load[j] + same;
            if (a.dweights) x[j] += mine[part * N + j];
            if (!on) x[j] = 0.f;
        }
        __syncwarp();
        using T = typename Elem<DT>::T;
        T *p = static_cast<T *>(a.dlogits.p) + t * a.dlogits.ld + part * N;
        const int left = experts - part * N;
        int valid = !in || left < 0 ? 0 : left < N ? left : N;
        if (valid && !fa_in_bounds(part * N, valid, experts)) valid = 0;
        if (vec) {
            if (valid == N) {
                store_n<DT, N>(p, x);
            } else {
#pragma unroll
                for (int j = 0; j < N; ++j)
                    if (j < valid) p[j] = Elem<DT>::round(x[j]);
            }
        } else {
            store_any<DT, N>(p, x, valid, 0xffffffffu, L);
        }
    }
}

// Calls f with the lanes of a token and the experts of a lane.
template <typename F>
cudaError_t for_lanes(int64_t experts, F f) {
    using std::integral_constant;
    const integral_constant<int, 8> n8{};
    if (experts <= 8) return f(integral_constant<int, 1>{}, n8);
    if (experts <= 16) return f(integral_constant<int, 2>{}, n8);
    if (experts <= 32) return f(integral_constant<int, 4>{}, n8);
    if (experts <= 64) return f(integral_constant<int, 8>{}, n8);
    if (experts <= 128) return f(integral_constant<int, 16>{}, n8);
    if (experts <= 256) return f(integral_constant<int, 32>{}, n8);
    if (experts <= 512) return f(integral_constant<int, 32>{}, integral_constant<int, 16>{});
    return f(integral_constant<int, 32>{}, integral_constant<int, 32>{});
}

int lanes_of(int64_t experts) {
    int lanes = 1;
    while (lanes < 32 && lanes * 8 < experts) lanes *= 2;
    return lanes;
}

}  // namespace

FA_BOUNDS_VIOLATIONS(route_bounds_violations, g_route_oob)

// CTAs of a pass: every warp with one turn of tokens until the SMs are full.
RoutePlan route_plan(int64_t tokens, int64_t experts) {
    RoutePlan p{0, 0};
    const int64_t turn = kRouteWarps * (32 / lanes_of(experts));
    p.ctas = (tokens + turn - 1) / turn;
    if (p.ctas > 2 * kSms) p.ctas = 2 * kSms;
    p.bytes = p.ctas * (experts + 1) * 8;
    return p;
}

cudaError_t launch_route(const RouteArgs &a, fa_dtype dt, cudaStream_t stream) {
    const bool vec = aligned_rows(a.logits, dt);
    const cudaError_t err = for_dtype(dt, [&](auto d) {
        return for_lanes(a.logits.cols, [&](auto l, auto n) {
            if (a.plan.ctas)
                route_kernel<d(), l(), n()><<<static_cast<unsigned>(a.plan.ctas), kRouteThreads,
                                             route_shared<l(), n()>(a), stream>>>(a, vec);
            return cudaGetLastError();
        });
    });
    if (err != cudaSuccess || !a.summary) return err;
    return launch_dependent(route_sums_kernel, dim3(1), dim3(1024), 0, stream, a);
}

cudaError_t launch_route_gradient(const RouteGradArgs &a, fa_dtype dt, cudaStream_t stream) {
    const bool vec = aligned_rows(a.r.logits, dt) && aligned_rows(a.dlogits, dt);
    const int64_t turn = kRouteWarps * (32 / lanes_of(a.r.logits.cols));
    int64_t ctas = (a.r.logits.rows + turn - 1) / turn;
    if (ctas > 8 * kSms) ctas = 8 * kSms;
    return for_dtype(dt, [&](auto d) {
        return for_lanes(a.r.logits.cols, [&](auto l, auto n) {
            route_gradient_kernel<d(), l(), n()>
                <<<static_cast<unsigned>(ctas), kRouteThreads, 0, stream>>>(a, vec);
            return cudaGetLastError();
        });
    });
}

}  // namespace fa
