// The gated activation h = act(gate) * up with an 8-bit checkpoint of its two inputs,
// and its backward pass from the checkpoint.
//
// Eight lanes take one block of kCheckpointBlock columns, two runs of eight consecutive
// columns each, 64 apart: 16-byte accesses for 16-bit types, and a block's largest
// magnitude is three shuffles away.  The four divisions of a block (127 / a and a / 127 of
// gate and up) are one division in four of its lanes.  Codes are rounded and taken apart
// without conversions: x * (127 / a) + 1.5 * 2^23 has the code in its low byte, and
// a code's byte below the exponent of 2^23 is the code + 128 + 2^23.
//
// Reads and writes bound both: 8 bytes an element forward and 10 backward with 16-bit types.
// 8192 x 5632 BF16 take 53 us (7.0 TB/s) and 66 us (7.0 TB/s), silu; the tanh form is as
// fast, but for the FP32 forward pass (105 us against 98).  Rows at odd addresses cost about twice the time (8192 x 5633: 246 us for both
// directions; 597 us with element accesses): their 16-byte lines are put together by lanes.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "internal.h"
#include "model_device.cuh"
#include "model_internal.h"

namespace fa {
namespace {

FA_BOUNDS_COUNTER(g_gated_oob)

constexpr int kGatedThreads = 256;
constexpr int kLanes = 8;                         // per block of columns
constexpr int kRun = 8;                           // consecutive columns of a lane
constexpr int kRunStride = kCheckpointBlock / 2;  // between its two runs
constexpr float kTiny = 0x1p-100f;                // blocks below it are stored as zeros
constexpr float kLog2E = 1.4426950408889634f;

__device__ __forceinline__ float reciprocal(float x) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ uint64_t both(float x) { return pair(x, x); }

// sigmoid(-t / log2(e)) of a pair: 1 / (1 + 2^t).  A result below 2^-126 is 0: what it costs is
// below 1.1e-36 (a reciprocal of subnormal results, and 2^t past 2^128, would lengthen every
// element for it).
__device__ __forceinline__ uint64_t sigmoid2(uint64_t t) {
    float lo, hi;
    unpair(t, lo, hi);
    unpair(add2(both(1.f), pair(exp2_fast(lo), exp2_fast(hi))), lo, hi);
    return pair(reciprocal(lo), reciprocal(hi));
}

// The activation of a pair and its derivative.  ``square``: 1, or 0 where the gate may be above
// 2^63 and is 2^55 at least or 0 (see gated_backward_kernel).
template <int ACT>
struct Activation;

template <>
struct Activation<FA_SILU> {
    static __device__ __forceinline__ uint64_t value(uint64_t g) {
        return mul2(g, sigmoid2(mul2(g, both(-kLog2E))));
    }
    static __device__ __forceinline__ void with_slope(uint64_t g, float, uint64_t &a,
                                                      uint64_t &da) {
        const uint64_t s = sigmoid2(mul2(g, both(-kLog2E)));
        a = mul2(g, s);
        da = fma2(a, fma2(s, both(-1.f), both(1.f)), s);  // s (1 + g (1 - s))
    }
};

template <>
struct Activation<FA_GELU_TANH> {
    // 2 sqrt(2/pi) (g + 0.044715 g^3) = g (kA + kB g^2)
    static constexpr float kA = 1.5957691216057308f, kB = 0.071354816272600250f;
    static __device__ __forceinline__ uint64_t gate(uint64_t g, uint64_t q) {
        return sigmoid2(mul2(g, fma2(q, both(-kB * kLog2E), both(-kA * kLog2E))));
    }
    static __device__ __forceinline__ uint64_t value(uint64_t g) {
        return mul2(g, gate(g, mul2(g, g)));
    }
    static __device__ __forceinline__ void with_slope(uint64_t g, float square, uint64_t &a,
                                                      uint64_t &da) {
        const uint64_t q = mul2(g, mul2(g, both(square))), s = gate(g, q);
        a = mul2(g, s);
        const uint64_t rest = mul2(a, fma2(s, both(-1.f), both(1.f)));
        da = fma2(rest, fma2(q, both(3.f * kB), both(kA)), s);
    }
};

// A lane's run of eight columns [c, c + 8) of a row.  ALIGNED: one 16-byte access (two for
// FP32) when the columns all exist, element accesses otherwise; else the 16-byte lines that the
// run touches (see RawAny, store_any).  Columns past the end read as 0 and are not written.
__device__ __forceinline__ int valid_cols(int64_t c, int64_t cols) {
    return c + kRun <= cols ? kRun : c < cols ? static_cast<int>(cols - c) : 0;
}
template <int DT, bool ALIGNED>
__device__ __forceinline__ Raw<DT, kRun> load_run(const MatrixArgs &m, int64_t row, int64_t c) {
    using E = Elem<DT>;
    const typename E::T *p = static_cast<const typename E::T *>(m.p) + row * m.ld + c;
    const int valid = valid_cols(c, m.cols);
    if (valid && !fa_in_bounds(c, valid, m.cols)) return {};
    if constexpr (ALIGNED) {
        Raw<DT, kRun> x;
        if (c + kRun <= m.cols) {
            x.load(p);
        } else {
            float y[kRun];
#pragma unroll
            for (int j = 0; j < kRun; ++j) y[j] = j < valid ? E::widen(p[j]) : 0.f;
            x.from(y);  // exact: they came from this type
        }
        return x;
    } else {
        RawAny<DT, kRun> x;
        x.load(p, valid, Span(m.p, ((m.rows - 1) * m.ld + m.cols) * sizeof(typename E::T)));
        return x.raw();
    }
}
template <int DT, bool ALIGNED>
__device__ __forceinline__ void store_run(const MatrixArgs &m, int64_t row, int64_t c,
                                          const float *x, unsigned lanes) {
    using E = Elem<DT>;
    typename E::T *p = static_cast<typename E::T *>(m.p) + row * m.ld + c;
    int valid = valid_cols(c, m.cols);
    if (valid && !fa_in_bounds(c, valid, m.cols)) valid = 0;
    if constexpr (ALIGNED) {
        if (c + kRun <= m.cols) {
            store_n<DT, kRun>(p, x);
        } else {
#pragma unroll
            for (int j = 0; j < kRun; ++j)
                if (j < valid) p[j] = E::round(x[j]);
        }
    } else {
        store_any<DT, kRun>(p, x, valid, lanes, kLanes);
    }
}

// The larger of two magnitudes; NaN where either is.
__device__ __forceinline__ float max_nan(float a, float b) {
    float y;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(b));
    return y;
}

// Eight codes of a run, packed.
__device__ __forceinline__ uint2 encode(const float *x, float inv) {
    uint32_t y[kRun];
#pragma unroll
    for (int j = 0; j < kRun; ++j)  // two roundings, as the rule says: the packed pair of
        // instructions was measured to round once
        y[j] = __float_as_uint(__fadd_rn(__fmul_rn(x[j], inv), 0x1.8p23f));
    const auto four = [](const uint32_t *q) {
        return __byte_perm(__byte_perm(q[0], q[1], 0x0040), __byte_perm(q[2], q[3], 0x0040),
                           0x5410);
    };
    return make_uint2(four(y), four(y + 4));
}

// What eight codes stand for, in pairs.
__device__ __forceinline__ void decode(uint2 codes, float scale, uint64_t *x) {
    const uint32_t w[2] = {codes.x ^ 0x80808080u, codes.y ^ 0x80808080u};
#pragma unroll
    for (int j = 0; j < kRun; j += 2) {
        const uint32_t b = w[j / 4];
        const uint32_t lo = __byte_perm(b, 0x4b000000u, j % 4 == 0 ? 0x7440 : 0x7442);
        const uint32_t hi = __byte_perm(b, 0x4b000000u, j % 4 == 0 ? 0x7441 : 0x7443);
        const uint64_t q = add2(pair(__uint_as_float(lo), __uint_as_float(hi)),
                                both(-(0x1p23f + 128.f)));  // exact
        x[j / 2] = mul2(q, both(scale));
    }
}

template <int DT, int ACT, bool ALIGNED, bool KEEP>
__global__ void __launch_bounds__(kGatedThreads, DT == FA_F32 ? 2 : ALIGNED ? 5 : 4)
gated_forward_kernel(GatedForwardArgs a) {
    const uint32_t b = (blockIdx.x * kGatedThreads + threadIdx.x) / kLanes;
    const int lane = threadIdx.x % kLanes;
    const int64_t n = a.rows * a.blocks;
    if (b >= n || !fa_in_bounds(b, 1, n)) return;  // all eight lanes of a block
    const uint32_t row = a.by_blocks.quotient(b);
    const int64_t c = static_cast<int64_t>(b - row * static_cast<uint32_t>(a.blocks)) *
                          kCheckpointBlock + lane * kRun;
    Raw<DT, kRun> g[2], u[2];
#pragma unroll
    for (int r = 0; r < 2; ++r) g[r] = load_run<DT, ALIGNED>(a.gate, row, c + r * kRunStride);
#pragma unroll
    for (int r = 0; r < 2; ++r) u[r] = load_run<DT, ALIGNED>(a.up, row, c + r * kRunStride);
    float inv_g = 0.f, inv_u = 0.f;
    const unsigned lanes = 0xffu << (threadIdx.x & 24);
    if (KEEP) {
        float tg = max_nan(g[0].magnitude(), g[1].magnitude());
        float tu = max_nan(u[0].magnitude(), u[1].magnitude());
#pragma unroll
        for (int o = kLanes / 2; o > 0; o >>= 1) {
            tg = max_nan(tg, __shfl_xor_sync(lanes, tg, o));
            tu = max_nan(tu, __shfl_xor_sync(lanes, tu, o));
        }
        // lane 0: 127 / tg, 1: tg / 127, 2 and 3: the same of tu (the others repeat them)
        const float top = lane & 2 ? tu : tg;
        const bool kept = top >= kTiny && top < INFINITY, scale = lane & 1;
        float q = __fdiv_rn(scale ? top : 127.f, scale ? 127.f : top);
        if (!kept) q = scale && !(top < INFINITY) ? NAN : 0.f;
        inv_g = __shfl_sync(lanes, q, 0, kLanes);
        inv_u = __shfl_sync(lanes, q, 2, kLanes);
        if (lane == 1) a.scales[b] = q;
        if (lane == 3) a.scales[n + b] = q;
    }
#pragma unroll
    for (int r = 0; r < 2; ++r) {
        float x[kRun], y[kRun];
        g[r].widen(x);
        u[r].widen(y);
        if (KEEP) {
            int8_t *code = a.codes + static_cast<int64_t>(b) * kCheckpointBlock + lane * kRun +
                           r * kRunStride;
            __stcs(reinterpret_cast<uint2 *>(code), encode(x, inv_g));
            __stcs(reinterpret_cast<uint2 *>(code + n * kCheckpointBlock), encode(y, inv_u));
        }
#pragma unroll
        for (int j = 0; j < kRun; j += 2)
            unpair(mul2(Activation<ACT>::value(pair(x[j], x[j + 1])), pair(y[j], y[j + 1])), x[j],
                   x[j + 1]);
        store_run<DT, ALIGNED>(a.h, row, c + r * kRunStride, x, lanes);
    }
}

template <int DT, int ACT, bool ALIGNED>
__global__ void __launch_bounds__(kGatedThreads, DT == FA_F32 && ACT == FA_GELU_TANH ? 3
                                                 : DT == FA_F32 || ALIGNED           ? 2
                                                                                     : 4)
gated_backward_kernel(GatedBackwardArgs a) {
    const uint32_t b = (blockIdx.x * kGatedThreads + threadIdx.x) / kLanes;
    const int lane = threadIdx.x % kLanes;
    const int64_t n = a.rows * a.blocks;
    if (b >= n || !fa_in_bounds(b, 1, n)) return;
    const uint32_t row = a.by_blocks.quotient(b);
    const int64_t c = static_cast<int64_t>(b - row * static_cast<uint32_t>(a.blocks)) *
                          kCheckpointBlock + lane * kRun;
    const int8_t *code = a.codes + static_cast<int64_t>(b) * kCheckpointBlock + lane * kRun;
    const unsigned lanes = 0xffu << (threadIdx.x & 24);
    uint2 qg[2], qu[2];
    Raw<DT, kRun> d[2];
#pragma unroll
    for (int r = 0; r < 2; ++r) {
        qg[r] = __ldcs(reinterpret_cast<const uint2 *>(code + r * kRunStride));
        qu[r] = __ldcs(reinterpret_cast<const uint2 *>(code + n * kCheckpointBlock + r * kRunStride));
        d[r] = load_run<DT, ALIGNED>(a.dh, row, c + r * kRunStride);
    }
    const float sg = a.scales[b], su = a.scales[n + b];
    // From 2^64 on a gate's square is infinite and its slope would be 0 * inf.  A scale of 2^55
    // makes every code but 0 so large that the sigmoid is 0 or 1 without the square.  (8192 x 5632,
    // tanh form: a bound on each square took BF16 73 us and FP32 160; a branch 81 and 145; this
    // takes 73 and 138, FP32 in 80 registers a thread, 159 in 92.)
    const float square = sg >= 0x1p55f ? 0.f : 1.f;
#pragma unroll
    for (int r = 0; r < 2; ++r) {
        uint64_t g[kRun / 2], u[kRun / 2];
        decode(qg[r], sg, g);
        decode(qu[r], su, u);
        float x[kRun], dg[kRun], du[kRun], h[kRun];
        d[r].widen(x);
#pragma unroll
        for (int j = 0; j < kRun; j += 2) {
            uint64_t act, slope;
            Activation<ACT>::with_slope(g[j / 2], square, act, slope);
            const uint64_t dh = pair(x[j], x[j + 1]);
            // |act'| < 1.13: overflows only where the gradient does
            unpair(mul2(mul2(dh, slope), u[j / 2]), dg[j], dg[j + 1]);
            unpair(mul2(dh, act), du[j], du[j + 1]);
            unpair(mul2(act, u[j / 2]), h[j], h[j + 1]);
        }
        store_run<DT, ALIGNED>(a.dgate, row, c + r * kRunStride, dg, lanes);
        store_run<DT, ALIGNED>(a.dup, row, c + r * kRunStride, du, lanes);
        if (a.h.p) store_run<DT, ALIGNED>(a.h, row, c + r * kRunStride, h, lanes);
    }
}

// Whether 16-byte accesses at multiples of eight columns are aligned in every row.
bool aligned_rows(const MatrixArgs &m, fa_dtype dt) {
    const int64_t row_bytes = m.ld * (dt == FA_F32 ? 4 : 2);
    return !m.p || (reinterpret_cast<uintptr_t>(m.p) % 16 == 0 &&
                    (m.rows < 2 || row_bytes % 16 == 0));
}

template <typename F>
cudaError_t for_activation(fa_activation act, F f) {
    return act == FA_SILU ? f(std::integral_constant<int, FA_SILU>{})
                          : f(std::integral_constant<int, FA_GELU_TANH>{});
}

}  // namespace

cudaError_t gated_bounds_violations(unsigned long long *count, bool clear) {
#if FA_BOUNDS_CHECK
    cudaError_t err = cudaMemcpyFromSymbol(count, g_gated_oob, sizeof(*count));
    if (err != cudaSuccess || !clear) return err;
    const unsigned long long zero = 0;
    return cudaMemcpyToSymbol(g_gated_oob, &zero, sizeof(zero));
#else
    (void)clear;
    *count = 0;
    return cudaSuccess;
#endif
}

cudaError_t launch_gated_forward(const GatedForwardArgs &a, fa_dtype dt, fa_activation act,
                                 cudaStream_t stream) {
    const int64_t ctas = (a.rows * a.blocks * kLanes + kGatedThreads - 1) / kGatedThreads;
    const bool vec = aligned_rows(a.gate, dt) && aligned_rows(a.up, dt) && aligned_rows(a.h, dt);
    return for_dtype(dt, [&](auto d) {
        return for_activation(act, [&](auto ac) {
            auto *kernel = vec ? a.codes ? gated_forward_kernel<d(), ac(), true, true>
                                         : gated_forward_kernel<d(), ac(), true, false>
                               : a.codes ? gated_forward_kernel<d(), ac(), false, true>
                                         : gated_forward_kernel<d(), ac(), false, false>;
            kernel<<<static_cast<unsigned>(ctas), kGatedThreads, 0, stream>>>(a);
            return cudaGetLastError();
        });
    });
}

cudaError_t launch_gated_backward(const GatedBackwardArgs &a, fa_dtype dt, fa_activation act,
                                  cudaStream_t stream) {
    const int64_t ctas = (a.rows * a.blocks * kLanes + kGatedThreads - 1) / kGatedThreads;
    const bool vec = aligned_rows(a.dh, dt) && aligned_rows(a.dgate, dt) &&
                     aligned_rows(a.dup, dt) && aligned_rows(a.h, dt);
    return for_dtype(dt, [&](auto d) {
        return for_activation(act, [&](auto ac) {
            auto *kernel = vec ? gated_backward_kernel<d(), ac(), true>
                               : gated_backward_kernel<d(), ac(), false>;
            kernel<<<static_cast<unsigned>(ctas), kGatedThreads, 0, stream>>>(a);
            return cudaGetLastError();
        });
    });
}

}  // namespace fa
