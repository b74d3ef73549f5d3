// The gated activation h = act(gate) * up with an 8-bit checkpoint of its two inputs,
// and its backward pass from the checkpoint.
//
// Sixteen lanes take one block of kCheckpointBlock columns, eight consecutive columns
// each: the block's largest magnitude is four shuffles away, and a lane's eight codes
// are one 8-byte store.
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
constexpr int kLanes = 16;                        // per block of columns
constexpr int kCols = kCheckpointBlock / kLanes;  // per lane
constexpr float kTiny = 0x1p-100f;                // blocks below it are stored as zeros

// sigmoid(z); 0 and 1 at the infinities.
__device__ __forceinline__ float sigmoid(float z) { return __fdividef(1.f, 1.f + __expf(-z)); }

template <int ACT>
struct Activation;

template <>
struct Activation<FA_SILU> {
    static __device__ __forceinline__ float value(float g) { return g * sigmoid(g); }
    static __device__ __forceinline__ void both(float g, float &a, float &da) {
        const float s = sigmoid(g);
        a = g * s;
        da = fmaf(a, 1.f - s, s);  // s (1 + g (1 - s))
    }
};

template <>
struct Activation<FA_GELU_TANH> {
    // 2 sqrt(2/pi) (g + 0.044715 g^3)
    static constexpr float kA = 1.5957691216057308f, kB = 0.071354816272600250f;
    static __device__ __forceinline__ float value(float g) {
        return g * sigmoid(g * fmaf(kB, g * g, kA));
    }
    static __device__ __forceinline__ void both(float g, float &a, float &da) {
        const float q = g * g, s = sigmoid(g * fmaf(kB, q, kA));
        a = g * s;
        da = fmaf(a * (1.f - s), fmaf(3.f * kB, q, kA), s);
    }
};

// A lane's eight columns [c, c + 8) of a row: one 16-byte access (two for FP32) when the
// rows are aligned and the columns all exist, element accesses otherwise; columns past
// the end read as 0 and are not written.
template <int DT, bool VEC>
__device__ __forceinline__ void load_cols(const void *base, int64_t row, int64_t ld, int64_t c,
                                          int64_t cols, float *x) {
    using E = Elem<DT>;
    const typename E::T *p = static_cast<const typename E::T *>(base) + row * ld + c;
    if (VEC && c + kCols <= cols) {
        if (fa_in_bounds(c, kCols, cols)) load_n<DT, kCols>(p, x);
    } else {
#pragma unroll
        for (int j = 0; j < kCols; ++j) x[j] = c + j < cols ? E::widen(p[j]) : 0.f;
    }
}
template <int DT, bool VEC>
__device__ __forceinline__ void store_cols(void *base, int64_t row, int64_t ld, int64_t c,
                                           int64_t cols, const float *x) {
    using E = Elem<DT>;
    typename E::T *p = static_cast<typename E::T *>(base) + row * ld + c;
    if (VEC && c + kCols <= cols) {
        if (fa_in_bounds(c, kCols, cols)) store_n<DT, kCols>(p, x);
    } else {
#pragma unroll
        for (int j = 0; j < kCols; ++j)
            if (c + j < cols) p[j] = E::round(x[j]);
    }
}

// Quantises a block held by the 16 lanes of the mask; the first stores the scale.
__device__ __forceinline__ void store_codes(const float *x, int8_t *codes, float *scale,
                                            bool first_lane, unsigned lanes) {
    float top = 0.f;
    bool bad = false;
#pragma unroll
    for (int j = 0; j < kCols; ++j) {
        top = fmaxf(top, fabsf(x[j]));
        bad |= !isfinite(x[j]);
    }
    if (bad) top = INFINITY;
#pragma unroll
    for (int o = kLanes / 2; o > 0; o >>= 1)
        top = fmaxf(top, __shfl_xor_sync(lanes, top, o, kLanes));
    const bool kept = top >= kTiny && top < INFINITY;
    const float inv = kept ? __fdiv_rn(127.f, top) : 0.f;
    uint32_t w[2] = {0u, 0u};
#pragma unroll
    for (int j = 0; j < kCols; ++j) {
        const int q = kept ? __float2int_rn(__fmul_rn(x[j], inv)) : 0;
        w[j / 4] |= (static_cast<uint32_t>(q) & 0xffu) << (8 * (j % 4));
    }
    __stcs(reinterpret_cast<uint2 *>(codes), make_uint2(w[0], w[1]));
    if (first_lane) *scale = kept ? __fdiv_rn(top, 127.f) : top == INFINITY ? NAN : 0.f;
}

__device__ __forceinline__ void load_codes(const int8_t *codes, float scale, float *x) {
    const uint2 r = __ldcs(reinterpret_cast<const uint2 *>(codes));
    const uint32_t w[2] = {r.x, r.y};
#pragma unroll
    for (int j = 0; j < kCols; ++j) {
        const int q = static_cast<int8_t>(w[j / 4] >> (8 * (j % 4)));
        x[j] = static_cast<float>(q) * scale;
    }
}

template <int DT, int ACT, bool VEC, bool KEEP>
__global__ void __launch_bounds__(kGatedThreads) gated_forward_kernel(GatedForwardArgs a) {
    const int64_t b = (static_cast<int64_t>(blockIdx.x) * kGatedThreads + threadIdx.x) / kLanes;
    const int lane = threadIdx.x % kLanes;
    const int64_t n = a.rows * a.blocks;
    if (b >= n || !fa_in_bounds(b, 1, n)) return;  // all sixteen lanes of a block
    const int64_t row = b / a.blocks;
    const int64_t c = (b - row * a.blocks) * kCheckpointBlock + lane * kCols;
    float g[kCols], u[kCols];
    load_cols<DT, VEC>(a.gate, row, a.gate_ld, c, a.cols, g);
    load_cols<DT, VEC>(a.up, row, a.up_ld, c, a.cols, u);
    float h[kCols];
#pragma unroll
    for (int j = 0; j < kCols; ++j) h[j] = Activation<ACT>::value(g[j]) * u[j];
    store_cols<DT, VEC>(a.h, row, a.h_ld, c, a.cols, h);
    if (KEEP) {
        const unsigned lanes = 0xffffu << (threadIdx.x & kLanes);
        int8_t *code = a.codes + b * kCheckpointBlock + lane * kCols;
        store_codes(g, code, a.scales + b, lane == 0, lanes);
        store_codes(u, code + n * kCheckpointBlock, a.scales + n + b, lane == 0, lanes);
    }
}

template <int DT, int ACT, bool VEC>
__global__ void __launch_bounds__(kGatedThreads) gated_backward_kernel(GatedBackwardArgs a) {
    const int64_t b = (static_cast<int64_t>(blockIdx.x) * kGatedThreads + threadIdx.x) / kLanes;
    const int lane = threadIdx.x % kLanes;
    const int64_t n = a.rows * a.blocks;
    if (b >= n || !fa_in_bounds(b, 1, n)) return;
    const int64_t row = b / a.blocks;
    const int64_t c = (b - row * a.blocks) * kCheckpointBlock + lane * kCols;
    const int8_t *code = a.codes + b * kCheckpointBlock + lane * kCols;
    float g[kCols], u[kCols], d[kCols];
    load_codes(code, a.scales[b], g);
    load_codes(code + n * kCheckpointBlock, a.scales[n + b], u);
    load_cols<DT, VEC>(a.dh, row, a.dh_ld, c, a.cols, d);
    float dg[kCols], du[kCols], h[kCols];
#pragma unroll
    for (int j = 0; j < kCols; ++j) {
        float act, dact;
        Activation<ACT>::both(g[j], act, dact);
        dg[j] = d[j] * dact * u[j];  // |act'| < 1.13: overflows only where the gradient does
        du[j] = d[j] * act;
        h[j] = act * u[j];
    }
    store_cols<DT, VEC>(a.dgate, row, a.dgate_ld, c, a.cols, dg);
    store_cols<DT, VEC>(a.dup, row, a.dup_ld, c, a.cols, du);
    if (a.h) store_cols<DT, VEC>(a.h, row, a.h_ld, c, a.cols, h);
}

// Whether 16-byte accesses at multiples of eight columns are aligned in every row.
bool vector_rows(const void *p, int64_t ld, fa_dtype dt) {
    const int64_t row_bytes = ld * (dt == FA_F32 ? 4 : 2);
    return !p || (reinterpret_cast<uintptr_t>(p) % 16 == 0 && row_bytes % 16 == 0);
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
    if (ctas > kMaxGridX) return cudaErrorInvalidConfiguration;
    const bool vec = vector_rows(a.gate, a.gate_ld, dt) && vector_rows(a.up, a.up_ld, dt) &&
                     vector_rows(a.h, a.h_ld, dt);
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
    if (ctas > kMaxGridX) return cudaErrorInvalidConfiguration;
    const bool vec = vector_rows(a.dh, a.dh_ld, dt) && vector_rows(a.dgate, a.dgate_ld, dt) &&
                     vector_rows(a.dup, a.dup_ld, dt) && vector_rows(a.h, a.h_ld, dt);
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
