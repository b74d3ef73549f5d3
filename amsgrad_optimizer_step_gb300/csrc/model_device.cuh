// Device helpers shared by the kernels of the model-side operators: the three element
// types in 16-byte vectors, block reductions and double-float sums.
#pragma once

#include <cstdint>

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "fa_model_ops.h"

namespace fa {

// One element type: kVec elements in 16 bytes, widened to and rounded from FP32.
template <int DT>
struct Elem;

template <>
struct Elem<FA_F32> {
    using T = float;
    static constexpr int kVec = 4;
    static __device__ __forceinline__ float widen(T x) { return x; }
    static __device__ __forceinline__ T round(float x) { return x; }
    static __device__ __forceinline__ void unpack(const uint4 &r, float *x) {
        x[0] = __uint_as_float(r.x);
        x[1] = __uint_as_float(r.y);
        x[2] = __uint_as_float(r.z);
        x[3] = __uint_as_float(r.w);
    }
    static __device__ __forceinline__ uint4 pack(const float *x) {
        return make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]),
                          __float_as_uint(x[3]));
    }
};

template <>
struct Elem<FA_F16> {
    using T = __half;
    static constexpr int kVec = 8;
    static __device__ __forceinline__ float widen(T x) { return __half2float(x); }
    static __device__ __forceinline__ T round(float x) { return __float2half_rn(x); }
    static __device__ __forceinline__ void unpack(const uint4 &r, float *x) {
        const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&w[k]));
            x[2 * k] = f.x;
            x[2 * k + 1] = f.y;
        }
    }
    static __device__ __forceinline__ uint4 pack(const float *x) {
        uint32_t w[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const __half2 h = __floats2half2_rn(x[2 * k], x[2 * k + 1]);
            w[k] = *reinterpret_cast<const uint32_t *>(&h);
        }
        return make_uint4(w[0], w[1], w[2], w[3]);
    }
};

template <>
struct Elem<FA_BF16> {
    using T = __nv_bfloat16;
    static constexpr int kVec = 8;
    static __device__ __forceinline__ float widen(T x) { return __bfloat162float(x); }
    static __device__ __forceinline__ T round(float x) { return __float2bfloat16_rn(x); }
    static __device__ __forceinline__ void unpack(const uint4 &r, float *x) {
        const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            x[2 * k] = __uint_as_float(w[k] << 16);
            x[2 * k + 1] = __uint_as_float(w[k] & 0xffff0000u);
        }
    }
    static __device__ __forceinline__ uint4 pack(const float *x) {
        uint32_t w[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const __nv_bfloat162 h = __floats2bfloat162_rn(x[2 * k], x[2 * k + 1]);
            w[k] = *reinterpret_cast<const uint32_t *>(&h);
        }
        return make_uint4(w[0], w[1], w[2], w[3]);
    }
};

// Stores N consecutive FP32 values as elements of DT: 16-byte stores when they fill
// whole vectors (p 16-byte aligned then), element stores otherwise.
template <int DT, int N>
__device__ __forceinline__ void store_n(typename Elem<DT>::T *p, const float *x) {
    constexpr int V = Elem<DT>::kVec;
    if constexpr (N % V == 0) {
#pragma unroll
        for (int j = 0; j < N; j += V) __stcs(reinterpret_cast<uint4 *>(p + j), Elem<DT>::pack(x + j));
    } else {
#pragma unroll
        for (int j = 0; j < N; ++j) p[j] = Elem<DT>::round(x[j]);
    }
}

// Loads N consecutive elements of DT as FP32 (the counterpart of store_n).
template <int DT, int N>
__device__ __forceinline__ void load_n(const typename Elem<DT>::T *p, float *x) {
    constexpr int V = Elem<DT>::kVec;
    if constexpr (N % V == 0) {
#pragma unroll
        for (int j = 0; j < N; j += V)
            Elem<DT>::unpack(__ldcs(reinterpret_cast<const uint4 *>(p + j)), x + j);
    } else {
#pragma unroll
        for (int j = 0; j < N; ++j) x[j] = Elem<DT>::widen(p[j]);
    }
}

template <int IT>
__device__ __forceinline__ int64_t load_id(const void *ids, int64_t i) {
    return IT == FA_I64 ? __ldg(static_cast<const long long *>(ids) + i)
                        : static_cast<int64_t>(__ldg(static_cast<const int *>(ids) + i));
}

// 2^x, within 2 ulp; 0 for -inf, inf above the range, NaN for NaN.
__device__ __forceinline__ float exp2_fast(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// A sum held as an FP32 value and its FP32 residual; each addition is error-free but
// for the residual's own rounding, so a sum of n terms is exact to about 2^-46.
struct Sum2 {
    float hi = 0.f, lo = 0.f;
    __device__ __forceinline__ void add(float x) {
        const float s = hi + x;
        const float b = s - hi;
        lo += (hi - (s - b)) + (x - b);
        hi = s;
    }
    __device__ __forceinline__ void add(const Sum2 &o) {
        add(o.hi);
        lo += o.lo;
    }
    // The sum in FP32 (an infinite or NaN sum has no residual).
    __device__ __forceinline__ float value() const { return isfinite(hi) ? hi + lo : hi; }
};

__device__ __forceinline__ Sum2 warp_sum2(Sum2 s) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        Sum2 t;
        t.hi = __shfl_down_sync(0xffffffffu, s.hi, o);
        t.lo = __shfl_down_sync(0xffffffffu, s.lo, o);
        s.add(t);
    }
    return s;  // valid in lane 0
}

}  // namespace fa
