// Device helpers shared by the kernels of the model-side operators: the three element
// types in 16-byte vectors, block reductions and double-float sums.
#pragma once

#include <cstdint>
#include <type_traits>

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
    // Largest magnitude in N vectors, NaN where any element is.
    template <int N>
    static __device__ __forceinline__ float magnitude(const uint4 *r) {
        float m = 0.f;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            float x[4];
            unpack(r[i], x);
#pragma unroll
            for (int j = 0; j < 4; ++j)
                asm("max.NaN.f32 %0, %0, %1;" : "+f"(m) : "f"(fabsf(x[j])));
        }
        return m;
    }
    // Largest element of N vectors, NaN ignored where there is another.
    template <int N>
    static __device__ __forceinline__ float largest(const uint4 *r) {
        float m = -INFINITY;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            m = fmaxf(fmaxf(m, __uint_as_float(r[i].x)), __uint_as_float(r[i].y));
            m = fmaxf(fmaxf(m, __uint_as_float(r[i].z)), __uint_as_float(r[i].w));
        }
        return m;
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
    template <int N>
    static __device__ __forceinline__ float magnitude(const uint4 *r) {
        const __half2 *p = reinterpret_cast<const __half2 *>(r);
        __half2 m = __habs2(p[0]);
#pragma unroll
        for (int i = 1; i < 4 * N; ++i) m = __hmax2_nan(m, __habs2(p[i]));
        return __half2float(__hmax_nan(__low2half(m), __high2half(m)));
    }
    template <int N>
    static __device__ __forceinline__ float largest(const uint4 *r) {
        const __half2 *p = reinterpret_cast<const __half2 *>(r);
        __half2 m = p[0];
#pragma unroll
        for (int i = 1; i < 4 * N; ++i) m = __hmax2(m, p[i]);
        return __half2float(__hmax(__low2half(m), __high2half(m)));
    }
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
    template <int N>
    static __device__ __forceinline__ float magnitude(const uint4 *r) {
        const __nv_bfloat162 *p = reinterpret_cast<const __nv_bfloat162 *>(r);
        __nv_bfloat162 m = __habs2(p[0]);
#pragma unroll
        for (int i = 1; i < 4 * N; ++i) m = __hmax2_nan(m, __habs2(p[i]));
        return __bfloat162float(__hmax_nan(__low2bfloat16(m), __high2bfloat16(m)));
    }
    template <int N>
    static __device__ __forceinline__ float largest(const uint4 *r) {
        const __nv_bfloat162 *p = reinterpret_cast<const __nv_bfloat162 *>(r);
        __nv_bfloat162 m = p[0];
#pragma unroll
        for (int i = 1; i < 4 * N; ++i) m = __hmax2(m, p[i]);
        return __bfloat162float(__hmax(__low2bfloat16(m), __high2bfloat16(m)));
    }
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

// N FP32 values (whole vectors) rounded and packed into words.
template <int DT, int N>
__device__ __forceinline__ void pack_words(const float *x, uint32_t *w) {
    using E = Elem<DT>;
#pragma unroll
    for (int k = 0; k < N / E::kVec; ++k) {
        const uint4 r = E::pack(x + k * E::kVec);
        w[4 * k] = r.x;
        w[4 * k + 1] = r.y;
        w[4 * k + 2] = r.z;
        w[4 * k + 3] = r.w;
    }
}

// N elements as they lie in memory, to be widened later: half the registers for 16-bit types.
template <int DT, int N>
struct Raw {
    using E = Elem<DT>;
    static constexpr bool kWhole = N % E::kVec == 0;
    static constexpr int kWords = kWhole ? N / E::kVec : N;
    std::conditional_t<kWhole, uint4, typename E::T> r[kWords];

    __device__ __forceinline__ void load(const typename E::T *p) {
#pragma unroll
        for (int k = 0; k < kWords; ++k) {
            if constexpr (kWhole)
                r[k] = __ldcs(reinterpret_cast<const uint4 *>(p) + k);
            else
                r[k] = p[k];
        }
    }
    __device__ __forceinline__ void widen(float *x) const {
#pragma unroll
        for (int k = 0; k < kWords; ++k) {
            if constexpr (kWhole)
                E::unpack(r[k], x + k * E::kVec);
            else
                x[k] = E::widen(r[k]);
        }
    }
    // From values of this type.
    __device__ __forceinline__ void from(const float *x) {
        static_assert(kWhole, "whole vectors");
#pragma unroll
        for (int k = 0; k < kWords; ++k) r[k] = E::pack(x + k * E::kVec);
    }
    // The largest magnitude; NaN where any element is.
    __device__ __forceinline__ float magnitude() const {
        static_assert(kWhole, "whole vectors");
        return E::template magnitude<kWords>(r);
    }
};

// ---- runs of elements at any element-aligned address ----------------------------------

// Words [0, W) of ``cat`` moved down by ``bytes`` (0 to 15, a multiple of two); cat holds W + 4.
template <int W>
__device__ __forceinline__ void move_down(const uint32_t *cat, int bytes, uint32_t *out) {
    uint32_t a[W + 3], b[W + 1];
#pragma unroll
    for (int i = 0; i < W + 3; ++i) a[i] = bytes & 4 ? cat[i + 1] : cat[i];
#pragma unroll
    for (int i = 0; i < W + 1; ++i) b[i] = bytes & 8 ? a[i + 2] : a[i];
#pragma unroll
    for (int i = 0; i < W; ++i) out[i] = __funnelshift_r(b[i], b[i + 1], 8 * (bytes & 2));
}

// Bytes that 16-byte reads may touch: those of the 16-byte lines inside an array.
struct Span {
    uintptr_t lo, hi;

    __host__ __device__ Span(const void *p, int64_t bytes)
        : lo(reinterpret_cast<uintptr_t>(p)), hi(lo + bytes) {}
};

// N elements (whole vectors) from any address, as they lie in memory: the 16-byte lines
// around them where those are inside the array (what else is in them is not used), else
// element by element.
template <int DT, int N>
struct RawAny {
    using E = Elem<DT>;
    static constexpr int kWords = N / E::kVec * 4;
    uint32_t cat[kWords + 4];
    int bytes;  // from the first word to the first element

    // The first ``valid`` of the elements exist; the others are 0.
    __device__ __forceinline__ void load(const typename E::T *p, int valid, const Span &in) {
        const uintptr_t at = reinterpret_cast<uintptr_t>(p), line = at & ~uintptr_t(15);
        bytes = static_cast<int>(at - line);
        if (valid == N && line >= in.lo && line + 4 * kWords + (bytes ? 16 : 0) <= in.hi) {
            const uint4 *q = reinterpret_cast<const uint4 *>(line);
#pragma unroll
            for (int k = 0; k <= kWords / 4; ++k) {
                uint4 r = make_uint4(0u, 0u, 0u, 0u);
                if (k < kWords / 4 || bytes) r = __ldg(q + k);
                cat[4 * k] = r.x;
                cat[4 * k + 1] = r.y;
                cat[4 * k + 2] = r.z;
                cat[4 * k + 3] = r.w;
            }
            return;
        }
        bytes = 0;
        float x[N];
#pragma unroll
        for (int j = 0; j < N; ++j) x[j] = j < valid ? E::widen(p[j]) : 0.f;
        pack_words<DT, N>(x, cat);  // exact: they came from this type
#pragma unroll
        for (int k = kWords; k < kWords + 4; ++k) cat[k] = 0u;
    }
    __device__ __forceinline__ Raw<DT, N> raw() const {
        uint32_t w[kWords];
        move_down<kWords>(cat, bytes, w);
        Raw<DT, N> x;
#pragma unroll
        for (int k = 0; k < kWords / 4; ++k)
            x.r[k] = make_uint4(w[4 * k], w[4 * k + 1], w[4 * k + 2], w[4 * k + 3]);
        return x;
    }
    __device__ __forceinline__ void widen(float *x) const { raw().widen(x); }
};

// Stores the runs of N elements that consecutive lanes hold of one row, lane after lane, from
// any address on: each lane writes the 16-byte lines that begin in the run before its own
// with what that lane has of them, and only the ends of the lanes' whole stretch go element
// by element.  ``p``: where this lane's run belongs; ``valid``: how many of its elements exist
// (N, but for the last lanes).  All lanes of ``lanes`` call it, in groups of ``width``.
template <int DT, int N>
__device__ __forceinline__ void store_any(typename Elem<DT>::T *p, const float *x, int valid,
                                          unsigned lanes, int width) {
    using E = Elem<DT>;
    constexpr int W = N / E::kVec * 4, kSize = sizeof(typename E::T);
    const int bytes = static_cast<int>(reinterpret_cast<uintptr_t>(p) & 15);
    uint32_t cat[W + 4];  // the end of the run before, then this one
    pack_words<DT, N>(x, cat + 4);
#pragma unroll
    for (int k = 0; k < 4; ++k) cat[k] = __shfl_up_sync(lanes, cat[W + k], 1, width);
    const int lane = (threadIdx.x & 31) & (width - 1);
    // whole: this lane writes its lines from the one that its run begins in
    const bool whole = valid == N && (lane > 0 || bytes == 0);
    const bool next_whole = __shfl_down_sync(lanes, whole, 1, width) && lane < width - 1 &&
                            (lanes >> ((threadIdx.x & 31) + 1) & 1u);
    int from = 0, to = valid;  // elements left to write one by one
    if (whole) {
        uint32_t w[W];
        // bytes == 0: the lines are the run's own
        if (bytes == 0) {
#pragma unroll
            for (int k = 0; k < W; ++k) w[k] = cat[4 + k];
        } else {
            move_down<W>(cat, 16 - bytes, w);
        }
        uint4 *q = reinterpret_cast<uint4 *>(reinterpret_cast<uintptr_t>(p) - bytes);
#pragma unroll
        for (int k = 0; k < W / 4; ++k)
            __stcs(q + k, make_uint4(w[4 * k], w[4 * k + 1], w[4 * k + 2], w[4 * k + 3]));
        from = N - bytes / kSize;  // what the next lane's first line holds
        to = next_whole ? from : N;
    } else if (valid == N && next_whole) {
        to = N - bytes / kSize;
    }
#pragma unroll
    for (int j = 0; j < N; ++j)
        if (j >= from && j < to) p[j] = E::round(x[j]);
}

// Loads N consecutive elements of DT as FP32 (the counterpart of store_n), of rows that others
// read too (kept in L2).
template <int DT, int N>
__device__ __forceinline__ void read_n(const typename Elem<DT>::T *p, float *x) {
    constexpr int V = Elem<DT>::kVec;
    if constexpr (N % V == 0) {
#pragma unroll
        for (int j = 0; j < N; j += V)
            Elem<DT>::unpack(__ldg(reinterpret_cast<const uint4 *>(p + j)), x + j);
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

// Asynchronous 16-byte copies from global to shared memory, by the thread that uses them.
__device__ __forceinline__ void copy_async16(void *shared, const void *global) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(
                     static_cast<uint32_t>(__cvta_generic_to_shared(shared))),
                 "l"(global)
                 : "memory");
}
__device__ __forceinline__ void copy_async_commit() {
    asm volatile("cp.async.commit_group;" ::: "memory");
}
// Waits until at most N of the thread's groups are in flight.
template <int N>
__device__ __forceinline__ void copy_async_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// 2^x, within 2 ulp; 0 for -inf, inf above the range, NaN for NaN.
__device__ __forceinline__ float exp2_fast(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// 2^t for t <= 0 within 1.5 ulp: 2^i times the series of 2^f, |f| <= 1/2 (the term left out
// is below 6e-9).  For the factors that whole sums are multiplied by, whose error does not
// average out: six exp2_fast in a row left the log-probabilities 2e-7 off, all the same way.
__device__ __forceinline__ float exp2_exact(float t) {
    if (!(t > -126.f)) return t <= -126.f ? 0.f : t;  // NaN stays
    const float i = rintf(t), f = t - i;
    float p = 1.5252733804059841e-05f;  // ln(2)^n / n!, n = 7 down to 0
    p = fmaf(p, f, 1.5403530393381609e-04f);
    p = fmaf(p, f, 1.3333558146428443e-03f);
    p = fmaf(p, f, 9.6181291076284772e-03f);
    p = fmaf(p, f, 5.5504108664821580e-02f);
    p = fmaf(p, f, 2.4022650695910072e-01f);
    p = fmaf(p, f, 6.9314718055994531e-01f);
    p = fmaf(p, f, 1.f);
    return p * __int_as_float((static_cast<int>(i) + 127) << 23);
}

// Pairs of FP32 values for the packed instructions (two lanes an instruction).
__device__ __forceinline__ uint64_t pair(float lo, float hi) {
    uint64_t d;
    asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "f"(lo), "f"(hi));
    return d;
}
__device__ __forceinline__ void unpair(uint64_t d, float &lo, float &hi) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(d));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
    uint64_t d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
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
