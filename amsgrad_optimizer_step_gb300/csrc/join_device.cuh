// What the kernels of a join and of its gradient share.  The including file invokes
// FA_BOUNDS_COUNTER first.
#pragma once

#include "block_internal.h"
#include "model_runs.cuh"
#include "philox.cuh"

namespace fa {

constexpr int kMaxThreads = 512;  // of a row of the gradient with several runs a thread

// Weights of a run: 1 where there are none; ``valid`` of them exist, the others are 0.
template <int DT>
__device__ __forceinline__ void load_weights(const JoinArgs &a, const void *p, int64_t at, int valid,
                                             float offset, float *w) {
    if (!p) {
#pragma unroll
        for (int j = 0; j < kRun; ++j) w[j] = 1.f;
        return;
    }
    using T = typename Elem<DT>::T;
    const bool wide = a.wide_weights;
    if (a.vec_weights && valid == kRun) {
        if (wide)
            read_n<FA_F32, kRun>(static_cast<const float *>(p) + at, w);
        else
            read_n<DT, kRun>(static_cast<const T *>(p) + at, w);
    } else {
#pragma unroll
        for (int j = 0; j < kRun; ++j) {
            w[j] = 0.f;
            if (j < valid)
                w[j] = wide ? static_cast<const float *>(p)[at + j]
                            : Elem<DT>::widen(static_cast<const T *>(p)[at + j]);
        }
    }
#pragma unroll
    for (int j = 0; j < kRun; ++j) w[j] += offset;
}

__device__ __forceinline__ float warp_sum(float x) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    return x;
}

// The lanes of a team (blockDim.x; the teams, 16 at most where they have several warps, are
// blockDim.y) wait for one another.  No barrier of the whole CTA may be open meanwhile.
__device__ __forceinline__ void team_sync() {
    asm volatile("bar.sync %0, %1;" ::"r"(threadIdx.y), "r"(blockDim.x) : "memory");
}

constexpr int kPairs = kRun / 2;

__device__ __forceinline__ uint64_t both(float x) { return pair(x, x); }

template <int DT>
__device__ __forceinline__ void widen_pairs(const Raw<DT, kRun> &x, uint64_t *p) {
    float v[kRun];
    x.widen(v);
#pragma unroll
    for (int j = 0; j < kPairs; ++j) p[j] = pair(v[2 * j], v[2 * j + 1]);
}

template <int DT>
__device__ __forceinline__ void zero(Raw<DT, kRun> &x) {
#pragma unroll
    for (int k = 0; k < Raw<DT, kRun>::kWords; ++k) x.r[k] = make_uint4(0u, 0u, 0u, 0u);
}

// Stores a run of whole, aligned vectors.
template <int DT>
__device__ __forceinline__ void store_raw(const MatrixArgs &m, int64_t row, int64_t c,
                                          const Raw<DT, kRun> &x) {
    if (!fa_in_bounds(c, kRun, m.cols)) return;
    auto *p = static_cast<typename Elem<DT>::T *>(m.p) + row * m.ld + c;
#pragma unroll
    for (int k = 0; k < Raw<DT, kRun>::kWords; ++k) __stcs(reinterpret_cast<uint4 *>(p) + k, x.r[k]);
}

// Run ``q`` of a row of ``runs``: whole vectors where VEC (zeros past the end), else from any
// address.
template <int DT, bool VEC>
__device__ __forceinline__ Raw<DT, kRun> read_run(const MatrixArgs &m, int64_t row, int q,
                                                  int runs) {
    if constexpr (VEC) {
        Raw<DT, kRun> x;
        zero(x);
        if (q < runs && fa_in_bounds(q * kRun, kRun, m.cols))
            x.load(static_cast<const typename Elem<DT>::T *>(m.p) + row * m.ld + q * kRun);
        return x;
    } else {
        return load_run<DT, false>(m, row, static_cast<int64_t>(q) * kRun);
    }
}

__device__ __forceinline__ void to_pairs(const float *x, uint64_t *p) {
#pragma unroll
    for (int j = 0; j < kPairs; ++j) p[j] = pair(x[2 * j], x[2 * j + 1]);
}
__device__ __forceinline__ void from_pairs(const uint64_t *p, float *x) {
#pragma unroll
    for (int j = 0; j < kPairs; ++j) unpair(p[j], x[2 * j], x[2 * j + 1]);
}

// Run ``q`` of a row (whole, aligned vectors) asked into a lane's slots, ``stride`` vectors apart,
// and taken from there.
template <int DT>
__device__ __forceinline__ void ask_run(const MatrixArgs &m, int64_t row, int q, uint4 *slot,
                                        int stride) {
    const auto *p = static_cast<const typename Elem<DT>::T *>(m.p) + row * m.ld + q * kRun;
#pragma unroll
    for (int k = 0; k < Raw<DT, kRun>::kWords; ++k)
        copy_async16(slot + k * stride, reinterpret_cast<const uint4 *>(p) + k);
}
template <int DT>
__device__ __forceinline__ void take_run(const uint4 *slot, int stride, Raw<DT, kRun> &x) {
#pragma unroll
    for (int k = 0; k < Raw<DT, kRun>::kWords; ++k) x.r[k] = slot[k * stride];
}

}  // namespace fa
