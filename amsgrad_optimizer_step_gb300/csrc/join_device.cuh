// What the kernels of a join and of its gradient share.  The including file invokes
// FA_BOUNDS_COUNTER first.
#pragma once

#include <initializer_list>

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

template <int DT>
__device__ __forceinline__ float one_weight(const JoinArgs &a, const void *p, int64_t at,
                                            float offset) {
    if (!p) return 1.f;
    return offset + (a.wide_weights ? static_cast<const float *>(p)[at]
                                    : Elem<DT>::widen(static_cast<const typename Elem<DT>::T *>(p)[at]));
}
// Of a run that begins at column ``c``, which may be negative: its weights, zeros in place of what is
// no column, and the stores of what is one.
__device__ __forceinline__ bool is_column(int c, int cols) {
    return static_cast<unsigned>(c) < static_cast<unsigned>(cols);
}
template <int DT>
__device__ __forceinline__ void load_columns(const JoinArgs &a, const void *p, int64_t row0, int c,
                                             int cols, float offset, float *w) {
#pragma unroll
    for (int j = 0; j < kRun; ++j)
        w[j] = is_column(c + j, cols) ? one_weight<DT>(a, p, row0 + c + j, offset) : 0.f;
}
template <int DT>
__device__ __forceinline__ void keep_columns(Raw<DT, kRun> &x, int c, int cols) {
    float v[kRun];
    x.widen(v);
#pragma unroll
    for (int j = 0; j < kRun; ++j) v[j] = is_column(c + j, cols) ? v[j] : 0.f;
    x.from(v);  // exact: they came from this type
}
template <int DT>
__device__ __forceinline__ void store_columns(typename Elem<DT>::T *p, const float *v, int c, int cols) {
#pragma unroll
    for (int j = 0; j < kRun; ++j)
        if (is_column(c + j, cols)) p[j] = Elem<DT>::round(v[j]);
}
template <int DT>
__device__ __forceinline__ void store_columns(const MatrixArgs &m, int64_t row, const float *v, int c) {
    if (fa_in_bounds(row, 1, m.rows))
        store_columns<DT>(static_cast<typename Elem<DT>::T *>(m.p) + row * m.ld + c, v, c,
                      static_cast<int>(m.cols));
}
// (c: where a line begins in memory)
template <int DT>
__device__ __forceinline__ Raw<DT, kRun> read_columns(const MatrixArgs &m, int64_t row, int c) {
    const auto *p = static_cast<const typename Elem<DT>::T *>(m.p) + row * m.ld + c;
    const int cols = static_cast<int>(m.cols);
    Raw<DT, kRun> x;
    const bool there = fa_in_bounds(row, 1, m.rows);
    if (there && c >= 0 && c + kRun <= cols) {
        x.load(p);
    } else {
        float v[kRun];
#pragma unroll
        for (int j = 0; j < kRun; ++j)
            v[j] = there && is_column(c + j, cols) ? Elem<DT>::widen(p[j]) : 0.f;
        x.from(v);  // exact: they came from this type
    }
    return x;
}
// Asks a vector of 16-bit columns into a slot: zeros behind the last one, the end of the row before in
// front of the first.
template <int DT>
__device__ __forceinline__ void ask_columns(const MatrixArgs &m, int64_t row, int c, uint4 *slot) {
    static_assert(Raw<DT, kRun>::kWords == 1, "a vector");
    const int left = static_cast<int>(m.cols) - c, n = left < kRun ? left : kRun;
    if (n <= 0 || !fa_in_bounds(row * m.ld + c, n, (m.rows - 1) * m.ld + m.cols)) return;
    copy_async16(slot, static_cast<const typename Elem<DT>::T *>(m.p) + row * m.ld + c, 2 * n);
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
    if (!fa_in_bounds(c, kRun, m.cols) || !fa_in_bounds(row, 1, m.rows)) return;
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
        if (q < runs && fa_in_bounds(q * kRun, kRun, m.cols) && fa_in_bounds(row, 1, m.rows))
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

// The row distance modulo eight that all of the matrices have that are there, where they begin on a
// 16-byte boundary; else -1.  Their 16-byte lines then begin at the same columns in a row of all of
// them, and at the same ones again eight rows on.
inline int common_ld8(std::initializer_list<const MatrixArgs *> matrices) {
    int64_t ld8 = -1;
    for (const MatrixArgs *m : matrices) {
        if (!m->p) continue;
        if (reinterpret_cast<uintptr_t>(m->p) % 16 || (ld8 >= 0 && m->ld % kRun != ld8)) return -1;
        ld8 = m->ld % kRun;
    }
    return static_cast<int>(ld8);
}

}  // namespace fa
