// What the kernels of a join and of its gradient share.  The including file invokes
// FA_BOUNDS_COUNTER first.
#pragma once

#include "block_internal.h"
#include "model_runs.cuh"
#include "philox.cuh"

namespace fa {

constexpr int kMaxThreads = 512;  // of a row

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

}  // namespace fa
