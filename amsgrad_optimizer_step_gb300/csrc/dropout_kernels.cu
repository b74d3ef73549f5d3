// Dropout whose mask is drawn again wherever it is needed and never stored.
//
// One Philox block of 128 bits serves a run of eight columns, so a thread that takes one
// 16-byte vector of 16-bit elements (two of FP32) draws once.  Rows that lie densely are one
// long row of runs; others go in blocks of 64 columns, eight lanes each, as whole 16-byte
// vectors where they are aligned and as the 16-byte lines around them where not.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "internal.h"

FA_BOUNDS_COUNTER(g_dropout_oob)

#include "model_runs.cuh"
#include "philox.cuh"

namespace fa {
namespace {

constexpr int kDropThreads = 256;
constexpr int kDropLanes = 8;  // per block of columns
constexpr int kDropBlock = kDropLanes * kRun;

__device__ __forceinline__ void drop(const DropArgs &d, const Kept &kept, float *x) {
#pragma unroll
    for (int j = 0; j < kRun; ++j) x[j] = kept(j, d.threshold) ? x[j] * d.scale : 0.f;
}

template <int DT, int R>
__global__ void __launch_bounds__(kDropThreads) dropout_dense_kernel(DropoutArgs a) {
    using T = typename Elem<DT>::T;
    const int64_t runs = a.x.rows * (a.x.cols / kRun);
    const int64_t first = static_cast<int64_t>(blockIdx.x) * (R * kDropThreads) + threadIdx.x;
    Raw<DT, kRun> raw[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
        const int64_t i = first + r * kDropThreads;
        if (i < runs && fa_in_bounds(i * kRun, kRun, a.x.rows * a.x.cols))
            raw[r].load(static_cast<const T *>(a.x.p) + i * kRun);
    }
    const uint64_t call = drop_call(a.drop);
#pragma unroll
    for (int r = 0; r < R; ++r) {
        const int64_t i = first + r * kDropThreads;
        if (i >= runs) return;
        Kept kept;
        kept.draw(a.drop, i, call);
        float x[kRun];
        raw[r].widen(x);
        drop(a.drop, kept, x);
        if (fa_in_bounds(i * kRun, kRun, a.out.rows * a.out.cols))
            store_n<DT, kRun>(static_cast<T *>(a.out.p) + i * kRun, x);
    }
}

template <int DT, bool ALIGNED>
__global__ void __launch_bounds__(kDropThreads) dropout_kernel(DropoutArgs a) {
    const int64_t b = static_cast<int64_t>(blockIdx.x) * (kDropThreads / kDropLanes) +
                      threadIdx.x / kDropLanes;
    if (b >= a.x.rows * a.blocks) return;  // all eight lanes of a block
    const int64_t row = a.by_blocks.quotient(static_cast<uint32_t>(b));
    const int64_t c = (b - row * a.blocks) * kDropBlock + threadIdx.x % kDropLanes * kRun;
    const Raw<DT, kRun> raw = load_run<DT, ALIGNED>(a.x, row, c);
    Kept kept;
    kept.draw(a.drop, row * ((a.x.cols + kRun - 1) / kRun) + c / kRun, drop_call(a.drop));
    float x[kRun];
    raw.widen(x);
    drop(a.drop, kept, x);
    store_run<DT, ALIGNED>(a.out, row, c, x, 0xffu << (threadIdx.x & 24), kDropLanes);
}

}  // namespace

FA_BOUNDS_VIOLATIONS(dropout_bounds_violations, g_dropout_oob)

cudaError_t launch_dropout(const DropoutArgs &a, fa_dtype dt, cudaStream_t stream) {
    const bool vec = aligned_rows(a.x, dt) && aligned_rows(a.out, dt);
    const bool dense = a.x.cols % kRun == 0 &&
                       (a.x.rows == 1 || (a.x.ld == a.x.cols && a.out.ld == a.out.cols));
    return for_dtype(dt, [&](auto d) {
        if (vec && dense) {
            constexpr int R = 2;
            const int64_t runs = a.x.rows * (a.x.cols / kRun);
            const int64_t ctas = (runs + R * kDropThreads - 1) / (R * kDropThreads);
            dropout_dense_kernel<d(), R>
                <<<static_cast<unsigned>(ctas), kDropThreads, 0, stream>>>(a);
        } else {
            constexpr int kBlocks = kDropThreads / kDropLanes;
            const int64_t ctas = (a.x.rows * a.blocks + kBlocks - 1) / kBlocks;
            auto *kernel = vec ? dropout_kernel<d(), true> : dropout_kernel<d(), false>;
            kernel<<<static_cast<unsigned>(ctas), kDropThreads, 0, stream>>>(a);
        }
        return cudaGetLastError();
    });
}

}  // namespace fa
