// The join of a block's output to the residual stream, with the norms behind and before it.
//
// A row belongs to one CTA (several short rows to one, a warp each); thread i holds the runs of
// eight columns i, i + threads, ... of it in registers, so the stream is read once and both
// norms' sums are taken from what is there.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "internal.h"

FA_BOUNDS_COUNTER(g_join_oob)

#include "join_device.cuh"

namespace fa {
namespace {

constexpr int kRowWarps = 4;       // short rows to a CTA
constexpr float kHuge = 0x1p-70f;  // rows whose squares pass FP32 are summed at this scale

// The sum over a row's threads (blockDim.x of them), in every one.  ``part``: one float per
// warp, not in use by the call before.
__device__ __forceinline__ float row_sum(float x, float *part) {
    x = warp_sum(x);
    if (blockDim.x == 32) return x;
    if (threadIdx.x % 32 == 0) part[threadIdx.x / 32] = x;
    __syncthreads();
    float s = 0.f;
    for (unsigned w = 0; w < blockDim.x / 32; ++w) s += part[w];
    return s;
}

__device__ __forceinline__ float inverse_root(float sum, float cols, float eps) {
    return __frsqrt_rn(__fdiv_rn(sum, cols) + eps);
}

// 1 / sqrt(mean square + eps) of the row that the threads hold.
template <int R>
__device__ __forceinline__ float row_rstd(const float (*x)[kRun], float cols, float eps,
                                          float *part, float *part_again) {
    float s = 0.f;
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
        for (int j = 0; j < kRun; ++j) s = fmaf(x[r][j], x[r][j], s);
    s = row_sum(s, part);
    if (s < INFINITY) return inverse_root(s, cols, eps);
    // squares past FP32 (or an infinity or NaN, which stays one); eps does not matter to them
    s = 0.f;
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
        for (int j = 0; j < kRun; ++j) {
            const float y = x[r][j] * kHuge;
            s = fmaf(y, y, s);
        }
    return inverse_root(row_sum(s, part_again), cols, 0.f) * kHuge;
}

template <int DT, int ST, int R, bool ALIGNED>
__global__ void __launch_bounds__(R == 1 ? 256 : kMaxThreads) join_kernel(JoinArgs a) {
    __shared__ float part[4][kMaxThreads / 32];
    const int64_t row = static_cast<int64_t>(blockIdx.x) * blockDim.y + threadIdx.y;
    if (row >= a.rows) return;  // a whole warp: rows share no barrier
    const float cols = static_cast<float>(a.cols);
    int64_t c[R];
    int valid[R];
    Raw<DT, kRun> ry[R];
    Raw<ST, kRun> rr[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
        c[r] = (static_cast<int64_t>(r) * blockDim.x + threadIdx.x) * kRun;
        valid[r] = valid_cols(c[r], a.cols);
        if (a.branch.p) ry[r] = load_run<DT, ALIGNED>(a.branch, row, c[r]);
    }
#pragma unroll
    for (int r = 0; r < R; ++r) rr[r] = load_run<ST, ALIGNED>(a.residual, row, c[r]);
    float y[R][kRun], x[R][kRun];
    if (a.branch.p) {
#pragma unroll
        for (int r = 0; r < R; ++r) ry[r].widen(y[r]);
        float rstd = 1.f;
        if (a.post_norm) {
            rstd = row_rstd<R>(y, cols, a.eps, part[0], part[1]);
            if (a.post_rstd && threadIdx.x == 0) a.post_rstd[row] = rstd;
        }
        const int64_t group = a.gate ? a.by_group.quotient(static_cast<uint32_t>(row)) : 0;
        const uint64_t call = a.dropped ? drop_call(a.drop) : 0;
        const float scale = a.dropped ? a.drop.scale * a.branch_scale : a.branch_scale;
        const int64_t blocks = (a.cols + kRun - 1) / kRun;
#pragma unroll
        for (int r = 0; r < R; ++r) {
            float w[kRun];
            if (a.post_norm) {
                load_weights<DT>(a, a.post_weight, c[r], valid[r],
                                          a.weight_offset, w);
#pragma unroll
                for (int j = 0; j < kRun; ++j) y[r][j] *= rstd * w[j];
            }
            if (a.gate) {
                load_weights<DT>(a, a.gate, group * a.gate_ld + c[r],
                                          valid[r], 0.f, w);
#pragma unroll
                for (int j = 0; j < kRun; ++j) y[r][j] *= w[j];
            }
            if (a.dropped) {
                Kept kept;
                kept.draw(a.drop, row * blocks + c[r] / kRun, call);
#pragma unroll
                for (int j = 0; j < kRun; ++j)
                    if (!kept(j, a.drop.threshold)) y[r][j] = 0.f;
            }
            rr[r].widen(x[r]);
#pragma unroll
            for (int j = 0; j < kRun; ++j)
                x[r][j] = fmaf(a.residual_scale, x[r][j], scale * y[r][j]);
        }
    } else {
#pragma unroll
        for (int r = 0; r < R; ++r) {
            rr[r].widen(x[r]);
#pragma unroll
            for (int j = 0; j < kRun; ++j) x[r][j] *= a.residual_scale;
        }
    }
    if (a.out.p) {
#pragma unroll
        for (int r = 0; r < R; ++r)
            store_run<ST, ALIGNED>(a.out, row, c[r], x[r], 0xffffffffu, 32);
    }
    if (!a.normed.p) return;
    // the norm is that of the stored values
#pragma unroll
    for (int r = 0; r < R; ++r) {
        rr[r].from(x[r]);
        rr[r].widen(x[r]);
    }
    const float rstd = row_rstd<R>(x, cols, a.eps, part[2], part[3]);
    if (a.pre_rstd && threadIdx.x == 0) a.pre_rstd[row] = rstd;
#pragma unroll
    for (int r = 0; r < R; ++r) {
        float w[kRun];
        load_weights<DT>(a, a.pre_weight, c[r], valid[r], a.weight_offset,
                                  w);
#pragma unroll
        for (int j = 0; j < kRun; ++j) x[r][j] *= rstd * w[j];
        store_run<DT, ALIGNED>(a.normed, row, c[r], x[r], 0xffffffffu, 32);
    }
}

// Threads of a row and runs of a thread.
struct Shape {
    int threads, runs;
};
Shape forward_shape(int64_t cols) {
    const int64_t runs = (cols + kRun - 1) / kRun;
    const int r = runs <= 256 ? 1 : runs <= 1024 ? 2 : 4;
    return {static_cast<int>(((runs + r - 1) / r + 31) / 32 * 32), r};
}

template <typename F>
cudaError_t for_runs(int runs, F f) {
    switch (runs) {
        case 1: return f(std::integral_constant<int, 1>{});
        case 2: return f(std::integral_constant<int, 2>{});
        default: return f(std::integral_constant<int, 4>{});
    }
}

}  // namespace

FA_BOUNDS_VIOLATIONS(join_bounds_violations, g_join_oob)

cudaError_t launch_block_join(const JoinArgs &a, fa_dtype dt, fa_dtype st, cudaStream_t stream) {
    const Shape shape = forward_shape(a.cols);
    const dim3 block(shape.threads, shape.threads == 32 ? kRowWarps : 1);
    const unsigned grid = static_cast<unsigned>((a.rows + block.y - 1) / block.y);
    const bool vec = aligned_rows(a.branch, dt) && aligned_rows(a.residual, st) &&
                     aligned_rows(a.out, st) && aligned_rows(a.normed, dt);
    return for_stream_dtype(dt, st, [&](auto d, auto s) {
        return for_runs(shape.runs, [&](auto r) {
            auto *kernel = vec ? join_kernel<d(), s(), r(), true>
                               : join_kernel<d(), s(), r(), false>;
            kernel<<<grid, block, 0, stream>>>(a);
            return cudaGetLastError();
        });
    });
}

}  // namespace fa
