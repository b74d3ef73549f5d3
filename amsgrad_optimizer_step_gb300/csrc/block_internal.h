// Internal interface between the C-ABI host layer of the residual blocks' operators
// (block_abi.cpp) and their kernels (dropout_kernels.cu, join_kernels.cu,
// route_kernels.cu).
#pragma once

#include <atomic>
#include <cstdint>

#include <cuda_runtime.h>

#include "fa_block_ops.h"
#include "internal.h"
#include "model_internal.h"

namespace fa {

// ---- dropout -------------------------------------------------------------------
constexpr int kPhiloxRounds = 10;
struct DropArgs {
    uint32_t threshold;  // 16 bits are kept from threshold >> 16 on; 2^32 - 1: none is
    uint32_t key[kPhiloxRounds][2];  // of each round
    uint64_t offset;
    const uint64_t *counter;  // or nullptr
    float scale;              // of what is kept
};
constexpr int kDropColumns = 128;  // whose blocks over all rows the grid's limit counts
struct DropoutArgs {
    MatrixArgs x, out;
    int64_t blocks;  // of a row, and the division by them (set by the launch)
    Divider by_blocks;
    DropArgs drop;
};
cudaError_t launch_dropout(const DropoutArgs &a, fa_dtype dt, cudaStream_t stream);

// ---- the join of a block to the residual stream -------------------------------------
struct JoinArgs {
    MatrixArgs branch, residual, out, normed;  // p nullptr where there is none
    const void *post_weight, *pre_weight, *gate;
    int64_t gate_ld;
    int64_t rows, cols;
    uint32_t group_rows;  // rows that share a row of the gate
    Divider by_group;
    bool wide_weights;  // FP32 (else the branch's type)
    bool vec_weights;   // every row of them starts on a 16-byte boundary
    bool post_norm, dropped;
    float residual_scale, branch_scale, eps, weight_offset;
    float *post_rstd, *pre_rstd;  // or nullptr
    DropArgs drop;
    int32_t ld8;  // the matrices' common_ld8 where rows are taken that begin anywhere, else -1
};
cudaError_t launch_block_join(const JoinArgs &a, fa_dtype dt, fa_dtype st, cudaStream_t stream);

// How the gradient cuts the rows into CTAs, each with FP32 sums of its own.  element_bytes: of a
// column over the four matrices that it reads (8 at least, which gives the most CTAs).
struct JoinPlan {
    int64_t chunk;  // rows of a CTA at most
    int64_t ctas;
    int64_t pitch;  // columns of one row of sums
    int64_t parts;  // rows of sums of a CTA
    int64_t bytes;
};
JoinPlan join_plan(int64_t rows, int64_t cols, int64_t groups, int element_bytes);

// Threads of a row of the gradient and runs of a thread: one up to 6144 columns, two up to 8192
// (the columns' sums are two registers a column); 0: more, in clusters, or from any address with the
// sums in shared memory.
struct JoinShape {
    int threads, runs;
};
JoinShape join_shape(int64_t cols);
constexpr int kJoinThreads = 768;  // of a row of one run a thread, and of an SM
// CTAs of the gradient on an SM, for rows of ``row_bytes`` over the four matrices that it reads:
// as many as have room for two rows each on their way, beside the weights (64 bytes a run).
constexpr int kSmShared = 228 * 1024;  // of an SM, of which a CTA has 2 KB for other things
inline int join_ctas_per_sm(const JoinShape &shape, int row_bytes) {
    int n = shape.threads < kJoinThreads ? kJoinThreads / shape.threads : 1;
    while (n > 1 && kSmShared / n - 2048 - 64 * shape.runs * shape.threads < 2 * row_bytes) --n;
    return n;
}

// CTAs of the gradient of ``rows``: as many as an SM has room for, but 16 rows each at least once there
// are 256 threads on an SM, since every CTA's sums are written and read again (5000 x 256 BF16: 23 us,
// 31 with two rows each; 4000 x 2048 35 and 41).
inline int64_t join_ctas(int64_t rows, const JoinShape &shape, int row_bytes) {
    const int64_t most = kSms * join_ctas_per_sm(shape, row_bytes);
    const int64_t filled = kSms * ((255 + shape.threads) / shape.threads);
    const int64_t n = rows / 16 > filled ? rows / 16 : filled;
    return n < most ? n : most;
}

struct JoinGradArgs {
    JoinArgs j;  // branch, weights, gate, scales; post_rstd and pre_rstd are read
    MatrixArgs out, dout, dnormed, dresidual, dbranch;  // p nullptr where there is none
    void *dpost_weight, *dpre_weight, *dgate;
    int64_t dgate_ld, groups;
    float *sums;
    JoinPlan plan;
    // set by the launch: of the kernel's ring; where a cluster has the row, its CTAs, the row's columns
    // and the first run of the part of them that this is
    int32_t stages, split, all_cols, first_run;
};
cudaError_t launch_block_join_gradient(const JoinGradArgs &a, fa_dtype dt, fa_dtype st,
                                       cudaStream_t stream);
cudaError_t launch_block_join_gradient_f32(const JoinGradArgs &a, fa_dtype dt,
                                           cudaStream_t stream);

// ---- the router ------------------------------------------------------------------------
struct RoutePlan {
    int64_t ctas;
    int64_t bytes;
};
RoutePlan route_plan(int64_t tokens, int64_t experts);

struct RouteArgs {
    MatrixArgs logits;
    const uint8_t *counted;
    int32_t top_k;
    bool renormalise;
    float weight_scale, balance_coef, z_coef;
    int32_t *chosen;
    float *weights, *lse;
    int32_t *counts;
    float *mean_prob, *summary;
    void *scratch;
    RoutePlan plan;
};
cudaError_t launch_route(const RouteArgs &a, fa_dtype dt, cudaStream_t stream);

struct RouteGradArgs {
    RouteArgs r;
    const float *dweights, *grad_loss;  // or nullptr
    MatrixArgs dlogits;
};
cudaError_t launch_route_gradient(const RouteGradArgs &a, fa_dtype dt, cudaStream_t stream);

// Reads (and optionally clears) the flag that the gradient of a join sets when a bounded wait for
// a row gives up.  Waits for the device.
cudaError_t join_gradient_error(int *flag, bool clear);
cudaError_t join_gradient_f32_error(int *flag, bool clear);

cudaError_t dropout_bounds_violations(unsigned long long *count, bool clear);
cudaError_t join_bounds_violations(unsigned long long *count, bool clear);
cudaError_t join_gradient_bounds_violations(unsigned long long *count, bool clear);
cudaError_t join_gradient_f32_bounds_violations(unsigned long long *count, bool clear);
cudaError_t route_bounds_violations(unsigned long long *count, bool clear);

// Calls f with the validated types of the branch and of the stream.
template <typename F>
inline cudaError_t for_stream_dtype(fa_dtype dt, fa_dtype st, F f) {
    return for_dtype(dt, [&](auto d) {
        return st == FA_F32 ? f(d, std::integral_constant<int, FA_F32>{}) : f(d, d);
    });
}

#if defined(__CUDACC__)
// Allows a kernel kMost bytes of dynamic shared memory, once on each device: what any of its calls
// needs, since the attribute is the kernel's and other threads launch it too.
template <auto kKernel, int kMost>
inline cudaError_t allow_shared() {
    static std::atomic<bool> allowed[64] = {};  // set twice by racing threads, it is the same
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess || (dev < 64 && allowed[dev].load(std::memory_order_acquire))) return e;
    e = cudaFuncSetAttribute(kKernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kMost);
    if (e == cudaSuccess && dev < 64) allowed[dev].store(true, std::memory_order_release);
    return e;
}
#endif

// Defines a file's ``name``_bounds_violations over its counter.
#if FA_BOUNDS_CHECK
#define FA_BOUNDS_VIOLATIONS(name, counter)                                    \
    cudaError_t name(unsigned long long *count, bool clear) {                  \
        cudaError_t err = cudaMemcpyFromSymbol(count, counter, sizeof(*count)); \
        if (err != cudaSuccess || !clear) return err;                          \
        const unsigned long long zero = 0;                                     \
        return cudaMemcpyToSymbol(counter, &zero, sizeof(zero));               \
    }
#else
#define FA_BOUNDS_VIOLATIONS(name, counter)                 \
    cudaError_t name(unsigned long long *count, bool) {     \
        *count = 0;                                         \
        return cudaSuccess;                                 \
    }
#endif

}  // namespace fa
