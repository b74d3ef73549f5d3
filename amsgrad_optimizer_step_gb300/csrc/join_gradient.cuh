// The gradient of a join: the kernels, as the files of the two kinds of stream include them
// (the branch's type, or FP32).
//
// A CTA takes rows that lie a grid apart (one after another under a gate of several groups) and keeps
// the columns' sums in registers.
// Per row it needs three sums over the columns, in one reduction: with d = dnormed * w_pre,
// t = dout + rstd_pre * d, a = branch_scale * gate * w_post and v = yh where it is kept,
//   s1 = sum d xh,  s2 = sum a v t,  s3 = sum a v xh
// the first norm's mean, which needs the second's gradient G = t - rstd_pre * mean(s1) * xh, is
// s2 - rstd_pre * mean(s1) * s3.  The gradients of the first weight and of the gate are both
// multiples, column by column, of K = sum over rows of v G: one sum serves both.
//
// 16384 x 2048 BF16, everything on, takes 74 us of which the bytes need 59 (66 without dropout): a
// row's reduction, whose wait the other CTAs of an SM hide, and issue slots bound it.  Copies of 16
// bytes by every thread took 89; two CTAs an SM instead of three, two runs a thread, or the next
// row's first half before a row's second where only one CTA fits (8192 x 4096: 89 against 78): no
// faster.  The CTAs' sums are joined in 6 to 11 us.
#pragma once

#include <cooperative_groups.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "internal.h"

FA_BOUNDS_COUNTER(g_join_gradient_oob)

#include "bulk_rows.cuh"
#include "join_device.cuh"

namespace fa {
namespace {

namespace cg = cooperative_groups;

// One row's four matrices as a thread holds them.
template <int DT, int ST, int R>
struct GradRow {
    Raw<ST, kRun> dout[R], x[R];
    Raw<DT, kRun> dn[R], y[R];
};

__device__ int g_join_gradient_error;  // a wait for a row ran out

// The rows on their way: a ring of up to four rows, the four matrices' one behind another, each as
// long as the threads' runs reach.  What nothing is copied to (columns past the end, matrices that
// are not there) stays 0, so that a thread reads its runs without asking.  The row's reduction is
// between the last read of a slot and the copies of a later row into it.
template <int DT, int ST, int R>
struct Ring {
    static constexpr int kMost = 4;
    static constexpr int kS = Raw<ST, kRun>::kWords, kD = Raw<DT, kRun>::kWords;  // of 16 bytes
    static constexpr int kVectors = 2 * R * (kS + kD);  // of a row, per thread

    static int bytes(int threads) { return 16 * kVectors * threads; }  // of a row
    // Rows that the ring has room for (below two there is none).
    static int stages(int threads, int ctas, int weights) {
        const int n = (kSmShared / ctas - 2048 - weights) / bytes(threads);
        return n < kMost ? n : kMost;
    }
    // Bytes to copy of a row whose first run begins ``shift`` columns before it: its 16-byte lines, of
    // the last row without one that ends behind the matrix.
    static __device__ __forceinline__ uint32_t lines(const JoinGradArgs &a, int64_t row, int shift,
                                                     int size) {
        const int bytes = (static_cast<int>(a.j.cols) + shift) * size;
        return (row + 1 < a.j.rows ? bytes + 15 : bytes) & ~15;
    }
    // By one thread: asks for a row.
    static __device__ __forceinline__ void issue(const JoinGradArgs &a, int64_t row, int shift,
                                                 uint4 *slot, uint64_t *bar) {
        if (!fa_in_bounds(row, 1, a.j.rows)) return;
        const int reach = R * blockDim.x;
        const uint32_t s = lines(a, row, shift, 2 * kS), d = lines(a, row, shift, 2 * kD);
        // (the lines lie in the matrix, in front of and behind the row too, and in the matrix's slots)
        const auto inside = [&](const MatrixArgs &m, int size, uint32_t bytes) {
            return m.p && fa_in_bounds(row * m.ld - shift, bytes / size, (m.rows - 1) * m.ld + m.cols) &&
                   fa_in_bounds(0, bytes, 8 * size * reach);
        };
        const bool dout = inside(a.dout, 2 * kS, s), out = inside(a.out, 2 * kS, s);
        const bool dnormed = inside(a.dnormed, 2 * kD, d), branch = inside(a.j.branch, 2 * kD, d);
        row_expect(bar, (dout ? s : 0) + (out ? s : 0) + (dnormed ? d : 0) + (branch ? d : 0));
        const auto copy = [&](bool it, const MatrixArgs &m, int size, uint32_t bytes, int at) {
            if (it)
                row_copy(slot + at * reach, static_cast<const char *>(m.p) + (row * m.ld - shift) * size,
                         bytes, bar);
        };
        copy(dout, a.dout, 2 * kS, s, 0);
        copy(out, a.out, 2 * kS, s, kS);
        copy(dnormed, a.dnormed, 2 * kD, d, 2 * kS);
        copy(branch, a.j.branch, 2 * kD, d, 2 * kS + kD);
    }
    // By the thread of the last row's last run: what ``lines`` left out.
    static __device__ void complete(const JoinGradArgs &a, int64_t row, int shift, uint4 *slot) {
        const int cols = static_cast<int>(a.j.cols), reach = R * blockDim.x;
        const auto copy = [&](const MatrixArgs &m, auto type, int at) {
            using T = typename Elem<decltype(type)::value>::T;
            T *const to = reinterpret_cast<T *>(slot + at * reach) + shift;
            const T *const from = static_cast<const T *>(m.p) + row * m.ld;
            const int there = static_cast<int>(lines(a, row, shift, sizeof(T)) / sizeof(T)) - shift;
            for (int c = there; m.p && c < cols; ++c)
                if (fa_in_bounds(c, 1, cols) && fa_in_bounds(shift + c, 1, kRun * reach)) to[c] = from[c];
        };
        copy(a.dout, std::integral_constant<int, ST>{}, 0);
        copy(a.out, std::integral_constant<int, ST>{}, kS);
        copy(a.dnormed, std::integral_constant<int, DT>{}, 2 * kS);
        copy(a.j.branch, std::integral_constant<int, DT>{}, 2 * kS + kD);
    }
    template <int W, typename T>
    static __device__ __forceinline__ void take(const uint4 *at, T &x) {
#pragma unroll
        for (int k = 0; k < W; ++k) x.r[k] = at[k];
    }
    static __device__ __forceinline__ void read(const uint4 *slot, GradRow<DT, ST, R> &g) {
        const int reach = R * blockDim.x;
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const int q = r * blockDim.x + threadIdx.x;
            take<kS>(slot + q * kS, g.dout[r]);
            take<kS>(slot + kS * reach + q * kS, g.x[r]);
            take<kD>(slot + 2 * kS * reach + q * kD, g.dn[r]);
            take<kD>(slot + (2 * kS + kD) * reach + q * kD, g.y[r]);
        }
    }
};

// Three sums over a warp, halving what a lane carries at each of the first steps: six shuffles
// instead of fifteen.  The sums end in lanes 0 to 7, 8 to 15 and 16 to 23.
__device__ __forceinline__ float warp_sum3(float s1, float s2, float s3) {
    const bool h16 = threadIdx.x & 16, h8 = threadIdx.x & 8;
    float a = h16 ? s3 : s1, b = h16 ? 0.f : s2;
    a += __shfl_xor_sync(0xffffffffu, h16 ? s1 : s3, 16);
    b += __shfl_xor_sync(0xffffffffu, h16 ? s2 : 0.f, 16);
    float c = h8 ? b : a;
    c += __shfl_xor_sync(0xffffffffu, h8 ? a : b, 8);
#pragma unroll
    for (int o = 4; o > 0; o >>= 1) c += __shfl_xor_sync(0xffffffffu, c, o);
    return c;
}

// The same over a row's threads, in every one.  ``part``: 24 floats for each sum and for nothing
// (those of no warp 0), not in use by the call before.  True where one of the threads says
// ``failed``.
constexpr int kPartWarps = kJoinThreads / 32;
__device__ __forceinline__ bool row_sum3(float &s1, float &s2, float &s3, float *part,
                                         bool failed) {
    float c = warp_sum3(s1, s2, s3);
    const int lane = threadIdx.x % 32, warps = blockDim.x / 32;
    if (warps > 1) {
        if (lane % 8 == 0) part[lane / 8 * kPartWarps + threadIdx.x / 32] = c;
        failed = __syncthreads_or(failed);
        // eight lanes take a sum's warps, eight at a time
        const float *const mine = part + lane / 8 * kPartWarps + lane % 8;
        c = mine[0];
        for (int w = 8; w < warps; w += 8) c += mine[w];
#pragma unroll
        for (int o = 4; o > 0; o >>= 1) c += __shfl_xor_sync(0xffffffffu, c, o);
    } else {
        failed = __any_sync(0xffffffffu, failed);
    }
    s1 = __shfl_sync(0xffffffffu, c, 0);
    s2 = __shfl_sync(0xffffffffu, c, 8);
    s3 = __shfl_sync(0xffffffffu, c, 16);
    return failed;
}

// The same over a row that a cluster of ``ctas`` holds: every warp writes its part into all of them.
constexpr int kMostSplit = 4;
constexpr int kSplitPlaces = 2 * kMostSplit * 4 * kPartWarps * static_cast<int>(sizeof(float));
__device__ __forceinline__ bool cluster_sum3(float &s1, float &s2, float &s3,
                                             float (*part)[4 * kPartWarps], int ctas, bool failed) {
    cg::cluster_group cluster = cg::this_cluster();
    float c = warp_sum3(s1, s2, s3);
    const int lane = threadIdx.x % 32, warps = blockDim.x / 32;
    failed = __any_sync(0xffffffffu, failed);
    if (lane / 8 == 3) c = failed ? 1.f : 0.f;  // in place of the sum of nothing
    if (lane % 8 == 0) {
        float *const mine = part[cluster.block_rank()] + lane / 8 * kPartWarps + threadIdx.x / 32;
        for (int r = 0; r < ctas; ++r) *cluster.map_shared_rank(mine, r) = c;
    }
    cluster.sync();
    c = 0.f;
    for (int r = 0; r < ctas; ++r)
        for (int w = lane % 8; w < warps; w += 8) c += part[r][lane / 8 * kPartWarps + w];
#pragma unroll
    for (int o = 4; o > 0; o >>= 1) c += __shfl_xor_sync(0xffffffffu, c, o);
    s1 = __shfl_sync(0xffffffffu, c, 0);
    s2 = __shfl_sync(0xffffffffu, c, 8);
    s3 = __shfl_sync(0xffffffffu, c, 16);
    return __shfl_sync(0xffffffffu, c, 24) != 0.f;
}

__device__ __forceinline__ float sum_of_pair(uint64_t p) {
    float lo, hi;
    unpair(p, lo, hi);
    return lo + hi;
}

template <int DT>
__device__ __forceinline__ void store_weight(void *p, bool wide, int64_t at, float x) {
    if (wide)
        static_cast<float *>(p)[at] = x;
    else
        static_cast<typename Elem<DT>::T *>(p)[at] = Elem<DT>::round(x);
}

// Parts of a CTA's sums, by row of its scratch.
enum { kPost = 0, kPre = 1, kHead = 2, kTail = 3 };

// RING: rows of whole, aligned runs that go through the ring; else each row is read when its turn
// comes, from any address.  ALL: both norms, the branch and every matrix's gradient are there
// (what a training step asks for, without a question a row).  DROP: false where nothing is dropped.
// SHIFT: rows of the ring that begin anywhere.  The 16-byte lines of matrices of one row distance begin at
// the same columns, and at the same ones again eight rows on.  A CTA's rows are a multiple of eight
// apart, so its run q is columns [8 q - shift, 8 q - shift + 8) in all of them: whole lines but
// for the row's two ends, and the columns' sums stay where they are.  SPLIT: ``a`` has the columns of
// one CTA, and a cluster has the row.
template <int DT, int ST, int R, bool RING, bool ALL, bool DROP, bool SHIFT, bool SPLIT>
__device__ __forceinline__ void join_gradient_rows(const JoinGradArgs &a) {
    static_assert(!SHIFT || (RING && R == 1), "a run a thread");
    extern __shared__ uint4 ring[];
    constexpr int kParts = SPLIT ? kMostSplit : 1;  // of the row's sums
    __shared__ __align__(16) float part[2][kParts][4 * kPartWarps];
    using Rows = Ring<DT, ST, R>;
    __shared__ uint64_t bars[Rows::kMost];
    // the CTA's rows: first, first + stride, ...
    const bool own_gate = a.j.gate && a.j.group_rows < a.j.rows;
    const int64_t cta = SPLIT ? blockIdx.x / a.split : blockIdx.x;  // or the cluster
    const int64_t stride = own_gate ? 1 : a.plan.ctas;
    const int64_t first = own_gate ? cta * a.plan.chunk : cta;
    const int64_t end = own_gate && first + a.plan.chunk < a.j.rows ? first + a.plan.chunk : a.j.rows;
    const int count = static_cast<int>((end - first + stride - 1) / stride);
    const bool pre = ALL || a.dnormed.p, branch = ALL || a.j.branch.p;
    const bool post = ALL || (a.j.post_norm && branch), dropped = DROP && (ALL || a.j.dropped);
    const int cols = static_cast<int>(a.j.cols), all_cols = SPLIT ? a.all_cols : cols;
    const int row_blocks = (all_cols + kRun - 1) / kRun, first_run = SPLIT ? a.first_run : 0;
    const int shift = SHIFT ? static_cast<int>(first) * a.j.ld8 % kRun : 0;
    const int runs = (cols + shift + kRun - 1) / kRun;
    const auto column = [&](int r) {  // the first of run r
        return static_cast<int>(r * blockDim.x + threadIdx.x) * kRun - shift;
    };
    const bool whole = !SHIFT || (column(0) >= 0 && column(0) + kRun <= cols);  // R == 1
    const float inv_cols = 1.f / static_cast<float>(all_cols);
    const int lane = threadIdx.x % 32;
    for (int i = threadIdx.x; i < 2 * kParts * 4 * kPartWarps; i += blockDim.x) part[0][0][i] = 0.f;
    const int row_vectors = RING ? Rows::kVectors * blockDim.x : 0;
    if (RING) {
        if (SHIFT || runs < R * static_cast<int>(blockDim.x) || !a.dout.p || !pre || !branch) {
            for (int i = threadIdx.x; i < a.stages * row_vectors; i += blockDim.x)
                ring[i] = make_uint4(0u, 0u, 0u, 0u);
            shared_writes_before_copies();
            __syncthreads();
        }
        if (threadIdx.x == 0) {
            for (int i = 0; i < a.stages; ++i) row_barrier_init(bars + i);
            row_barriers_ready();
            for (int i = 0; i < a.stages && i < count; ++i)
                Rows::issue(a, first + i * stride, shift, ring + i * row_vectors, bars + i);
        }
    }
    if constexpr (SPLIT)
        cg::this_cluster().sync();
    else
        __syncthreads();
    const float scale = dropped ? a.j.branch_scale * a.j.drop.scale : a.j.branch_scale;
    const uint64_t call = dropped ? drop_call(a.j.drop) : 0;
    // the thread's weights, in slots of its own: w_pre, then scale * gate * w_post, of each run
    float4 *const kept_weights =
        reinterpret_cast<float4 *>(ring + a.stages * row_vectors) + threadIdx.x;
    const auto keep = [&](int which, int r, const float *w) {
        float4 *const at = kept_weights + (4 * r + 2 * which) * blockDim.x;
        at[0] = make_float4(w[0], w[1], w[2], w[3]);
        at[blockDim.x] = make_float4(w[4], w[5], w[6], w[7]);
    };
    const auto fetch = [&](int which, int r, uint64_t *w) {
        const float4 *const at = kept_weights + (4 * r + 2 * which) * blockDim.x;
        const float4 lo = at[0], hi = at[blockDim.x];
        w[0] = pair(lo.x, lo.y);
        w[1] = pair(lo.z, lo.w);
        w[2] = pair(hi.x, hi.y);
        w[3] = pair(hi.z, hi.w);
    };
    uint64_t sum_k[R][kPairs] = {}, sum_p[R][kPairs] = {};
    // the weights of run r: what: a weight or the gate's row, ``offset`` added
    const auto weights = [&](const void *p, int64_t row0, int r, float offset, float *w) {
        const int c = column(r);
        if constexpr (SHIFT)
            load_columns<DT>(a.j, p, row0, c, cols, offset, w);
        else
            load_weights<DT>(a.j, p, row0 + c, valid_cols(c, cols), offset, w);
    };
#pragma unroll
    for (int r = 0; r < R; ++r) {
        float w[kRun];
        weights(pre ? a.j.pre_weight : nullptr, 0, r, a.j.weight_offset, w);
        keep(0, r, w);
    }
    float *const sums = a.sums + cta * a.plan.parts * a.plan.pitch;
    const auto in_sums = [&](int which, int c) {  // of the CTA's sums, in what they have room for
        const int64_t at = (cta * a.plan.parts + which) * a.plan.pitch + first_run * kRun + c;
        return is_column(c, cols) && fa_in_bounds(at, 1, a.plan.bytes / 4);
    };
    // the gate's group of the row, and the turns that its rows begin and end with
    int64_t group = own_gate ? a.j.by_group.quotient(static_cast<uint32_t>(first)) : 0;
    int64_t group_begin = own_gate ? group * a.j.group_rows - first : 0;
    int64_t group_end = own_gate ? group_begin + a.j.group_rows : count + 1;
    bool flushed = false;

    const auto new_group = [&] {
#pragma unroll
        for (int r = 0; r < R; ++r) {
            float w[kRun], g[kRun];
            weights(post ? a.j.post_weight : nullptr, 0, r, a.j.weight_offset, w);
            weights(a.j.gate, group * a.j.gate_ld, r, 0.f, g);
#pragma unroll
            for (int j = 0; j < kRun; ++j) w[j] *= scale * g[j];
            keep(1, r, w);
        }
    };
    // The group's sums: whole where all its rows are this CTA's, else a part of them.
    const auto flush = [&] {
        if (!own_gate) {  // K itself: what it is times is the same for all CTAs
#pragma unroll
            for (int r = 0; r < R; ++r) {
                const int c = column(r);
                float k[kRun];
                from_pairs(sum_k[r], k);
                float *const at = sums + kPost * a.plan.pitch + c;
#pragma unroll
                for (int j = 0; j < kRun; ++j)
                    if (in_sums(kPost, c + j)) at[j] = scale * k[j];
            }
            return;
        }
        const bool begun_here = group_begin >= 0, whole = begun_here && group_end <= count;
        float *const gate_part = sums + (begun_here ? kTail : kHead) * a.plan.pitch;
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const int c = column(r);
            float w[kRun], k[kRun];
            from_pairs(sum_k[r], k);
            if (a.dpost_weight) {
                weights(a.j.gate, group * a.j.gate_ld, r, 0.f, w);
                float *const at = sums + kPost * a.plan.pitch + c;
#pragma unroll
                for (int j = 0; j < kRun; ++j)
                    if (in_sums(kPost, c + j)) {
                        const float x = scale * w[j] * k[j];
                        at[j] = flushed ? at[j] + x : x;
                    }
            }
            if (a.dgate) {
                weights(post ? a.j.post_weight : nullptr, 0, r, a.j.weight_offset, w);
#pragma unroll
                for (int j = 0; j < kRun; ++j)
                    if (is_column(c + j, cols)) {
                        const float x = scale * w[j] * k[j];
                        if (whole)
                            store_weight<DT>(a.dgate, a.j.wide_weights,
                                             group * a.dgate_ld + c + j, x);
                        else if (in_sums(begun_here ? kTail : kHead, c + j))
                            gate_part[c + j] = x;
                    }
            }
#pragma unroll
            for (int j = 0; j < kPairs; ++j) sum_k[r][j] = 0;
        }
        flushed = true;
    };

    if (branch) new_group();
    float rp_lane = 0.f, rq_lane = 1.f;
    int stage = 0;
    uint32_t parity = 0;
    bool failed = false;
    fa_allow_dependents();
    int64_t row = first;
    using S = typename Elem<ST>::T;
    using D = typename Elem<DT>::T;
    S *to_residual = static_cast<S *>(a.dresidual.p) + first * a.dresidual.ld + column(0);
    D *to_branch = static_cast<D *>(a.dbranch.p) + first * a.dbranch.ld + column(0);
    const int64_t residual_step = stride * a.dresidual.ld, branch_step = stride * a.dbranch.ld;
    for (int n = 0; n < count;
         ++n, row += stride, to_residual += residual_step, to_branch += branch_step) {
        if (n % 32 == 0) {  // the inverse roots of 32 rows, a lane each
            const int64_t at = row + lane * stride;
            if (pre) rp_lane = at < end ? a.j.pre_rstd[at] : 0.f;
            if (post) rq_lane = at < end ? a.j.post_rstd[at] : 0.f;
        }
        const float rp = __shfl_sync(0xffffffffu, rp_lane, n % 32);
        const float rq = __shfl_sync(0xffffffffu, rq_lane, n % 32);
        if (n == group_end) {
            if (branch) flush();
            ++group;
            group_begin = group_end;
            group_end += a.j.group_rows;
            if (branch) new_group();
        }
        GradRow<DT, ST, R> g;
        if (RING) {
            failed = !row_wait(bars + stage, parity);
            if (SHIFT && row == a.j.rows - 1 && static_cast<int>(threadIdx.x) == runs - 1)
                Rows::complete(a, row, shift, ring + stage * row_vectors);
            Rows::read(ring + stage * row_vectors, g);
            if (SHIFT && !whole) {  // a neighbour's elements
                keep_columns<ST>(g.dout[0], column(0), cols);
                keep_columns<ST>(g.x[0], column(0), cols);
                keep_columns<DT>(g.dn[0], column(0), cols);
                keep_columns<DT>(g.y[0], column(0), cols);
            }
        } else {
#pragma unroll
            for (int r = 0; r < R; ++r) {
                const int c = (r * blockDim.x + threadIdx.x) * kRun;
                zero(g.dout[r]);
                zero(g.x[r]);
                zero(g.dn[r]);
                zero(g.y[r]);
                if (a.dout.p) g.dout[r] = load_run<ST, false>(a.dout, row, c);
                if (a.out.p) g.x[r] = load_run<ST, false>(a.out, row, c);
                if (pre) g.dn[r] = load_run<DT, false>(a.dnormed, row, c);
                if (branch) g.y[r] = load_run<DT, false>(a.j.branch, row, c);
            }
        }
        // ym: the kept yh; am: the weights of the kept ones
        uint64_t t[R][kPairs], ym[R][kPairs], am[R][kPairs];
        uint64_t s1 = 0, s2 = 0, s3 = 0;
#pragma unroll
        for (int r = 0; r < R; ++r) {
            uint64_t x[kPairs];
            widen_pairs<ST>(g.dout[r], t[r]);
            widen_pairs<ST>(g.x[r], x);
#pragma unroll
            for (int j = 0; j < kPairs; ++j) x[j] = mul2(x[j], both(rp));
            if (pre) {
                uint64_t d[kPairs], wp[kPairs];
                widen_pairs<DT>(g.dn[r], d);
                fetch(0, r, wp);
#pragma unroll
                for (int j = 0; j < kPairs; ++j) {
                    sum_p[r][j] = fma2(d[j], x[j], sum_p[r][j]);
                    d[j] = mul2(d[j], wp[j]);
                    t[r][j] = fma2(d[j], both(rp), t[r][j]);
                    s1 = fma2(d[j], x[j], s1);
                }
            }
            widen_pairs<DT>(g.y[r], ym[r]);
            fetch(1, r, am[r]);
#pragma unroll
            for (int j = 0; j < kPairs; ++j) ym[r][j] = mul2(ym[r][j], both(rq));
            if (dropped) {
                Kept kept;
                const uint64_t block =
                    static_cast<uint64_t>(row) * row_blocks + first_run + (r * blockDim.x + threadIdx.x);
                kept.draw(a.j.drop, block, call);
                if (SHIFT && shift) kept.begin_before(a.j.drop, block, call, shift);
                kept.mask(ym[r], a.j.drop.threshold);
                kept.mask(am[r], a.j.drop.threshold);
            }
            if (post) {
#pragma unroll
                for (int j = 0; j < kPairs; ++j) {
                    const uint64_t q = mul2(ym[r][j], am[r][j]);
                    s2 = fma2(q, t[r][j], s2);
                    s3 = fma2(q, x[j], s3);
                }
            }
        }
        float back = 0.f, mean = 0.f;  // times xh: taken off t; times yh: taken off dbranch
        float f1 = sum_of_pair(s1), f2 = sum_of_pair(s2), f3 = sum_of_pair(s3);
        // (the other part is still being read)
        if constexpr (SPLIT)
            failed = cluster_sum3(f1, f2, f3, part[n % 2], a.split, failed);
        else
            failed = row_sum3(f1, f2, f3, part[n % 2][0], failed);
        if (RING) {
            if (failed) break;
            // every thread has read its part of the slot
            if (threadIdx.x == 0 && n + a.stages < count)
                Rows::issue(a, row + a.stages * stride, shift, ring + stage * row_vectors,
                            bars + stage);
            if (++stage == a.stages) {
                stage = 0;
                parity ^= 1;
            }
        }
        if (pre || post) {
            back = rp * (f1 * inv_cols);
            mean = (f2 - back * f3) * inv_cols * rq;
        }
#pragma unroll
        for (int r = 0; r < R; ++r) {
            uint64_t x[kPairs], y[kPairs], dr[kPairs], db[kPairs];
            widen_pairs<ST>(g.x[r], x);
            widen_pairs<DT>(g.y[r], y);
#pragma unroll
            for (int j = 0; j < kPairs; ++j) {
                const uint64_t total =
                    pre ? fma2(mul2(x[j], both(rp)), both(-back), t[r][j]) : t[r][j];
                dr[j] = mul2(total, both(a.j.residual_scale));
                sum_k[r][j] = fma2(ym[r][j], total, sum_k[r][j]);
                db[j] = mul2(total, am[r][j]);
                if (post)
                    db[j] = fma2(mul2(y[j], both(rq)), both(-mean), mul2(db[j], both(rq)));
            }
            const int q = r * blockDim.x + threadIdx.x;
            const bool there = fa_in_bounds(row, 1, a.j.rows);
            float v[kRun];
            if (ALL || a.dresidual.p) {
                from_pairs(dr, v);
                if (!RING)
                    store_run<ST, false>(a.dresidual, row, q * kRun, v, 0xffffffffu, 32);
                else if (SHIFT && !whole)
                    store_columns<ST>(to_residual, v, column(0), there ? cols : 0);
                else if (q < runs && there && fa_in_bounds(column(r), kRun, cols))
                    store_n<ST, kRun>(to_residual + r * blockDim.x * kRun, v);
            }
            if (ALL || a.dbranch.p) {
                from_pairs(db, v);
                if (!RING)
                    store_run<DT, false>(a.dbranch, row, q * kRun, v, 0xffffffffu, 32);
                else if (SHIFT && !whole)
                    store_columns<DT>(to_branch, v, column(0), there ? cols : 0);
                else if (q < runs && there && fa_in_bounds(column(r), kRun, cols))
                    store_n<DT, kRun>(to_branch + r * blockDim.x * kRun, v);
            }
        }
    }
    if (RING && failed) {  // the same in every thread
        if (threadIdx.x == 0) {
            atomicExch(&g_join_gradient_error, 1);
            // the copies that are still on their way to this CTA's memory
            for (int i = 0; i < a.stages; ++i) row_wait(bars + i, i < stage ? parity ^ 1 : parity);
        }
        return;
    }
    if (branch && (a.dpost_weight || a.dgate)) flush();
    if (a.dpre_weight) {
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const int c = column(r);
            float v[kRun];
            from_pairs(sum_p[r], v);
#pragma unroll
            for (int j = 0; j < kRun; ++j)
                if (in_sums(kPre, c + j)) sums[kPre * a.plan.pitch + c + j] = v[j];
        }
    }
}

template <int DT, int ST, int R, bool RING, bool ALL, bool DROP, bool SHIFT>
__global__ void __launch_bounds__(R == 1 ? kJoinThreads : kMaxThreads)
join_gradient_kernel(const __grid_constant__ JoinGradArgs a) {
    join_gradient_rows<DT, ST, R, RING, ALL, DROP, SHIFT, false>(a);
}

// Rows wider than a CTA holds: a cluster's CTAs have a part of the columns each, and what a row's sums
// are is exchanged.  2048 x 16384 BF16 by fours: 159 us, 2730 x 12288 by twos 121; in one CTA that reads
// the row twice 451 and more.
struct SplitArgs {
    JoinGradArgs of[kMostSplit];
};
template <int DT, int ST>
__global__ void __launch_bounds__(kJoinThreads)
join_gradient_split_kernel(const __grid_constant__ SplitArgs a) {
    join_gradient_rows<DT, ST, 1, true, false, true, false, true>(
        a.of[cg::this_cluster().block_rank()]);
}

// Rows of more than two runs a thread, at any addresses: their columns' sums lie in shared memory, and a
// row is read again from L2 once its three sums are there.
template <int DT, int ST>
__global__ void __launch_bounds__(kMaxThreads) join_gradient_wide_kernel(JoinGradArgs a) {
    extern __shared__ float wide_sums[];
    __shared__ float part[2][3][kMaxThreads / 32];
    float *const sum_k = wide_sums, *const sum_p = wide_sums + a.plan.pitch;
    const int64_t first = blockIdx.x * a.plan.chunk;
    const int64_t last = first + a.plan.chunk < a.j.rows ? first + a.plan.chunk : a.j.rows;
    const bool pre = a.dnormed.p, branch = a.j.branch.p, post = a.j.post_norm && branch;
    const int64_t blocks = (a.j.cols + kRun - 1) / kRun;
    const float inv_cols = 1.f / static_cast<float>(a.j.cols);
    const float scale = a.j.dropped ? a.j.branch_scale * a.j.drop.scale : a.j.branch_scale;
    const uint64_t call = a.j.dropped ? drop_call(a.j.drop) : 0;
    // lanes of one warp hold consecutive runs, and all of them take every turn
    const int64_t turns = (blocks + blockDim.x - 1) / blockDim.x;
    float *const sums = a.sums + blockIdx.x * a.plan.parts * a.plan.pitch;
    const auto in_sums = [&](int which, int64_t c) {
        return fa_in_bounds((blockIdx.x * a.plan.parts + which) * a.plan.pitch + c, 1, a.plan.bytes / 4);
    };
    const bool own_gate = a.j.gate && a.j.group_rows < a.j.rows;
    int64_t group = own_gate ? a.j.by_group.quotient(static_cast<uint32_t>(first)) : 0;
    int64_t group_first = own_gate ? group * a.j.group_rows : first;
    int64_t group_last = own_gate ? group_first + a.j.group_rows : last;
    bool flushed = false;
    fa_allow_dependents();

    // what a run of the row is and what follows from it; aw = scale * gate * w_post
    struct Run {
        float t[kRun], dn[kRun], xh[kRun], yh[kRun], wp[kRun], aw[kRun];
        Kept kept;
    };
    const auto read = [&](int64_t row, int64_t c, float rp, float rq, Run &u) {
        const int valid = valid_cols(c, a.j.cols);
        Raw<ST, kRun> s;
        Raw<DT, kRun> d;
        if (a.dout.p) s = load_run<ST, false>(a.dout, row, c);
        else zero(s);
        s.widen(u.t);
        if (a.out.p) s = load_run<ST, false>(a.out, row, c);
        else zero(s);
        s.widen(u.xh);
        if (pre) d = load_run<DT, false>(a.dnormed, row, c);
        else zero(d);
        d.widen(u.dn);
        if (branch) d = load_run<DT, false>(a.j.branch, row, c);
        else zero(d);
        d.widen(u.yh);
        float w[kRun];
        load_weights<DT>(a.j, pre ? a.j.pre_weight : nullptr, c, valid,
                                a.j.weight_offset, u.wp);
        load_weights<DT>(a.j, post ? a.j.post_weight : nullptr, c, valid,
                                a.j.weight_offset, u.aw);
        load_weights<DT>(a.j, a.j.gate, group * a.j.gate_ld + c, valid, 0.f, w);
        if (a.j.dropped)
            u.kept.draw(a.j.drop, row * blocks + c / kRun, call);
        else
            u.kept.all();
#pragma unroll
        for (int j = 0; j < kRun; ++j) {
            u.xh[j] *= rp;
            u.yh[j] *= rq;
            u.aw[j] *= scale * w[j];
            u.t[j] = fmaf(rp, u.dn[j] * u.wp[j], u.t[j]);
        }
    };
    const auto flush = [&] {
        if (!own_gate) {  // K itself
            for (int64_t q = threadIdx.x; q < blocks; q += blockDim.x)
                for (int j = 0; j < valid_cols(q * kRun, a.j.cols); ++j)
                    if (in_sums(kPost, q * kRun + j))
                        sums[kPost * a.plan.pitch + q * kRun + j] = scale * sum_k[q * kRun + j];
            return;
        }
        const bool begun_here = group_first >= first, whole = begun_here && group_last <= last;
        float *const gate_part = sums + (begun_here ? kTail : kHead) * a.plan.pitch;
        for (int64_t q = threadIdx.x; q < blocks; q += blockDim.x) {
            const int64_t c = q * kRun;
            const int valid = valid_cols(c, a.j.cols);
            float g[kRun], w[kRun];
            load_weights<DT>(a.j, a.j.gate, group * a.j.gate_ld + c, valid,
                                    0.f, g);
            load_weights<DT>(a.j, post ? a.j.post_weight : nullptr, c, valid,
                                    a.j.weight_offset, w);
            for (int j = 0; j < valid; ++j) {
                const float k = scale * sum_k[c + j];
                sum_k[c + j] = 0.f;
                float *at = sums + kPost * a.plan.pitch + c + j;
                if (a.dpost_weight && in_sums(kPost, c + j)) *at = flushed ? *at + g[j] * k : g[j] * k;
                if (a.dgate && whole)
                    store_weight<DT>(a.dgate, a.j.wide_weights, group * a.dgate_ld + c + j,
                                     w[j] * k);
                else if (a.dgate && in_sums(begun_here ? kTail : kHead, c + j))
                    gate_part[c + j] = w[j] * k;
            }
        }
        flushed = true;
    };
    // every thread reads and writes the sums of its own runs only
    for (int64_t q = threadIdx.x; q < blocks; q += blockDim.x)
#pragma unroll
        for (int j = 0; j < kRun; ++j) sum_k[q * kRun + j] = sum_p[q * kRun + j] = 0.f;
    for (int64_t row = first; row < last; ++row) {
        if (row == group_last) {
            if (branch) flush();
            ++group;
            group_first = group_last;
            group_last += a.j.group_rows;
        }
        const float rp = pre ? a.j.pre_rstd[row] : 0.f, rq = post ? a.j.post_rstd[row] : 1.f;
        float s1 = 0.f, s2 = 0.f, s3 = 0.f;
        Run u;
        for (int64_t turn = 0; turn < turns && (pre || post); ++turn) {
            read(row, (turn * blockDim.x + threadIdx.x) * kRun, rp, rq, u);
#pragma unroll
            for (int j = 0; j < kRun; ++j) {
                s1 = fmaf(u.dn[j] * u.wp[j], u.xh[j], s1);
                const float q = u.kept(j, a.j.drop.threshold) ? u.yh[j] * u.aw[j] : 0.f;
                s2 = fmaf(q, u.t[j], s2);
                s3 = fmaf(q, u.xh[j], s3);
            }
        }
        s1 = warp_sum(s1);
        s2 = warp_sum(s2);
        s3 = warp_sum(s3);
        float(*p)[kMaxThreads / 32] = part[(row - first) % 2];
        if (threadIdx.x % 32 == 0) {
            p[0][threadIdx.x / 32] = s1;
            p[1][threadIdx.x / 32] = s2;
            p[2][threadIdx.x / 32] = s3;
        }
        __syncthreads();
        s1 = s2 = s3 = 0.f;
        for (unsigned w = 0; w < blockDim.x / 32; ++w) {
            s1 += p[0][w];
            s2 += p[1][w];
            s3 += p[2][w];
        }
        const float back = rp * (s1 * inv_cols), mean = (s2 - back * s3) * inv_cols * rq;
        for (int64_t turn = 0; turn < turns; ++turn) {
            const int64_t c = (turn * blockDim.x + threadIdx.x) * kRun;
            const int valid = valid_cols(c, a.j.cols);
            read(row, c, rp, rq, u);
            float dr[kRun], db[kRun];
#pragma unroll
            for (int j = 0; j < kRun; ++j) {
                const float total = pre ? fmaf(-back, u.xh[j], u.t[j]) : u.t[j];
                const bool on = u.kept(j, a.j.drop.threshold);
                dr[j] = a.j.residual_scale * total;
                db[j] = on ? total * u.aw[j] : 0.f;
                if (post) db[j] = fmaf(db[j], rq, -u.yh[j] * mean);
                if (j < valid) {
                    sum_p[c + j] = fmaf(u.dn[j], u.xh[j], sum_p[c + j]);
                    if (on) sum_k[c + j] = fmaf(u.yh[j], total, sum_k[c + j]);
                }
            }
            if (a.dresidual.p) store_run<ST, false>(a.dresidual, row, c, dr, 0xffffffffu, 32);
            if (a.dbranch.p) store_run<DT, false>(a.dbranch, row, c, db, 0xffffffffu, 32);
        }
    }
    if (branch && (a.dpost_weight || a.dgate)) flush();
    if (a.dpre_weight)
        for (int64_t q = threadIdx.x; q < blocks; q += blockDim.x)
            for (int j = 0; j < valid_cols(q * kRun, a.j.cols); ++j)
                if (in_sums(kPre, q * kRun + j))
                    sums[kPre * a.plan.pitch + q * kRun + j] = sum_p[q * kRun + j];
}

// Joins the CTAs' sums in order: K for the first weight and a gate that all rows share, the second
// weight's, then the gate's groups, or (where there are more groups than CTAs) the border before each
// CTA, whose group it joins if it is the group's first border.  A block takes 32 columns and 16 runs
// of CTAs side by side, or 128 and four of a group, whose rows few CTAs share.
constexpr int kSumThreads = 512;
template <int DT>
__global__ void __launch_bounds__(kSumThreads) join_sums_kernel(JoinGradArgs a) {
    __shared__ float part[kSumThreads];
    fa_grid_dependency_wait();
    const JoinPlan &p = a.plan;
    const int cols = static_cast<int>(a.j.cols), blocks = (cols + 31) / 32;
    const int wide_blocks = (cols + 127) / 128;
    const int b = blockIdx.x;
    const int what = b < blocks ? kPost : b < 2 * blocks ? kPre : kHead;
    const int width = what == kHead ? 128 : 32, slices = kSumThreads / width;
    const int x = threadIdx.x % width, y = threadIdx.x / width;
    int64_t c0 = 0, c1 = p.ctas - 1, group = 0;
    int col = b % blocks * 32 + x;
    // a gate of several groups is in the first weight's sum already, and has sums of its own
    const bool own_gate = a.j.gate && a.j.group_rows < a.j.rows;
    if (what == kPre && !a.dpre_weight) return;
    if (what == kPost && !a.dpost_weight && (own_gate || !a.dgate)) return;
    if (what == kHead) {
        const int64_t at = (b - 2 * blocks) / wide_blocks;
        col = (b - 2 * blocks) % wide_blocks * 128 + x;
        group = at;
        if (a.groups > p.ctas) {
            const int64_t row = (at + 1) * p.chunk;
            if (row >= a.j.rows || row % a.j.group_rows == 0) return;
            group = row / a.j.group_rows;
        }
        c0 = group * a.j.group_rows / p.chunk;
        c1 = ((group + 1) * a.j.group_rows - 1) / p.chunk;
        if (c0 == c1) return;  // written by its CTA
        if (a.groups > p.ctas && c0 != at) return;
    }
    float s = 0.f;
    if (col < cols) {
        // a group's first CTA began it: its part is the tail
#pragma unroll 8
        for (int64_t c = c0 + y; c <= c1; c += slices) {
            const int row = what == kHead && c == c0 ? kTail : what;
            const int64_t at = (c * p.parts + row) * p.pitch + col;
            if (fa_in_bounds(at, 1, p.ctas * p.parts * p.pitch)) s += a.sums[at];
        }
    }
    part[threadIdx.x] = s;
    __syncthreads();
    if (y || col >= cols) return;
    s = 0.f;
    for (int k = 0; k < slices; ++k) s += part[k * width + x];
    const bool wide = a.j.wide_weights;
    if (what == kHead) {
        store_weight<DT>(a.dgate, wide, group * a.dgate_ld + col, s);
    } else if (what == kPre) {
        store_weight<DT>(a.dpre_weight, wide, col, s);
    } else if (own_gate) {
        store_weight<DT>(a.dpost_weight, wide, col, s);
    } else {
        if (a.dpost_weight)
            store_weight<DT>(a.dpost_weight, wide, col, s * one_weight<DT>(a.j, a.j.gate, col, 0.f));
        if (a.dgate)
            store_weight<DT>(a.dgate, wide, col,
                             s * one_weight<DT>(a.j, a.j.post_norm ? a.j.post_weight : nullptr, col,
                                                a.j.weight_offset));
    }
}

// What a CTA alone on its SM has beside a kernel's own arrays (see Ring::stages).
constexpr int kMostShared = kSmShared - 2048;

template <auto kKernel>
cudaError_t launch_rows(const JoinGradArgs &a, int threads, size_t smem, cudaStream_t stream) {
    const cudaError_t e = allow_shared<kKernel, kMostShared>();
    if (e != cudaSuccess) return e;
    kKernel<<<static_cast<unsigned>(a.plan.ctas), threads, smem, stream>>>(a);
    return cudaGetLastError();
}

// Rows that the ring of a CTA of this many threads has room for.
template <int DT, int ST, int R>
int ring_stages(int threads) {
    const int row_bytes = Ring<DT, ST, R>::bytes(threads);
    return Ring<DT, ST, R>::stages(threads, join_ctas_per_sm({threads, R}, row_bytes),
                                   4 * R * threads * static_cast<int>(sizeof(float4)));
}

template <int DT, int ST, int R>
cudaError_t launch_gradient_rows(const JoinGradArgs &a, bool vec, int threads,
                                 cudaStream_t stream) {
    JoinGradArgs args = a;
    const size_t weights = 4 * R * threads * sizeof(float4);
    args.stages = ring_stages<DT, ST, R>(threads);
    if constexpr (R == 1 || DT != FA_F32) {  // (no ring has two rows of FP32 that wide)
        if (vec && args.stages >= 2) {
            const size_t smem = weights + args.stages * Ring<DT, ST, R>::bytes(threads);
            const bool all =
                a.j.post_norm && a.dnormed.p && a.dout.p && a.dresidual.p && a.dbranch.p;
            const auto launch = [&](auto shift) {
                const auto as = [&](auto every, auto drop) {
                    return launch_rows<join_gradient_kernel<DT, ST, R, true, every(), drop(), shift()>>(
                        args, threads, smem, stream);
                };
                const std::true_type yes{};
                const std::false_type no{};
                return !all ? as(no, yes) : a.j.dropped ? as(yes, yes) : as(yes, no);
            };
            if constexpr (R == 1)
                if (a.j.ld8 >= 0) return launch(std::true_type{});
            return launch(std::false_type{});
        }
    }
    args.stages = 0;
    return launch_rows<join_gradient_kernel<DT, ST, R, false, false, true, false>>(args, threads, weights,
                                                                                  stream);
}

// Whole runs of rows that no CTA holds.  ``a.plan`` becomes the clusters'.
template <int DT, int ST>
cudaError_t launch_split(JoinGradArgs &a, cudaStream_t stream) {
    const int runs = static_cast<int>(a.j.cols) / kRun;
    SplitArgs args;
    int threads = 0, mine = 0, weights = 0, stages = 0;
    for (a.split = 2; a.split <= kMostSplit; a.split *= 2) {
        mine = (runs + a.split - 1) / a.split;
        threads = (mine + 31) / 32 * 32;
        weights = 4 * threads * static_cast<int>(sizeof(float4));
        stages = Ring<DT, ST, 1>::stages(threads, 1, weights + kSplitPlaces);
        if (threads <= kJoinThreads && stages >= 2) break;
    }
    if (a.split > kMostSplit) return cudaErrorInvalidConfiguration;
    const size_t smem = weights + stages * Ring<DT, ST, 1>::bytes(threads);
    constexpr auto kernel = join_gradient_split_kernel<DT, ST>;
    const cudaError_t e = allow_shared<kernel, kMostShared - kSplitPlaces>();
    if (e != cudaSuccess) return e;
    // As many as ran side by side on the measured GPU, 76 of two and 36 of four (38 are two rounds: 277 us
    // for 159), and not what this one has room for: the rows' sums are grouped by them, and their bits
    // are to be every GPU's.
    const int clusters = a.split == 2 ? kSms / 2 : 36;
    a.plan.chunk = (a.j.rows + clusters - 1) / clusters;
    a.plan.ctas = (a.j.rows + a.plan.chunk - 1) / a.plan.chunk;
    a.stages = stages;
    a.all_cols = static_cast<int32_t>(a.j.cols);
    const int weight_bytes = a.j.wide_weights ? 4 : sizeof(typename Elem<DT>::T);
    for (int i = 0; i < a.split; ++i) {
        JoinGradArgs &p = args.of[i];
        p = a;
        const int64_t first = static_cast<int64_t>(i) * mine * kRun;
        p.first_run = i * mine;
        p.j.cols = first + mine * kRun < a.j.cols ? mine * kRun : a.j.cols - first;
        for (MatrixArgs *m : {&p.j.branch, &p.out, &p.dout, &p.dnormed, &p.dresidual, &p.dbranch}) {
            const bool of_branch = m == &p.j.branch || m == &p.dnormed || m == &p.dbranch;
            const int size = of_branch ? sizeof(typename Elem<DT>::T) : sizeof(typename Elem<ST>::T);
            if (m->p) m->p = static_cast<char *>(m->p) + first * size;
            m->cols = p.j.cols;
        }
        const auto along = [&](auto &w) {
            if (w) w = static_cast<char *>(const_cast<void *>(w)) + first * weight_bytes;
        };
        along(p.j.post_weight);
        along(p.j.pre_weight);
        along(p.j.gate);
        along(p.dgate);
        p.sums = a.sums + first;
    }
    return launch_clusters(kernel, dim3(static_cast<unsigned>(a.plan.ctas * a.split)), dim3(threads), smem,
                           a.split, false, stream, args);
}

template <int DT, int ST>
cudaError_t launch_gradient(const JoinGradArgs &given, cudaStream_t stream) {
    JoinGradArgs a = given;
    a.j.ld8 = -1;
    const fa_dtype dt = static_cast<fa_dtype>(DT), st = static_cast<fa_dtype>(ST);
    JoinShape shape = join_shape(a.j.cols);
    const bool vec = a.j.cols % kRun == 0 && aligned_rows(a.j.branch, dt) && aligned_rows(a.out, st) &&
                     aligned_rows(a.dout, st) && aligned_rows(a.dnormed, dt) &&
                     aligned_rows(a.dresidual, st) && aligned_rows(a.dbranch, dt);
    // Rows that begin anywhere, at least one a CTA, go through the ring too, if all matrices' do alike
    // (16384 x 2047 BF16: 99 us, 188 with every run put together from two lines).  A gate's
    // groups need a CTA's rows one after another.
    const JoinShape wider = join_shape(a.j.cols + kRun - 1);
    if (!vec && wider.runs == 1 && a.j.cols >= 2 * kRun && !(a.j.gate && a.j.group_rows < a.j.rows)) {
        static_assert(kSms % kRun == 0, "a CTA's rows are a multiple of eight apart");
        const int64_t ctas =
            join_ctas(a.j.rows, wider, Ring<DT, ST, 1>::bytes(wider.threads)) / kRun * kRun;
        if (a.j.rows >= ctas && ctas * a.plan.parts * a.plan.pitch * 4 <= a.plan.bytes)
            a.j.ld8 = common_ld8({&a.j.branch, &a.out, &a.dout, &a.dnormed, &a.dresidual, &a.dbranch});
        if (a.j.ld8 >= 0) {
            shape = wider;
            a.plan.ctas = ctas;
        }
    }
    // Whole rows of which no two fit beside each other are a cluster's (2048 x 8192 FP32: 107 us, 158 in
    // one CTA without a ring; 2730 x 6144: 115 and 125).
    const int stages = shape.runs == 1   ? ring_stages<DT, ST, 1>(shape.threads)
                       : shape.runs == 2 ? ring_stages<DT, ST, 2>(shape.threads)
                                         : 0;
    cudaError_t err;
    if (vec && stages < 2)
        err = launch_split<DT, ST>(a, stream);
    else if (shape.runs == 1)
        err = launch_gradient_rows<DT, ST, 1>(a, vec || a.j.ld8 >= 0, shape.threads, stream);
    else if (shape.runs == 2)
        err = launch_gradient_rows<DT, ST, 2>(a, vec, shape.threads, stream);
    else
        err = launch_rows<join_gradient_wide_kernel<DT, ST>>(a, shape.threads,
                                                             2 * a.plan.pitch * sizeof(float), stream);
    if (err != cudaSuccess || (!a.dpost_weight && !a.dpre_weight && !a.dgate)) return err;
    const bool own_gate = a.dgate && a.j.group_rows < a.j.rows;
    const int64_t groups = !own_gate ? 0 : a.groups > a.plan.ctas ? a.plan.ctas - 1 : a.groups;
    const int64_t blocks = 2 * ((a.j.cols + 31) / 32) + groups * ((a.j.cols + 127) / 128);
    return launch_dependent(join_sums_kernel<DT>, dim3(static_cast<unsigned>(blocks)),
                            dim3(kSumThreads), 0, stream, a);
}

cudaError_t read_row_error(int *flag, bool clear) {
    const cudaError_t e = cudaMemcpyFromSymbol(flag, g_join_gradient_error, sizeof(int));
    if (e != cudaSuccess || !clear) return e;
    const int zero = 0;
    return cudaMemcpyToSymbol(g_join_gradient_error, &zero, sizeof(int));
}

}  // namespace
}  // namespace fa
