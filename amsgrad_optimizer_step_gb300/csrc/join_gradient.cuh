// The gradient of a join: the kernels, as the files of the two kinds of stream include them
// (the branch's type, or FP32).
//
// A CTA takes a run of consecutive rows and keeps the columns' sums in registers.
// Per row it needs three sums over the columns, in one reduction: with d = dnormed * w_pre,
// t = dout + rstd_pre * d, a = branch_scale * gate * w_post and v = yh where it is kept,
//   s1 = sum d xh,  s2 = sum a v t,  s3 = sum a v xh
// the first norm's mean, which needs the second's gradient G = t - rstd_pre * mean(s1) * xh, is
// s2 - rstd_pre * mean(s1) * s3.  The gradients of the first weight and of the gate are both
// multiples, column by column, of K = sum over rows of v G: one sum serves both.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "internal.h"

FA_BOUNDS_COUNTER(g_join_gradient_oob)

#include "join_device.cuh"

namespace fa {
namespace {

constexpr int kRingBytes = 220 * 1024;

// One row's four matrices as a thread holds them.
template <int DT, int ST, int R>
struct GradRow {
    Raw<ST, kRun> dout[R], x[R];
    Raw<DT, kRun> dn[R], y[R];
};

template <int DT>
__device__ __forceinline__ void zero(Raw<DT, kRun> &x) {
#pragma unroll
    for (int k = 0; k < Raw<DT, kRun>::kWords; ++k) x.r[k] = make_uint4(0u, 0u, 0u, 0u);
}

// The rows on their way: a ring in shared memory of two to four rows, every thread's vectors in
// slots of its own, copied asynchronously by the thread that reads them (no barrier is needed).
template <int DT, int ST, int R>
struct Ring {
    static constexpr int kMost = 4;
    static constexpr int kS = Raw<ST, kRun>::kWords, kD = Raw<DT, kRun>::kWords;
    static constexpr int kVectors = 2 * R * (kS + kD);  // of 16 bytes, a thread's for one row

    static int bytes(int threads) { return kVectors * threads * 16; }  // of one row
    // Rows that the ring has room for (below two there is none).
    static int stages(int threads) {
        const int n = kRingBytes / bytes(threads);
        return n < kMost ? n : kMost;
    }
    // Waits for the oldest row but ``stages`` - 2 later ones.
    static __device__ __forceinline__ void wait(int stages) {
        if (stages == 4)
            copy_async_wait<2>();
        else if (stages == 3)
            copy_async_wait<1>();
        else
            copy_async_wait<0>();
    }
    template <int DD>
    static __device__ __forceinline__ void ask(const MatrixArgs &m, int64_t row, int64_t c,
                                               uint4 *slot) {
        constexpr int W = Raw<DD, kRun>::kWords;
        if (!m.p || c >= m.cols || !fa_in_bounds(c, kRun, m.cols)) return;
        const auto *p = static_cast<const typename Elem<DD>::T *>(m.p) + row * m.ld + c;
#pragma unroll
        for (int k = 0; k < W; ++k)
            copy_async16(slot + k * blockDim.x, reinterpret_cast<const uint4 *>(p) + k);
    }
    static __device__ __forceinline__ uint4 *stage(uint4 *ring, int s) {
        return ring + static_cast<size_t>(s) * kVectors * blockDim.x + threadIdx.x;
    }
    // Asks for a row (nothing past the last one) and closes the group.
    static __device__ __forceinline__ void issue(const JoinGradArgs &a, int64_t row, int64_t last,
                                                 uint4 *slot) {
        if (row < last) {
#pragma unroll
            for (int r = 0; r < R; ++r) {
                const int64_t c = (static_cast<int64_t>(r) * blockDim.x + threadIdx.x) * kRun;
                uint4 *at = slot + r * 2 * (kS + kD) * blockDim.x;
                ask<ST>(a.dout, row, c, at);
                ask<ST>(a.out, row, c, at + kS * blockDim.x);
                ask<DT>(a.dnormed, row, c, at + 2 * kS * blockDim.x);
                ask<DT>(a.j.branch, row, c, at + (2 * kS + kD) * blockDim.x);
            }
        }
        copy_async_commit();
    }
    template <int DD>
    static __device__ __forceinline__ void take(bool there, const uint4 *slot,
                                                Raw<DD, kRun> &x) {
        zero(x);
        if (!there) return;
#pragma unroll
        for (int k = 0; k < Raw<DD, kRun>::kWords; ++k) x.r[k] = slot[k * blockDim.x];
    }
    static __device__ __forceinline__ void read(const JoinGradArgs &a, const uint4 *slot,
                                                GradRow<DT, ST, R> &g) {
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const bool in = (static_cast<int64_t>(r) * blockDim.x + threadIdx.x) * kRun < a.j.cols;
            const uint4 *at = slot + r * 2 * (kS + kD) * blockDim.x;
            take(in && a.dout.p, at, g.dout[r]);
            take(in && a.out.p, at + kS * blockDim.x, g.x[r]);
            take(in && a.dnormed.p, at + 2 * kS * blockDim.x, g.dn[r]);
            take(in && a.j.branch.p, at + (2 * kS + kD) * blockDim.x, g.y[r]);
        }
    }
};

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
// comes, from any address.
template <int DT, int ST, int R, bool RING>
__global__ void __launch_bounds__(kMaxThreads) join_gradient_kernel(JoinGradArgs a) {
    extern __shared__ uint4 ring[];
    __shared__ float part[2][3][kMaxThreads / 32];
    using Rows = Ring<DT, ST, R>;
    const int64_t first = blockIdx.x * a.plan.chunk;
    const int64_t last = first + a.plan.chunk < a.j.rows ? first + a.plan.chunk : a.j.rows;
    const bool pre = a.dnormed.p, branch = a.j.branch.p, post = a.j.post_norm && branch;
    const int64_t blocks = (a.j.cols + kRun - 1) / kRun;
    const float inv_cols = 1.f / static_cast<float>(a.j.cols);
    const int lane = threadIdx.x % 32, warps = blockDim.x / 32;
    int64_t c[R];
    int valid[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
        c[r] = (static_cast<int64_t>(r) * blockDim.x + threadIdx.x) * kRun;
        valid[r] = valid_cols(c[r], a.j.cols);
    }
    if (RING) {
#pragma unroll
        for (int s = 0; s < Rows::kMost - 1; ++s)
            if (s < a.stages - 1) Rows::issue(a, first + s, last, Rows::stage(ring, s));
    }
    const float scale = a.j.dropped ? a.j.branch_scale * a.j.drop.scale : a.j.branch_scale;
    const uint64_t call = a.j.dropped ? drop_call(a.j.drop) : 0;
    float wp[R][kRun], aw[R][kRun];  // w_pre; scale * gate * w_post
    float sum_k[R][kRun] = {}, sum_p[R][kRun] = {};
#pragma unroll
    for (int r = 0; r < R; ++r)
        load_weights<DT>(a.j, pre ? a.j.pre_weight : nullptr, c[r], valid[r],
                               a.j.weight_offset, wp[r]);
    float *const sums = a.sums + blockIdx.x * a.plan.parts * a.plan.pitch;
    // the gate's group of the first row, and how many of its rows are left
    int64_t group = a.j.gate ? a.j.by_group.quotient(static_cast<uint32_t>(first)) : 0;
    int64_t group_first = a.j.gate ? group * a.j.group_rows : first;
    int64_t group_last = a.j.gate ? group_first + a.j.group_rows : last;
    bool flushed = false;

    const auto new_group = [&] {
#pragma unroll
        for (int r = 0; r < R; ++r) {
            float w[kRun];
            load_weights<DT>(a.j, post ? a.j.post_weight : nullptr, c[r],
                                   valid[r], a.j.weight_offset, aw[r]);
            load_weights<DT>(a.j, a.j.gate, group * a.j.gate_ld + c[r],
                                   valid[r], 0.f, w);
#pragma unroll
            for (int j = 0; j < kRun; ++j) aw[r][j] *= scale * w[j];
        }
    };
    // The group's sums: whole where all its rows are this CTA's, else a part of them.
    const auto flush = [&] {
        const bool begun_here = group_first >= first, whole = begun_here && group_last <= last;
        float *const gate_part = sums + (begun_here ? kTail : kHead) * a.plan.pitch;
#pragma unroll
        for (int r = 0; r < R; ++r) {
            float w[kRun];
            if (a.dpost_weight) {
                load_weights<DT>(a.j, a.j.gate, group * a.j.gate_ld + c[r],
                                       valid[r], 0.f, w);
#pragma unroll
                for (int j = 0; j < kRun; ++j)
                    if (j < valid[r]) {
                        float *at = sums + kPost * a.plan.pitch + c[r] + j;
                        const float x = scale * w[j] * sum_k[r][j];
                        *at = flushed ? *at + x : x;
                    }
            }
            if (a.dgate) {
                load_weights<DT>(a.j, post ? a.j.post_weight : nullptr, c[r],
                                       valid[r], a.j.weight_offset, w);
#pragma unroll
                for (int j = 0; j < kRun; ++j)
                    if (j < valid[r]) {
                        const float x = scale * w[j] * sum_k[r][j];
                        if (whole)
                            store_weight<DT>(a.dgate, a.j.wide_weights,
                                             group * a.dgate_ld + c[r] + j, x);
                        else
                            gate_part[c[r] + j] = x;
                    }
            }
#pragma unroll
            for (int j = 0; j < kRun; ++j) sum_k[r][j] = 0.f;
        }
        flushed = true;
    };

    if (branch) new_group();
    float rp_lane = 0.f, rq_lane = 1.f;
    int stage = 0;
    fa_allow_dependents();
    for (int64_t row = first; row < last; ++row) {
        const int64_t n = row - first;
        if (n % 32 == 0) {  // the inverse roots of 32 rows, a lane each
            const bool in = row + lane < last;
            if (pre) rp_lane = in ? a.j.pre_rstd[row + lane] : 0.f;
            if (post) rq_lane = in ? a.j.post_rstd[row + lane] : 0.f;
        }
        const float rp = __shfl_sync(0xffffffffu, rp_lane, n % 32);
        const float rq = __shfl_sync(0xffffffffu, rq_lane, n % 32);
        if (row == group_last) {
            if (branch) flush();
            ++group;
            group_first = group_last;
            group_last += a.j.group_rows;
            if (branch) new_group();
        }
        GradRow<DT, ST, R> g;
        if (RING) {
            Rows::wait(a.stages);
            Rows::read(a, Rows::stage(ring, stage), g);
            // the slot read a row ago is free
            Rows::issue(a, row + a.stages - 1, last,
                        Rows::stage(ring, stage == 0 ? a.stages - 1 : stage - 1));
            stage = stage == a.stages - 1 ? 0 : stage + 1;
        } else {
#pragma unroll
            for (int r = 0; r < R; ++r) {
                if (a.dout.p) g.dout[r] = load_run<ST, RING>(a.dout, row, c[r]);
                else zero(g.dout[r]);
                if (a.out.p) g.x[r] = load_run<ST, RING>(a.out, row, c[r]);
                else zero(g.x[r]);
                if (pre) g.dn[r] = load_run<DT, RING>(a.dnormed, row, c[r]);
                else zero(g.dn[r]);
                if (branch) g.y[r] = load_run<DT, RING>(a.j.branch, row, c[r]);
                else zero(g.y[r]);
            }
        }
        float s1 = 0.f, s2 = 0.f, s3 = 0.f;
        float t[R][kRun];
        Kept kept[R];
#pragma unroll
        for (int r = 0; r < R; ++r) {
            if (a.j.dropped)
                kept[r].draw(a.j.drop, row * blocks + c[r] / kRun, call);
            else
                kept[r].all();
            float dn[kRun], x[kRun], y[kRun];
            g.dout[r].widen(t[r]);
            g.dn[r].widen(dn);
            g.x[r].widen(x);
            g.y[r].widen(y);
#pragma unroll
            for (int j = 0; j < kRun; ++j) {
                const float d = dn[j] * wp[r][j], xh = x[j] * rp;
                s1 = fmaf(d, xh, s1);
                t[r][j] = fmaf(rp, d, t[r][j]);
                if (post) {
                    const float v = kept[r](j, a.j.drop.threshold) ? y[j] * rq : 0.f;
                    const float q = v * aw[r][j];
                    s2 = fmaf(q, t[r][j], s2);
                    s3 = fmaf(q, xh, s3);
                }
            }
        }
        if (pre || post) {
            s1 = warp_sum(s1);
            if (post) {
                s2 = warp_sum(s2);
                s3 = warp_sum(s3);
            }
            if (warps > 1) {
                float(*p)[kMaxThreads / 32] = part[n % 2];  // the other one is still being read
                if (lane == 0) {
                    p[0][threadIdx.x / 32] = s1;
                    p[1][threadIdx.x / 32] = s2;
                    p[2][threadIdx.x / 32] = s3;
                }
                __syncthreads();
                s1 = s2 = s3 = 0.f;
                for (int w = 0; w < warps; ++w) {
                    s1 += p[0][w];
                    s2 += p[1][w];
                    s3 += p[2][w];
                }
            }
        }
        const float back = rp * (s1 * inv_cols);            // times xh: taken off t
        const float mean = (s2 - back * s3) * inv_cols * rq;  // times yh: taken off dbranch
#pragma unroll
        for (int r = 0; r < R; ++r) {
            float dn[kRun], x[kRun], y[kRun], dr[kRun], db[kRun];
            g.dn[r].widen(dn);
            g.x[r].widen(x);
            g.y[r].widen(y);
#pragma unroll
            for (int j = 0; j < kRun; ++j) {
                const float xh = x[j] * rp;
                const float total = pre ? fmaf(-back, xh, t[r][j]) : t[r][j];
                sum_p[r][j] = fmaf(dn[j], xh, sum_p[r][j]);
                dr[j] = a.j.residual_scale * total;
                const bool on = kept[r](j, a.j.drop.threshold);
                const float yh = y[j] * rq;
                sum_k[r][j] = fmaf(on ? yh : 0.f, on ? total : 0.f, sum_k[r][j]);
                db[j] = on ? total * aw[r][j] : 0.f;
                if (post) db[j] = fmaf(db[j], rq, -yh * mean);
            }
            if (a.dresidual.p)
                store_run<ST, RING>(a.dresidual, row, c[r], dr, 0xffffffffu, 32);
            if (a.dbranch.p) store_run<DT, RING>(a.dbranch, row, c[r], db, 0xffffffffu, 32);
        }
    }
    if (branch && (a.dpost_weight || a.dgate)) flush();
    if (a.dpre_weight) {
#pragma unroll
        for (int r = 0; r < R; ++r)
#pragma unroll
            for (int j = 0; j < kRun; ++j)
                if (j < valid[r]) sums[kPre * a.plan.pitch + c[r] + j] = sum_p[r][j];
    }
}

// Rows of more than two runs a thread: their columns' sums lie in shared memory, and a row is
// read again from L2 once its three sums are there.
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
    int64_t group = a.j.gate ? a.j.by_group.quotient(static_cast<uint32_t>(first)) : 0;
    int64_t group_first = a.j.gate ? group * a.j.group_rows : first;
    int64_t group_last = a.j.gate ? group_first + a.j.group_rows : last;
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
                if (a.dpost_weight) *at = flushed ? *at + g[j] * k : g[j] * k;
                if (a.dgate && whole)
                    store_weight<DT>(a.dgate, a.j.wide_weights, group * a.dgate_ld + c + j,
                                     w[j] * k);
                else if (a.dgate)
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
                sums[kPre * a.plan.pitch + q * kRun + j] = sum_p[q * kRun + j];
}

// Joins the CTAs' sums in order.  A block takes 32 columns of one result, eight runs of CTAs
// side by side.  blockIdx.y: the first weight, the second, then the gate's groups, or (where
// there are more groups than CTAs) the border before each CTA, whose group it joins if it is
// the group's first border.
constexpr int kJoinSlices = 8;
template <int DT>
__global__ void __launch_bounds__(32 * kJoinSlices) join_sums_kernel(JoinGradArgs a) {
    __shared__ float part[kJoinSlices][32];
    fa_grid_dependency_wait();
    const int64_t col = blockIdx.x * 32 + threadIdx.x;
    const JoinPlan &p = a.plan;
    int64_t c0 = 0, c1 = p.ctas - 1, group = 0;
    const int what = blockIdx.y < 2 ? static_cast<int>(blockIdx.y) : kHead;
    if (what == kPost && !a.dpost_weight) return;
    if (what == kPre && !a.dpre_weight) return;
    if (what == kHead) {
        group = blockIdx.y - 2;
        if (a.groups > p.ctas) {
            const int64_t row = (group + 1) * p.chunk;
            if (row >= a.j.rows || row % a.j.group_rows == 0) return;
            group = row / a.j.group_rows;
        }
        c0 = group * a.j.group_rows / p.chunk;
        c1 = ((group + 1) * a.j.group_rows - 1) / p.chunk;
        if (c0 == c1) return;  // written by its CTA
        if (a.groups > p.ctas && c0 != static_cast<int64_t>(blockIdx.y) - 2) return;
    }
    float s = 0.f;
    if (col < a.j.cols) {
        // a group's first CTA began it: its part is the tail
        for (int64_t c = c0 + threadIdx.y; c <= c1; c += kJoinSlices) {
            const int row = what == kHead && c == c0 ? kTail : what;
            const int64_t at = (c * p.parts + row) * p.pitch + col;
            if (fa_in_bounds(at, 1, p.ctas * p.parts * p.pitch)) s += a.sums[at];
        }
    }
    part[threadIdx.y][threadIdx.x] = s;
    __syncthreads();
    if (threadIdx.y || col >= a.j.cols) return;
    s = 0.f;
#pragma unroll
    for (int k = 0; k < kJoinSlices; ++k) s += part[k][threadIdx.x];
    void *out = what == kPost ? a.dpost_weight : what == kPre ? a.dpre_weight : a.dgate;
    store_weight<DT>(out, a.j.wide_weights, (what == kHead ? group * a.dgate_ld : 0) + col, s);
}

template <typename Kernel>
cudaError_t launch_rows(Kernel kernel, const JoinGradArgs &a, int threads, size_t smem,
                        cudaStream_t stream) {
    const cudaError_t e = cudaFuncSetAttribute(
        kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
    if (e != cudaSuccess) return e;
    kernel<<<static_cast<unsigned>(a.plan.ctas), threads, smem, stream>>>(a);
    return cudaGetLastError();
}

template <int DT, int ST, int R>
cudaError_t launch_gradient_rows(const JoinGradArgs &a, bool vec, int threads,
                                 cudaStream_t stream) {
    JoinGradArgs args = a;
    args.stages = Ring<DT, ST, R>::stages(threads);
    if (vec && args.stages >= 2)
        return launch_rows(join_gradient_kernel<DT, ST, R, true>, args, threads,
                           args.stages * Ring<DT, ST, R>::bytes(threads), stream);
    return launch_rows(join_gradient_kernel<DT, ST, R, false>, args, threads, 0, stream);
}

template <int DT, int ST>
cudaError_t launch_gradient(const JoinGradArgs &a, cudaStream_t stream) {
    const fa_dtype dt = static_cast<fa_dtype>(DT), st = static_cast<fa_dtype>(ST);
    const JoinShape shape = join_shape(a.j.cols);
    const bool vec = a.j.cols % kRun == 0 && aligned_rows(a.j.branch, dt) && aligned_rows(a.out, st) &&
                     aligned_rows(a.dout, st) && aligned_rows(a.dnormed, dt) &&
                     aligned_rows(a.dresidual, st) && aligned_rows(a.dbranch, dt);
    cudaError_t err;
    if (shape.runs == 1)
        err = launch_gradient_rows<DT, ST, 1>(a, vec, shape.threads, stream);
    else if (shape.runs == 2)
        err = launch_gradient_rows<DT, ST, 2>(a, vec, shape.threads, stream);
    else
        err = launch_rows(join_gradient_wide_kernel<DT, ST>, a, shape.threads,
                          2 * a.plan.pitch * sizeof(float), stream);
    if (err != cudaSuccess || (!a.dpost_weight && !a.dpre_weight && !a.dgate)) return err;
    const int64_t groups = !a.dgate ? 0 : a.groups > a.plan.ctas ? a.plan.ctas - 1 : a.groups;
    const dim3 grid(static_cast<unsigned>((a.j.cols + 31) / 32),
                    static_cast<unsigned>(2 + groups));
    return launch_dependent(join_sums_kernel<DT>, grid, dim3(32, kJoinSlices), 0, stream, a);
}

}  // namespace
}  // namespace fa
