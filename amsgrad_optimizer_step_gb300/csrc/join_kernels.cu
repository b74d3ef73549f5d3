// The join of a block's output to the residual stream, with the norms behind and before it.
//
// A row belongs to a team of warps.  The work is bound by issue slots before it is by memory (a
// row a CTA and a run of eight columns a lane took 684 instructions a warp's run, 90 us for 16384 x
// 2048 BF16 of which the memory needs 40), so what is done once a row is spread over two
// runs a lane, the arithmetic is in packed pairs, what a row could ask is a template's argument, and
// the weights lie widened and multiplied together in shared memory for all rows of a CTA.  A lane's
// runs of the next row are on their way to shared memory, to slots that nobody else reads, while it
// works on those of this one.  The same rows take 51 us now, 41 (the memory's rate) without dropout;
// more runs a lane in loops over shared memory took 55, and 47 to 104 at other widths.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "internal.h"

FA_BOUNDS_COUNTER(g_join_oob)

#include "join_device.cuh"

namespace fa {
namespace {

constexpr int kTeamThreads = 1024;  // of a CTA and an SM at most, in 64 registers each
constexpr int kMaxWarps = 32;
constexpr int kMostShared = 220 * 1024;
// Rows whose squares pass FP32 are summed at this scale: 2^14 squares of up to 2^96 do not, and the root
// of such a row is 2^57 at least, so that what is lost below adds nothing to it.
constexpr float kHuge = 0x1p-80f;

// The sum over a team's lanes, in every one.  ``part``: four floats for each four warps, not in
// use by the call before.
__device__ __forceinline__ float team_sum(float x, float *part) {
    x = warp_sum(x);
    if (blockDim.x == 32) return x;
    const unsigned warps = blockDim.x / 32;
    if (threadIdx.x % 32 == 0) part[threadIdx.x / 32] = x;
    team_sync();
    float s = 0.f;
    for (unsigned w = 0; w < warps; w += 4) {  // (what no warp wrote is 0)
        const float4 v = *reinterpret_cast<const float4 *>(part + w);
        s += (v.x + v.y) + (v.z + v.w);
    }
    return s;
}

// 1 / sqrt(mean) within two units in the last place.
__device__ __forceinline__ float inverse_root(float mean) {
    const float y = rsqrtf(mean);
    const float e = fmaf(-mean * y, y, 1.f);
    return mean < INFINITY ? fmaf(0.5f * y, e, y) : y;
}

__device__ __forceinline__ float sum_of_pairs(uint64_t a, uint64_t b) {
    float x, y;
    unpair(add2(a, b), x, y);
    return x + y;
}

__device__ __forceinline__ void add_squares(const uint64_t *p, uint64_t *s) {
#pragma unroll
    for (int j = 0; j < kPairs; ++j) s[j % 2] = fma2(p[j], p[j], s[j % 2]);
}

// 1 / sqrt(mean square + eps) of the row that a team holds, R runs a lane.
template <int DT, int R>
__device__ __forceinline__ float team_rstd(const Raw<DT, kRun> *x, float inv_cols, float eps,
                                           float *part) {
    uint64_t s[2] = {}, p[kPairs];
#pragma unroll
    for (int r = 0; r < R; ++r) {
        widen_pairs<DT>(x[r], p);
        add_squares(p, s);
    }
    float sum = team_sum(sum_of_pairs(s[0], s[1]), part);
    if (sum < INFINITY) return inverse_root(fmaf(sum, inv_cols, eps));
    // squares past FP32 (or an infinity or NaN, which stays one); eps does not matter to them
    s[0] = s[1] = 0;
#pragma unroll
    for (int r = 0; r < R; ++r) {
        widen_pairs<DT>(x[r], p);
#pragma unroll
        for (int j = 0; j < kPairs; ++j) p[j] = mul2(p[j], both(kHuge));
        add_squares(p, s);
    }
    sum = team_sum(sum_of_pairs(s[0], s[1]), part + 4 * kMaxWarps);
    return inverse_root(sum * inv_cols) * kHuge;
}

// Two sums' places in turn: one is written again only after a wait for those who read it.
struct Parts {
    float at[2][2 * 4 * kMaxWarps];
};
__device__ __forceinline__ void clear_parts(Parts &parts, int thread, int threads) {
    for (int i = thread; i < 2 * 2 * 4 * kMaxWarps; i += threads) parts.at[0][i] = 0.f;
}

// out and the branch's share of it, of one run: p = alpha * p + f.
__device__ __forceinline__ void join_pairs(uint64_t alpha, uint64_t *p, const uint64_t *f) {
#pragma unroll
    for (int j = 0; j < kPairs; ++j) p[j] = fma2(alpha, p[j], f[j]);
}

// Many rows.  blockDim: the lanes of a team, the teams; R runs a lane.  VEC: rows of whole, aligned
// runs (else they are read from any address).  RING: the runs of the team's next row are asked for
// while it works on this one.  ALL: a branch, a gate that all rows share or none, and both results
// (asked once, not in every row).  DROP: false where nothing is dropped.  SHIFT: rows of VEC that begin
// anywhere, in matrices of one common_ld8.  The rows of a CTA are a multiple of eight apart, so its
// run q is columns [8 q - shift, 8 q - shift + 8) in all of them, whole lines but for the row's
// two ends.
template <int DT, int ST, int R, bool VEC, bool RING, bool ALL, bool DROP, bool SHIFT>
__global__ void __launch_bounds__(kTeamThreads) join_kernel(JoinArgs a) {
    constexpr int kD = Raw<DT, kRun>::kWords, kS = Raw<ST, kRun>::kWords;
    extern __shared__ float4 staged[];
    __shared__ Parts parts;
    const int cols = static_cast<int>(a.cols), row_blocks = (cols + kRun - 1) / kRun;
    const int shift = SHIFT ? static_cast<int>(blockIdx.x) % kRun * a.ld8 % kRun : 0;
    const int runs = SHIFT ? (cols + shift + kRun - 1) / kRun : row_blocks;
    const auto whole = [&](int q) {  // a run of columns alone
        return !SHIFT || (q * kRun >= shift && q * kRun - shift + kRun <= cols);
    };
    const float inv_cols = 1.f / static_cast<float>(cols);
    const int q0 = threadIdx.x, lanes = blockDim.x;  // this lane's runs: q0, q0 + lanes, ...
    const int threads = blockDim.x * blockDim.y, thread = threadIdx.y * lanes + q0;
    const bool branch = ALL || a.branch.p, dropped = DROP && (ALL || a.dropped);
    const bool own_gate = !ALL && a.gate && a.group_rows < a.rows;  // row by row
    // the weights, as two planes of four columns of each run: the scale of the branch with its
    // norm's weight and a gate that all rows share, and the second norm's weight
    float4 *const plane_post = staged, *const plane_pre = staged + 2 * runs;
    const float scale = dropped ? a.drop.scale * a.branch_scale : a.branch_scale;
    for (int q = thread; q < runs; q += threads) {
        float w[kRun], g[kRun];
        const auto load = [&](const void *p, float offset, float *to) {
            if constexpr (SHIFT)
                load_columns<DT>(a, p, 0, q * kRun - shift, cols, offset, to);
            else
                load_weights<DT>(a, p, q * kRun, valid_cols(q * kRun, cols), offset, to);
        };
        load(a.post_norm ? a.post_weight : nullptr, a.weight_offset, w);
        load(own_gate ? nullptr : a.gate, 0.f, g);
#pragma unroll
        for (int j = 0; j < kRun; ++j) w[j] *= scale * g[j];
        plane_post[q] = make_float4(w[0], w[1], w[2], w[3]);
        plane_post[q + runs] = make_float4(w[4], w[5], w[6], w[7]);
        load(a.pre_weight, a.weight_offset, w);
        plane_pre[q] = make_float4(w[0], w[1], w[2], w[3]);
        plane_pre[q + runs] = make_float4(w[4], w[5], w[6], w[7]);
    }
    clear_parts(parts, thread, threads);
    // a lane's slots: the branch's and the stream's runs, of two rows; those of no run stay 0
    uint4 *const ring = reinterpret_cast<uint4 *>(staged + 4 * runs) + thread;
    const int run_stride = (kD + kS) * threads;
    if (RING)
        for (int k = 0; k < 2 * R * (kD + kS); ++k)
            ring[k * threads] = make_uint4(0u, 0u, 0u, 0u);
    __syncthreads();
    const auto weights = [&](const float4 *plane, int q, uint64_t *w) {
        // (what is not there is not read: read all the same, a join without its second norm spilled
        // registers, 39 us for 33 at 16384 x 2048 BF16)
        const bool post = plane == plane_post;
        if (VEC && !ALL && !SHIFT &&
            !(post ? a.gate || (a.post_norm && a.post_weight) : a.pre_weight != nullptr)) {
#pragma unroll
            for (int j = 0; j < kPairs; ++j) w[j] = both(post ? scale : 1.f);
            return;
        }
        if (q >= runs) q = 0;  // not used
        const float4 lo = plane[q], hi = plane[q + runs];
        w[0] = pair(lo.x, lo.y);
        w[1] = pair(lo.z, lo.w);
        w[2] = pair(hi.x, hi.y);
        w[3] = pair(hi.z, hi.w);
    };
    const auto ask = [&](int64_t row, int slot) {
        if (row < a.rows) {
            uint4 *at = ring + slot * R * run_stride;
#pragma unroll
            for (int r = 0; r < R; ++r, at += run_stride) {
                const int q = q0 + r * lanes;
                if constexpr (SHIFT && RING) {
                    if (branch) ask_columns<DT>(a.branch, row, q * kRun - shift, at);
                    ask_columns<ST>(a.residual, row, q * kRun - shift, at + kD * threads);
                } else {
                    if (q >= runs || !fa_in_bounds(q * kRun, kRun, cols)) continue;
                    if (branch) ask_run<DT>(a.branch, row, q, at, threads);
                    ask_run<ST>(a.residual, row, q, at + kD * threads, threads);
                }
            }
        }
        copy_async_commit();
    };
    const uint64_t call = dropped ? drop_call(a.drop) : 0;
    const uint64_t alpha = both(a.residual_scale);
    const int64_t step = static_cast<int64_t>(gridDim.x) * blockDim.y;
    int64_t row = static_cast<int64_t>(blockIdx.x) * blockDim.y + threadIdx.y;
    if (SHIFT)
        row = blockIdx.x % kRun + static_cast<int64_t>(blockIdx.x / kRun * blockDim.y + threadIdx.y) * kRun;
    const int team_part = threadIdx.y * ((lanes / 32 + 3) / 4 * 4);
    int turn = 0, slot = 0;  // of the sums' places; of this row
    if (RING) ask(row, slot);
    for (; row < a.rows; row += step) {
        Raw<DT, kRun> y[R];
        Raw<ST, kRun> x[R];
        if (RING) {
            ask(row + step, slot ^ 1);  // that slot was read a row ago
            copy_async_wait<1>();
            const uint4 *at = ring + slot * R * run_stride;
            slot ^= 1;
#pragma unroll
            for (int r = 0; r < R; ++r, at += run_stride) {
                take_run(at, threads, y[r]);
                take_run(at + kD * threads, threads, x[r]);
                if (SHIFT && q0 + r * lanes == 0 && shift) {  // the end of the row before
                    keep_columns<DT>(y[r], -shift, cols);
                    keep_columns<ST>(x[r], -shift, cols);
                }
            }
        } else {
#pragma unroll
            for (int r = 0; r < R; ++r) {
                zero(y[r]);
                if constexpr (SHIFT) {
                    const int c = (q0 + r * lanes) * kRun - shift;
                    if (branch) y[r] = read_columns<DT>(a.branch, row, c);
                    x[r] = read_columns<ST>(a.residual, row, c);
                } else {
                    if (branch) y[r] = read_run<DT, VEC>(a.branch, row, q0 + r * lanes, runs);
                    x[r] = read_run<ST, VEC>(a.residual, row, q0 + r * lanes, runs);
                }
            }
        }
        float rstd = 1.f;
        if (a.post_norm) {
            rstd = team_rstd<DT, R>(y, inv_cols, a.eps, parts.at[turn] + team_part);
            turn ^= 1;
            if (a.post_rstd && q0 == 0) a.post_rstd[row] = rstd;
        }
        const uint64_t root = both(rstd);
        const int64_t group = own_gate ? a.by_group.quotient(static_cast<uint32_t>(row)) : 0;
        uint64_t block = static_cast<uint64_t>(row) * row_blocks + q0;
#pragma unroll
        for (int r = 0; r < R; ++r, block += lanes) {
            const int q = q0 + r * lanes;
            uint64_t p[kPairs];
            widen_pairs<ST>(x[r], p);
            if (branch) {
                uint64_t f[kPairs], w[kPairs];
                widen_pairs<DT>(y[r], f);
                weights(plane_post, q, w);
#pragma unroll
                for (int j = 0; j < kPairs; ++j) f[j] = mul2(mul2(f[j], root), w[j]);
                if (own_gate) {
                    float g[kRun];
                    if constexpr (SHIFT)
                        load_columns<DT>(a, a.gate, group * a.gate_ld, q * kRun - shift, cols, 0.f, g);
                    else
                        load_weights<DT>(a, a.gate, group * a.gate_ld + q * kRun,
                                         valid_cols(q * kRun, cols), 0.f, g);
                    to_pairs(g, w);
#pragma unroll
                    for (int j = 0; j < kPairs; ++j) f[j] = mul2(f[j], w[j]);
                }
                if (dropped) {
                    Kept kept;
                    kept.draw(a.drop, block, call);
                    if (SHIFT && shift) kept.begin_before(a.drop, block, call, shift);
                    kept.mask(f, a.drop.threshold);
                }
                join_pairs(alpha, p, f);
            } else {
#pragma unroll
                for (int j = 0; j < kPairs; ++j) p[j] = mul2(alpha, p[j]);
            }
            float v[kRun];
            from_pairs(p, v);
            x[r].from(v);  // as it is stored
            if (SHIFT && !whole(q)) {
                if (a.out.p) store_columns<ST>(a.out, row, v, q * kRun - shift);
                keep_columns<ST>(x[r], q * kRun - shift, cols);
            } else if (VEC) {
                if ((ALL || a.out.p) && q < runs) store_raw<ST>(a.out, row, q * kRun - shift, x[r]);
            } else {
#pragma unroll
                for (int j = 0; j < kRun; ++j)  // what is not there adds nothing to the sum
                    if (q * kRun + j >= cols) v[j] = 0.f;
                x[r].from(v);
                if (a.out.p) store_run<ST, false>(a.out, row, q * kRun, v, 0xffffffffu, 32);
            }
            if (VEC && !SHIFT && q >= runs) zero(x[r]);
        }
        if (!ALL && !a.normed.p) continue;
        // the norm is that of the stored values
        rstd = team_rstd<ST, R>(x, inv_cols, a.eps, parts.at[turn] + team_part);
        turn ^= 1;
        if (a.pre_rstd && q0 == 0) a.pre_rstd[row] = rstd;
        const uint64_t root_pre = both(rstd);
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const int q = q0 + r * lanes;
            uint64_t p[kPairs], w[kPairs];
            widen_pairs<ST>(x[r], p);
            weights(plane_pre, q, w);
#pragma unroll
            for (int j = 0; j < kPairs; ++j) p[j] = mul2(mul2(p[j], root_pre), w[j]);
            float v[kRun];
            from_pairs(p, v);
            if (SHIFT && !whole(q)) {
                store_columns<DT>(a.normed, row, v, q * kRun - shift);
            } else if (VEC) {
                Raw<DT, kRun> n;
                n.from(v);
                if (q < runs) store_raw<DT>(a.normed, row, q * kRun - shift, n);
            } else {
                store_run<DT, false>(a.normed, row, q * kRun, v, 0xffffffffu, 32);
            }
        }
    }
}

// Few rows: a row a CTA and a run a lane, the shortest way through a row.
template <int DT, int ST>
__global__ void __launch_bounds__(32 * kMaxWarps) join_few_kernel(JoinArgs a, bool vec) {
    __shared__ Parts parts;
    const int cols = static_cast<int>(a.cols), runs = (cols + kRun - 1) / kRun;
    const float inv_cols = 1.f / static_cast<float>(cols);
    const float scale = a.dropped ? a.drop.scale * a.branch_scale : a.branch_scale;
    const int64_t row = blockIdx.x;
    const int q = threadIdx.x, c = q * kRun, valid = valid_cols(c, cols);
    Raw<DT, kRun> y;
    zero(y);
    if (a.branch.p)
        y = vec ? read_run<DT, true>(a.branch, row, q, runs)
                : read_run<DT, false>(a.branch, row, q, runs);
    const Raw<ST, kRun> x = vec ? read_run<ST, true>(a.residual, row, q, runs)
                                : read_run<ST, false>(a.residual, row, q, runs);
    const int64_t group = a.gate ? a.by_group.quotient(static_cast<uint32_t>(row)) : 0;
    float w[kRun], g[kRun], w_pre[kRun];
    load_weights<DT>(a, a.post_norm ? a.post_weight : nullptr, c, valid, a.weight_offset, w);
    load_weights<DT>(a, a.gate, group * a.gate_ld + c, valid, 0.f, g);
    load_weights<DT>(a, a.pre_weight, c, valid, a.weight_offset, w_pre);
    clear_parts(parts, threadIdx.x, blockDim.x);
    __syncthreads();
    uint64_t p[kPairs], f[kPairs];
    float rstd = 1.f;
    widen_pairs<DT>(y, f);
    if (a.post_norm) {
        rstd = team_rstd<DT, 1>(&y, inv_cols, a.eps, parts.at[0]);
        if (a.post_rstd && q == 0) a.post_rstd[row] = rstd;
    }
    widen_pairs<ST>(x, p);
    if (a.branch.p) {
#pragma unroll
        for (int j = 0; j < kPairs; ++j)
            f[j] = mul2(mul2(f[j], both(rstd)), pair(w[2 * j] * (scale * g[2 * j]),
                                                     w[2 * j + 1] * (scale * g[2 * j + 1])));
        if (a.dropped) {
            Kept kept;
            kept.draw(a.drop, static_cast<uint64_t>(row) * runs + q, drop_call(a.drop));
            kept.mask(f, a.drop.threshold);
        }
        join_pairs(both(a.residual_scale), p, f);
    } else {
#pragma unroll
        for (int j = 0; j < kPairs; ++j) p[j] = mul2(both(a.residual_scale), p[j]);
    }
    float v[kRun];
    from_pairs(p, v);
#pragma unroll
    for (int j = 0; j < kRun; ++j)
        if (j >= valid) v[j] = 0.f;
    const auto store = [&](const MatrixArgs &m, auto type) {
        if (vec)
            store_run<decltype(type)::value, true>(m, row, c, v, 0xffffffffu, 32);
        else
            store_run<decltype(type)::value, false>(m, row, c, v, 0xffffffffu, 32);
    };
    if (a.out.p) store(a.out, std::integral_constant<int, ST>{});
    if (!a.normed.p) return;
    Raw<ST, kRun> stored;
    stored.from(v);
    widen_pairs<ST>(stored, p);
    rstd = team_rstd<ST, 1>(&stored, inv_cols, a.eps, parts.at[1]);
    if (a.pre_rstd && q == 0) a.pre_rstd[row] = rstd;
#pragma unroll
    for (int j = 0; j < kPairs; ++j)
        p[j] = mul2(mul2(p[j], both(rstd)), pair(w_pre[2 * j], w_pre[2 * j + 1]));
    from_pairs(p, v);
    store(a.normed, std::integral_constant<int, DT>{});
}

template <int DT, int ST, int R, bool VEC, bool RING, bool ALL, bool DROP, bool SHIFT = false>
cudaError_t launch_as(const JoinArgs &a, dim3 block, size_t smem, cudaStream_t stream) {
    constexpr auto kernel = join_kernel<DT, ST, R, VEC, RING, ALL, DROP, SHIFT>;
    const cudaError_t e = allow_shared<kernel, kMostShared>();
    if (e != cudaSuccess) return e;
    int64_t grid = (a.rows + block.y - 1) / block.y;
    // the SMs are full, and the weights are staged once (SHIFT: every eighth CTA has rows of one kind)
    if (SHIFT || grid > kSms) grid = kSms;
    kernel<<<static_cast<unsigned>(grid), block, smem, stream>>>(a);
    return cudaGetLastError();
}

template <int DT, int ST, int R, bool RING, bool SHIFT>
cudaError_t launch_parts(const JoinArgs &a, dim3 block, size_t smem, cudaStream_t stream) {
    const bool all = a.branch.p && a.out.p && a.normed.p &&
                     (!a.gate || a.group_rows >= a.rows);
    return !all ? launch_as<DT, ST, R, true, RING, false, true, SHIFT>(a, block, smem, stream)
           : a.dropped ? launch_as<DT, ST, R, true, RING, true, true, SHIFT>(a, block, smem, stream)
                       : launch_as<DT, ST, R, true, RING, true, false, SHIFT>(a, block, smem, stream);
}

// VEC, SHIFT: as the kernel has them.
template <int DT, int ST, int R, bool VEC, bool SHIFT>
cudaError_t launch_many(const JoinArgs &a, cudaStream_t stream) {
    // (SHIFT: the most that a row can have)
    const int runs = static_cast<int>((a.cols + (SHIFT ? 2 : 1) * (kRun - 1)) / kRun);
    const int warps = (runs + 32 * R - 1) / (32 * R), teams = kTeamThreads / 32 / warps;
    constexpr int kRunWeights = 4 * static_cast<int>(sizeof(float4));
    static_assert(FA_JOIN_MAX_COLS / kRun * kRunWeights <= kMostShared, "the weights of any row fit");
    const int weights = kRunWeights * runs;
    const dim3 block(32 * warps, warps > 1 && teams > 16 ? 16 : teams);  // 16: a barrier each
    if constexpr (VEC && ST != FA_F32) {
        // The ring, where it has room for three quarters of the teams.  16384 x 2048 BF16 took 57 us
        // with it and 63 without.  Runs of FP32 are two vectors 32 bytes apart, which the copies
        // to shared memory fetch as half sectors: 10922 x 2048 of BF16 and FP32 took 65 and 53.
        const int team = 2 * 16 * R * 32 * warps *
                         (Raw<DT, kRun>::kWords + Raw<ST, kRun>::kWords);
        int room = (kMostShared - weights) / team;
        if (room > static_cast<int>(block.y)) room = block.y;
        if (4 * room >= 3 * static_cast<int>(block.y)) {
            const dim3 fewer(block.x, room);
            const size_t smem = weights + static_cast<size_t>(team) * room;
            // (ALL, for rows that begin anywhere: 65153 x 515 BF16, a run a lane, 94 us and 104 without; with
            // two it is as fast without)
            if constexpr (SHIFT && R > 1)
                return launch_as<DT, ST, R, true, true, false, true, true>(a, fewer, smem, stream);
            else
                return launch_parts<DT, ST, R, true, SHIFT>(a, fewer, smem, stream);
        }
    }
    if constexpr (SHIFT) {
        if constexpr (ST == FA_F32)
            return launch_as<DT, ST, R, true, false, false, true, true>(a, block, weights, stream);
        else
            return launch_many<DT, ST, R, false, false>(a, stream);
    } else if constexpr (VEC && ST == FA_F32) {
        return launch_parts<DT, ST, R, false, false>(a, block, weights, stream);
    } else {
        return launch_as<DT, ST, R, VEC, false, false, true>(a, block, weights, stream);
    }
}

}  // namespace

FA_BOUNDS_VIOLATIONS(join_bounds_violations, g_join_oob)

cudaError_t launch_block_join(const JoinArgs &a, fa_dtype dt, fa_dtype st, cudaStream_t stream) {
    const bool vec = a.cols % kRun == 0 && aligned_rows(a.branch, dt) &&
                     aligned_rows(a.residual, st) && aligned_rows(a.out, st) &&
                     aligned_rows(a.normed, dt);
    // Rows that begin anywhere, in all matrices alike (16384 x 2047 BF16: 64 us, and 90 with eight
    // gates; 110 and 123 with every run put together from two lines).
    static_assert(kSms % kRun == 0, "a CTA's rows are a multiple of eight apart");
    JoinArgs shifted = a;
    const bool fits = a.cols >= 2 * kRun && a.cols + 2 * (kRun - 1) <= 2 * kRun * kTeamThreads;
    shifted.ld8 =
        vec || !fits ? -1 : common_ld8({&a.branch, &a.residual, &a.out, &a.normed});
    // few rows: fewer than four warps an SM with a run a lane
    const int64_t warps = ((a.cols + kRun - 1) / kRun + 31) / 32;
    return for_stream_dtype(dt, st, [&](auto d, auto s) {
        if (warps <= kMaxWarps && a.rows * warps < 4 * kSms) {
            join_few_kernel<d(), s()><<<static_cast<unsigned>(a.rows),
                                        static_cast<unsigned>(32 * warps), 0, stream>>>(a, vec);
            return cudaGetLastError();
        }
        // two runs a lane are what 64 registers hold of the work on them
        const auto many = [&](auto r) {
            return vec ? launch_many<d(), s(), r(), true, false>(a, stream)
                   : shifted.ld8 >= 0 ? launch_many<d(), s(), r(), true, true>(shifted, stream)
                                      : launch_many<d(), s(), r(), false, false>(a, stream);
        };
        // three warps' runs fill four warps by twos: 65153 x 515 BF16 took 94 us with one a lane and 114
        // with two; whole runs, which wait for memory, 63 and 62 (64528 x 520)
        return warps == 1 || (warps == 3 && shifted.ld8 >= 0)
                   ? many(std::integral_constant<int, 1>{})
                   : many(std::integral_constant<int, 2>{});
    });
}

}  // namespace fa
