// Dropout whose mask is drawn again wherever it is needed and never stored.
//
// One Philox block of 128 bits serves a run of eight columns, so a thread that takes one
// 16-byte vector of 16-bit elements (two of FP32) draws once.  Rows that lie densely and aligned are
// one long row of runs.  Rows at other addresses are taken in the vectors that memory has, and it is
// the random bits that are moved to where their columns lie in them, from the lane before; where
// input and output lie differently in their vectors, the data are moved too, by eight lanes with
// two runs each.
//
// Reads and writes bound the first (16384 x 5632 BF16: 56 us, 6.6 TB/s); issue slots bound
// odd rows, most of them the generator's (4099 x 5633 FP16: 25 us, of which the bytes need 14; moving
// all data with a run a lane took 37, with two 33).
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
constexpr int kPair = 2 * kRun;  // consecutive columns of a lane
constexpr int kDropBlock = kDropLanes * kPair;
static_assert(kDropBlock == kDropColumns, "the host limits the blocks");

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

// Rows whose vectors hold the same columns of input and output.  A warp takes twice 31 vectors
// (pairs of them for FP32) of eight elements of a row; its first lane draws the bits that the second
// needs of the run before.
constexpr int kShiftedLanes = 31, kShiftedTurns = 2;
constexpr int kShiftedVectors = kShiftedTurns * kShiftedLanes;
template <int DT>
__global__ void __launch_bounds__(kDropThreads) dropout_shifted_kernel(DropoutArgs a) {
    using T = typename Elem<DT>::T;
    const int64_t w = static_cast<int64_t>(blockIdx.x) * (kDropThreads / 32) + threadIdx.x / 32;
    if (w >= a.x.rows * a.blocks) return;  // a whole warp
    const int lane = threadIdx.x % 32;
    const int64_t row = a.by_blocks.quotient(static_cast<uint32_t>(w));
    const int64_t part = w - row * a.blocks, run0 = part * kShiftedVectors, col0 = run0 * kRun;
    const T *row_from = static_cast<const T *>(a.x.p) + row * a.x.ld;
    // columns of the row's first vector that are before it
    const int shift = static_cast<int>(reinterpret_cast<uintptr_t>(row_from) & 15) / sizeof(T);
    // a lane's elements, counted from col0: c to c + 8 (a turn further on in the second turn), as
    // far as the row has them
    const int c0 = (lane - 1) * kRun - shift, low = part ? -kRun : 0;
    const int left = static_cast<int>(min(a.x.cols - col0, static_cast<int64_t>(1) << 20));
    const T *from = row_from + col0 + c0;
    T *to = static_cast<T *>(a.out.p) + row * a.out.ld + col0 + c0;
    Raw<DT, kRun> raw[kShiftedTurns];
    bool any[kShiftedTurns], whole[kShiftedTurns];
#pragma unroll
    for (int r = 0; r < kShiftedTurns; ++r) {
        const int c = c0 + r * kShiftedLanes * kRun, begin = max(c, low), end = min(c + kRun, left);
        any[r] = lane > 0 && begin < end && fa_in_bounds(col0 + begin, end - begin, a.x.cols);
        whole[r] = any[r] && end - begin == kRun;
        if (whole[r]) raw[r].load(from + r * kShiftedLanes * kRun);
    }
    const uint64_t call = drop_call(a.drop);
    const int64_t block = row * ((a.x.cols + kRun - 1) / kRun) + run0 + (lane - 1);
#pragma unroll
    for (int r = 0; r < kShiftedTurns; ++r) {
        const int c = c0 + r * kShiftedLanes * kRun;
        if (c - c0 >= left + kRun) return;  // all lanes: nothing of the row is left
        Kept kept;
        kept.draw(a.drop, block + r * kShiftedLanes, call);
        if (shift) {  // the same for all lanes
            uint32_t cat[8];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                cat[k] = __shfl_up_sync(0xffffffffu, kept.w[k], 1);
                cat[4 + k] = kept.w[k];
            }
            move_down<4>(cat, 2 * (kRun - shift), kept.w);
        }
        const T *p = from + r * kShiftedLanes * kRun;
        T *q = to + r * kShiftedLanes * kRun;
        if (whole[r]) {
            float x[kRun];
            raw[r].widen(x);
            drop(a.drop, kept, x);
            store_n<DT, kRun>(q, x);
        } else if (any[r]) {
#pragma unroll
            for (int j = 0; j < kRun; ++j)
                if (c + j >= max(c, low) && c + j < min(c + kRun, left))
                    q[j] = Elem<DT>::round(kept(j, a.drop.threshold)
                                               ? Elem<DT>::widen(p[j]) * a.drop.scale : 0.f);
        }
    }
}

template <int DT>
__global__ void __launch_bounds__(kDropThreads) dropout_kernel(DropoutArgs a) {
    using T = typename Elem<DT>::T;
    const int64_t b = static_cast<int64_t>(blockIdx.x) * (kDropThreads / kDropLanes) +
                      threadIdx.x / kDropLanes;
    if (b >= a.x.rows * a.blocks) return;  // all eight lanes of a block
    const int64_t row = a.by_blocks.quotient(static_cast<uint32_t>(b));
    const int64_t c = (b - row * a.blocks) * kDropBlock + threadIdx.x % kDropLanes * kPair;
    const int64_t left = a.x.cols - c;
    int valid = left < 0 ? 0 : left < kPair ? static_cast<int>(left) : kPair;
    if (valid && !fa_in_bounds(c, valid, a.x.cols)) valid = 0;
    RawAny<DT, kPair> raw;
    raw.load(static_cast<const T *>(a.x.p) + row * a.x.ld + c, valid,
             Span(a.x.p, ((a.x.rows - 1) * a.x.ld + a.x.cols) * sizeof(T)));
    float x[kPair];
    raw.widen(x);
    const uint64_t call = drop_call(a.drop);
    const int64_t block = row * ((a.x.cols + kRun - 1) / kRun) + c / kRun;
#pragma unroll
    for (int r = 0; r < 2; ++r) {
        Kept kept;
        kept.draw(a.drop, block + r, call);
        drop(a.drop, kept, x + r * kRun);
    }
    store_any<DT, kPair>(static_cast<T *>(a.out.p) + row * a.out.ld + c, x, valid,
                         0xffu << (threadIdx.x & 24), kDropLanes);
}

// Whether every row of the two starts at the same place of a vector.
bool alike(const MatrixArgs &x, const MatrixArgs &y, int64_t size) {
    const auto at = [](const MatrixArgs &m) { return reinterpret_cast<uintptr_t>(m.p) % 16; };
    return at(x) == at(y) && (x.rows == 1 || (x.ld - y.ld) * size % 16 == 0);
}

}  // namespace

FA_BOUNDS_VIOLATIONS(dropout_bounds_violations, g_dropout_oob)

cudaError_t launch_dropout(const DropoutArgs &args, fa_dtype dt, cudaStream_t stream) {
    DropoutArgs a = args;
    const int64_t runs = (a.x.cols + kRun - 1) / kRun;
    const bool dense = a.x.cols % kRun == 0 &&
                       (a.x.rows == 1 || (a.x.ld == a.x.cols && a.out.ld == a.out.cols)) &&
                       aligned_rows(a.x, dt) && aligned_rows(a.out, dt);
    return for_dtype(dt, [&](auto d) {
        const auto grid = [](int64_t units, int64_t each) {
            return static_cast<unsigned>((units + each - 1) / each);
        };
        if (dense) {
            constexpr int R = 2;
            dropout_dense_kernel<d(), R>
                <<<grid(a.x.rows * runs, R * kDropThreads), kDropThreads, 0, stream>>>(a);
            return cudaGetLastError();
        }
        const bool shifted = alike(a.x, a.out, sizeof(typename Elem<d()>::T));
        // (a row that begins inside a vector may have one more than its runs)
        a.blocks = shifted ? runs / kShiftedVectors + 1 : (a.x.cols + kDropBlock - 1) / kDropBlock;
        a.by_blocks = Divider(static_cast<uint32_t>(a.blocks));
        if (shifted)
            dropout_shifted_kernel<d()>
                <<<grid(a.x.rows * a.blocks, kDropThreads / 32), kDropThreads, 0, stream>>>(a);
        else
            dropout_kernel<d()><<<grid(a.x.rows * a.blocks, kDropThreads / kDropLanes),
                                  kDropThreads, 0, stream>>>(a);
        return cudaGetLastError();
    });
}

}  // namespace fa
