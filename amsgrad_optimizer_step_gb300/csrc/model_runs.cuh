// Runs of eight columns of a row, as the kernels of whole matrices read and write them.  The
// including file invokes FA_BOUNDS_COUNTER first: its counter takes the accesses out of range.
#pragma once

#include "model_device.cuh"
#include "model_internal.h"

namespace fa {

constexpr int kRun = 8;  // consecutive columns of a lane: 16 bytes of 16-bit types

// A lane's run of eight columns [c, c + 8) of a row.  ALIGNED: one 16-byte access (two for
// FP32) when the columns all exist, element accesses otherwise; else the 16-byte lines that the
// run touches (see RawAny, store_any).  Columns past the end read as 0 and are not written.
__device__ __forceinline__ int valid_cols(int64_t c, int64_t cols) {
    return c + kRun <= cols ? kRun : c < cols ? static_cast<int>(cols - c) : 0;
}
template <int DT, bool ALIGNED>
__device__ __forceinline__ Raw<DT, kRun> load_run(const MatrixArgs &m, int64_t row, int64_t c) {
    using E = Elem<DT>;
    const typename E::T *p = static_cast<const typename E::T *>(m.p) + row * m.ld + c;
    const int valid = valid_cols(c, m.cols);
    if (valid && !(fa_in_bounds(c, valid, m.cols) && fa_in_bounds(row, 1, m.rows))) return {};
    if constexpr (ALIGNED) {
        Raw<DT, kRun> x;
        if (c + kRun <= m.cols) {
            x.load(p);
        } else {
            float y[kRun];
#pragma unroll
            for (int j = 0; j < kRun; ++j) y[j] = j < valid ? E::widen(p[j]) : 0.f;
            x.from(y);  // exact: they came from this type
        }
        return x;
    } else {
        RawAny<DT, kRun> x;
        x.load(p, valid, Span(m.p, ((m.rows - 1) * m.ld + m.cols) * sizeof(typename E::T)));
        return x.raw();
    }
}
// ``lanes`` call it in groups of ``width``, which hold consecutive runs of one row.
template <int DT, bool ALIGNED>
__device__ __forceinline__ void store_run(const MatrixArgs &m, int64_t row, int64_t c,
                                          const float *x, unsigned lanes, int width) {
    using E = Elem<DT>;
    typename E::T *p = static_cast<typename E::T *>(m.p) + row * m.ld + c;
    int valid = valid_cols(c, m.cols);
    if (valid && !(fa_in_bounds(c, valid, m.cols) && fa_in_bounds(row, 1, m.rows))) valid = 0;
    if constexpr (ALIGNED) {
        if (c + kRun <= m.cols) {
            store_n<DT, kRun>(p, x);
        } else {
#pragma unroll
            for (int j = 0; j < kRun; ++j)
                if (j < valid) p[j] = E::round(x[j]);
        }
    } else {
        store_any<DT, kRun>(p, x, valid, lanes, width);
    }
}

// Whether 16-byte accesses at multiples of eight columns are aligned in every row.
inline bool aligned_rows(const MatrixArgs &m, fa_dtype dt) {
    const int64_t row_bytes = m.ld * (dt == FA_F32 ? 4 : 2);
    return !m.p || (reinterpret_cast<uintptr_t>(m.p) % 16 == 0 &&
                    (m.rows < 2 || row_bytes % 16 == 0));
}

}  // namespace fa
