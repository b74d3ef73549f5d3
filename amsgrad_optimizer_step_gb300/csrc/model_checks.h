// Host-side argument rules that the model-side operators share (model_abi.cpp and
// block_abi.cpp): matrices, aliases, limits and the status of a launch.
#pragma once

#include <cmath>
#include <cstdint>

#include <cuda_runtime.h>

#include "fa_model_ops.h"

namespace fa {

constexpr int64_t kMaxCount = 0x7fffffff;        // tokens, ids, rows: the grid's limit
constexpr int64_t kMaxElements = int64_t(1) << 56;  // of one matrix: byte offsets stay in 64 bits

// A matrix argument: rows of row_bytes at distance ld_bytes.  A vector is one row.
struct Matrix {
    const void *p;
    int64_t rows;
    int64_t row_bytes;
    int64_t ld_bytes;
};

inline Matrix vec(const void *p, int64_t bytes) { return {p, 1, bytes, bytes}; }
inline Matrix mat(const void *p, int64_t rows, int64_t cols, int64_t ld, size_t elem) {
    const int64_t e = static_cast<int64_t>(elem);
    return {p, rows, cols * e, ld * e};
}

// Whether two matrices share a byte.  Rows of the same pitch may interleave (the two
// halves of one matrix); of different pitches, overlapping spans count as shared.
inline bool overlap(const Matrix &a, const Matrix &b) {
    if (!a.p || !b.p || !a.rows || !b.rows || !a.row_bytes || !b.row_bytes) return false;
    const auto first = [](const Matrix &m) { return reinterpret_cast<uintptr_t>(m.p); };
    const auto end = [&](const Matrix &m) {
        return first(m) + static_cast<uintptr_t>(m.rows - 1) * m.ld_bytes + m.row_bytes;
    };
    if (first(a) >= end(b) || first(b) >= end(a)) return false;
    const int64_t pitch = a.rows > 1 ? a.ld_bytes : b.ld_bytes;
    if ((a.rows > 1 && a.ld_bytes != pitch) || (b.rows > 1 && b.ld_bytes != pitch)) return true;
    if (a.rows == 1 && b.rows == 1) return true;
    if (a.row_bytes > pitch || b.row_bytes > pitch) return true;
    // b's rows start ``d`` bytes into a's pitch
    const int64_t d = first(b) >= first(a)
                          ? static_cast<int64_t>((first(b) - first(a)) % pitch)
                          : (pitch - static_cast<int64_t>((first(a) - first(b)) % pitch)) % pitch;
    return d < a.row_bytes || d + b.row_bytes > pitch;
}

// Every output against every other buffer.
inline fa_status check_outputs(const Matrix *out, int nout, const Matrix *in, int nin) {
    for (int i = 0; i < nout; ++i) {
        for (int j = i + 1; j < nout; ++j)
            if (overlap(out[i], out[j])) return FA_ERR_ALIAS;
        for (int j = 0; j < nin; ++j)
            if (overlap(out[i], in[j])) return FA_ERR_ALIAS;
    }
    return FA_OK;
}

inline bool float_ok(double x) { return std::isfinite(static_cast<float>(x)); }

// Shared argument rules of a matrix [rows, cols] with row distance ld.
inline fa_status check_matrix(int64_t rows, int64_t cols, int64_t ld) {
    if (rows < 0 || cols < 0 || ld < cols) return FA_ERR_SIZE;
    if (rows && ld > kMaxElements / rows) return FA_ERR_SIZE;
    return FA_OK;
}

inline fa_status cuda_status(cudaError_t e) {
    if (e == cudaSuccess) return FA_OK;
    cudaGetLastError();
    return FA_ERR_CUDA;
}

#define FA_TRY(expr)                          \
    do {                                      \
        const fa_status st_ = (expr);         \
        if (st_ != FA_OK) return st_;         \
    } while (0)

}  // namespace fa
