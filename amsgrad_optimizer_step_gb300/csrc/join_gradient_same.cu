// The gradient of a join whose stream has the branch's type, and how it cuts the rows.
#include "join_gradient.cuh"

namespace fa {

FA_BOUNDS_VIOLATIONS(join_gradient_bounds_violations, g_join_gradient_oob)

cudaError_t join_gradient_error(int *flag, bool clear) { return read_row_error(flag, clear); }

JoinShape join_shape(int64_t cols) {
    const int runs = static_cast<int>((cols + kRun - 1) / kRun);
    if (runs <= kJoinThreads) return {(runs + 31) / 32 * 32, 1};
    if (runs <= 2 * kMaxThreads) return {(runs + 63) / 64 * 32, 2};
    return {kMaxThreads, 0};
}

JoinPlan join_plan(int64_t rows, int64_t cols, int64_t groups, int element_bytes) {
    JoinPlan p{0, 0, 0, 0, 0};
    if (rows == 0 || cols == 0) return p;
    const JoinShape shape = join_shape(cols);
    const int reach = kRun * shape.threads * (shape.runs ? shape.runs : 1);
    const int64_t ctas = join_ctas(rows, shape, reach * element_bytes);
    p.chunk = (rows + ctas - 1) / ctas;
    p.ctas = (rows + p.chunk - 1) / p.chunk;
    p.pitch = (cols + kRun - 1) / kRun * kRun;
    p.parts = groups > 0 ? 4 : 2;
    p.bytes = (ctas < rows ? ctas : rows) * p.parts * p.pitch * 4;
    return p;
}

cudaError_t launch_block_join_gradient(const JoinGradArgs &a, fa_dtype dt, fa_dtype st,
                                       cudaStream_t stream) {
    if (st == FA_F32) return launch_block_join_gradient_f32(a, dt, stream);
    return dt == FA_F16 ? launch_gradient<FA_F16, FA_F16>(a, stream)
                        : launch_gradient<FA_BF16, FA_BF16>(a, stream);
}

}  // namespace fa
