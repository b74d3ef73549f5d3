// The gradient of a join whose stream is FP32.
#include "join_gradient.cuh"

namespace fa {

FA_BOUNDS_VIOLATIONS(join_gradient_f32_bounds_violations, g_join_gradient_oob)

cudaError_t join_gradient_f32_error(int *flag, bool clear) { return read_row_error(flag, clear); }

cudaError_t launch_block_join_gradient_f32(const JoinGradArgs &a, fa_dtype dt,
                                           cudaStream_t stream) {
    return for_dtype(dt, [&](auto d) { return launch_gradient<d(), FA_F32>(a, stream); });
}

}  // namespace fa
