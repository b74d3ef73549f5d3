// Internal interface between the C-ABI host layer of the model-side operators
// (model_abi.cpp) and their kernels (embedding_kernels.cu, logprob_kernels.cu,
// gated_kernels.cu).
#pragma once

#include <cstdint>
#include <type_traits>

#include <cuda_runtime.h>

#include "fa_model_ops.h"

namespace fa {

constexpr int kCheckpointBlock = FA_CHECKPOINT_BLOCK;
constexpr int kSms = 152;  // a GB300's, which the sizes of grids and their thresholds count in

// Division of a number below 2^31 by a constant: the high word of a product with the
// divisor's inverse, rounded up, at 31 + ceil(log2 d) fractional bits.
struct Divider {
    uint32_t mul = 0, shift = 0;  // mul 0: the divisor is 1

    Divider() = default;
    explicit Divider(uint32_t d) {
        if (d < 2) return;
        uint32_t bits = 1;
        while (bits < 31 && (uint64_t(1) << bits) < d) ++bits;
        mul = static_cast<uint32_t>(((uint64_t(1) << (31 + bits)) + d - 1) / d);
        shift = bits - 1;
    }
#if defined(__CUDACC__)
    __device__ __forceinline__ uint32_t quotient(uint32_t n) const {
        return mul ? __umulhi(n, mul) >> shift : n;
    }
#endif
};

// ---- embedding ---------------------------------------------------------------
struct LookupArgs {
    const void *ids;
    const void *table;
    void *out;
    int64_t tokens, vocab, dim, table_ld, out_ld;
    float scale;
};
cudaError_t launch_embedding_lookup(const LookupArgs &a, fa_itype idt, fa_dtype tdt, fa_dtype odt,
                                    cudaStream_t stream);

// Scratch of the embedding gradient, in this order (each part 16-byte aligned).
struct EmbeddingScratch {
    int64_t chunks;  // runs of kSortChunk tokens that one cluster sorts
    int64_t units;   // runs of kSumUnit sorted tokens that one CTA adds
    int64_t claim_words;   // a token of each id
    int64_t run_words;     // the list of long runs
    int64_t sorted_words;  // 32-bit words of one sorted array (tokens, rounded up to 4)
    int64_t bytes;
};
constexpr int kSortSlots = 4096;             // tokens in one CTA's shared memory
constexpr int kSortChunk = 16 * kSortSlots;  // in a cluster's
constexpr int kSumUnit = 32;
EmbeddingScratch embedding_scratch_layout(int64_t tokens, int64_t vocab, int64_t dim);

struct EmbeddingGradArgs {
    const void *ids;
    const void *dout;
    void *dtable;
    void *scratch;
    int64_t tokens, vocab, dim, dout_ld, table_ld, padding_idx;
    float scale;
    bool accumulate;
};
cudaError_t launch_embedding_gradient(const EmbeddingGradArgs &a, fa_itype idt, fa_dtype ddt,
                                      fa_dtype tdt, cudaStream_t stream);

// ---- losses from the logits -----------------------------------------------------
struct LogitsArgs {
    const void *logits;
    const void *labels;
    bool wide_labels;  // int64
    int64_t tokens, vocab, ld;
    float scale, scale_lo;  // logit_scale as an FP32 value and its residual
    float k, k_lo;          // logit_scale * log2(e) in the same way
};
cudaError_t launch_token_logprobs(const LogitsArgs &x, fa_dtype dt, float *logp, float *lse,
                                  cudaStream_t stream);

struct LogitGradArgs {
    LogitsArgs x;
    const float *lse;
    const float *dlogp;
    const float *grad_loss;
    float factor;  // logit_scale * grad_scale
    void *dlogits;
    int64_t dlogits_ld;
};
cudaError_t launch_token_logprobs_gradient(const LogitGradArgs &a, fa_dtype dt,
                                           cudaStream_t stream);

struct PreferenceArgs {
    const void *labels;
    int64_t tokens, vocab, pairs;
    const int64_t *seq_offsets;
    const float *logp, *ref_logp;
    float beta, smoothing;
    bool average;
    float *loss, *pair_loss, *rewards, *dlogp;
};
cudaError_t launch_preference(const PreferenceArgs &a, fa_itype lt, cudaStream_t stream);

struct PolicyArgs {
    LogitsArgs x;
    const float *old_logp, *advantages, *ref_logp, *weights;
    float clip_lo, clip_hi;  // 1 - clip_low, 1 + clip_high
    float kl_coef;
    float denominator;  // 0: the number of counted tokens, from summary[3]
    float grad_factor;  // logit_scale * grad_scale
    float *summary, *logp, *token_loss, *token_kl;
    float *lse, *dlogp;  // or nullptr
    void *dlogits;
    int64_t dlogits_ld;
};
cudaError_t launch_policy(const PolicyArgs &a, fa_dtype dt, cudaStream_t stream);

// ---- gated activation -------------------------------------------------------------
struct MatrixArgs {
    void *p;
    int64_t rows, cols, ld;
};
struct GatedForwardArgs {
    MatrixArgs gate, up, h;
    int8_t *codes;  // nullptr: no checkpoint
    float *scales;
    int64_t rows, blocks;
    Divider by_blocks;
};
cudaError_t launch_gated_forward(const GatedForwardArgs &a, fa_dtype dt, fa_activation act,
                                 cudaStream_t stream);

struct GatedBackwardArgs {
    const int8_t *codes;
    const float *scales;
    MatrixArgs dh, dgate, dup, h;  // h.p may be nullptr
    int64_t rows, blocks;
    Divider by_blocks;
};
cudaError_t launch_gated_backward(const GatedBackwardArgs &a, fa_dtype dt, fa_activation act,
                                  cudaStream_t stream);

// Out-of-range accesses counted by each file's kernels in the bounds-checked build
// (0 in the normal build).  Wait for the device.
cudaError_t embedding_bounds_violations(unsigned long long *count, bool clear);
cudaError_t logprob_bounds_violations(unsigned long long *count, bool clear);
cudaError_t gated_bounds_violations(unsigned long long *count, bool clear);

#if defined(__CUDACC__)
// Launches ``kernel`` in clusters of ``cluster`` CTAs (1: none), as a programmatic
// dependent of the kernel before it or not.  A dependent waits (fa_grid_dependency_wait)
// before its first access to global memory, as those of launch_dependent do, with two
// exceptions: policy_row_kernel waits only to read the count of the kernel before it, and
// the sorting CTAs of sort_chunk_kernel do not wait at all.  Both are launched so behind a
// kernel of the same call that is itself an ordinary launch, so that all earlier work of the
// stream has ended when it begins, and that reads nothing they write and writes nothing they
// read without waiting.
template <typename... Params, typename... Args>
inline cudaError_t launch_clusters(void (*kernel)(Params...), dim3 grid, dim3 block, size_t smem,
                                   unsigned cluster, bool dependent, cudaStream_t stream,
                                   const Args &...args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    unsigned n = 0;
    if (cluster > 1) {
        attr[n].id = cudaLaunchAttributeClusterDimension;
        attr[n].val.clusterDim.x = cluster;
        attr[n].val.clusterDim.y = 1;
        attr[n++].val.clusterDim.z = 1;
    }
    if (dependent) {
        attr[n].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[n++].val.programmaticStreamSerializationAllowed = 1;
    }
    cfg.attrs = attr;
    cfg.numAttrs = n;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}
#endif

// Calls f with the validated type as a compile-time constant.
template <typename F>
inline cudaError_t for_dtype(fa_dtype dt, F f) {
    switch (dt) {
        case FA_F32: return f(std::integral_constant<int, FA_F32>{});
        case FA_F16: return f(std::integral_constant<int, FA_F16>{});
        default: return f(std::integral_constant<int, FA_BF16>{});
    }
}
template <typename F>
inline cudaError_t for_itype(fa_itype it, F f) {
    return it == FA_I64 ? f(std::integral_constant<int, FA_I64>{})
                        : f(std::integral_constant<int, FA_I32>{});
}

}  // namespace fa
