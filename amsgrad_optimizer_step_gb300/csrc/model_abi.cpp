// C-ABI host layer of the model-side operators: validation and launches of the kernels
// in embedding_kernels.cu, logprob_kernels.cu and gated_kernels.cu.  The contract is
// fused_adamw.h's: everything is checked before anything is enqueued.
#include <cmath>
#include <cstdint>

#include <cuda_runtime.h>

#include "abi_checks.h"
#include "fa_model_ops.h"
#include "internal.h"
#include "model_checks.h"
#include "model_internal.h"

namespace {

using namespace fa;

constexpr int64_t kMaxDim = int64_t(1) << 21;       // of an embedding: the grid's other limit
constexpr int64_t kMaxBlocks = int64_t(1) << 28;    // of a checkpoint: 8 lanes each, in one grid
constexpr double kLog2E = 1.4426950408889634;

bool valid_itype(fa_itype t) { return t == FA_I32 || t == FA_I64; }
size_t itype_bytes(fa_itype t) { return t == FA_I64 ? 8 : 4; }

// The host-side rules of a logits record.
fa_status check_logits(const fa_logits *x) {
    if (!x) return FA_ERR_NULL;
    if (!valid_dtype(x->dtype) || !valid_itype(x->ltype)) return FA_ERR_DTYPE;
    FA_TRY(check_matrix(x->tokens, x->vocab, x->ld));
    if (x->tokens > kMaxCount || x->vocab > kMaxCount) return FA_ERR_SIZE;
    if (x->tokens > 0 && x->vocab < 1) return FA_ERR_SIZE;
    // (k and its residual are normal FP32 numbers)
    if (!(x->logit_scale >= 1e-4) || !(x->logit_scale <= 1e4)) return FA_ERR_OPTION;
    return FA_OK;
}
// Its device pointers.
fa_status check_logits_ptrs(const fa_logits *x, int dev) {
    FA_TRY(check_device_ptr(x->logits, dev, dtype_bytes(x->dtype)));
    return check_device_ptr(x->labels, dev, itype_bytes(x->ltype));
}
Matrix logits_matrix(const fa_logits *x) {
    return mat(x->logits, x->tokens, x->vocab, x->ld, dtype_bytes(x->dtype));
}
Matrix labels_vec(const fa_logits *x) {
    return vec(x->labels, x->tokens * static_cast<int64_t>(itype_bytes(x->ltype)));
}
fa::LogitsArgs logits_args(const fa_logits *x) {
    fa::LogitsArgs a;
    a.logits = x->logits;
    a.labels = x->labels;
    a.wide_labels = x->ltype == FA_I64;
    a.tokens = x->tokens;
    a.vocab = x->vocab;
    a.ld = x->ld;
    a.scale = static_cast<float>(x->logit_scale);
    a.scale_lo = static_cast<float>(x->logit_scale - a.scale);
    // k rounded down, so that its residual is positive: -inf times either part is -inf
    const double k = x->logit_scale * kLog2E;
    a.k = static_cast<float>(k);
    if (a.k > k) a.k = std::nextafter(a.k, 0.0f);
    a.k_lo = std::fmax(static_cast<float>(k - a.k), 1e-30f * a.k);
    return a;
}
// dlogits: the logits' type; the logits themselves, or no overlap with them.
fa_status check_dlogits(const fa_logits *x, const void *dlogits, int64_t ld, int dev) {
    FA_TRY(check_device_ptr(dlogits, dev, dtype_bytes(x->dtype)));
    if (dlogits == x->logits && ld == x->ld) return FA_OK;
    return overlap(logits_matrix(x), mat(dlogits, x->tokens, x->vocab, ld, dtype_bytes(x->dtype)))
               ? FA_ERR_ALIAS
               : FA_OK;
}

}  // namespace

extern "C" {

// ---- embedding ---------------------------------------------------------------

fa_status fa_embedding_lookup(int64_t tokens, const void *ids, fa_itype idt, const void *table,
                              fa_dtype tdt, int64_t vocab, int64_t dim, int64_t table_ld,
                              double scale, void *out, fa_dtype odt, int64_t out_ld,
                              void *stream) {
    if (!valid_dtype(tdt) || !valid_dtype(odt) || !valid_itype(idt)) return FA_ERR_DTYPE;
    FA_TRY(check_matrix(vocab, dim, table_ld));
    FA_TRY(check_matrix(tokens, dim, out_ld));
    if (tokens > kMaxCount || dim > kMaxDim) return FA_ERR_SIZE;
    if (!float_ok(scale)) return FA_ERR_OPTION;
    if (tokens == 0 || dim == 0) return FA_OK;
    int dev;
    FA_TRY(stream_device(stream, &dev));
    FA_TRY(check_device_ptr(ids, dev, itype_bytes(idt)));
    if (vocab > 0) FA_TRY(check_device_ptr(table, dev, dtype_bytes(tdt)));
    FA_TRY(check_device_ptr(out, dev, dtype_bytes(odt)));
    const Matrix outs[] = {mat(out, tokens, dim, out_ld, dtype_bytes(odt))};
    const Matrix ins[] = {vec(ids, tokens * static_cast<int64_t>(itype_bytes(idt))),
                          mat(table, vocab, dim, table_ld, dtype_bytes(tdt))};
    FA_TRY(check_outputs(outs, 1, ins, 2));
    TraceRange trace("fa_embedding_lookup");
    fa::LookupArgs a;
    a.ids = ids;
    a.table = table;
    a.out = out;
    a.tokens = tokens;
    a.vocab = vocab;
    a.dim = dim;
    a.table_ld = table_ld;
    a.out_ld = out_ld;
    a.scale = static_cast<float>(scale);
    return cuda_status(
        fa::launch_embedding_lookup(a, idt, tdt, odt, static_cast<cudaStream_t>(stream)));
}

fa_status fa_embedding_scratch(int64_t tokens, int64_t vocab, int64_t dim, int64_t *bytes) {
    if (!bytes) return FA_ERR_NULL;
    if (tokens < 0 || vocab < 0 || dim < 0 || tokens > kMaxCount || vocab >= kMaxCount ||
        dim > kMaxDim)
        return FA_ERR_SIZE;
    *bytes = fa::embedding_scratch_layout(tokens, vocab, dim).bytes;
    return FA_OK;
}

fa_status fa_embedding_gradient(int64_t tokens, const void *ids, fa_itype idt, const void *dout,
                                fa_dtype ddt, int64_t dout_ld, double scale, int64_t padding_idx,
                                int32_t accumulate, void *dtable, fa_dtype tdt, int64_t vocab,
                                int64_t dim, int64_t table_ld, void *scratch,
                                int64_t scratch_bytes, void *stream) {
    if (!valid_dtype(tdt) || !valid_dtype(ddt) || !valid_itype(idt)) return FA_ERR_DTYPE;
    FA_TRY(check_matrix(vocab, dim, table_ld));
    FA_TRY(check_matrix(tokens, dim, dout_ld));
    int64_t need = 0;
    FA_TRY(fa_embedding_scratch(tokens, vocab, dim, &need));
    if (!float_ok(scale) || (accumulate != 0 && accumulate != 1)) return FA_ERR_OPTION;
    if (vocab == 0 || dim == 0 || (accumulate && tokens == 0)) return FA_OK;
    if (scratch_bytes < need) return FA_ERR_SIZE;
    int dev;
    FA_TRY(stream_device(stream, &dev));
    if (tokens > 0) {
        FA_TRY(check_device_ptr(ids, dev, itype_bytes(idt)));
        FA_TRY(check_device_ptr(dout, dev, dtype_bytes(ddt)));
        FA_TRY(check_device_ptr(scratch, dev, 16));
    }
    FA_TRY(check_device_ptr(dtable, dev, dtype_bytes(tdt)));
    const Matrix outs[] = {mat(dtable, vocab, dim, table_ld, dtype_bytes(tdt)),
                           vec(scratch, need)};
    const Matrix ins[] = {vec(ids, tokens * static_cast<int64_t>(itype_bytes(idt))),
                          mat(dout, tokens, dim, dout_ld, dtype_bytes(ddt))};
    FA_TRY(check_outputs(outs, 2, ins, 2));
    TraceRange trace("fa_embedding_gradient");
    fa::EmbeddingGradArgs a;
    a.ids = ids;
    a.dout = dout;
    a.dtable = dtable;
    a.scratch = scratch;
    a.tokens = tokens;
    a.vocab = vocab;
    a.dim = dim;
    a.dout_ld = dout_ld;
    a.table_ld = table_ld;
    a.padding_idx = padding_idx;
    a.scale = static_cast<float>(scale);
    a.accumulate = accumulate != 0;
    return cuda_status(
        fa::launch_embedding_gradient(a, idt, ddt, tdt, static_cast<cudaStream_t>(stream)));
}

// ---- losses from the logits -----------------------------------------------------

fa_status fa_token_logprobs(const fa_logits *x, float *logp, float *lse, void *stream) {
    FA_TRY(check_logits(x));
    if (x->tokens == 0) return FA_OK;
    int dev;
    FA_TRY(stream_device(stream, &dev));
    FA_TRY(check_logits_ptrs(x, dev));
    FA_TRY(check_device_ptr(logp, dev, 4));
    if (lse) FA_TRY(check_device_ptr(lse, dev, 8));
    const Matrix outs[] = {vec(logp, x->tokens * 4), vec(lse, x->tokens * 8)};
    const Matrix ins[] = {logits_matrix(x), labels_vec(x)};
    FA_TRY(check_outputs(outs, 2, ins, 2));
    TraceRange trace("fa_token_logprobs");
    return cuda_status(fa::launch_token_logprobs(logits_args(x), x->dtype, logp, lse,
                                                 static_cast<cudaStream_t>(stream)));
}

fa_status fa_token_logprobs_gradient(const fa_logits *x, const float *lse, const float *dlogp,
                                     double grad_scale, const float *grad_loss, void *dlogits,
                                     int64_t dlogits_ld, void *stream) {
    FA_TRY(check_logits(x));
    FA_TRY(check_matrix(x->tokens, x->vocab, dlogits_ld));
    if (!float_ok(grad_scale * x->logit_scale)) return FA_ERR_OPTION;
    if (x->tokens == 0) return FA_OK;
    int dev;
    FA_TRY(stream_device(stream, &dev));
    FA_TRY(check_logits_ptrs(x, dev));
    FA_TRY(check_device_ptr(lse, dev, 8));
    FA_TRY(check_device_ptr(dlogp, dev, 4));
    if (grad_loss) FA_TRY(check_device_ptr(grad_loss, dev, 4));
    FA_TRY(check_dlogits(x, dlogits, dlogits_ld, dev));
    const Matrix outs[] = {
        mat(dlogits, x->tokens, x->vocab, dlogits_ld, dtype_bytes(x->dtype))};
    const Matrix ins[] = {labels_vec(x), vec(lse, x->tokens * 8), vec(dlogp, x->tokens * 4),
                          vec(grad_loss, 4)};
    FA_TRY(check_outputs(outs, 1, ins, 4));
    TraceRange trace("fa_token_logprobs_gradient");
    fa::LogitGradArgs a;
    a.x = logits_args(x);
    a.lse = lse;
    a.dlogp = dlogp;
    a.grad_loss = grad_loss;
    a.factor = static_cast<float>(grad_scale * x->logit_scale);
    a.dlogits = dlogits;
    a.dlogits_ld = dlogits_ld;
    return cuda_status(fa::launch_token_logprobs_gradient(a, x->dtype, static_cast<cudaStream_t>(stream)));
}

fa_status fa_preference_loss(const fa_logits *x, const fa_preference *p, void *stream) {
    FA_TRY(check_logits(x));
    if (!p) return FA_ERR_NULL;
    if (p->pairs < 0 || p->pairs > kMaxCount) return FA_ERR_SIZE;
    if (!(p->beta > 0) || !float_ok(p->beta) || !(p->label_smoothing >= 0) ||
        p->label_smoothing > 0.5 || (p->average != 0 && p->average != 1))
        return FA_ERR_OPTION;
    int dev;
    FA_TRY(stream_device(stream, &dev));
    FA_TRY(check_device_ptr(p->loss, dev, 4));
    if (p->pairs > 0) {
        FA_TRY(check_device_ptr(p->seq_offsets, dev, 8));
        FA_TRY(check_device_ptr(p->pair_loss, dev, 4));
        FA_TRY(check_device_ptr(p->rewards, dev, 4));
    }
    if (x->tokens > 0) {
        FA_TRY(check_logits_ptrs(x, dev));
        FA_TRY(check_device_ptr(p->ref_logp, dev, 4));
        FA_TRY(check_device_ptr(p->logp, dev, 4));
        FA_TRY(check_device_ptr(p->lse, dev, 8));
        FA_TRY(check_device_ptr(p->dlogp, dev, 4));
    }
    const Matrix outs[] = {vec(p->loss, 4),           vec(p->pair_loss, p->pairs * 4),
                           vec(p->rewards, p->pairs * 8), vec(p->logp, x->tokens * 4),
                           vec(p->lse, x->tokens * 8), vec(p->dlogp, x->tokens * 4)};
    const Matrix ins[] = {logits_matrix(x), labels_vec(x),
                          vec(p->seq_offsets, (2 * p->pairs + 1) * 8),
                          vec(p->ref_logp, x->tokens * 4)};
    FA_TRY(check_outputs(outs, 6, ins, 4));
    TraceRange trace("fa_preference_loss");
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (x->tokens > 0)
        FA_TRY(cuda_status(fa::launch_token_logprobs(logits_args(x), x->dtype, p->logp, p->lse, s)));
    fa::PreferenceArgs a;
    a.labels = x->labels;
    a.tokens = x->tokens;
    a.vocab = x->vocab;
    a.pairs = p->pairs;
    a.seq_offsets = p->seq_offsets;
    a.logp = p->logp;
    a.ref_logp = p->ref_logp;
    a.beta = static_cast<float>(p->beta);
    a.smoothing = static_cast<float>(p->label_smoothing);
    a.average = p->average != 0;
    a.loss = p->loss;
    a.pair_loss = p->pair_loss;
    a.rewards = p->rewards;
    a.dlogp = p->dlogp;
    return cuda_status(fa::launch_preference(a, x->ltype, s));
}

fa_status fa_policy_loss(const fa_logits *x, const fa_policy *p, void *stream) {
    FA_TRY(check_logits(x));
    if (!p) return FA_ERR_NULL;
    if (p->dlogits) FA_TRY(check_matrix(x->tokens, x->vocab, p->dlogits_ld));
    if (!(p->clip_low >= 0) || p->clip_low > 1 || !(p->clip_high >= 0) ||
        !float_ok(1.0 + p->clip_high) || !(p->kl_coef >= 0) || !float_ok(p->kl_coef) ||
        !(p->denominator >= 0) || !float_ok(p->denominator) ||
        (p->denominator > 0 && static_cast<float>(p->denominator) == 0.f) ||
        !float_ok(p->grad_scale * x->logit_scale))
        return FA_ERR_OPTION;
    if (p->kl_coef > 0 && !p->ref_logp) return FA_ERR_NULL;
    int dev;
    FA_TRY(stream_device(stream, &dev));
    FA_TRY(check_device_ptr(p->summary, dev, 4));
    if (x->tokens > 0) {
        FA_TRY(check_logits_ptrs(x, dev));
        FA_TRY(check_device_ptr(p->old_logp, dev, 4));
        FA_TRY(check_device_ptr(p->advantages, dev, 4));
        if (p->ref_logp) FA_TRY(check_device_ptr(p->ref_logp, dev, 4));
        if (p->weights) FA_TRY(check_device_ptr(p->weights, dev, 4));
        FA_TRY(check_device_ptr(p->logp, dev, 4));
        FA_TRY(check_device_ptr(p->token_loss, dev, 4));
        FA_TRY(check_device_ptr(p->token_kl, dev, 4));
        if (p->lse) FA_TRY(check_device_ptr(p->lse, dev, 8));
        if (p->dlogp) FA_TRY(check_device_ptr(p->dlogp, dev, 4));
        if (p->dlogits) FA_TRY(check_dlogits(x, p->dlogits, p->dlogits_ld, dev));
    }
    const int64_t b = x->tokens * 4;
    const Matrix outs[] = {
        vec(p->summary, 16), vec(p->logp, b), vec(p->token_loss, b), vec(p->token_kl, b),
        vec(p->lse, 2 * b), vec(p->dlogp, b),
        mat(p->dlogits, x->tokens, x->vocab, p->dlogits_ld, dtype_bytes(x->dtype))};
    const Matrix ins[] = {labels_vec(x),       vec(p->old_logp, b), vec(p->advantages, b),
                          vec(p->ref_logp, b), vec(p->weights, b)};
    FA_TRY(check_outputs(outs, 7, ins, 5));
    const Matrix logits[] = {logits_matrix(x)};
    FA_TRY(check_outputs(outs, 6, logits, 1));  // dlogits: checked above
    TraceRange trace("fa_policy_loss");
    fa::PolicyArgs a;
    a.x = logits_args(x);
    a.old_logp = p->old_logp;
    a.advantages = p->advantages;
    a.ref_logp = p->ref_logp;
    a.weights = p->weights;
    a.clip_lo = static_cast<float>(1.0 - p->clip_low);
    a.clip_hi = static_cast<float>(1.0 + p->clip_high);
    a.kl_coef = static_cast<float>(p->kl_coef);
    a.denominator = static_cast<float>(p->denominator);
    a.grad_factor = static_cast<float>(p->grad_scale * x->logit_scale);
    a.summary = p->summary;
    a.logp = p->logp;
    a.token_loss = p->token_loss;
    a.token_kl = p->token_kl;
    a.lse = p->lse;
    a.dlogp = p->dlogp;
    a.dlogits = p->dlogits;
    a.dlogits_ld = p->dlogits_ld;
    return cuda_status(fa::launch_policy(a, x->dtype, static_cast<cudaStream_t>(stream)));
}

// ---- gated activation -------------------------------------------------------------

fa_status fa_checkpoint_size(int64_t rows, int64_t cols, int64_t *code_bytes,
                             int64_t *scale_elements) {
    if (!code_bytes || !scale_elements) return FA_ERR_NULL;
    if (rows < 0 || cols < 0 || cols > kMaxElements) return FA_ERR_SIZE;
    const int64_t blocks = (cols + fa::kCheckpointBlock - 1) / fa::kCheckpointBlock;
    if (rows && blocks > kMaxBlocks / rows) return FA_ERR_SIZE;
    *code_bytes = 2 * rows * blocks * fa::kCheckpointBlock;
    *scale_elements = 2 * rows * blocks;
    return FA_OK;
}

fa_status fa_gated_forward(int64_t rows, int64_t cols, const void *gate, int64_t gate_ld,
                           const void *up, int64_t up_ld, fa_dtype dtype,
                           fa_activation activation, void *h, int64_t h_ld, int8_t *codes,
                           float *scales, void *stream) {
    if (!valid_dtype(dtype)) return FA_ERR_DTYPE;
    if (activation != FA_SILU && activation != FA_GELU_TANH) return FA_ERR_OPTION;
    FA_TRY(check_matrix(rows, cols, gate_ld));
    FA_TRY(check_matrix(rows, cols, up_ld));
    FA_TRY(check_matrix(rows, cols, h_ld));
    int64_t code_bytes, scale_elements;
    FA_TRY(fa_checkpoint_size(rows, cols, &code_bytes, &scale_elements));
    if ((codes == nullptr) != (scales == nullptr)) return FA_ERR_NULL;
    if (rows == 0 || cols == 0) return FA_OK;
    int dev;
    FA_TRY(stream_device(stream, &dev));
    const size_t e = dtype_bytes(dtype);
    FA_TRY(check_device_ptr(gate, dev, e));
    FA_TRY(check_device_ptr(up, dev, e));
    FA_TRY(check_device_ptr(h, dev, e));
    if (codes) {
        FA_TRY(check_device_ptr(codes, dev, 16));
        FA_TRY(check_device_ptr(scales, dev, 4));
    }
    const Matrix outs[] = {mat(h, rows, cols, h_ld, e), vec(codes, code_bytes),
                           vec(scales, scale_elements * 4)};
    const Matrix ins[] = {mat(gate, rows, cols, gate_ld, e), mat(up, rows, cols, up_ld, e)};
    FA_TRY(check_outputs(outs, 3, ins, 2));
    TraceRange trace("fa_gated_forward");
    fa::GatedForwardArgs a;
    a.gate = {const_cast<void *>(gate), rows, cols, gate_ld};
    a.up = {const_cast<void *>(up), rows, cols, up_ld};
    a.h = {h, rows, cols, h_ld};
    a.codes = codes;
    a.scales = scales;
    a.rows = rows;
    a.blocks = (cols + fa::kCheckpointBlock - 1) / fa::kCheckpointBlock;
    a.by_blocks = fa::Divider(static_cast<uint32_t>(a.blocks));
    return cuda_status(
        fa::launch_gated_forward(a, dtype, activation, static_cast<cudaStream_t>(stream)));
}

fa_status fa_gated_backward(int64_t rows, int64_t cols, const int8_t *codes, const float *scales,
                            fa_activation activation, const void *dh, int64_t dh_ld,
                            fa_dtype dtype, void *dgate, int64_t dgate_ld, void *dup,
                            int64_t dup_ld, void *h, int64_t h_ld, void *stream) {
    if (!valid_dtype(dtype)) return FA_ERR_DTYPE;
    if (activation != FA_SILU && activation != FA_GELU_TANH) return FA_ERR_OPTION;
    FA_TRY(check_matrix(rows, cols, dh_ld));
    FA_TRY(check_matrix(rows, cols, dgate_ld));
    FA_TRY(check_matrix(rows, cols, dup_ld));
    if (h) FA_TRY(check_matrix(rows, cols, h_ld));
    int64_t code_bytes, scale_elements;
    FA_TRY(fa_checkpoint_size(rows, cols, &code_bytes, &scale_elements));
    if (rows == 0 || cols == 0) return FA_OK;
    int dev;
    FA_TRY(stream_device(stream, &dev));
    const size_t e = dtype_bytes(dtype);
    FA_TRY(check_device_ptr(codes, dev, 16));
    FA_TRY(check_device_ptr(scales, dev, 4));
    FA_TRY(check_device_ptr(dh, dev, e));
    FA_TRY(check_device_ptr(dgate, dev, e));
    FA_TRY(check_device_ptr(dup, dev, e));
    if (h) FA_TRY(check_device_ptr(h, dev, e));
    const Matrix outs[] = {mat(dgate, rows, cols, dgate_ld, e), mat(dup, rows, cols, dup_ld, e),
                           mat(h, rows, cols, h_ld, e)};
    const Matrix ins[] = {vec(codes, code_bytes), vec(scales, scale_elements * 4),
                          mat(dh, rows, cols, dh_ld, e)};
    FA_TRY(check_outputs(outs, 3, ins, 3));
    TraceRange trace("fa_gated_backward");
    fa::GatedBackwardArgs a;
    a.codes = codes;
    a.scales = scales;
    a.dh = {const_cast<void *>(dh), rows, cols, dh_ld};
    a.dgate = {dgate, rows, cols, dgate_ld};
    a.dup = {dup, rows, cols, dup_ld};
    a.h = {h, rows, cols, h_ld};
    a.rows = rows;
    a.blocks = (cols + fa::kCheckpointBlock - 1) / fa::kCheckpointBlock;
    a.by_blocks = fa::Divider(static_cast<uint32_t>(a.blocks));
    return cuda_status(
        fa::launch_gated_backward(a, dtype, activation, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
