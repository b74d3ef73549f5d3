// C-ABI host layer of the residual blocks' operators: validation and launches of the kernels
// in dropout_kernels.cu, join_kernels.cu, join_gradient.cuh and route_kernels.cu.  The
// contract is fused_adamw.h's: everything is checked before anything is enqueued.
#include <cmath>
#include <cstdint>

#include <cuda_runtime.h>

#include "abi_checks.h"
#include "block_internal.h"
#include "fa_block_ops.h"
#include "internal.h"
#include "model_checks.h"

namespace {

using namespace fa;

// A dropout record on the host, and its device scalar.
fa_status check_key(const fa_dropout_key *k) {
    return k->p >= 0.0 && k->p <= 1.0 ? FA_OK : FA_ERR_OPTION;
}
fa_status check_key_ptr(const fa_dropout_key *k, int dev) {
    return k->counter ? check_device_ptr(k->counter, dev, 8) : FA_OK;
}
Matrix key_vec(const fa_dropout_key *k) { return vec(k ? k->counter : nullptr, 8); }
DropArgs drop_args(const fa_dropout_key *k) {
    const auto q = static_cast<uint32_t>(std::nearbyint(65536.0 * k->p));
    DropArgs d;
    d.threshold = q < 65536 ? q << 16 : 0xffffffffu;
    for (uint32_t r = 0; r < static_cast<uint32_t>(kPhiloxRounds); ++r) {
        d.key[r][0] = static_cast<uint32_t>(k->seed) + r * 0x9E3779B9u;
        d.key[r][1] = static_cast<uint32_t>(k->seed >> 32) + r * 0xBB67AE85u;
    }
    d.offset = k->offset;
    d.counter = k->counter;
    d.scale = q < 65536 ? static_cast<float>(65536.0 / (65536.0 - q)) : 0.f;
    return d;
}

MatrixArgs matrix_args(const void *p, int64_t rows, int64_t cols, int64_t ld) {
    return {const_cast<void *>(p), rows, cols, ld};
}

// The host-side rules of a join.
fa_status check_join(const fa_join *j) {
    if (!j) return FA_ERR_NULL;
    if (!valid_dtype(j->dtype) || !valid_dtype(j->stream_dtype) || !valid_dtype(j->weight_dtype))
        return FA_ERR_DTYPE;
    if ((j->stream_dtype != j->dtype && j->stream_dtype != FA_F32) ||
        (j->weight_dtype != j->dtype && j->weight_dtype != FA_F32))
        return FA_ERR_DTYPE;
    if (j->rows < 0 || j->rows > kMaxCount || j->cols < 0 || j->cols > FA_JOIN_MAX_COLS)
        return FA_ERR_SIZE;
    if (j->branch) FA_TRY(check_matrix(j->rows, j->cols, j->branch_ld));
    if (j->gate) {
        if (j->groups < 1 || j->rows % j->groups) return FA_ERR_SIZE;
        FA_TRY(check_matrix(j->groups, j->cols, j->gate_ld));
    }
    if ((j->post_norm != 0 && j->post_norm != 1) || !float_ok(j->residual_scale) ||
        !float_ok(j->branch_scale) || !float_ok(j->weight_offset) || !float_ok(j->eps) ||
        !(static_cast<float>(j->eps) > 0.f))
        return FA_ERR_OPTION;
    if (j->dropout) FA_TRY(check_key(j->dropout));
    return FA_OK;
}
// Its device pointers.
fa_status check_join_ptrs(const fa_join *j, int dev) {
    const size_t e = dtype_bytes(j->dtype), w = dtype_bytes(j->weight_dtype);
    if (j->branch) FA_TRY(check_device_ptr(j->branch, dev, e));
    if (j->post_weight) FA_TRY(check_device_ptr(j->post_weight, dev, w));
    if (j->pre_weight) FA_TRY(check_device_ptr(j->pre_weight, dev, w));
    if (j->gate) FA_TRY(check_device_ptr(j->gate, dev, w));
    return j->dropout ? check_key_ptr(j->dropout, dev) : FA_OK;
}
JoinArgs join_args(const fa_join *j) {
    JoinArgs a{};
    a.branch = matrix_args(j->branch, j->rows, j->cols, j->branch_ld);
    a.post_weight = j->post_weight;
    a.pre_weight = j->pre_weight;
    a.gate = j->branch ? j->gate : nullptr;
    a.gate_ld = j->gate_ld;
    a.rows = j->rows;
    a.cols = j->cols;
    a.group_rows = a.gate ? static_cast<uint32_t>(j->rows / j->groups) : 1;
    a.by_group = Divider(a.group_rows);
    a.wide_weights = j->weight_dtype == FA_F32 && j->dtype != FA_F32;
    const auto at16 = [](const void *p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; };
    a.vec_weights = at16(j->post_weight) && at16(j->pre_weight) && at16(a.gate) &&
                    (!a.gate || j->groups == 1 ||
                     j->gate_ld * static_cast<int64_t>(dtype_bytes(j->weight_dtype)) % 16 == 0);
    a.post_norm = j->post_norm && j->branch;
    a.residual_scale = static_cast<float>(j->residual_scale);
    a.branch_scale = static_cast<float>(j->branch_scale);
    a.eps = static_cast<float>(j->eps);
    a.weight_offset = static_cast<float>(j->weight_offset);
    if (j->dropout && j->branch) {
        a.drop = drop_args(j->dropout);
        a.dropped = a.drop.threshold != 0;
    }
    return a;
}

// The host-side rules of a router.
fa_status check_router(const fa_router *x) {
    if (!x) return FA_ERR_NULL;
    if (!valid_dtype(x->dtype)) return FA_ERR_DTYPE;
    FA_TRY(check_matrix(x->tokens, x->experts, x->ld));
    if (x->tokens > kMaxCount || x->experts < 1 || x->experts > FA_ROUTE_MAX_EXPERTS ||
        x->top_k < 1 || x->top_k > x->experts || x->top_k > FA_ROUTE_MAX_CHOSEN)
        return FA_ERR_SIZE;
    if ((x->renormalise != 0 && x->renormalise != 1) || !(x->weight_scale > 0) ||
        !float_ok(x->weight_scale) || !(static_cast<float>(x->weight_scale) >= 0x1p-126f) ||
        !(x->balance_coef >= 0) || !float_ok(x->balance_coef) || !(x->z_coef >= 0) ||
        !float_ok(x->z_coef))
        return FA_ERR_OPTION;
    return FA_OK;
}
fa_status check_router_ptrs(const fa_router *x, int dev) {
    FA_TRY(check_device_ptr(x->logits, dev, dtype_bytes(x->dtype)));
    return x->counted ? check_device_ptr(x->counted, dev, 1) : FA_OK;
}
RouteArgs route_args(const fa_router *x, const fa_routing *r) {
    RouteArgs a{};
    a.logits = matrix_args(x->logits, x->tokens, x->experts, x->ld);
    a.counted = x->counted;
    a.top_k = x->top_k;
    a.renormalise = x->renormalise != 0;
    a.weight_scale = static_cast<float>(x->weight_scale);
    a.balance_coef = static_cast<float>(x->balance_coef);
    a.z_coef = static_cast<float>(x->z_coef);
    a.chosen = r->chosen;
    a.weights = r->weights;
    a.lse = r->lse;
    a.counts = r->counts;
    a.mean_prob = r->mean_prob;
    a.summary = r->summary;
    a.scratch = r->scratch;
    a.plan = route_plan(x->tokens, x->experts);
    return a;
}

}  // namespace

extern "C" {

// ---- dropout -----------------------------------------------------------------------

fa_status fa_dropout(int64_t rows, int64_t cols, const void *x, int64_t x_ld, fa_dtype dtype,
                     const fa_dropout_key *key, void *out, int64_t out_ld, void *stream) {
    if (!valid_dtype(dtype)) return FA_ERR_DTYPE;
    FA_TRY(check_matrix(rows, cols, x_ld));
    FA_TRY(check_matrix(rows, cols, out_ld));
    const int64_t blocks = cols / kDropColumns + (cols % kDropColumns != 0);
    if (rows && blocks > kMaxCount / rows) return FA_ERR_SIZE;
    if (!key) return FA_ERR_NULL;
    FA_TRY(check_key(key));
    if (rows == 0 || cols == 0) return FA_OK;
    int dev;
    FA_TRY(stream_device(stream, &dev));
    const size_t e = dtype_bytes(dtype);
    FA_TRY(check_device_ptr(x, dev, e));
    FA_TRY(check_device_ptr(out, dev, e));
    FA_TRY(check_key_ptr(key, dev));
    const Matrix outs[] = {mat(out, rows, cols, out_ld, e)};
    const Matrix ins[] = {key_vec(key), mat(x, rows, cols, x_ld, e)};
    FA_TRY(check_outputs(outs, 1, ins, x == out && x_ld == out_ld ? 1 : 2));
    TraceRange trace("fa_dropout");
    DropoutArgs a{};
    a.x = matrix_args(x, rows, cols, x_ld);
    a.out = matrix_args(out, rows, cols, out_ld);
    a.drop = drop_args(key);
    return cuda_status(launch_dropout(a, dtype, static_cast<cudaStream_t>(stream)));
}

// ---- the join of a block to the residual stream ------------------------------------------

fa_status fa_block_join(const fa_join *j, const void *residual, int64_t residual_ld, void *out,
                        int64_t out_ld, void *normed, int64_t normed_ld, float *post_rstd,
                        float *pre_rstd, void *stream) {
    FA_TRY(check_join(j));
    FA_TRY(check_matrix(j->rows, j->cols, residual_ld));
    if (out) FA_TRY(check_matrix(j->rows, j->cols, out_ld));
    if (normed) FA_TRY(check_matrix(j->rows, j->cols, normed_ld));
    if (j->rows == 0 || j->cols == 0) return FA_OK;
    int dev;
    FA_TRY(stream_device(stream, &dev));
    const size_t e = dtype_bytes(j->dtype), s = dtype_bytes(j->stream_dtype),
                 w = dtype_bytes(j->weight_dtype);
    FA_TRY(check_join_ptrs(j, dev));
    FA_TRY(check_device_ptr(residual, dev, s));
    if (out) FA_TRY(check_device_ptr(out, dev, s));
    if (normed) FA_TRY(check_device_ptr(normed, dev, e));
    if (post_rstd) FA_TRY(check_device_ptr(post_rstd, dev, 4));
    if (pre_rstd) FA_TRY(check_device_ptr(pre_rstd, dev, 4));
    const Matrix outs[] = {mat(out, j->rows, j->cols, out_ld, s),
                           mat(normed, j->rows, j->cols, normed_ld, e),
                           vec(post_rstd, j->rows * 4), vec(pre_rstd, j->rows * 4)};
    const int64_t c = j->cols;
    const Matrix ins[] = {mat(j->branch, j->rows, c, j->branch_ld, e),
                          vec(j->post_weight, c * static_cast<int64_t>(w)),
                          vec(j->pre_weight, c * static_cast<int64_t>(w)),
                          mat(j->gate, j->groups, c, j->gate_ld, w), key_vec(j->dropout)};
    FA_TRY(check_outputs(outs, 4, ins, 5));
    const Matrix stream_in[] = {mat(residual, j->rows, c, residual_ld, s)};
    // the stream may be joined in place
    const int own = out == residual && out_ld == residual_ld ? 1 : 0;
    FA_TRY(check_outputs(outs + own, 4 - own, stream_in, 1));
    TraceRange trace("fa_block_join");
    JoinArgs a = join_args(j);
    a.residual = matrix_args(residual, j->rows, c, residual_ld);
    a.out = matrix_args(out, j->rows, c, out_ld);
    a.normed = matrix_args(normed, j->rows, c, normed_ld);
    a.post_rstd = post_rstd;
    a.pre_rstd = pre_rstd;
    return cuda_status(launch_block_join(a, j->dtype, j->stream_dtype,
                                         static_cast<cudaStream_t>(stream)));
}

fa_status fa_block_join_scratch(int64_t rows, int64_t cols, int64_t groups, int64_t *bytes) {
    if (!bytes) return FA_ERR_NULL;
    if (rows < 0 || rows > kMaxCount || cols < 0 || cols > FA_JOIN_MAX_COLS || groups < 0)
        return FA_ERR_SIZE;
    *bytes = join_plan(rows, cols, groups, 8).bytes;
    return FA_OK;
}

fa_status fa_block_join_gradient(const fa_join *j, const fa_join_gradient *g, void *stream) {
    FA_TRY(check_join(j));
    if (!g) return FA_ERR_NULL;
    const int64_t rows = j->rows, cols = j->cols;
    const bool pre = g->dnormed != nullptr, post = j->post_norm && j->branch;
    // what is asked for has to be there to have a gradient (of no rows there is nothing)
    if (rows > 0 &&
        ((g->dbranch && !j->branch) || (g->dpost_weight && !(j->post_weight && post)) ||
         (g->dpre_weight && !(j->pre_weight && pre)) ||
         (g->dgate && !(j->gate && j->branch))))
        return FA_ERR_NULL;
    if (g->out) FA_TRY(check_matrix(rows, cols, g->out_ld));
    if (g->dout) FA_TRY(check_matrix(rows, cols, g->dout_ld));
    if (g->dnormed) FA_TRY(check_matrix(rows, cols, g->dnormed_ld));
    if (g->dresidual) FA_TRY(check_matrix(rows, cols, g->dresidual_ld));
    if (g->dbranch) FA_TRY(check_matrix(rows, cols, g->dbranch_ld));
    if (g->dgate) FA_TRY(check_matrix(j->groups, cols, g->dgate_ld));
    if (cols == 0) return FA_OK;
    const int element_bytes =
        2 * static_cast<int>(dtype_bytes(j->dtype) + dtype_bytes(j->stream_dtype));
    const JoinPlan plan = join_plan(rows, cols, g->dgate ? j->groups : 0, element_bytes);
    const bool sums = g->dpost_weight || g->dpre_weight || g->dgate;
    int64_t need = 0;
    FA_TRY(fa_block_join_scratch(rows, cols, g->dgate ? j->groups : 0, &need));
    if (rows > 0 && sums && g->scratch_bytes < need) return FA_ERR_SIZE;
    int dev;
    FA_TRY(stream_device(stream, &dev));
    const size_t e = dtype_bytes(j->dtype), s = dtype_bytes(j->stream_dtype),
                 w = dtype_bytes(j->weight_dtype);
    const int64_t row_bytes = cols * static_cast<int64_t>(w);
    if (g->dpost_weight) FA_TRY(check_device_ptr(g->dpost_weight, dev, w));
    if (g->dpre_weight) FA_TRY(check_device_ptr(g->dpre_weight, dev, w));
    if (g->dgate) FA_TRY(check_device_ptr(g->dgate, dev, w));
    if (rows > 0) {
        FA_TRY(check_join_ptrs(j, dev));
        if (pre) {
            FA_TRY(check_device_ptr(g->dnormed, dev, e));
            FA_TRY(check_device_ptr(g->out, dev, s));
            FA_TRY(check_device_ptr(g->pre_rstd, dev, 4));
        }
        if (post) FA_TRY(check_device_ptr(g->post_rstd, dev, 4));
        if (g->dout) FA_TRY(check_device_ptr(g->dout, dev, s));
        if (g->dresidual) FA_TRY(check_device_ptr(g->dresidual, dev, s));
        if (g->dbranch) FA_TRY(check_device_ptr(g->dbranch, dev, e));
        if (sums) FA_TRY(check_device_ptr(g->scratch, dev, 16));
    }
    const Matrix outs[] = {mat(g->dresidual, rows, cols, g->dresidual_ld, s),
                           mat(g->dbranch, rows, cols, g->dbranch_ld, e),
                           vec(g->dpost_weight, row_bytes),
                           vec(g->dpre_weight, row_bytes),
                           mat(g->dgate, j->groups, cols, g->dgate_ld, w),
                           vec(sums ? g->scratch : nullptr, need)};
    const Matrix ins[] = {mat(j->branch, rows, cols, j->branch_ld, e),
                          mat(pre ? g->out : nullptr, rows, cols, g->out_ld, s),
                          mat(g->dout, rows, cols, g->dout_ld, s),
                          mat(g->dnormed, rows, cols, g->dnormed_ld, e),
                          vec(j->post_weight, row_bytes),
                          vec(j->pre_weight, row_bytes),
                          mat(j->gate, j->groups, cols, j->gate_ld, w),
                          vec(post ? g->post_rstd : nullptr, rows * 4),
                          vec(pre ? g->pre_rstd : nullptr, rows * 4), key_vec(j->dropout)};
    FA_TRY(check_outputs(outs, 6, ins, 10));
    TraceRange trace("fa_block_join_gradient");
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (rows == 0) {  // sums of nothing
        const auto clear = [&](void *p, int64_t ld, int64_t n) {
            return p ? cuda_status(cudaMemset2DAsync(p, ld * w, 0, row_bytes, n, st)) : FA_OK;
        };
        FA_TRY(clear(g->dpost_weight, cols, 1));
        FA_TRY(clear(g->dpre_weight, cols, 1));
        return clear(g->dgate, g->dgate_ld, j->groups);
    }
    JoinGradArgs a{};
    a.j = join_args(j);
    a.j.post_rstd = post ? const_cast<float *>(g->post_rstd) : nullptr;
    a.j.pre_rstd = pre ? const_cast<float *>(g->pre_rstd) : nullptr;
    a.out = matrix_args(pre ? g->out : nullptr, rows, cols, g->out_ld);
    a.dout = matrix_args(g->dout, rows, cols, g->dout_ld);
    a.dnormed = matrix_args(g->dnormed, rows, cols, g->dnormed_ld);
    a.dresidual = matrix_args(g->dresidual, rows, cols, g->dresidual_ld);
    a.dbranch = matrix_args(g->dbranch, rows, cols, g->dbranch_ld);
    a.dpost_weight = g->dpost_weight;
    a.dpre_weight = g->dpre_weight;
    a.dgate = g->dgate;
    a.dgate_ld = g->dgate_ld;
    a.groups = j->groups;
    a.sums = static_cast<float *>(g->scratch);
    a.plan = plan;
    return cuda_status(launch_block_join_gradient(a, j->dtype, j->stream_dtype, st));
}

// ---- the router --------------------------------------------------------------------------

fa_status fa_route_scratch(int64_t tokens, int64_t experts, int64_t *bytes) {
    if (!bytes) return FA_ERR_NULL;
    if (tokens < 0 || tokens > kMaxCount || experts < 0 || experts > FA_ROUTE_MAX_EXPERTS)
        return FA_ERR_SIZE;
    *bytes = route_plan(tokens, experts).bytes;
    return FA_OK;
}

fa_status fa_route(const fa_router *x, const fa_routing *r, void *stream) {
    FA_TRY(check_router(x));
    if (!r) return FA_ERR_NULL;
    const bool loss = r->summary != nullptr;
    if (loss != (r->lse != nullptr) || loss != (r->counts != nullptr) ||
        loss != (r->mean_prob != nullptr) || loss != (r->scratch != nullptr)) {
        if (x->tokens > 0 || !loss || !r->counts || !r->mean_prob) return FA_ERR_NULL;
    }
    if (x->tokens == 0 && !loss) return FA_OK;
    const RoutePlan plan = route_plan(x->tokens, x->experts);
    if (loss && r->scratch_bytes < plan.bytes) return FA_ERR_SIZE;
    int dev;
    FA_TRY(stream_device(stream, &dev));
    if (loss) {
        FA_TRY(check_device_ptr(r->counts, dev, 4));
        FA_TRY(check_device_ptr(r->mean_prob, dev, 4));
        FA_TRY(check_device_ptr(r->summary, dev, 4));
    }
    if (x->tokens > 0) {
        FA_TRY(check_router_ptrs(x, dev));
        FA_TRY(check_device_ptr(r->chosen, dev, 4));
        FA_TRY(check_device_ptr(r->weights, dev, 4));
        if (loss) {
            FA_TRY(check_device_ptr(r->lse, dev, 8));
            FA_TRY(check_device_ptr(r->scratch, dev, 16));
        }
    }
    const int64_t pairs = x->tokens * x->top_k * 4;
    const Matrix outs[] = {vec(r->chosen, pairs), vec(r->weights, pairs),
                           vec(r->lse, x->tokens * 8), vec(r->counts, x->experts * 4),
                           vec(r->mean_prob, x->experts * 4), vec(r->summary, 16),
                           vec(r->scratch, plan.bytes)};
    const Matrix ins[] = {mat(x->logits, x->tokens, x->experts, x->ld, dtype_bytes(x->dtype)),
                          vec(x->counted, x->tokens)};
    FA_TRY(check_outputs(outs, 7, ins, 2));
    TraceRange trace("fa_route");
    return cuda_status(
        launch_route(route_args(x, r), x->dtype, static_cast<cudaStream_t>(stream)));
}

fa_status fa_route_gradient(const fa_router *x, const fa_routing *r, const float *dweights,
                            const float *grad_loss, void *dlogits, int64_t dlogits_ld,
                            void *stream) {
    FA_TRY(check_router(x));
    if (!r) return FA_ERR_NULL;
    FA_TRY(check_matrix(x->tokens, x->experts, dlogits_ld));
    if (x->tokens == 0) return FA_OK;
    int dev;
    FA_TRY(stream_device(stream, &dev));
    FA_TRY(check_router_ptrs(x, dev));
    FA_TRY(check_device_ptr(r->lse, dev, 8));
    FA_TRY(check_device_ptr(r->counts, dev, 4));
    if (dweights) {
        FA_TRY(check_device_ptr(r->chosen, dev, 4));
        FA_TRY(check_device_ptr(r->weights, dev, 4));
        FA_TRY(check_device_ptr(dweights, dev, 4));
    }
    if (grad_loss) FA_TRY(check_device_ptr(grad_loss, dev, 4));
    const size_t e = dtype_bytes(x->dtype);
    FA_TRY(check_device_ptr(dlogits, dev, e));
    const int64_t pairs = x->tokens * x->top_k * 4;
    const Matrix outs[] = {mat(dlogits, x->tokens, x->experts, dlogits_ld, e)};
    const Matrix ins[] = {mat(x->logits, x->tokens, x->experts, x->ld, e),
                          vec(x->counted, x->tokens),
                          vec(r->lse, x->tokens * 8),
                          vec(r->counts, x->experts * 4),
                          vec(dweights ? r->chosen : nullptr, pairs),
                          vec(dweights ? r->weights : nullptr, pairs),
                          vec(dweights, pairs),
                          vec(grad_loss, 4)};
    FA_TRY(check_outputs(outs, 1, ins, 8));
    TraceRange trace("fa_route_gradient");
    RouteGradArgs a{};
    a.r = route_args(x, r);
    a.dweights = dweights;
    a.grad_loss = grad_loss;
    a.dlogits = matrix_args(dlogits, x->tokens, x->experts, dlogits_ld);
    return cuda_status(launch_route_gradient(a, x->dtype, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
