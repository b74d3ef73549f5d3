/*
 * fa_block_ops.h -- C ABI of the operators of a model's residual blocks: the join of a
 * block's output to the residual stream with the norms behind and before it, dropout
 * from a counter-based generator, and the router of gated experts with its balance
 * loss.  Each comes with its gradient.  The RUDA documentation pages cover the
 * optimizer only: every entry point below is this library's, and the pages have no
 * counterpart to any of them.
 *
 * Contract: as in fa_model_ops.h (device pointers of the current device, validation
 * first, the caller owns every buffer, outputs overlap no other buffer unless a call
 * says otherwise, matrices are row-major with unit stride along a row and distance
 * ``ld`` between rows, FP32 arithmetic, no floating-point value is added atomically,
 * every call may be captured into a CUDA graph).
 */
#ifndef FA_BLOCK_OPS_H
#define FA_BLOCK_OPS_H

#include <stdint.h>

#include "fa_model_ops.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ---- dropout ------------------------------------------------------------------- */

/*
 * Which elements of a [rows, cols] matrix a dropout keeps.  Element (t, c) has the
 * 16 bits number c % 8 (bits 16 * (c % 2) of word (c % 8) / 2) of the Philox 4x32-10
 * block (Salmon, Moraes, Dror and Shaw, "Parallel random numbers: as easy as 1, 2, 3",
 * 2011) with key ``seed`` and counter (t * ceil(cols / 8) + c / 8, offset + *counter),
 * 64 bits each, low words first.  With q = rint(65536 * p) it is kept where they are
 * q at least, and then multiplied by 65536 / (65536 - q): p is a multiple of 2^-16, and
 * the mean is kept for it exactly.  A dropped element is 0 whatever it was.  The mask
 * depends on the element's place in the matrix alone, not on the layout, so that the same
 * record gives it again to the backward pass.
 */
typedef struct fa_dropout_key {
    double p;                /* in [0, 1] */
    uint64_t seed;
    uint64_t offset;         /* the call's own: two calls with the same drop the same places */
    const uint64_t *counter; /* device scalar added to offset (modulo 2^64), or NULL: what a
                                captured graph reads anew in every replay */
} fa_dropout_key;

/*
 * out = x with dropped elements 0 and the others multiplied, in FP32, rounded to the type
 * (the pages have no counterpart).  The gradient is the same call on the
 * output's gradient.  out may be x itself (same pointer and ld).  rows == 0 or
 * cols == 0: nothing is launched or checked.  FA_ERR_SIZE for more than 2^31 - 1 blocks
 * of 128 columns (rows * ceil(cols / 128)).
 */
fa_status fa_dropout(int64_t rows, int64_t cols, const void *x, int64_t x_ld, fa_dtype dtype,
                     const fa_dropout_key *key, void *out, int64_t out_ld, void *stream);

/* ---- the join of a block to the residual stream ------------------------------------ */

/* Columns that a join takes at most. */
#define FA_JOIN_MAX_COLS 16384

/*
 * A join: with r a row of the residual stream, y of the block's output (the branch),
 *   yh   = y / sqrt(mean(y^2) + eps)
 *   b    = (post_weight + weight_offset) * yh   (post_norm; b = y without)
 *   out  = residual_scale * r + branch_scale * gate * D(b), rounded to the stream's type
 *   xh   = out / sqrt(mean(out^2) + eps)
 *   normed = (pre_weight + weight_offset) * xh
 * D drops elements (see fa_dropout_key; NULL: none).  The second norm is that of ``out``
 * as it is stored, so it can be taken again from it bit for bit (a join without a branch, of the same
 * rows in matrices that lie alike: of one row distance, from 16-byte boundaries).
 * Weights that are NULL are 1 (and have no offset added).
 */
typedef struct fa_join {
    int64_t rows;
    int64_t cols;               /* at most FA_JOIN_MAX_COLS */
    fa_dtype dtype;             /* of branch, normed and their gradients */
    fa_dtype stream_dtype;      /* of residual, out and their gradients: dtype, or FA_F32 */
    fa_dtype weight_dtype;      /* of the weights, the gate and their gradients: dtype or FA_F32 */
    int32_t post_norm;          /* 1: the branch is normed before it is added */
    const void *branch;         /* [rows, cols], or NULL: out = residual_scale * residual */
    int64_t branch_ld;
    const void *post_weight;    /* [cols] or NULL */
    const void *pre_weight;     /* [cols] or NULL */
    const void *gate;           /* [groups, cols], or NULL: 1.  Row t takes row t / (rows / groups) */
    int64_t gate_ld;
    int64_t groups;             /* a divisor of rows: 1 for a gate per channel, the number of equally
                                   long sequences for one per sequence, rows for one per token */
    double residual_scale;      /* finite */
    double branch_scale;        /* finite */
    double eps;                 /* > 0, finite */
    double weight_offset;       /* finite: 1 for weights stored around 0 */
    const fa_dropout_key *dropout;
} fa_join;

/*
 * The join (the pages have no counterpart).  out NULL: the stream is not written (a last
 * norm); normed NULL: there is no second norm.  out may be the residual itself (same
 * pointer and ld).  post_rstd and pre_rstd (FP32 [rows], or NULL) receive the inverse
 * roots, which the gradient takes.  A row whose squares pass FP32 is normed all the same.
 * rows == 0 or cols == 0: nothing is launched or checked.
 */
fa_status fa_block_join(const fa_join *j, const void *residual, int64_t residual_ld, void *out,
                        int64_t out_ld, void *normed, int64_t normed_ld, float *post_rstd,
                        float *pre_rstd, void *stream);

/* Scratch of fa_block_join_gradient in bytes, into *bytes (the pages have no counterpart):
 * FP32 sums of the columns' gradients.  groups: the gate's, 0 for none.  Host only;
 * FA_ERR_SIZE as for the gradient. */
fa_status fa_block_join_scratch(int64_t rows, int64_t cols, int64_t groups, int64_t *bytes);

/* Gradients of a join. */
typedef struct fa_join_gradient {
    const void *out;            /* the stream as the join stored it; NULL without a second norm */
    int64_t out_ld;
    const float *post_rstd;     /* as the join wrote them; NULL without that norm */
    const float *pre_rstd;
    const void *dout;           /* gradient of out, or NULL: 0 */
    int64_t dout_ld;
    const void *dnormed;        /* gradient of normed, or NULL: there is no second norm */
    int64_t dnormed_ld;
    void *dresidual;            /* gradient of the residual, or NULL */
    int64_t dresidual_ld;
    void *dbranch;              /* gradient of the branch, or NULL */
    int64_t dbranch_ld;
    void *dpost_weight;         /* [cols] or NULL */
    void *dpre_weight;          /* [cols] or NULL */
    void *dgate;                /* [groups, cols] or NULL */
    int64_t dgate_ld;
    void *scratch;              /* fa_block_join_scratch's bytes, 16-byte aligned; NULL where none */
    int64_t scratch_bytes;      /* of the three gradients above is asked for                       */
} fa_join_gradient;

/*
 * Gradients of fa_block_join (the pages have no counterpart): with G the gradient of out
 * in all,
 *   d = dnormed * (pre_weight + weight_offset),  G = dout + pre_rstd * (d - xh * mean(d * xh))
 *   dresidual = residual_scale * G,  db = branch_scale * gate * D(G)
 *   dgate = sum over the group's rows of branch_scale * D(b) * G
 *   dpre_weight = sum of dnormed * xh,  dpost_weight = sum of db * yh
 *   dbranch = post_rstd * (e - yh * mean(e * yh)),  e = db * (post_weight + weight_offset)
 * (dbranch = db without the first norm: a dropped element then has no gradient, whatever the
 * branch holds there; with the norm it is part of its row's mean, forward and back).  Sums over rows are FP32, in groups whose sums are joined in order:
 * reproducible bit for bit.  Weights' gradients are written, not added to.  rows == 0:
 * they are set to 0; cols == 0: nothing is launched or checked.
 */
fa_status fa_block_join_gradient(const fa_join *j, const fa_join_gradient *g, void *stream);

/* ---- the router of gated experts --------------------------------------------------- */

#define FA_ROUTE_MAX_EXPERTS 1024
#define FA_ROUTE_MAX_CHOSEN 32

/*
 * Routing of tokens to experts from their logits: with p = softmax(logits[t]), a token
 * takes the top_k experts with the largest logits (of equal ones, those with the lower
 * index first; NaN counts as the largest), in that order, with weights
 *   w_j = weight_scale * p_j   (/ the sum of the chosen p with renormalise)
 * A token with counted[t] == 0 (padding) has chosen -1 and weights 0, and its row is
 * never read.  With n the number of counted tokens, f_e = counts_e / (n top_k) and
 * P_e the mean of p_e over them:
 *   balance = experts * sum_e f_e P_e          (1 where the load is even)
 *   z       = mean of (log sum exp logits)^2
 *   loss    = balance_coef * balance + z_coef * z      (0 where no token is counted)
 * -Inf logits have probability zero (and weight 0 if chosen for want of others); a row
 * with no finite logit, or with a NaN or +Inf, gives NaN.
 */
typedef struct fa_router {
    int64_t tokens;
    int64_t experts;          /* 1 to FA_ROUTE_MAX_EXPERTS */
    const void *logits;       /* device, [tokens, experts] of type dtype */
    fa_dtype dtype;
    int64_t ld;
    const uint8_t *counted;   /* device, [tokens], or NULL: every token counts */
    int32_t top_k;            /* 1 to the experts, at most FA_ROUTE_MAX_CHOSEN */
    int32_t renormalise;      /* 0 or 1 */
    double weight_scale;      /* > 0, finite */
    double balance_coef;      /* >= 0, finite */
    double z_coef;            /* >= 0, finite */
} fa_router;

/* Outputs of fa_route.  summary, counts, mean_prob, lse and scratch may be NULL together:
 * a pass that takes no loss and keeps nothing for a gradient. */
typedef struct fa_routing {
    int32_t *chosen;          /* device, [tokens][top_k] */
    float *weights;           /* [tokens][top_k] */
    float *lse;               /* [tokens][2] the log-sum-exp as m + ln(s), 8-byte aligned */
    int32_t *counts;          /* [experts] tokens that chose each */
    float *mean_prob;         /* [experts] P */
    float *summary;           /* [4]: loss, balance, z, counted tokens */
    void *scratch;            /* fa_route_scratch's bytes, 16-byte aligned */
    int64_t scratch_bytes;
} fa_routing;

/* Scratch of fa_route in bytes, into *bytes (the pages have no counterpart).  Host only;
 * FA_ERR_SIZE for a negative count, more than 2^31 - 1 tokens or too many experts. */
fa_status fa_route_scratch(int64_t tokens, int64_t experts, int64_t *bytes);

/* Experts, weights, counts and losses (the pages have no counterpart).  Sums over tokens
 * are FP32, joined in order.  tokens == 0: counts, mean_prob and summary are set to 0. */
fa_status fa_route(const fa_router *x, const fa_routing *r, void *stream);

/*
 * Gradient of fa_route for the logits (the pages have no counterpart), from what it wrote:
 * that of grad_loss * loss + sum of dweights * weights.  The counts have no gradient.
 *   dlogits_e = p_e * grad_loss * (balance_coef * experts / n * (f_e - sum f p)
 *                                  + z_coef * 2 lse / n) + the weights' part,
 * zeros for a token that is not counted.  dweights FP32 [tokens][top_k] or NULL; grad_loss
 * a device FP32 scalar, or NULL: the loss has no gradient.  dlogits has the logits' type.
 * r's chosen, weights, lse and counts are read, and nothing else of it.  tokens == 0: nothing is launched or checked.
 */
fa_status fa_route_gradient(const fa_router *x, const fa_routing *r, const float *dweights,
                            const float *grad_loss, void *dlogits, int64_t dlogits_ld,
                            void *stream);

#ifdef __cplusplus
}
#endif

#endif /* FA_BLOCK_OPS_H */
