/*
 * fa_model_ops.h -- C ABI of the model-side operators of a training step: the
 * embedding lookup and its gradient, the token log-probabilities with the
 * preference and the clipped policy loss, and the gated activation with its
 * 8-bit checkpoint.  They produce the gradients that fused_adamw.h consumes.
 * The RUDA documentation pages cover the optimizer only: every entry point
 * below is this library's, and the pages have no counterpart to any of them.
 *
 * Contract: as in fused_adamw.h.  Device pointers of the current device (else
 * FA_ERR_POINTER), aligned to their element size (FA_ERR_ALIGN); everything is
 * enqueued on ``stream`` in call order and FA_OK means enqueued; validation
 * comes first, and on any error nothing is enqueued or written; the library
 * allocates nothing, and scratch belongs to the caller (its contents on entry
 * do not matter).  Outputs overlap no other buffer (FA_ERR_ALIAS) unless a
 * call says otherwise.  Every call may be captured into a CUDA graph.
 *
 * Matrices are row-major with unit stride along a row; ``ld`` is the distance
 * between two rows in elements (>= the row's length; FA_ERR_SIZE else).  Rows
 * that start on 16-byte boundaries take 16-byte accesses; others are correct
 * and slower.  Values are FP32, FP16 or BF16 (fa_dtype); sums, softmax
 * statistics and losses are held in FP32, and each 16-bit output is
 * rounded once, to nearest even.  Results do not depend on the order in which
 * blocks run: no floating-point value is added atomically.
 */
#ifndef FA_MODEL_OPS_H
#define FA_MODEL_OPS_H

#include <stdint.h>

#include "fused_adamw.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Type of token ids and labels. */
typedef enum fa_itype { FA_I32 = 0, FA_I64 = 1 } fa_itype;

/* Activations of a gated MLP: x * sigmoid(x), and the tanh form of GELU,
 * x * sigmoid(2 sqrt(2/pi) (x + 0.044715 x^3)). */
typedef enum fa_activation { FA_SILU = 0, FA_GELU_TANH = 1 } fa_activation;

/* Columns that share one scale of an 8-bit checkpoint. */
#define FA_CHECKPOINT_BLOCK 128

/* ---- embedding -------------------------------------------------------------- */

/*
 * out[t, :] = scale * table[ids[t], :] for t < tokens, in FP32, rounded to odt
 * (the pages have no counterpart).  An id outside [0, vocab) gives a row of
 * zeros.  table [vocab, dim] and out [tokens, dim] may have different types.
 * scale is finite.  tokens == 0 or dim == 0: nothing is launched or checked.
 */
fa_status fa_embedding_lookup(int64_t tokens, const void *ids, fa_itype idt, const void *table,
                              fa_dtype tdt, int64_t vocab, int64_t dim, int64_t table_ld,
                              double scale, void *out, fa_dtype odt, int64_t out_ld,
                              void *stream);

/* Scratch of fa_embedding_gradient in bytes, into *bytes (the pages
 * have no counterpart): the tokens sorted by id, and FP32 partial sums of the ids
 * whose tokens several blocks share.  Host only; FA_ERR_SIZE for a negative count, more
 * than 2^31 - 1 tokens, 2^31 - 2 ids or 2^21 columns (of a lookup: the same tokens and
 * columns, and any vocab). */
fa_status fa_embedding_scratch(int64_t tokens, int64_t vocab, int64_t dim, int64_t *bytes);

/*
 * Gradient of fa_embedding_lookup for the table (the pages have no counterpart):
 *   dtable[v, :] = (accumulate ? dtable[v, :] : 0) + scale * sum_{t: ids[t] = v} dout[t, :]
 * Ids outside [0, vocab), and those equal to padding_idx (< 0: none), add
 * nothing.  The tokens are sorted by id first (stable, by the library's own
 * kernels); each id's rows are then added in FP32 in ascending t, in groups
 * whose sums are joined in order, so the result is reproducible bit for bit.
 * accumulate == 0 writes every row of dtable, with zeros for ids that no token
 * has; accumulate == 1 reads and writes only the rows of ids that occur (a
 * parameter bucket's gradient, or a table that is also the output head's).
 * scratch: device memory of at least fa_embedding_scratch's bytes, 16-byte
 * aligned.  vocab == 0 or dim == 0, or accumulate with tokens == 0: nothing is
 * launched or checked.
 */
fa_status fa_embedding_gradient(int64_t tokens, const void *ids, fa_itype idt, const void *dout,
                                fa_dtype ddt, int64_t dout_ld, double scale, int64_t padding_idx,
                                int32_t accumulate, void *dtable, fa_dtype tdt, int64_t vocab,
                                int64_t dim, int64_t table_ld, void *scratch,
                                int64_t scratch_bytes, void *stream);

/* ---- losses from the logits ---------------------------------------------------- */

/* Logits of a batch of tokens with their labels: row t is a distribution over
 * vocab ids after multiplication by logit_scale (an inverse temperature, from 1e-4
 * to 1e4).  A label outside [0, vocab) marks a token that is not counted (a prompt,
 * padding): its row is never read, so it may hold anything.  -Inf logits have
 * probability zero; a row with no finite logit, or with a NaN or +Inf, gives NaN. */
typedef struct fa_logits {
    int64_t tokens;
    int64_t vocab;
    const void *logits;  /* device, [tokens, vocab] of type dtype */
    fa_dtype dtype;
    int64_t ld;
    const void *labels;  /* device, [tokens] */
    fa_itype ltype;
    double logit_scale;
} fa_logits;

/*
 * logp[t] = log softmax(logit_scale * logits[t])[labels[t]], FP32 (the pages have
 * no counterpart); 0 for a token that is not counted.  lse (FP32 [tokens][2], may
 * be NULL; 8-byte aligned) receives the row's log-sum-exp in two parts (m, s), as the
 * gradient takes it: logit_scale * m + ln(s), with m the row's largest logit; (0, 1)
 * for a token that is not counted.  tokens == 0: nothing is launched
 * or checked.  vocab >= 1 else.
 */
fa_status fa_token_logprobs(const fa_logits *x, float *logp, float *lse, void *stream);

/*
 * Gradient of fa_token_logprobs (the pages have no counterpart):
 *   dlogits[t, v] = c * (1[v = labels[t]] - softmax(logit_scale * logits[t])[v]),
 *   c = dlogp[t] * logit_scale * grad_scale * (grad_loss ? *grad_loss : 1)
 * and zeros for a token that is not counted.  lse as fa_token_logprobs wrote it;
 * dlogp FP32 [tokens]; grad_scale finite (a loss scale); grad_loss a device FP32
 * scalar or NULL.  dlogits has the logits' type; it may be the logits themselves
 * (same pointer and ld) and must not overlap them otherwise.
 */
fa_status fa_token_logprobs_gradient(const fa_logits *x, const float *lse, const float *dlogp,
                                     double grad_scale, const float *grad_loss, void *dlogits,
                                     int64_t dlogits_ld, void *stream);

/* Arguments of fa_preference_loss besides the logits. */
typedef struct fa_preference {
    int64_t pairs;
    const int64_t *seq_offsets; /* device, 2 * pairs + 1 offsets into the tokens, non-decreasing;
                                   sequence 2k was preferred to sequence 2k + 1 */
    const float *ref_logp;      /* device, [tokens]: the reference model's log-probabilities */
    double beta;                /* > 0, finite */
    double label_smoothing;     /* in [0, 0.5]: probability that a preference is the wrong way */
    int32_t average;            /* 1: a sequence counts with its mean over tokens, not the sum */
    float *loss;                /* device outputs: [1] the mean over the pairs (0 for none),  */
    float *pair_loss;           /* [pairs],                                                   */
    float *rewards;             /* [pairs][2]: beta * log ratio of the preferred, the other,  */
    float *logp;                /* [tokens] and                                               */
    float *lse;                 /* [tokens][2]: as fa_token_logprobs,                         */
    float *dlogp;               /* [tokens]: dloss / dlogp, for fa_token_logprobs_gradient    */
} fa_preference;

/*
 * Preference loss from paired log ratios (the pages have no counterpart): with
 *   s_j = sum (or mean) over the counted tokens of sequence j of (logp - ref_logp),
 *   z_k = beta * (s_2k - s_2k+1),
 *   pair_loss_k = -(1 - e) log sigmoid(z_k) - e log sigmoid(-z_k),  e = label_smoothing.
 * Sums over tokens and pairs are held as an FP32 value and its residual.  A
 * sequence without a counted token has s = 0.  Offsets are clamped to [0, tokens]; tokens of no sequence have
 * dlogp 0.  pairs == 0 or tokens == 0 are allowed.
 */
fa_status fa_preference_loss(const fa_logits *x, const fa_preference *a, void *stream);

/* Arguments of fa_policy_loss besides the logits; [tokens] FP32 on the device. */
typedef struct fa_policy {
    const float *old_logp;    /* log-probabilities under the policy that drew the tokens     */
    const float *advantages;
    const float *ref_logp;    /* the reference model's, or NULL (then kl_coef must be 0)      */
    const float *weights;     /* a weight per token, or NULL (1)                              */
    double clip_low;          /* in [0, 1]                                                   */
    double clip_high;         /* >= 0, finite                                                */
    double kl_coef;           /* >= 0, finite                                                */
    double denominator;       /* the weighted sum's divisor; 0: the number of counted tokens */
    double grad_scale;        /* a loss scale on dlogits (finite)                            */
    float *summary;           /* [4]: the loss, the mean KL term and the clipped share over  */
                              /* the counted tokens, and their number                        */
    float *logp;              /* [tokens], as fa_token_logprobs                               */
    float *token_loss;        /* [tokens], 0 where not counted                                */
    float *token_kl;          /* [tokens], 0 where not counted                                */
    float *lse;               /* [tokens][2] as fa_token_logprobs, or NULL                    */
    float *dlogp;             /* [tokens]: dloss / dlogp, or NULL: with lse, the gradient can */
                              /* be taken later, by fa_token_logprobs_gradient                */
    void *dlogits;            /* [tokens, vocab] of the logits' type, or NULL: no gradient;   */
    int64_t dlogits_ld;       /* may be the logits themselves (same pointer and ld)           */
} fa_policy;

/*
 * Clipped policy loss with a KL term, and its gradient in the same pass (the pages
 * have no counterpart): with r = exp(logp - old_logp), A the advantage, d = ref_logp
 * - logp,
 *   token_kl = exp(d) - d - 1 (infinite where d is),
 *   token_loss = -min(r A, clamp(r, 1 - clip_low, 1 + clip_high) A) + kl_coef * token_kl,
 *   loss = sum_t weights_t * token_loss_t / denominator,
 *   dlogits as fa_token_logprobs_gradient with dlogp = weights / denominator *
 *     (kl_coef * (1 - exp(d)) - (r A where r A <= the clamped product, else 0)).
 * A token whose clamped product is the smaller counts as clipped.  A token with
 * advantage or weight 0 adds nothing by it where its ratio, its loss or its slope is
 * infinite (past FP32, or a label whose logit is -Inf); a NaN stays.  Sums over
 * tokens are held as an FP32 value and its residual.  The logits are read once.  tokens == 0: summary 0.
 */
fa_status fa_policy_loss(const fa_logits *x, const fa_policy *a, void *stream);

/* ---- gated activation with an 8-bit checkpoint ------------------------------------ */

/* Size of the checkpoint of a [rows, cols] gated activation (the pages
 * have no counterpart): its codes in bytes, 2 * rows * pitch with pitch = cols rounded up to
 * 128 (gate [rows, pitch], then up), and its scales in FP32 elements, 2 * rows *
 * pitch / 128 (in the same order).  Host only; FA_ERR_SIZE for a negative count or
 * more than 2^28 blocks (rows * pitch / 128), which the calls below refuse too. */
fa_status fa_checkpoint_size(int64_t rows, int64_t cols, int64_t *code_bytes,
                             int64_t *scale_elements);

/*
 * h = act(gate) * up (in FP32, rounded to the type), keeping gate and up as an 8-bit
 * checkpoint for the backward pass (the pages have no counterpart).  Each 128
 * consecutive columns of a row are one block: with a its largest magnitude,
 *   scale = a / 127,  code = rint(x * (127 / a))
 * in FP32 (ties to even), so a code stands for code * scale, within a / 254 of x (and
 * FP32 rounding, by which 127 * scale is infinite where a is FP32's largest number).  A block with a < 2^-100 is stored as zeros; one with a NaN or an
 * infinity has scale NaN, so that what the backward pass makes of it is NaN and the
 * gradient statistics skip the step.  The sigmoid's values below 2^-126 count as
 * zero: act and act' are 0 for silu gates below -87.3 (|act| < 1.1e-36 there) and tanh-GELU
 * gates below -10 (1.2e-37).  Columns past cols hold code 0.  codes NULL (and
 * scales NULL): no checkpoint is kept.  gate and up may be halves of one matrix.
 * rows == 0 or cols == 0: nothing is launched or checked.
 */
fa_status fa_gated_forward(int64_t rows, int64_t cols, const void *gate, int64_t gate_ld,
                           const void *up, int64_t up_ld, fa_dtype dtype,
                           fa_activation activation, void *h, int64_t h_ld, int8_t *codes,
                           float *scales, void *stream);

/*
 * Backward of fa_gated_forward from the checkpoint (the pages have no counterpart):
 * with g and u the values that the codes stand for,
 *   dgate = dh * u * act'(g),  dup = dh * act(g),
 * and, where h is not NULL, h = act(g) * u again (what the weight gradient of the
 * projection after it needs).  codes are 16-byte aligned, scales 4-byte.
 */
fa_status fa_gated_backward(int64_t rows, int64_t cols, const int8_t *codes, const float *scales,
                            fa_activation activation, const void *dh, int64_t dh_ld,
                            fa_dtype dtype, void *dgate, int64_t dgate_ld, void *dup,
                            int64_t dup_ld, void *h, int64_t h_ld, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* FA_MODEL_OPS_H */
