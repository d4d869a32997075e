/*
 * adamw_losses.h -- C ABI of the fine-tuning operators that feed the AdamW
 * step: per-token log-probabilities from logits, the clipped policy loss with
 * a KL term, the preference loss over pairs, each with its gradient, and the
 * clip of a list of gradients by their global norm.
 *
 * Together they are what happens between a model's logits and adamw_step:
 *     logits -> token log-probabilities -> preference loss -> their gradient,
 *     logits -> policy loss and the logits' gradient in one pass, and
 *     gradients (of any of three types, of every parameter group) -> one
 *     global norm -> the clipped gradients that the step reads.
 *
 * Conventions, as in adamw_sm.h: every entry point is asynchronous on the
 * given stream of the current device unless stated, returns one of the
 * ADAMW_* status codes, and launches nothing when it returns an error that
 * its arguments caused.  Buffers belong to the caller and are not kept.
 * Pointers are not looked up (a call costs microseconds): they must be
 * dereferenceable by the current device.  Two calls may run at the same time
 * when they share no output and no workspace.
 *
 * Values: sums, softmax statistics and gradients are computed in fp32 or
 * more and rounded once, to nearest even, when they are stored.
 */
#ifndef ADAMW_LOSSES_H
#define ADAMW_LOSSES_H

#include "adamw_sm.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Element types of logits and gradients. */
#define ADAMW_DTYPE_BF16 0
#define ADAMW_DTYPE_FP16 1
#define ADAMW_DTYPE_FP32 2

/* A matrix of `rows` rows of `cols` elements (the vocabulary), in two levels
 * of strides, so that a view such as logits[:, :-1] of a [batch, tokens,
 * vocabulary] tensor needs no copy: row r starts at element
 * (r / inner) * outer_stride + (r % inner) * row_stride of `data`.  The
 * elements of a row are consecutive.  Strides are in elements and not
 * negative; inner >= 1 divides rows.  rows and cols up to 2^31 - 1; offsets
 * are 64-bit.  Rows at any element alignment are accepted; rows whose
 * addresses have the same remainder modulo 16 bytes in the logits and in
 * their gradient take 16-byte accesses in both. */
typedef struct {
    void* data;
    int64_t rows;
    int64_t inner;
    int64_t outer_stride;
    int64_t row_stride;
    int32_t cols;
    int32_t dtype; /* ADAMW_DTYPE_* */
} adamw_rows_t;

/* Log-probability of one target per row under the softmax of the row.
 *
 * With x_j = scale * logits[r][j] (scale = 1 / temperature, > 0), m the
 * largest x_j and s = sum_j exp(x_j - m):
 *     logp[r]    = x_t - m - log(s),  t = targets[r]
 *     entropy[r] = log(s) - sum_j exp(x_j - m) (x_j - m) / s
 *     stats[r]   = what the backward pass needs: the row's largest logit and
 *                  its sum relative to it.
 * targets: device int64, one per row.  A row whose target is ignore_index is
 *   not read: logp 0, entropy 0, no gradient.  A target outside [0, cols)
 *   gives NaN for the row and its gradient (a step whose gradients hold NaN
 *   is what the optimizer's non-finite flag reports).
 * Logits of -inf (masked entries) have probability 0 and take no part in the
 *   entropy; masks by finite numbers are ordinary logits, a row of one such
 *   number throughout is uniform.  A row that is -inf throughout has no distribution: logp -inf,
 *   entropy 0, gradient 0.  A +inf or NaN logit gives NaN.
 * logp: device fp32 [rows].  entropy: device fp32 [rows] or NULL.  stats:
 *   device fp32 [rows][2], 8-byte aligned, or NULL when no backward follows.
 * Errors: INVALID_ARG (NULL logits, targets or logp with rows > 0, negative
 * or inconsistent sizes or strides, unknown dtype, scale not positive and
 * finite), MISALIGNED, TOO_LARGE (rows above 2^31 - 1, a stride above 2^40),
 * CUDA. */
int adamw_token_logprob(const adamw_rows_t* logits, const int64_t* targets, int64_t ignore_index,
                        float scale, float* logp, float* entropy, float* stats,
                        adamw_stream_t stream);

/* The gradient of adamw_token_logprob with respect to the logits:
 *     d_logits[r][j] = scale * (d_logp[r] ([j = t] - p_j)
 *                               - d_entropy[r] p_j (log p_j + entropy[r]))
 * stats: as written by the forward call with the same logits, targets,
 *   ignore_index and scale.
 * d_logp: fp32 [rows].  d_entropy: fp32 [rows] or NULL; then entropy (the
 *   forward's) is required too.
 * d_logits: the same rows, cols and dtype as logits, rows not overlapping;
 *   may be the logits themselves (same data and strides: in place) but must
 *   not overlap them otherwise.  Every element of the rows is written, zeros
 *   for ignored rows.
 * Errors: as adamw_token_logprob. */
int adamw_token_logprob_backward(const adamw_rows_t* logits, const int64_t* targets,
                                 int64_t ignore_index, float scale, const float* stats,
                                 const float* entropy, const float* d_logp,
                                 const float* d_entropy, const adamw_rows_t* d_logits,
                                 adamw_stream_t stream);

/* How a flat array of n tokens is cut into sequences.
 * offsets: device int64 [sequences + 1], ascending: sequence i is tokens
 *   offsets[i] .. offsets[i + 1] - 1 (it may be empty; tokens outside every
 *   sequence do not count); or NULL: n / sequences tokens each.
 * mask: device bytes [n], 0 = the token does not count, or NULL.  Values at
 *   tokens that do not count are not used, whatever they hold; their
 *   gradients are 0.
 * n up to 2^31 - 1. */
typedef struct {
    int64_t n;
    int64_t sequences;
    const int64_t* offsets;
    const uint8_t* mask;
} adamw_tokens_t;

/* KL estimators of adamw_policy_t, k = logp - ref_logp. */
#define ADAMW_KL_K1 1 /* k                  */
#define ADAMW_KL_K2 2 /* k^2 / 2            */
#define ADAMW_KL_K3 3 /* exp(-k) - 1 + k    */
/* Token weights w of adamw_policy_t. */
#define ADAMW_REDUCE_TOKEN 0    /* 1 / tokens that count                          */
#define ADAMW_REDUCE_SEQUENCE 1 /* 1 / (its sequence's tokens * non-empty sequences) */
#define ADAMW_REDUCE_FIXED 2    /* 1 / divisor                                    */

/* The clipped policy loss.  Per token that counts, with d = logp - old_logp,
 * r = exp(d) and advantage A:
 *     clipped r: 1 + clip_high where d > log(1 + clip_high), 1 - clip_low
 *       where d < log(1 - clip_low), else r
 *     pg = max(-A r, -A clipped r), and with dual_clip c > 1 and A < 0 at
 *       most -A c
 *     loss = sum w (pg + kl_coef KL - entropy_coef entropy)
 * The comparisons are on d, so the gradient is 0 exactly where the clipped
 * branch holds: A > 0 and d > log(1 + clip_high), A < 0 and d < log(1 -
 * clip_low), A < 0 and d > log(c).  A token with A = 0 has pg = 0, past fp32's
 * range of r too. */
typedef struct {
    float clip_low;     /* in [0, 1]                                   */
    float clip_high;    /* >= 0                                        */
    float dual_clip;    /* 0 (off) or > 1                              */
    float kl_coef;      /* any finite; needs ref_logp when not 0       */
    float entropy_coef; /* any finite; needs the entropy when not 0    */
    float divisor;      /* ADAMW_REDUCE_FIXED: > 0                     */
    float grad_scale;   /* multiplies the gradients, not the statistics */
    int32_t kl;         /* ADAMW_KL_*                                  */
    int32_t reduce;     /* ADAMW_REDUCE_*                              */
    int32_t advantage_per_token; /* 1: advantages [n], 0: [sequences]  */
} adamw_policy_t;

/* Loss, statistics and gradients from log-probabilities.
 * logp, old_logp: fp32 [n]; ref_logp, entropy: fp32 [n] or NULL; advantages.
 * stats: fp32 [6]: loss, and the weighted means (weights w) of pg, the KL
 *   estimate (0 without ref_logp), the entropy (0 without), tokens whose
 *   gradient the clip removed, and r - 1 - d (the KL from the old policy).
 * counts: int64 [2]: tokens that count, sequences with at least one.
 * d_logp: fp32 [n]; d_entropy: fp32 [n], or NULL (required with entropy and
 *   entropy_coef != 0).
 * workspace: adamw_policy_workspace(n, sequences) bytes of device memory,
 *   16-byte aligned, contents undefined before and after.
 * Sums run in a fixed order: the same call gives the same bits.
 * Errors: INVALID_ARG, MISALIGNED, TOO_LARGE (n or sequences above 2^31 - 1),
 * CUDA. */
int adamw_policy_loss(const adamw_tokens_t* tokens, const adamw_policy_t* policy,
                      const float* logp, const float* old_logp, const float* ref_logp,
                      const float* advantages, const float* entropy, float* stats,
                      int64_t* counts, float* d_logp, float* d_entropy, void* workspace,
                      adamw_stream_t stream);
/* Bytes of workspace, 0 for sizes that the call refuses. */
int64_t adamw_policy_workspace(int64_t n, int64_t sequences);

/* The same loss from logits, with the logits' gradient, in one pass over the
 * logits: a row stays on chip between its softmax sums and its gradient, so
 * the logits are read once and the gradient written once (rows above 8 times
 * 200 KB take adamw_token_logprob, adamw_policy_loss and the backward pass
 * instead, inside this call).
 * tokens->n = logits->rows; tokens->mask must be NULL: a token counts unless
 *   its target is ignore_index.  scale as in adamw_token_logprob.
 * logp: fp32 [n], written.  entropy: fp32 [n], written, or NULL (required
 *   when entropy_coef != 0).
 * d_logits: as in adamw_token_logprob_backward.
 * workspace: adamw_policy_logits_workspace(n, sequences) bytes.
 * Errors: as above. */
int adamw_policy_loss_logits(const adamw_rows_t* logits, const int64_t* targets,
                             int64_t ignore_index, float scale, const adamw_tokens_t* tokens,
                             const adamw_policy_t* policy, const float* old_logp,
                             const float* ref_logp, const float* advantages, float* stats,
                             int64_t* counts, float* logp, float* entropy,
                             const adamw_rows_t* d_logits, void* workspace,
                             adamw_stream_t stream);
int64_t adamw_policy_logits_workspace(int64_t n, int64_t sequences);

/* Preference losses. */
#define ADAMW_PREF_SIGMOID 0 /* -(1-e) log sigmoid(h) - e log sigmoid(-h)   */
#define ADAMW_PREF_HINGE 1   /* max(0, 1 - h)                               */
#define ADAMW_PREF_IPO 2     /* (D - 1 / (2 beta))^2                        */
/* The reference's log-probabilities. */
#define ADAMW_REF_NONE 0
#define ADAMW_REF_TOKEN 1    /* fp32 [n]            */
#define ADAMW_REF_SEQUENCE 2 /* fp32 [sequences]: each sequence's sum */
typedef struct {
    float beta;            /* > 0                                        */
    float margin;          /* subtracted from beta D (0 with IPO)        */
    float label_smoothing; /* e in [0, 0.5], sigmoid only                */
    float grad_scale;      /* multiplies the gradient only               */
    int32_t kind;          /* ADAMW_PREF_*                               */
    int32_t length_average;/* 1: each sequence's sum over its tokens that count */
    int32_t ref;           /* ADAMW_REF_*                                */
} adamw_preference_t;

/* The loss over pairs of sequences: of 2 B sequences, i is preferred over
 * B + i.  S = sum over a sequence's tokens that count of (logp - ref), or its
 * mean (length_average); D = S_i - S_{B+i}, h = beta D - margin; the loss is
 * the mean over the B pairs.
 * stats: fp32 [3]: loss, share of pairs with D > 0, mean of h.
 * D is the difference of the error-free sums, rounded once.
 * losses: fp32 [B].  rewards: fp32 [2 B], beta S.  d_logp: fp32 [n].
 * A sequence with no token that counts has S = 0 (less its reference's sum).
 * Errors: INVALID_ARG (an odd or zero number of sequences among them),
 * MISALIGNED, TOO_LARGE, CUDA. */
int adamw_preference_loss(const adamw_tokens_t* tokens, const adamw_preference_t* pref,
                          const float* logp, const float* ref_logp, float* stats, float* losses,
                          float* rewards, float* d_logp, adamw_stream_t stream);

/* One gradient of a list to clip.  src is read; dst receives the clipped
 * gradient, rounded to dst_dtype: another buffer, src itself (in place; then
 * the types must be equal), or NULL (only the norm is wanted).  numel may be
 * 0.  Buffers of different entries must not overlap, those that are only read
 * among them (a gradient listed twice would count twice).  They are aligned to
 * their element size; tensors whose src and dst are 16-byte aligned take
 * 16-byte accesses. */
typedef struct {
    const void* src;
    void* dst;
    int64_t numel;
    int32_t src_dtype;
    int32_t dst_dtype;
} adamw_grad_t;

/* Norms of adamw_clip_grads. */
#define ADAMW_NORM_L2 0
#define ADAMW_NORM_MAX 1

/* What adamw_clip_grads writes, in device memory. */
typedef struct {
    float norm;        /* the global norm, rounded once to fp32 (infinity
                          where a finite norm is above fp32's range; coef is
                          still its own)                                    */
    float coef;        /* min(1, max_norm / (norm + 1e-6)); 1 for a
                          non-finite norm                                   */
    int32_t nonfinite; /* 1 when a gradient is inf or NaN                    */
    int32_t pad_;
} adamw_clip_result_t;

typedef struct adamw_clip_plan* adamw_clip_plan_t;

/* Builds a plan over a list of gradients on the current device: checks the
 * list, cuts it into tiles, uploads their table and allocates the norm's
 * workspace.  Synchronous.  Used from one host thread at a time; calls on one
 * plan must not overlap on the GPU.
 * Errors: INVALID_ARG (NULL out or table with n > 0, n < 0, numel < 0, NULL
 * src with numel > 0, unknown dtype, dst overlapping src without being it, in
 * place with two types, buffers of two entries that overlap), MISALIGNED, NOT_ACCESSIBLE, TOO_LARGE (more than
 * 2^40 elements), CUDA. */
int adamw_clip_plan_create(const adamw_grad_t* host_table, int32_t n, adamw_clip_plan_t* out);

/* Clips the plan's gradients by their global norm: dst = coef * src for every
 * tensor with a dst (rounded once; coef 1 copies the values, and an in-place
 * tensor is then not touched).  A non-finite gradient leaves coef 1, so that
 * it reaches the optimizer, whose step reports it or is skipped.
 * max_norm > 0 (infinity: no clipping).  norm: ADAMW_NORM_*.
 * result: device adamw_clip_result_t, 16-byte aligned.
 * A launch for the norm and one for each pair of types in the list; no host
 * synchronisation; sums run in a fixed order.
 * Errors: INVALID_ARG, MISALIGNED, CUDA. */
int adamw_clip_grads(adamw_clip_plan_t plan, float max_norm, int32_t norm,
                     adamw_clip_result_t* result, adamw_stream_t stream);

/* Releases the plan's device memory (synchronises its device first).  NULL is
 * accepted. */
int adamw_clip_plan_destroy(adamw_clip_plan_t plan);

#ifdef __cplusplus
}
#endif

#endif /* ADAMW_LOSSES_H */
