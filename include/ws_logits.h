/*
 * ws_logits.h -- C ABI of the operators over rows of logits for MI355X
 * (gfx950): what a classifier or a language model answers with, one row of V
 * logits per image or token position, many rows per call.
 *
 *   ws_logprobs       log probabilities of given tokens, entropy, and the K
 *                     best alternatives with their log probabilities
 *   ws_logprobs_grad  the gradient of all of those with respect to the logits
 *   ws_distill        distillation loss against a teacher's top entries, and
 *                     on request its gradient in the same call
 *   ws_distill_grad   that gradient alone, from the loss call's statistics
 *
 * The alternatives ws_logprobs reports for a teacher's logits are, as they
 * lie in memory, the teacher entries ws_distill takes.
 *
 * Notation, per row: z the V logits, tau the temperature, x_j = z_j / tau,
 * lse = log sum_j exp(x_j), p_j = exp(x_j - lse).
 *
 * Calls: each enqueues its kernels on `stream` (a hipStream_t of
 * rows->device, or NULL for that device's null stream), reads and writes only
 * the caller's buffers, allocates nothing, does not synchronise and can be
 * captured into a graph.  rows->device must be the calling thread's current
 * device.  Arguments are read during the call and not retained; the buffers
 * must stay until the stream has passed the call.  No output may overlap an
 * input, the workspace or another output, but for gradients as said there.
 * Calls share no state: two may run at once from any threads and streams as
 * long as neither writes what the other uses, the workspace included (two
 * captured graphs that may run at once need a workspace each).  A workspace
 * needs no initialisation and its contents do not matter between calls.
 *
 * Numbers: logits are FP32, FP16 or BF16; everything else, and every sum, is
 * FP32 or wider.  Gradients are computed in FP32 and rounded once to the
 * logits' type.  The same call on the same inputs gives the same bits; a
 * change of shape, alignment or K may change the order of a sum.
 *
 * Rows that have no distribution: a logit of -inf has probability 0.  A row
 * of nothing else has lse = -inf: its log probabilities are -inf, its entropy
 * 0, its distillation loss +inf (0 where q is 0 throughout) and its
 * gradient 0.  A row that holds a NaN or +inf has NaN for its log
 * probabilities, entropy, loss and gradient.
 *
 * Indices: -1 stands for no token.  Any other index outside [0, V) is never
 * used as an address; it makes what depends on it NaN (the row's log
 * probability or loss, and its whole gradient).
 *
 * Errors: as in ws.h.  Everything the host can see is checked before anything
 * is enqueued; a call with 0 rows checks its arguments and enqueues nothing.
 */
#ifndef WS_LOGITS_H
#define WS_LOGITS_H

#include "ws.h"

#ifdef __cplusplus
extern "C" {
#endif

#define WS_MAX_ROWS           (1 << 22)
#define WS_MAX_ROW_STRIDE     (1ll << 32)
#define WS_MIN_TEMPERATURE    1e-3f
#define WS_MAX_TEMPERATURE    1e3f
#define WS_DISTILL_MAX_K      128

#define WS_DISTILL_RENORM 0   /* the teacher's listed entries, renormalised   */
#define WS_DISTILL_TAIL   1   /* the listed entries and one event for the rest */

/* 2^-16, above what FP32 scores of a list that holds all of the mass leave of 1
 * minus their sum: with E = 2^-24 at most 128 E for the additions of a sum over
 * 128 tokens, 4 E log 128 for its logarithm, 3 E log 128 for the exponents (the
 * weighted mean of their size), E log 128 for the scores' own rounding and 4 E
 * for the exponentials: 171 E of 256 E. */
#define WS_DISTILL_ROUNDING 1.52587890625e-5f

/* A matrix of logits: `rows` rows of `vocab` elements, `row_stride` elements
 * from one row's start to the next.  Rows may start at any element address;
 * the elements between vocab and row_stride are neither read nor written.
 * Rows whose starts are 16-byte aligned are read fastest. */
typedef struct ws_rows {
    int32_t device;       /* HIP device ordinal                               */
    int32_t dtype;        /* WS_DTYPE_* of the logits and of their gradient   */
    int32_t rows;         /* 0..WS_MAX_ROWS                                   */
    int32_t vocab;        /* V, 1..WS_MAX_SCORES                              */
    int64_t row_stride;   /* >= vocab, <= WS_MAX_ROW_STRIDE                   */
    float   temperature;  /* tau, WS_MIN_TEMPERATURE..WS_MAX_TEMPERATURE      */
    int32_t reserved;     /* must be 0                                        */
} ws_rows;

/* What a gradient needs of its row: lse = max / tau + logsum.  A row of -inf
 * only has {-inf, -inf}. */
typedef struct ws_row_stats {
    float max;      /* largest logit of the row                               */
    float logsum;   /* log sum_j exp((z_j - max) / tau)                       */
} ws_row_stats;

/* ---- log probabilities ---------------------------------------------------
 *   logprob[r]  x_t - lse for t = targets[r]; 0 where targets[r] is -1
 *   entropy[r]  lse - sum_j p_j x_j, in nats
 *   top[r][i]   the top_k best tokens by logit, rank order: equal logits
 *               prefer the lower index, -0 equals +0, NaN counts as -inf (the
 *               lane's Top-K order); score = x - lse
 *   stats[r]    for ws_logprobs_grad
 * Every output may be NULL (left out); logprob and targets come together, top
 * and top_k > 0 come together. */
typedef struct ws_logprobs_args {
    const void    *logits;
    const int32_t *targets;          /* [rows]                                */
    float         *logprob;          /* [rows]                                */
    float         *entropy;          /* [rows]                                */
    ws_topk_entry *top;              /* [rows][top_k], 8-byte aligned         */
    ws_row_stats  *stats;            /* [rows], 8-byte aligned                */
    void          *workspace;        /* ws_logprobs_workspace bytes, 16-byte
                                        aligned; NULL when 0                  */
    size_t         workspace_bytes;
    int32_t        top_k;            /* 0..min(WS_MAX_K, vocab)               */
    int32_t        reserved;         /* must be 0                             */
} ws_logprobs_args;

/* Workspace bytes of ws_logprobs for this shape (0 for many shapes). */
int ws_logprobs_workspace(const ws_rows *rows, int32_t top_k, size_t *bytes);

int ws_logprobs(const ws_rows *rows, const ws_logprobs_args *args, void *stream);

/* ---- gradient of the log probabilities -----------------------------------
 * With gl, gh and g the upstream gradients of logprob, entropy and top scores,
 *   dz_j = 1/tau [ gl (1[j = t] - p_j) + sum_k g_k (1[j = id_k] - p_j)
 *                  - gh p_j (log p_j + entropy) ]
 * targets and grad_logprob come together, top (of which only the indices are
 * read; -1 adds nothing) with grad_top and top_k, entropy (the forward's
 * output) with grad_entropy; each may be left out.  grad_logits may be the
 * logits themselves (same address and stride): each element is read before it
 * is written.  Otherwise no element may belong to both: apart, or with equal
 * strides in one buffer, each row of one in the other's padding. */
typedef struct ws_logprobs_grad_args {
    const void          *logits;
    const ws_row_stats  *stats;         /* [rows]                             */
    const int32_t       *targets;       /* [rows]                             */
    const float         *grad_logprob;  /* [rows]                             */
    const float         *entropy;       /* [rows]                             */
    const float         *grad_entropy;  /* [rows]                             */
    const ws_topk_entry *top;           /* [rows][top_k]                      */
    const float         *grad_top;      /* [rows][top_k]                      */
    void                *grad_logits;   /* [rows] of stride grad_stride       */
    int64_t              grad_stride;   /* >= vocab, <= WS_MAX_ROW_STRIDE     */
    int32_t              top_k;         /* 0..WS_MAX_K                        */
    int32_t              reserved;      /* must be 0                          */
} ws_logprobs_grad_args;

int ws_logprobs_grad(const ws_rows *rows, const ws_logprobs_grad_args *args, void *stream);

/* ---- distillation --------------------------------------------------------
 * teacher[r] lists up to teacher_k tokens with the teacher's log
 * probabilities (at the temperature in use; with WS_DISTILL_RENORM any values
 * that differ from them by one constant a row, such as the teacher's logits
 * over tau).  An index of -1 is an absent entry, so lists may differ in
 * length.  A score of -inf is a listed token of probability 0.
 *
 *   WS_DISTILL_RENORM  q = softmax of the listed scores,
 *                      loss = sum_k q_k (log q_k - log p_id(k))
 *   WS_DISTILL_TAIL    q_k = exp(score_k), q_t = max(0, 1 - sum_k q_k),
 *                      p_t = the sum of p over the tokens not listed,
 *                      loss = sum_k q_k (log q_k - log p_id(k))
 *                             + q_t (log q_t - log p_t)
 * with terms of q = 0 counted as 0 (so a row without entries has loss 0, unless
 * it holds a NaN or +inf: its loss and gradient are NaN whatever is listed); in
 * WS_DISTILL_TAIL, a list that names every token of the vocabulary has no
 * q_t.  Where a list holds all of the teacher's mass, FP32 scores leave a q_t of
 * either sign and about 1e-7; against a p_t of 0 (every unlisted token masked,
 * by -inf or the type's lowest value) half of such rows would have an infinite
 * loss.  So where p_t is 0 in FP32 (log p_t below log 2^-150), a q_t of at most
 * WS_DISTILL_ROUNDING counts as 0.  A token listed twice is two terms of the
 * loss, but one listed token to p_t and to the gradient, which is
 *   dz_j = g / tau (M p_j - sum_{k: id(k) = j} q_k)   for a listed token
 *   dz_j = g / tau (M - q_t / p_t) p_j                otherwise
 * with g = grad_loss[r] and M = sum_k q_k + q_t.  Where the student gives a
 * positive q no probability the loss is +inf and the gradient still that of
 * the formula, 0 for an unlisted token when p_t = 0.  grad_logits may be the
 * logits themselves, as for ws_logprobs_grad.
 *
 * ws_distill returns the loss, and the gradient as well when grad_logits is
 * set (grad_loss is then needed and grad_stride read).  ws_distill_grad is
 * for upstream gradients not known before the loss: it takes the stats and,
 * with WS_DISTILL_TAIL, the tail of an earlier ws_distill call. */
typedef struct ws_distill_args {
    const void          *logits;
    const ws_topk_entry *teacher;       /* [rows][teacher_k], 8-byte aligned  */
    float               *loss;          /* [rows]                             */
    ws_row_stats        *stats;         /* [rows] or NULL                     */
    float               *tail;          /* [rows] or NULL: log p_t
                                           (WS_DISTILL_TAIL only)             */
    const float         *grad_loss;     /* [rows], with grad_logits           */
    void                *grad_logits;   /* [rows] of stride grad_stride, or
                                           NULL: no gradient                  */
    int64_t              grad_stride;   /* >= vocab, <= WS_MAX_ROW_STRIDE     */
    void                *workspace;     /* ws_distill_workspace bytes, 16-byte
                                           aligned; NULL when 0               */
    size_t               workspace_bytes;
    int32_t              teacher_k;     /* 1..WS_DISTILL_MAX_K                */
    int32_t              mode;          /* WS_DISTILL_*                       */
    int32_t              reserved[2];   /* must be 0                          */
} ws_distill_args;

/* Workspace bytes of ws_distill for this shape and mode, `gradient` being
 * whether grad_logits will be set. */
int ws_distill_workspace(const ws_rows *rows, int32_t mode, int32_t gradient, size_t *bytes);

int ws_distill(const ws_rows *rows, const ws_distill_args *args, void *stream);

typedef struct ws_distill_grad_args {
    const void          *logits;
    const ws_topk_entry *teacher;       /* [rows][teacher_k]                  */
    const ws_row_stats  *stats;         /* [rows]                             */
    const float         *tail;          /* [rows]; WS_DISTILL_TAIL only       */
    const float         *grad_loss;     /* [rows]                             */
    void                *grad_logits;   /* [rows] of stride grad_stride       */
    int64_t              grad_stride;   /* >= vocab, <= WS_MAX_ROW_STRIDE     */
    int32_t              teacher_k;     /* 1..WS_DISTILL_MAX_K                */
    int32_t              mode;          /* WS_DISTILL_*                       */
} ws_distill_grad_args;

int ws_distill_grad(const ws_rows *rows, const ws_distill_grad_args *args, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* WS_LOGITS_H */
