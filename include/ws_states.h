/*
 * ws_states.h -- C ABI of the operators over rows of hidden states for MI355X
 * (gfx950): what a language model computes on between its tokens and its
 * logits, one row of `width` elements per token position, many rows per call.
 *
 *   ws_embed           rows of a table looked up by token, scaled
 *   ws_embed_grad      the table's gradient: the rows of every token summed
 *   ws_layernorm       layer norm of every row, with weight and bias
 *   ws_layernorm_grad  the gradients of its rows, its weight and its bias
 *
 * Tokens are those of ws_logits.h: what ws_sample draws is what ws_embed looks
 * up, and -1 is no token in both.
 *
 * Calls: as in ws_logits.h.  Each enqueues its kernels on `stream` (a
 * hipStream_t of states->device, or NULL for that device's null stream), reads
 * and writes only the caller's buffers, allocates nothing, does not synchronise
 * and can be captured into a graph.  states->device must be the calling
 * thread's current device.  Arguments are read during the call and not
 * retained; the buffers must stay until the stream has passed the call.  No
 * output may overlap an input, the workspace or another output, but where said
 * so.  The elements between a matrix's rows are not its own: an array may lie
 * there, and another matrix of the same stride in bytes (matrices of different
 * strides must lie apart, one wholly behind the other).  Calls share no state:
 * two may run at once from any threads and streams as long as neither writes
 * what the other uses, the workspace included (two captured graphs that may run
 * at once need a workspace each).  A workspace needs no initialisation and its
 * contents do not matter between calls.
 *
 * Numbers: rows are FP32, FP16 or BF16.  Sums, means and deviations are FP32;
 * every output is rounded once to its type.  The same call on the same inputs
 * gives the same bits (no sum's order depends on timing); another shape,
 * alignment or order of tokens may change the order of a sum.  NaN and
 * infinities go where the formulas carry them, and so do sums that pass FP32's
 * range: a row whose sum does (its mean need not) has a norm of NaN, one whose
 * deviations' squares do an inverse of 0.
 *
 * Errors: as in ws.h.  Everything the host can see is checked before anything
 * is enqueued; a call with 0 rows checks its arguments and does what the
 * formulas say of no rows (ws_embed_grad and ws_layernorm_grad then write
 * gradients of 0, or leave what they add to as it is).
 */
#ifndef WS_STATES_H
#define WS_STATES_H

#include "ws_logits.h"

#ifdef __cplusplus
extern "C" {
#endif

#define WS_MAX_WIDTH  (1 << 20)
#define WS_MAX_TOKENS (1 << 24)

/* A matrix of hidden states: `rows` rows of `width` elements, `row_stride`
 * elements from one row's start to the next.  Rows may start at any element
 * address; the elements between width and row_stride are neither read nor
 * written. */
typedef struct ws_states {
    int32_t device;       /* HIP device ordinal                               */
    int32_t dtype;        /* WS_DTYPE_* of the rows                           */
    int32_t rows;         /* 0..WS_MAX_ROWS                                   */
    int32_t width;        /* 1..WS_MAX_WIDTH                                  */
    int64_t row_stride;   /* >= width, <= WS_MAX_ROW_STRIDE                   */
} ws_states;

/* ---- embedding lookup ------------------------------------------------------
 *   out[r] = scale * table[ids[r]]
 * 0 where ids[r] is -1; any other index outside [0, vocab) is never used as an
 * address and makes the row NaN.  `states` describes out. */
typedef struct ws_embed_args {
    const void    *table;         /* [vocab] rows of states->dtype            */
    int64_t        table_stride;  /* >= width, <= WS_MAX_ROW_STRIDE           */
    const int32_t *ids;           /* [rows]                                   */
    void          *out;           /* [rows] of stride states->row_stride      */
    int32_t        vocab;         /* 1..WS_MAX_TOKENS                         */
    float          scale;         /* finite                                   */
} ws_embed_args;

int ws_embed(const ws_states *states, const ws_embed_args *args, void *stream);

/* ---- its gradient ----------------------------------------------------------
 *   grad_table[v] = scale * sum of grad_out[r] over the rows with ids[r] = v
 * for every v of the vocabulary (0 for a token no row names), or, with
 * accumulate = 1, that sum added to what grad_table holds (rows no token names
 * are then neither read nor written).  Indices outside [0, vocab) add nothing.
 * The tokens are sorted by index, equal ones by row, and each token's rows are
 * added in that order, in blocks.  `states` describes grad_out. */
typedef struct ws_embed_grad_args {
    const void    *grad_out;      /* [rows] of stride states->row_stride      */
    const int32_t *ids;           /* [rows]                                   */
    void          *grad_table;    /* [vocab] rows of grad_dtype               */
    int64_t        grad_stride;   /* >= width, <= WS_MAX_ROW_STRIDE           */
    void          *workspace;     /* ws_embed_grad_workspace bytes, 16-byte
                                     aligned; NULL when 0                     */
    size_t         workspace_bytes;
    int32_t        vocab;         /* 1..WS_MAX_TOKENS                         */
    int32_t        grad_dtype;    /* states->dtype or WS_DTYPE_F32            */
    int32_t        accumulate;    /* 0 or 1                                   */
    float          scale;         /* finite                                   */
} ws_embed_grad_args;

/* Workspace bytes of ws_embed_grad for these rows and this vocabulary.  (Few rows
 * are added without a sort and leave it untouched, but it is asked for all the
 * same.) */
int ws_embed_grad_workspace(const ws_states *states, int32_t vocab, size_t *bytes);

int ws_embed_grad(const ws_states *states, const ws_embed_grad_args *args, void *stream);

/* ---- layer norm --------------------------------------------------------------
 *   mean = sum_c x_c / width,  inverse = 1 / sqrt(sum_c (x_c - mean)^2 / width + eps)
 *   y_c  = (x_c - mean) * inverse * weight_c + bias_c
 * Without weight its factor is 1, without bias its term 0.  y may be x itself
 * (same address and stride); otherwise no element may belong to both: apart, or
 * with equal strides in one buffer, each row of one in the other's padding.
 * `states` describes x. */
typedef struct ws_norm_stats {
    float mean;      /* rounded to FP32, which ws_layernorm itself does not see:
                        of a row whose mean is n times its deviation the
                        gradient's u is off by up to n 2^-24                  */
    float inverse;
} ws_norm_stats;

typedef struct ws_layernorm_args {
    const void    *x;
    const void    *weight;        /* [width] of weight_dtype, or NULL         */
    const void    *bias;          /* [width] of weight_dtype, or NULL         */
    void          *y;             /* [rows] of states->dtype                  */
    int64_t        y_stride;      /* >= width, <= WS_MAX_ROW_STRIDE           */
    ws_norm_stats *stats;         /* [rows], 8-byte aligned, or NULL: for
                                     ws_layernorm_grad                        */
    int32_t        weight_dtype;  /* states->dtype or WS_DTYPE_F32            */
    float          eps;           /* >= 0, finite                             */
} ws_layernorm_args;

int ws_layernorm(const ws_states *states, const ws_layernorm_args *args, void *stream);

/* ---- its gradients -----------------------------------------------------------
 * With g = grad_y, u_c = (x_c - mean) * inverse and d_c = g_c weight_c, per row
 *   grad_x_c = inverse (d_c - sum_i d_i / width - u_c sum_i d_i u_i / width)
 * and over the rows
 *   grad_weight_c = sum_r g_c u_c,   grad_bias_c = sum_r g_c
 * Each of the three may be NULL (left out), not all.  grad_x may be grad_y or x
 * itself (same address and stride); otherwise it lies apart from both, as y
 * from x above. */
typedef struct ws_layernorm_grad_args {
    const void          *x;
    const ws_norm_stats *stats;           /* [rows], from ws_layernorm        */
    const void          *weight;          /* [width], or NULL: 1              */
    const void          *grad_y;          /* [rows] of states->dtype          */
    int64_t              grad_y_stride;   /* >= width, <= WS_MAX_ROW_STRIDE   */
    void                *grad_x;          /* [rows] of states->dtype, or NULL */
    int64_t              grad_x_stride;   /* with grad_x                      */
    void                *grad_weight;     /* [width] of weight_dtype, or NULL */
    void                *grad_bias;       /* [width] of weight_dtype, or NULL */
    void                *workspace;       /* ws_layernorm_grad_workspace
                                             bytes, 16-byte aligned; NULL
                                             without both                     */
    size_t               workspace_bytes;
    int32_t              weight_dtype;    /* states->dtype or WS_DTYPE_F32    */
    int32_t              reserved;        /* must be 0                        */
} ws_layernorm_grad_args;

/* Workspace bytes of ws_layernorm_grad for these rows, with the weight's or the
 * bias's gradient (without both it needs none). */
int ws_layernorm_grad_workspace(const ws_states *states, size_t *bytes);

int ws_layernorm_grad(const ws_states *states, const ws_layernorm_grad_args *args, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* WS_STATES_H */
