/*
 * psgd_lm.h -- the two ends of a language model around its tied table, on the packed
 * buffers of psgd.h: embedding and softmax cross entropy, each with the table gradient it
 * writes into every worker's gradient slice, and dropout.
 *
 * The table T is one matrix of the model (vocab x dim): tensor `table` of the layer list
 * the compressors' plans are made from.  W workers have `rows` tokens each.  What the
 * calls compute, for worker w, row t and word v:
 *   psgd_lm_embed       out_wt = drop(T[token_wt])
 *   psgd_lm_embed_grad  G_w[v] (+)= sum over rows t with token_wt = v of drop(dout_wt)
 *   psgd_lm_loss        s_wtv = drop(x_wt) . T[v]
 *                       lse_wt = log sum_v exp(s_wtv),  loss_wt = lse_wt - s_wt,target
 *                       mean_w = mean of loss_wt over the rows that count
 *   psgd_lm_loss_grad   the gradients of scale_w * mean_w:
 *                       g_wtv = scale_w / counted_w * (exp(s_wtv - lse_wt) - [v = target_wt])
 *                       dx_wt = drop(sum_v g_wtv T[v]),  G_w[v] (+)= sum_t g_wtv drop(x_wt)
 *   psgd_dropout        out = residual + drop(x)
 * G_w is the table's part of worker w's gradient slice; (+)= sets it, or adds to it with
 * PSGD_LM_ACCUMULATE: a tied table's gradient is psgd_lm_loss_grad's plus
 * psgd_lm_embed_grad's.  The rest of a slice, padding included, is neither read nor written.
 *
 * Rows that do not count.  A target outside 0..vocab-1 (-100, say) takes its row out: loss,
 * lse and dx are 0 there and x is not used, whatever it holds.  A worker without counted
 * rows has mean 0 and gradient 0.  A token outside that range has an embedding of zeros and
 * no gradient.
 *
 * Dropout.  Entry i of a call's x, out or dout (row-major, all workers' rows one after the
 * other) is kept if word i % 4 of Philox4x32-10 (Salmon et al., "Parallel random numbers:
 * as easy as 1, 2, 3", 2011) with counter (i / 4, *step) and key `seed` is at least
 * floor(p * 2^32), and multiplied by 1 / (1 - p); a dropped entry is 0 whatever it was.  No
 * mask is stored: the backward pass is the same call, with the same seed and step, on the
 * gradient.  psgd_lm_loss_grad and psgd_lm_embed_grad take the configuration of the forward
 * call.  The step lives in device memory (AdamW's step count, say), so that replays of a
 * graph draw new masks; layers are told apart by their seeds.
 *
 * Precision.  Activations (x, out, dout, dx) and params have one type, gradients another or
 * the same, float32 or bfloat16 each.  Products are summed in float32.
 * - float32 activations.  For the scores x and the table enter the matrix cores as two fp16
 *   parts of rows scaled by their own powers of two: 22 bits of an entry down to 2^-28 of the
 *   largest finite entry of its row (of those that dropout keeps), fewer below that and none
 *   below 2^-49; what other rows hold does not matter.  For the gradients they and g have all
 *   their 24 bits (16 for a bfloat16 table gradient), whatever the other entries are; entries
 *   below 2^-102 fewer.
 * - bfloat16 activations.  x and the table are taken as they are.  g is rounded to bfloat16 for
 *   dx, and for the table gradient unless that is float32.
 * Everything else is float32, means are taken in float64, results are rounded once.  Sums have
 * a fixed order: equal calls give equal bits.  Non-finite entries are not errors: one in the
 * table, or in a counted row of x, makes what depends on it infinite or NaN (that row's loss,
 * or every counted row's).
 *
 * No logits are kept: psgd_lm_loss reduces each tile of them where it is computed, and
 * psgd_lm_loss_grad holds g for one piece of the vocabulary at a time in the workspace.
 *
 * Pointers, errors and ownership are those of psgd.h, and argument problems are found
 * before anything is enqueued.  Whole packed buffers and the workspace are 16-byte aligned,
 * everything else to its type.  No two buffers of a call may overlap (from their first
 * element to their last), except where in place is stated.
 *
 * Concurrency.  A plan may be used by one host thread at a time (several streams may), a
 * workspace by one stream at a time; two captured graphs that may run at the same time need
 * a workspace each.  The contents of a workspace need not be preserved between calls.
 *
 * Graphs.  Every call can be captured, with kernel timing off; nothing has to run first.
 */
#ifndef PSGD_LM_H_
#define PSGD_LM_H_

#include "psgd.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef struct psgd_lm_plan psgd_lm_plan;

typedef struct psgd_dropout_config {
  double p;            /* probability that an entry is dropped, in [0, 1] */
  uint64_t seed;       /* Philox key */
  const int64_t* step; /* [1] int64 in device memory, read only; NULL = 0 */
} psgd_dropout_config;

typedef struct psgd_lm_sizes {
  int32_t n_layers, n_workers, table, act_dtype, grad_dtype, reserved;
  int64_t vocab, dim, rows; /* rows: per worker */
  int64_t worker_stride;    /* elements per slice of params and grads */
  int64_t table_offset;     /* element offset of the table in a slice */
  uint64_t workspace_bytes;
} psgd_lm_sizes;

/* Build a plan for a model of `n_layers` tensors (1 <= rows*cols < 2^31 each) of which
 * tensor `table` is the vocab x dim table, n_workers in 1..65535 workers and `rows` tokens
 * per worker, n_workers * rows in 1..2^23.  dim is at most 2^23, and the table and
 * the workers' rows (every worker's rounded up to 64) have at most 2^23 blocks of 64 x 64.  act_dtype: type of
 * params and activations; grad_dtype: type of grads.  flags must be 0 (PSGD_ERR_UNSUPPORTED otherwise, as for an
 * unknown dtype).  Host only. */
psgd_status psgd_lm_plan_create(const psgd_layer* layers, int32_t n_layers, int32_t table, int32_t n_workers,
                                int64_t rows, psgd_dtype act_dtype, psgd_dtype grad_dtype, uint32_t flags,
                                psgd_lm_plan** out);
psgd_status psgd_lm_plan_sizes(const psgd_lm_plan* plan, psgd_lm_sizes* out);
/* Free the plan.  NULL is accepted.  No timed call of the plan may still be running. */
psgd_status psgd_lm_plan_destroy(psgd_lm_plan* plan);

/* Add to the table's gradient instead of setting it. */
#define PSGD_LM_ACCUMULATE 0x1u

/* Rows of the table:
 *   params   [worker_stride] act_dtype, read only (the table's part)
 *   tokens   [n_workers][rows] int64
 *   dropout  NULL: none
 *   out      [n_workers][rows][dim] act_dtype out
 * Asynchronous on `stream` (a hipStream_t; NULL = default stream), as every call below. */
psgd_status psgd_lm_embed(psgd_lm_plan* plan, const void* params, const int64_t* tokens,
                          const psgd_dropout_config* dropout, void* out, void* stream);

/* The table gradient of psgd_lm_embed:
 *   dout       [n_workers][rows][dim] act_dtype: gradient of out
 *   grads      [n_workers][worker_stride] grad_dtype, the table's part set or added to
 *   flags      0 or PSGD_LM_ACCUMULATE (PSGD_ERR_UNSUPPORTED for others)
 *   workspace  workspace_bytes of device memory */
psgd_status psgd_lm_embed_grad(psgd_lm_plan* plan, const int64_t* tokens, const void* dout,
                               const psgd_dropout_config* dropout, void* grads, uint32_t flags, void* workspace,
                               void* stream);

/* Loss of every row and every worker's mean:
 *   x        [n_workers][rows][dim] act_dtype
 *   targets  [n_workers][rows] int64
 *   losses   [n_workers][rows] float32 out
 *   lse      [n_workers][rows] float32 out: what psgd_lm_loss_grad takes
 *   mean     [n_workers] float32 out */
psgd_status psgd_lm_loss(psgd_lm_plan* plan, const void* x, const void* params, const int64_t* targets,
                         const psgd_dropout_config* dropout, float* losses, float* lse, float* mean, void* workspace,
                         void* stream);

/* Gradients of every worker's scale * mean:
 *   lse     [n_workers][rows] float32, of psgd_lm_loss on the same x, params and dropout
 *   scale   [n_workers] float32, or NULL for 1
 *   dx      [n_workers][rows][dim] act_dtype out, or NULL
 *   grads   [n_workers][worker_stride] grad_dtype, the table's part set or added to, or NULL
 * One of dx and grads at least is given. */
psgd_status psgd_lm_loss_grad(psgd_lm_plan* plan, const void* x, const void* params, const int64_t* targets,
                              const float* lse, const float* scale, const psgd_dropout_config* dropout, void* dx,
                              void* grads, uint32_t flags, void* workspace, void* stream);

/* Dropout of a matrix, with the addition of a residual:
 *   x, out    [rows][cols] of `dtype`, rows x_stride and out_stride elements apart
 *   residual  the same, residual_stride apart, or NULL
 *   config    required
 * rows, cols >= 0, rows * cols < 2^41, strides >= cols (not read for a single row).  out
 * may be x or residual (same pointer and stride).  No plan and no workspace are needed. */
psgd_status psgd_dropout(const void* x, int64_t x_stride, const void* residual, int64_t residual_stride, void* out,
                         int64_t out_stride, int64_t rows, int64_t cols, psgd_dtype dtype,
                         const psgd_dropout_config* config, void* stream);

/* Kernel timing as psgd_plan_set_timing / psgd_plan_kernel_stats. */
psgd_status psgd_lm_plan_set_timing(psgd_lm_plan* plan, int32_t enable);
psgd_status psgd_lm_plan_kernel_stats(psgd_lm_plan* plan, psgd_kernel_stat* out, int32_t capacity, int32_t* count,
                                      int32_t reset);

#ifdef __cplusplus
}
#endif

#endif /* PSGD_LM_H_ */
