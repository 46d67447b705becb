/*
 * psgd_clip.h -- gradient norms over many tensors, clipping by them, and the AdamW step
 * on a clipped update: the work of a training step around the compressors of psgd.h,
 * psgd_rtopk.h and psgd_atomo.h, on the same packed buffers.
 *
 * What the calls compute, for a buffer of S slices (the workers' gradients, or one
 * update) and N elements per slice over the plan's tensors i:
 *   psgd_grad_norm     PSGD_NORM_L2:  |g_s| = sqrt(sum_ij g_sij^2)
 *                      PSGD_NORM_MAX: |g_s| = max_ij |g_sij|
 *                      and, if asked, the same over every single tensor
 *   psgd_grad_clip     c_s = 1 if |g_s| <= max_norm, else max_norm / |g_s|
 *                      out_s = c_s * g_s
 *   psgd_adamw_apply   t <- t + 1,  g = c * U  (c from U's norm as above; 1 without clipping)
 *                      m <- beta1 * m + (1 - beta1) * g
 *                      v <- beta2 * v + (1 - beta2) * g^2
 *                      x <- x - lr * weight_decay * x
 *                             - lr * (m / (1 - beta1^t)) / (sqrt(v / (1 - beta2^t)) + eps)
 *
 * Precision.  Sums of squares are held in float64, so no float32 gradient overflows or
 * underflows them, and are added in a fixed order: equal calls give equal bits.  That order
 * depends on the call and the plan's sizes, so norms of one buffer from two different calls
 * (psgd_grad_norm and psgd_grad_clip, say) may differ in their last bit.  Norms
 * and coefficients are rounded once to float32 (a norm past its largest number becomes
 * infinite); a coefficient is taken from the float64 norm.  out is c * g in float32,
 * rounded once to the gradient type.  The AdamW state is float32 and its step size and
 * bias corrections are formed in float64.  A moment's weights beta and 1 - beta are not
 * rounded against each other: they add up to 1 far below a rounding of the moment.  A
 * moment at its steady value takes no change below half a float32 step, so for 1 - beta
 * below about 2^-24 (6e-8) it stands still there.
 *
 * Non-finite gradients are not errors: an infinite entry gives an infinite norm, hence
 * c = 0 for every finite max_norm (finite entries become 0, infinite ones NaN); a NaN
 * entry gives a NaN norm of either kind, and NaN everywhere in what is scaled by it.
 * With PSGD_ADAMW_SKIP_NONFINITE such an update changes nothing instead.  A finite update is
 * never skipped by the flag unless its norm is past float32's largest number; where it makes
 * v infinite (|c U| above about sqrt(3.4e38 / (1 - beta2)), 5.8e20 at beta2 = 0.999), v stays
 * so and the weight takes no further step but its decay.
 *
 * Memory layout, pointers, errors and ownership are those of psgd.h: a clip plan made
 * from a layer list has the layout (offsets, worker_stride) of every other plan made from
 * that list, padding between tensors is never read for results and never written, and
 * argument problems are found before anything is enqueued.  Buffers of whole slices and
 * the workspace are 16-byte aligned; norms, coefficients and the step count need only
 * their type's alignment.  No two buffers of a call may overlap, except where in place is
 * stated.
 *
 * Concurrency.  A plan, and a workspace, may be used by one stream and one host thread at
 * a time; two captured graphs that may run at the same time need a workspace each.  The
 * contents of a workspace need not be preserved between calls.
 *
 * Graphs.  Every call can be captured once the plan has run one call eagerly on that
 * device (the first call uploads the plan's tables) and with kernel timing off; other
 * captures are refused with PSGD_ERR_INVALID_ARG.  The AdamW step count lives in device
 * memory, so replays count.  A graph reads the plan's tables and the buffers of the call
 * it captured: all of them must outlive it.
 */
#ifndef PSGD_CLIP_H_
#define PSGD_CLIP_H_

#include "psgd.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef struct psgd_clip_plan psgd_clip_plan;

typedef enum psgd_norm_kind {
  PSGD_NORM_L2 = 0, /* Euclidean norm */
  PSGD_NORM_MAX = 1 /* largest magnitude */
} psgd_norm_kind;

typedef struct psgd_clip_layer_info {
  int64_t rows, cols, numel;
  int64_t offset; /* element offset inside a slice */
} psgd_clip_layer_info;

typedef struct psgd_clip_sizes {
  int32_t n_layers, n_slices, grad_dtype, reserved;
  int64_t worker_stride; /* elements per slice */
  int64_t numel;         /* sum of rows*cols over all tensors */
  uint64_t workspace_bytes;
  /* minimal bytes of a call: psgd_grad_norm reads every slice once; psgd_grad_clip also
     writes it; psgd_adamw_apply reads the update, and reads and writes params and both
     moments (without the bfloat16 copy) */
  uint64_t norm_bytes, clip_bytes, adamw_bytes;
} psgd_clip_sizes;

/* Build a plan for `n_layers` tensors (1 <= rows*cols < 2^31 each), n_slices in 1..65535
 * slices and gradients of grad_dtype.  flags must be 0 (PSGD_ERR_UNSUPPORTED otherwise,
 * as for an unknown dtype).  Host only. */
psgd_status psgd_clip_plan_create(const psgd_layer* layers, int32_t n_layers, int32_t n_slices,
                                  psgd_dtype grad_dtype, uint32_t flags, psgd_clip_plan** out);
psgd_status psgd_clip_plan_sizes(const psgd_clip_plan* plan, psgd_clip_sizes* out);
psgd_status psgd_clip_plan_layer_info(const psgd_clip_plan* plan, int32_t layer, psgd_clip_layer_info* out);
/* Free the plan and its device tables.  NULL is accepted.  No call using the plan may
 * still be running, and no graph that captured one may be replayed afterwards. */
psgd_status psgd_clip_plan_destroy(psgd_clip_plan* plan);

/* Norm of every slice, and of every tensor of every slice:
 *   grads         [n_slices][worker_stride] grad_dtype, read only
 *   norms         [n_slices] float32 out
 *   tensor_norms  [n_slices][n_layers] float32 out, or NULL
 *   workspace     workspace_bytes of device memory
 * Asynchronous on `stream` (a hipStream_t; NULL = default stream). */
psgd_status psgd_grad_norm(psgd_clip_plan* plan, const void* grads, psgd_norm_kind kind, float* norms,
                           float* tensor_norms, void* workspace, void* stream);

/* Scale every slice down to norm max_norm where its norm exceeds it:
 *   grads      [n_slices][worker_stride] grad_dtype
 *   out        the same shape and type; may be grads (in place: slices with c = 1 are not
 *              written)
 *   max_norm   > 0; +infinity leaves every slice whose norm is not NaN as it is
 *   norms      [n_slices] float32 out: the norms before clipping
 *   coefs      [n_slices] float32 out: c
 * Asynchronous on `stream`.  PSGD_ERR_INVALID_ARG for a max_norm that is not > 0. */
psgd_status psgd_grad_clip(psgd_clip_plan* plan, const void* grads, void* out, psgd_norm_kind kind, float max_norm,
                           float* norms, float* coefs, void* workspace, void* stream);

/* Decay only matrices: tensors with rows == 1 or cols == 1 take weight_decay 0. */
#define PSGD_ADAMW_DECAY_MATRICES_ONLY 0x1u
/* An update whose norm (as float32) is infinite or NaN changes nothing: params, moments,
 * copy and step count stay as they are, and the norm output says so.  Needs max_norm > 0. */
#define PSGD_ADAMW_SKIP_NONFINITE 0x2u

typedef struct psgd_adamw_config {
  double lr;           /* >= 0 */
  double beta1, beta2; /* in [0, 1) */
  double eps;          /* > 0, also in float32 */
  double weight_decay; /* >= 0 */
  double max_norm;     /* > 0: clip the update by its norm (+infinity: only measure it); 0: no norm is taken */
  int32_t norm_kind;   /* psgd_norm_kind, read when max_norm > 0 */
  uint32_t flags;      /* PSGD_ADAMW_* */
} psgd_adamw_config;

/* One AdamW step (decoupled weight decay) over every tensor of a plan with one slice:
 *   update      [worker_stride] grad_dtype: U (or any gradient), read only
 *   params, exp_avg, exp_avg_sq   [worker_stride] float32, in place: x, m, v
 *   params_bf16 [worker_stride] bfloat16 out: the new params rounded to nearest, or NULL
 *   step        [1] int64 in device memory, in place: t, the steps taken so far (>= 0)
 *   norm        [1] float32 out: U's norm; required if max_norm > 0, otherwise NULL
 * Asynchronous on `stream`.  PSGD_ERR_INVALID_ARG for a plan with several slices or a
 * config value outside its range, PSGD_ERR_UNSUPPORTED for unknown flags or norm kinds. */
psgd_status psgd_adamw_apply(psgd_clip_plan* plan, const psgd_adamw_config* config, const void* update, float* params,
                             float* exp_avg, float* exp_avg_sq, void* params_bf16, int64_t* step, float* norm,
                             void* workspace, void* stream);

/* Kernel timing as psgd_plan_set_timing / psgd_plan_kernel_stats.  Kernel names:
 * "cl_norm", "cl_final", "cl_scale", "cl_adamw", "cl_small", "cl_small_adamw". */
psgd_status psgd_clip_plan_set_timing(psgd_clip_plan* plan, int32_t enable);
psgd_status psgd_clip_plan_kernel_stats(psgd_clip_plan* plan, psgd_kernel_stat* out, int32_t capacity,
                                        int32_t* count, int32_t reset);

#ifdef __cplusplus
}
#endif

#endif /* PSGD_CLIP_H_ */
