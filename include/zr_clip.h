/*
 * zr_clip.h -- clipping by the global gradient norm, between the gradient reduce and the
 * AdamW step of zr.h.
 *
 *   zr_grad_norm           sum of squares, norm and clip factor of many tensors
 *   zr_clip_grads          tensors scaled by the factor, in place
 *   zr_adamw_step_clip     zr_adamw_step on the clipped gradient, which is not written
 *   zr_adamw_step_clip_f16 zr_adamw_step_f16 on the clipped gradient
 *
 * The norm of a model's whole gradient is the root of the sum of the squares that its
 * ranks hold ([TUT] 2.1: each rank owns one contiguous slice; the mean of the slice is
 * zr_reduce_slice's), and every rank has to scale by the same factor.  A rank's share is
 * its slice; tensors that every rank holds whole ([ART] small-parameter residency) count
 * once:
 *   zr_grad_norm(slice, accumulate 0)        the rank's own sum
 *   ... all-reduce of clip->sum_squares over the ranks (one fp64 value) ...
 *   zr_grad_norm(whole tensors, accumulate 1)   adds them; norm and factor of everything
 *   zr_adamw_step_clip(slice ...), zr_adamw_step_clip(whole tensors ...)
 * With no tensors (n = 0) and accumulate 1 the call only works out norm and factor
 * again, as after an all-reduce.
 *
 * The conventions of zr.h hold for every call: validation first, nothing launched and
 * nothing written on an error, asynchronous on `stream`, no device allocation,
 * capturable into a zr_graph.  The same call gives the same bits every time, wherever the
 * tensors lie and whatever grid runs it: sums are fp64, in an order that goes by the
 * tensors' sizes alone, so that ranks that hold the same tensors work out the same factor.
 */
#ifndef ZR_CLIP_H
#define ZR_CLIP_H

#include "zr_fp8.h" /* zr_dtype */

#ifdef __cplusplus
extern "C" {
#endif

/* fp64 sums in zr_grad_norm's workspace. */
#define ZR_GRAD_NORM_PARTIALS 2048

/* The outcome of a norm, in device memory (caller-allocated, 8-byte aligned), read and
 * written in stream order. */
typedef struct zr_clip {
    double sum_squares;  /* of the elements as they are (scaled gradients: before any scale) */
    float  norm;         /* |grad_scale| * sqrt(sum_squares) / loss scale */
    float  factor;       /* min(1, max_norm / (norm + eps)) */
} zr_clip;

typedef struct zr_clip_hparams {
    double max_norm;     /* > 0; infinity: never clip */
    double eps;          /* finite, >= 0 (1e-6 is customary) */
    double grad_scale;   /* finite; what the step multiplies the gradient by (1.0 for a mean) */
} zr_clip_hparams;

/*
 * clip->sum_squares = sum of x^2 over the elements of n tensors (plus what it held, with
 * accumulate), and from it
 *   norm   = |grad_scale| * sqrt(sum_squares) / S     (S = ls->scale, 1 without ls)
 *   factor = min(1, max_norm / (norm + eps))
 * worked out in fp64 and rounded once to fp32.  Clipping by the global norm: Pascanu,
 * Mikolov & Bengio, ICML 2013.  An infinity among the elements makes the norm infinite and the
 * factor 0, a NaN makes both NaN (with max_norm infinite the factor is 1 whatever the norm is);
 * finite elements never overflow the sum.  With ls,
 * ls->found_inf is set if the sum is not finite, so that the fp16 step is skipped -- on
 * every rank, once the sum has been all-reduced.
 *
 * grads: host array of n device pointers (n >= 0; an entry may be NULL where numels is
 * 0); numels: host array of n element counts (0 ... 2^42).  dtype: ZR_BF16, ZR_F16 or ZR_F32.
 * hp: host pointer.  ls may be NULL.  workspace: device fp64 [ZR_GRAD_NORM_PARTIALS],
 * contents undefined before and after; two calls that may run at once need workspaces and
 * records of their own, and so do two graphs whose replays may.  The tensors may overlap
 * one another (each counts), not the record, the workspace or ls.
 * In a captured step: zr_graph_set_adamw gives its grad_scale to every zr_grad_norm that was
 * captured with the grad_scale of an AdamW-family call of the same graph (compared as
 * doubles), so that the norm stays that of the step's gradient.  A norm captured with
 * another scale keeps it; max_norm and eps are fixed at capture.
 * Errors: ZR_EINVAL, ZR_EALIGN, ZR_EHIP.
 */
ZR_API zr_status zr_grad_norm(const void *const *grads, const int64_t *numels, int32_t n, zr_dtype dtype,
                              const zr_clip_hparams *hp, int32_t accumulate, zr_loss_scale *ls, zr_clip *clip,
                              double *workspace, void *stream);

/*
 * x = T(x * clip->factor) for every element of n tensors of type T = dtype, in place (the
 * product is fp32, rounded once).  Where the factor is 1 nothing is written.  No two
 * tensors may overlap.  grads and numels as for zr_grad_norm.
 * Errors: ZR_EINVAL, ZR_EALIGN, ZR_ENOMEM, ZR_EHIP.
 */
ZR_API zr_status zr_clip_grads(void *const *grads, const int64_t *numels, int32_t n, zr_dtype dtype,
                               const zr_clip *clip, void *stream);

/*
 * zr_adamw_step on the gradient multiplied by clip->factor: its update with grad_scale *
 * factor (one fp64 product) in the place of grad_scale, bit for bit.  The clipped
 * gradient is not written: clipping costs the step no pass over memory.  A factor of NaN
 * makes every state NaN, as a gradient of NaN does; only the fp16 form skips such a step.
 * The graph calls of zr.h treat it as a call of the AdamW family.  Buffer rules as
 * zr_adamw_step; the record must not overlap a buffer.  Errors: ZR_EINVAL, ZR_EALIGN, ZR_EHIP.
 */
ZR_API zr_status zr_adamw_step_clip(const void *grad, float *master, float *exp_avg, float *exp_avg_sq,
                                    void *param_out, int64_t numel, const zr_adamw_hparams *hp, const zr_clip *clip,
                                    void *stream);

/* The same for zr_adamw_step_f16: the fp16 gradient is divided by ls->scale, then
 * multiplied by grad_scale * factor; skipped entirely while ls->found_inf is set.
 * Errors: ZR_EINVAL, ZR_EALIGN, ZR_EHIP. */
ZR_API zr_status zr_adamw_step_clip_f16(const void *grad, float *master, float *exp_avg, float *exp_avg_sq,
                                        void *param_out, int64_t numel, const zr_adamw_hparams *hp,
                                        const zr_loss_scale *ls, const zr_clip *clip, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* ZR_CLIP_H */
