/*
 * zr_rope.h -- the norm of queries and keys for each head and the rotation by their
 * positions, in one pass, between the query/key/value product of zr_fp8.h and
 * attention.
 *
 *   zr_qk_norm_rope            norm and rotation
 *   zr_qk_norm_rope_backward   their gradients
 *
 * For every token t and head the row x of head_dim elements is normed and turned:
 *   rstd = 1 / sqrt(mean of x^2 + eps),  y = x * rstd * weight
 * (y = x where the weight is NULL), then for each pair j < rot_dim / 2
 *   angle = positions[axis(j)][t] * inv_freq[j]
 *   (y_a, y_b) -> (y_a cos - y_b sin, y_b cos + y_a sin)
 * with (a, b) = (j, j + rot_dim / 2), or (2j, 2j + 1) where pairs are interleaved.
 * Elements from rot_dim on keep y.  Rotary positions: Su et al., 2021; root mean square
 * norm: Zhang & Sennrich, NeurIPS 2019.  With several axes (time, height, width of an image's
 * or a video's patch) each pair is turned by the position of its axis.
 *
 * The angle is an fp64 product, reduced to one turn in fp64 before its sine and cosine
 * are taken in fp32: positions of 2^31 at a frequency of 1 still have angles right to 2^-20.
 * All other arithmetic is fp32, each output rounded once; a finite row whose squares pass
 * fp32's range (magnitudes from about 1e19 on) has rstd 0, and outputs and gradients 0 with
 * it.  An infinity or a NaN in a normed row makes NaN where the formulas do, in that row and
 * in the weight's gradient.  Squares below fp32's normal range (magnitudes under about 1e-19)
 * lose bits or count as zeros: rows of them take an eps well above 1e-38.
 *
 * The conventions of zr.h hold for every call: validation first, nothing launched and
 * nothing written on an error, asynchronous on `stream`, no device allocation,
 * capturable into a zr_graph.  Buffers need their element's natural alignment only.  The
 * same call gives the same bits every time, wherever its buffers lie.
 */
#ifndef ZR_ROPE_H
#define ZR_ROPE_H

#include "zr_fp8.h" /* zr_dtype */

#ifdef __cplusplus
extern "C" {
#endif

/* Largest head_dim, most axes, and rows of fp32 partial sums in the backward pass's
 * workspace. */
#define ZR_MAX_HEAD_DIM 512
#define ZR_MAX_ROPE_AXES 4
#define ZR_QK_PARTIALS 512

/* Heads of all tokens in device memory: the row of token t and head h is the head_dim
 * elements from ptr + t * token_stride + h * head_stride on (strides in elements).  Rows
 * must not overlap: with the strides of the axes longer than 1 in ascending order, the
 * smaller is at least head_dim and the larger at least what the other axis spans.
 * heads 0 stands for no heads (ptr is ignored). */
typedef struct zr_heads {
    void   *ptr;
    int64_t heads;
    int64_t token_stride;
    int64_t head_stride;
} zr_heads;

/* How pairs are turned. */
typedef struct zr_rope {
    const float   *inv_freq;    /* device fp32 [rot_dim / 2] */
    const uint8_t *pair_axis;   /* host [rot_dim / 2]: the axis of each pair; NULL: axis 0 */
    int32_t        rot_dim;     /* even, 0 <= rot_dim <= head_dim; 0: no rotation */
    int32_t        axes;        /* 1 ... ZR_MAX_ROPE_AXES */
    int32_t        interleaved; /* 0 or 1 */
} zr_rope;

/*
 * q_out, k_out = norm and rotation of q, k (dtype ZR_BF16 or ZR_F16; q_weight and
 * k_weight [head_dim] of the same type, or NULL: that tensor is turned and not normed).
 * q_out and k_out have the heads of q and k; q_out may be exactly q (same strides along the
 * axes longer than 1), k_out exactly k.  Otherwise no output may overlap another buffer; heads of one fused row
 * (equal token strides, ranges of the row that do not meet) do not count as overlapping.
 * positions: device int64 [axes][position_stride] with position_stride >= tokens where
 * axes > 1, or 0 where all axes share the first's; any values.  0 <= tokens <= 2^40 (0 is a
 * no-op), heads <= 65536, 1 <= head_dim <= ZR_MAX_HEAD_DIM, eps finite and >= 0.  positions
 * may be NULL where rot_dim is 0.
 * Errors: ZR_EINVAL, ZR_EALIGN, ZR_EHIP.
 */
ZR_API zr_status zr_qk_norm_rope(const zr_heads *q, const zr_heads *k, const void *q_weight, const void *k_weight,
                                 zr_dtype dtype, int64_t tokens, int64_t head_dim, double eps,
                                 const int64_t *positions, int64_t position_stride, const zr_rope *rope,
                                 const zr_heads *q_out, const zr_heads *k_out, void *stream);

/*
 * Gradients from dq, dk (of q_out and k_out) and the forward pass's q, k, weights, eps and
 * positions.  With g = the output's gradient turned back and xh = x * rstd (rstd is worked
 * out again from x, which is read anyway):
 *   dweight = sum over tokens and heads of g * xh
 *   dx      = rstd * (g * weight - xh * mean of g * weight * xh)
 * and dx = g, with x not read, where the weight is NULL.  dq_in may be exactly dq or
 * exactly q (same strides), dk_in exactly dk or k; otherwise as above.  dq_weight, dk_weight
 * [head_dim] of type dtype, needed with q_weight, k_weight and ignored without.
 * workspace: fp32 [ZR_QK_PARTIALS * head_dim], contents undefined before and after, needed
 * with a weight; two calls that may run at once need workspaces of their own, and so do two
 * graphs whose replays may.  tokens == 0 writes dq_weight = dk_weight = 0 and nothing else;
 * so does a tensor without heads for its weight.
 * Errors: ZR_EINVAL, ZR_EALIGN, ZR_EHIP.
 */
ZR_API zr_status zr_qk_norm_rope_backward(const zr_heads *dq, const zr_heads *dk, const zr_heads *q, const zr_heads *k,
                                          const void *q_weight, const void *k_weight, zr_dtype dtype, int64_t tokens,
                                          int64_t head_dim, double eps, const int64_t *positions,
                                          int64_t position_stride, const zr_rope *rope, const zr_heads *dq_in,
                                          const zr_heads *dk_in, void *dq_weight, void *dk_weight, float *workspace,
                                          void *stream);

#ifdef __cplusplus
}
#endif

#endif /* ZR_ROPE_H */
