/*
 * zr_fp8.h -- the 8-bit floating-point operators of libzr: what a training
 * step runs between the parameter gather and the gradient reduce of zr.h when
 * its linear layers multiply 8-bit codes.
 *
 *   zr_quantize_fp8       codes and block scales of a matrix, and of its
 *                         transpose from the same read
 *   zr_matmul_fp8         product of two matrices of codes: the forward, input
 *                         gradient and weight gradient products of a linear
 *                         layer
 *   zr_rmsnorm_fp8        residual addition, root-mean-square norm and 8-bit
 *                         output in one pass
 *   zr_rmsnorm_backward   gradients of that norm
 *
 * Codes and scales.  A code is one byte, OCP e4m3 (largest value 448, one NaN
 * per sign, no infinity) or OCP e5m2 (largest value 57344).  A group of
 * ZR_FP8_GROUP = 128 consecutive elements of a row (or a block of 128 x 128
 * elements) shares one scale, a power of two held as one E8M0 byte s, which
 * stands for 2^(s - 127); s = 255 stands for NaN.  An element's value is code *
 * scale.  The scale of a group with largest magnitude amax is the smallest 2^e,
 * e >= -127, with amax <= MAX * 2^e (MAX the format's largest value; e = -127 for
 * a group of zeros), and the code is x * 2^-e rounded once, to nearest even:
 * codes and scales are exact functions of the input bits.  A group that holds
 * an infinity or a NaN gets scale 255 and NaN codes (0x7f), so that every sum
 * that uses it is NaN.  A row of `cols` elements has ceil(cols / 128) groups,
 * the last possibly short, and scales are row-major with no gaps: a flat shard
 * quantized as one row has its scales in flat order, and where row lengths are
 * multiples of 128 those are the scales of its rows.
 *
 * The conventions of zr.h hold for every call: validation first, nothing
 * launched and nothing written on an error, asynchronous on `stream`, no device
 * allocation, capturable into a zr_graph.  Matrices are row-major; `ld` arguments
 * are the distance between rows in elements (>= the row length).  Buffers need
 * their element's natural alignment only; products of matrices of codes whose base
 * and row distance are multiples of 16 bytes are the fast ones.  zr_matmul_fp8 may read up
 * to 15 bytes behind a matrix's last code, inside the aligned 16 bytes that hold it, and up to
 * 3 on either side of an array of scales, inside aligned words; what is there does not
 * count.  The same call gives
 * the same bits every time; the order of a product's fp32 sums, and with it their
 * last bit, goes by the call's sizes and by that alignment, never by the machine's
 * state.
 * Buffers that a call writes must not overlap any other of its buffers (as
 * address ranges from the first to the last element) except where stated.
 * Calls with disjoint outputs may run at once on different streams.
 */
#ifndef ZR_FP8_H
#define ZR_FP8_H

#include "zr.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Elements that share a scale along a row. */
#define ZR_FP8_GROUP 128

/* Rows of fp32 partial sums in zr_rmsnorm_backward's workspace. */
#define ZR_RMSNORM_PARTIALS 512

/* Element types of unquantized matrices. */
typedef int32_t zr_dtype;
#define ZR_BF16 0
#define ZR_F16  1
#define ZR_F32  2

/* Code formats. */
typedef int32_t zr_fp8_format;
#define ZR_E4M3 0
#define ZR_E5M2 1

/*
 * Codes of src [rows, cols] (ZR_BF16 or ZR_F16).
 *
 * block_rows 1: q [rows, cols] with scales [rows, ceil(cols / 128)], a scale
 * for each group of 128 along a row; qt [cols, rows] with scales_t
 * [cols, ceil(rows / 128)] are the codes of src's transpose, grouped along
 * its own rows (the operands of a weight gradient, whose sum runs over tokens).
 * block_rows 128: q with scales [ceil(rows / 128), ceil(cols / 128)], a scale
 * for each 128 x 128 block; qt and scales_t are the transposes of q and scales
 * (one quantization serves a weight's forward and input gradient products).
 *
 * Either pair (q, scales) or (qt, scales_t) may be NULL, not both.  rows or
 * cols == 0 is a no-op.  Errors: ZR_EINVAL, ZR_EALIGN, ZR_EHIP.
 */
ZR_API zr_status zr_quantize_fp8(const void *src, zr_dtype dtype, int64_t rows, int64_t cols, int64_t ld,
                                 int32_t block_rows, zr_fp8_format format, uint8_t *q, int64_t ldq, uint8_t *scales,
                                 uint8_t *qt, int64_t ldqt, uint8_t *scales_t, void *stream);

/*
 * out[i][j] = sum over k of A[i][k] * B[j][k] (+ out[i][j] with accumulate), for
 * A [m, k] with a scale per group of a row and B [n, k] with a scale per group of
 * a row (b_block_rows 1: b_scales [n, ceil(k / 128)]) or per 128 x 128 block
 * (b_block_rows 128: b_scales [ceil(n / 128), ceil(k / 128)]).  Sums are taken in a
 * fixed order and the result is rounded once to out_dtype (ZR_BF16, ZR_F16 or
 * ZR_F32; values past fp16's range become infinities).  With a 16-bit out the matrix
 * unit's 8-bit path adds each run of 8 products, aligned to the largest of them
 * with 13 bits below it, and the runs in fp32: on normal data 1.4e-5 of the result,
 * far below the rounding to 16 bits; sums that cancel keep the error of their terms.
 * With ZR_F32 the codes are widened to bf16 and every addition is fp32, at half the
 * rate; an element (code * scale) below 2^-126 may count as 0 there, large ones count
 * whatever their size.  A's codes are a_format, B's are e4m3.
 *
 * The three products of a linear layer y = x W^T with W [n, k], x [t, k]:
 *   y  = zr_matmul_fp8(x, W)                      m, n, k = t, n, k
 *   dx = zr_matmul_fp8(dy, W's transpose)         m, n, k = t, k, n
 *   dW = zr_matmul_fp8(dy's transpose, x's transpose)  m, n, k = n, k, t
 * out may be a weight's piece of the flat gradient buffer (a contribution of
 * zr_reduce_slice); accumulate adds a further micro-batch.
 *
 * k == 0: out = 0 (unchanged with accumulate).  m or n == 0 is a no-op.  k is at most
 * 2^31 - 65 groups.
 * Errors: ZR_EINVAL, ZR_EALIGN, ZR_EHIP.
 */
ZR_API zr_status zr_matmul_fp8(const uint8_t *a, int64_t lda, const uint8_t *a_scales, zr_fp8_format a_format,
                               const uint8_t *b, int64_t ldb, const uint8_t *b_scales, int32_t b_block_rows, int64_t m,
                               int64_t n, int64_t k, void *out, zr_dtype out_dtype, int64_t ldo, int32_t accumulate,
                               void *stream);

/*
 * Residual addition, root-mean-square norm (Zhang & Sennrich, NeurIPS 2019) and
 * 8-bit output of rows x cols elements of type T = dtype (ZR_BF16 or ZR_F16):
 *   h    = T(x + residual)     (h = x when residual is NULL)
 *   rstd = 1 / sqrt(mean of h^2 over the row + eps)
 *   y    = h * rstd * weight   in fp32
 * The sum of squares is fp32 in a fixed order (a row whose sum passes fp32's range, with
 * magnitudes from about 1e19 on, has rstd 0).  h, which the next layer adds to
 * and the backward pass reads, is rounded to T before the norm, so that both
 * passes use the same h.  Outputs, each optional (NULL) but y and q not both:
 *   h          the stream (requires residual); may be exactly x or residual with
 *              the same row distance;
 *   y          T(y);
 *   q, scales  e4m3 codes of y with a scale per group of 128 of a row, made from
 *              the fp32 y (not from T(y));
 *   rstd       fp32 [rows].
 * cols >= 1; rows == 0 is a no-op.  eps finite and >= 0.  Row distances of absent
 * matrices are ignored.  Errors: ZR_EINVAL, ZR_EALIGN, ZR_EHIP.
 */
ZR_API zr_status zr_rmsnorm_fp8(const void *x, int64_t ldx, const void *residual, int64_t ldr, const void *weight,
                                zr_dtype dtype, int64_t rows, int64_t cols, double eps, void *h, int64_t ldh, void *y,
                                int64_t ldy, uint8_t *q, int64_t ldq, uint8_t *scales, float *rstd, void *stream);

/*
 * Gradients of zr_rmsnorm_fp8 from dy = the gradient of y and the h and rstd of
 * the forward pass (all matrices of type dtype, ZR_BF16 or ZR_F16):
 *   xh = h * rstd,  g = dy * weight
 *   dx = rstd * (g - xh * mean of g * xh over the row) + dh
 *   dweight[j] = sum over rows of dy * xh
 * dh (NULL for none) is the gradient that reaches the stream h from the layers
 * above; dx is the gradient of x and of residual alike.  dx may be exactly dy or
 * dh with the same row distance.  Sums are fp32; each output is rounded once.
 * workspace: fp32 [ZR_RMSNORM_PARTIALS * cols], contents undefined before and
 * after; two calls that may run at once need workspaces of their own, and so do
 * two graphs whose replays may.  rows == 0 writes dweight = 0 and nothing else.  cols >= 1.
 * Errors: ZR_EINVAL, ZR_EALIGN, ZR_EHIP.
 */
ZR_API zr_status zr_rmsnorm_backward(const void *dy, int64_t lddy, const void *h, int64_t ldh, const void *weight,
                                     const float *rstd, const void *dh, int64_t lddh, zr_dtype dtype, int64_t rows,
                                     int64_t cols, void *dx, int64_t lddx, void *dweight, float *workspace,
                                     void *stream);

#ifdef __cplusplus
}
#endif

#endif /* ZR_FP8_H */
