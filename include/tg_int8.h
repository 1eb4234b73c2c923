/*
 * tg_int8.h -- linear layers in 8-bit integers on the tile GEMM library
 * (libtg.so, MI355X / gfx950): matrices quantized to int8 with a scale for
 * each row, and their product with the epilogue of tg_linear.  The conventions
 * of tg.h and tg_ops.h hold: device pointers owned by the caller, row-major
 * matrices 16-byte aligned with leading dimensions (in elements) of whole 16
 * bytes, asynchronous execution on `stream`, synchronous validation before any
 * HIP call, status codes, sizes up to 2^31 - 1, enums read as ints.  Nothing is
 * allocated and no state is kept; a call may be captured in a HIP graph.
 */
#ifndef TG_INT8_H
#define TG_INT8_H

#include "tg.h"
#include "tg_ops.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Rows of x to int8, symmetric: scale[m] = max over k of |x[m][k]| times 1/127
 * (the fp32 number) and q[m][k] = x[m][k] / scale[m], each rounded to fp32, the
 * quotient then to the nearest whole number (ties to even) and held within
 * -127 .. 127.  A
 * row of zeros has the scale 0 and q 0.  A NaN or an infinity in a row makes
 * its scale NaN or infinity (q of such values 0), so that products of it do not
 * look finite.  Activations of M tokens give a scale per token, a weight N x K
 * one per channel.
 *   x     : M x K of x_dtype (TG_F32, TG_F16 or TG_BF16)
 *   q     : int8, M x K;   scale : fp32 [M], 4-byte aligned
 * Columns of q between K and ldq are left as they are. */
tg_status tg_quantize_i8(tg_dtype x_dtype, int64_t M, int64_t K, const void *x, int64_t ldx,
                         int8_t *q, int64_t ldq, float *scale, void *stream);

/* Y = act(scale_x[m] scale_w[n] (x . W^T) + bias) + residual
 *   x : int8 M x K, W : int8 N x K (the nn.Linear layout); K a multiple of 16
 *       and below 131072, else TG_ERR_NOT_SUPPORTED: the sums are exact int32
 *       (so are more than 32 rows with 256 ldx + K or 256 ldw + K at 2^31 - 16 or
 *       above: offsets within a tile are 32 bits wide)
 *   scale_x : fp32 [M], scale_w : fp32 [N];  bias : fp32 [N] or NULL
 *   residual : M x N of y_dtype, or NULL; may be Y itself (same pointer and ld)
 * The sum is rounded to fp32 once, scales, bias, activation and residual are
 * fp32, and Y is rounded once to y_dtype (any).  The workspace is tg_ops.h's,
 * or NULL.  M == 0 or N == 0 is a no-op; K == 0 takes an empty sum. */
tg_status tg_linear_i8(int64_t M, int64_t N, int64_t K, const int8_t *x, int64_t ldx,
                       const int8_t *W, int64_t ldw, const float *scale_x, const float *scale_w,
                       const float *bias, tg_act act, const void *residual, int64_t ldr,
                       void *Y, int64_t ldy, tg_dtype y_dtype,
                       void *workspace, int64_t workspace_bytes, void *stream);

int64_t tg_linear_i8_workspace_bytes(int64_t M, int64_t N, int64_t K);

#ifdef __cplusplus
}
#endif

#endif /* TG_INT8_H */
