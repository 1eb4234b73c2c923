/*
 * tg_ops.h -- feed-forward operators of language models on the tile GEMM
 * library (libtg.so, MI355X / gfx950): matrix products with a fused epilogue,
 * their gradients, and gradient clipping.  The conventions of tg.h hold for
 * every call here: device pointers owned by the caller, row-major matrices
 * with a leading dimension in elements, every base pointer 16-byte aligned
 * and every leading dimension times the element size a multiple of 16,
 * asynchronous execution on `stream`, synchronous validation before any HIP
 * call, status codes, sizes up to 2^31 - 1, enums read as ints.  Nothing is
 * allocated and no state is kept; a call may be captured in a HIP graph.
 *
 * Notation: x is M x K activations (M tokens), W an N x K weight (the
 * nn.Linear layout, as TG_COL_MAJOR in tg.h).  All sums, activations and
 * their derivatives are fp32 on the unrounded accumulator; every stored value
 * is rounded once, to nearest even.  fp8 inputs (OCP e4m3) carry per-tensor
 * scales; their matrix instructions sum each group of 8 products to about 13
 * bits below the largest, so fp32 outputs of fp8 inputs hold about four
 * digits.
 *
 * Speed: sums that run along a matrix's rows take fast kernels where the rows
 * fill whole 16-byte chunks (multiples of 8 elements, 16 for fp8), and so do
 * the column counts of the gradients' products; other sizes run a tile kernel
 * that is several times slower.  So does a backward pass's product with a
 * row-major weight (dX = dZ . W, dH = dY . Wd) that spans 2 GiB or nearly, which
 * one buffer descriptor does not hold: at 24, 256 and 2048 tokens and K = 8192,
 * 130560 rows of bf16 W take 0.38, 0.70 and 3.4 ms, 131072 rows 5.3, 5.3 and 32.
 *
 * workspace: as for tg_gemm_ex (256-byte aligned device memory, first 64 KiB
 * zero before first use and left zero, one per concurrently running call, or
 * NULL with workspace_bytes 0: less is split then).  One workspace of the
 * largest size that the queries report serves every call.  A non-NULL
 * workspace smaller than the call's query reports is TG_ERR_INVALID_VALUE,
 * one not 256-byte aligned TG_ERR_MISALIGNED.  Results do not depend on the
 * order in which workgroups finish: repeated calls are bit-identical.
 */
#ifndef TG_OPS_H
#define TG_OPS_H

#include "tg.h"

#ifdef __cplusplus
extern "C" {
#endif

/* none x; relu max(x, 0); gelu x Phi(x); gelu_tanh x/2 (1 + tanh(sqrt(2/pi)
 * (x + 0.044715 x^3))); silu x / (1 + e^-x).  Derivatives are those of these
 * formulas, relu's taken as 0 at 0.  gelu's Phi is evaluated to 1.5e-7, and in
 * its negative tail to 3e-6 + 9e-8 x^2 of its value (1.2e-5 at -10).  The
 * formulas hold for every finite x; at infinity they are taken as they stand
 * (silu, gelu and gelu_tanh give inf at inf and NaN, 0 times inf, at -inf). */
typedef enum {
    TG_ACT_NONE = 0,
    TG_ACT_RELU = 1,
    TG_ACT_GELU = 2,
    TG_ACT_GELU_TANH = 3,
    TG_ACT_SILU = 4
} tg_act;

/* Y = act(Z) + residual with Z = scale_x scale_w (x . W^T) + bias.
 *   bias     : fp32 [N], 4-byte aligned, or NULL
 *   residual : M x N of y_dtype, or NULL; may be Y itself (same pointer and ld)
 *   preact   : M x N of y_dtype, or NULL: Z, kept for tg_linear_backward
 *   scales   : used for TG_IN_FP8 only (finite), ignored otherwise
 *   y_dtype  : TG_F32 or the input type for 16-bit inputs, any for fp8; else
 *              TG_ERR_NOT_SUPPORTED
 * M == 0 or N == 0 is a no-op; K == 0 takes an empty sum. */
tg_status tg_linear(tg_input in, int64_t M, int64_t N, int64_t K,
                    const void *x, int64_t ldx, const void *W, int64_t ldw,
                    const float *bias, tg_act act,
                    const void *residual, int64_t ldr,
                    float scale_x, float scale_w,
                    void *Y, int64_t ldy, tg_dtype y_dtype,
                    void *preact, int64_t ldz,
                    void *workspace, int64_t workspace_bytes, void *stream);

int64_t tg_linear_workspace_bytes(tg_input in, int64_t M, int64_t N, int64_t K);

/* Gradients of Y = act(Z) + residual (16-bit inputs; the residual's gradient
 * is dY itself):
 *   dZ = dY * act'(Z);   dX = dZ . W;   dW = dZ^T . x;   dbias = column sums of dZ
 *   dY     : M x N of the input type
 *   preact : Z, M x N of the input type; read only with an activation
 *   dZ     : M x N of the input type, written (rounded: the products below
 *            take it as their 16-bit operand); with TG_ACT_NONE dZ is dY, and
 *            preact and dZ are ignored.  May be dY itself (same pointer and ld).
 *   dX     : M x K of the input type, or NULL
 *   dW     : N x K of dw_dtype (TG_F32 or the input type), or NULL
 *   dbias  : fp32 [N], 4-byte aligned, or NULL (sums of the unrounded dZ)
 * Each output that is given is overwritten; with M == 0 dW and dbias are zero. */
tg_status tg_linear_backward(tg_input in, int64_t M, int64_t N, int64_t K,
                             const void *dY, int64_t lddy, const void *x, int64_t ldx,
                             const void *W, int64_t ldw,
                             const void *preact, int64_t ldz, tg_act act,
                             void *dZ, int64_t lddz,
                             void *dX, int64_t lddx,
                             void *dW, int64_t lddw, tg_dtype dw_dtype,
                             float *dbias,
                             void *workspace, int64_t workspace_bytes, void *stream);

int64_t tg_linear_backward_workspace_bytes(tg_input in, int64_t M, int64_t N, int64_t K);

/* The gated pair of a feed-forward block: g = s x . Wg^T, u = s x . Wu^T with
 * s = scale_x scale_w (fp8 only), H = act(g) * u.
 *   x       : M x D
 *   W       : 2F x D, the F rows of Wg and then those of Wu
 *   H       : M x F of h_dtype: the input type for 16-bit inputs, TG_F16 or
 *             TG_BF16 for fp8; else TG_ERR_NOT_SUPPORTED
 *   gate_up : M x 2F of h_dtype, or NULL: [g | u], kept for tg_glu_backward */
tg_status tg_glu(tg_input in, int64_t M, int64_t F, int64_t D,
                 const void *x, int64_t ldx, const void *W, int64_t ldw, tg_act act,
                 float scale_x, float scale_w,
                 void *H, int64_t ldh, tg_dtype h_dtype,
                 void *gate_up, int64_t ldgu,
                 void *workspace, int64_t workspace_bytes, void *stream);

int64_t tg_glu_workspace_bytes(tg_input in, int64_t M, int64_t F, int64_t D);

/* Gradients of the gated block y = H . Wd^T (16-bit inputs):
 *   dH = dY . Wd (not stored);  dg = dH * u * act'(g);  du = dH * act(g);
 *   dX = [dg | du] . W;   dW = [dg | du]^T . x;   dWd = dY^T . H
 *   dY       : M x D of the input type        Wd : D x F (the nn.Linear layout)
 *   gate_up  : [g | u], M x 2F                H  : M x F, read only for dWd
 *   dgate_up : M x 2F of the input type, written: [dg | du] (rounded: the
 *              16-bit operand of the two products); may be gate_up itself
 *   dX       : M x D of the input type, or NULL
 *   dW       : 2F x D of dw_dtype, or NULL;  dWd : D x F of dw_dtype, or NULL
 *              (TG_F32 or the input type)
 * Each output that is given is overwritten; with M == 0 dW and dWd are zero. */
tg_status tg_glu_backward(tg_input in, int64_t M, int64_t F, int64_t D,
                          const void *dY, int64_t lddy, const void *Wd, int64_t ldwd,
                          const void *x, int64_t ldx, const void *W, int64_t ldw,
                          const void *gate_up, int64_t ldgu, const void *H, int64_t ldh,
                          tg_act act,
                          void *dgate_up, int64_t lddgu,
                          void *dX, int64_t lddx,
                          void *dW, int64_t lddw, void *dWd, int64_t lddwd, tg_dtype dw_dtype,
                          void *workspace, int64_t workspace_bytes, void *stream);

int64_t tg_glu_backward_workspace_bytes(tg_input in, int64_t M, int64_t F, int64_t D);

/* Clip `count` gradients by their global norm:
 *   norm = sqrt(sum over all tensors of g^2)
 *   out  = g * min(1, max_norm / (norm + eps))
 *   grads, outs, sizes, dtypes : HOST arrays of `count` entries, read before
 *            the call returns: device pointers of contiguous tensors (aligned
 *            to their elements), their numbers of elements (0: skipped), and
 *            tg_dtype values.  outs[i] == grads[i] clips in place; tensors
 *            must not overlap otherwise.
 *   norm   : device fp32 [1] written with the norm before clipping, or NULL
 * Squares and their sum are fp64, the factor is rounded to fp32 and each
 * product once more to the tensor's type.  A norm of infinity gives the
 * factor 0 (and NaN where a gradient is infinite), a NaN makes every output
 * NaN.  max_norm >= 0 and eps >= 0, else TG_ERR_INVALID_VALUE.  Nothing is
 * clipped with norm + eps == 0, nor with max_norm infinity, an infinite norm
 * included.  The workspace is required (when count > 0 or norm is given). */
tg_status tg_clip_grads(int64_t count, const void *const *grads, void *const *outs,
                        const int64_t *sizes, const int32_t *dtypes,
                        float max_norm, float eps, float *norm,
                        void *workspace, int64_t workspace_bytes, void *stream);

int64_t tg_clip_grads_workspace_bytes(int64_t count);

#ifdef __cplusplus
}
#endif

#endif /* TG_OPS_H */
