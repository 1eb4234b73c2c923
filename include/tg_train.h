/*
 * tg_train.h -- the two ends of a training step of language models on the
 * tile GEMM library (libtg.so, MI355X / gfx950): the loss over a vocabulary
 * with its gradient, whose logits are never stored, and the AdamW update.
 * The conventions of tg.h and tg_ops.h hold for every call here: device
 * pointers owned by the caller, row-major matrices with a leading dimension
 * in elements, matrices 16-byte aligned with leading dimensions of whole 16
 * bytes, asynchronous execution on `stream`, synchronous validation before
 * any HIP call, status codes, sizes up to 2^31 - 1, enums read as ints.
 * Nothing is allocated and no state is kept; a call may be captured in a HIP
 * graph.  Results do not depend on the order in which workgroups finish:
 * repeated calls are bit-identical.
 *
 * workspace: 256-byte aligned device memory whose first 64 KiB are zero
 * before first use and left zero, one per concurrently running call (as for
 * tg_gemm_ex: one workspace serves every call of the library that it is large
 * enough for).
 */
#ifndef TG_TRAIN_H
#define TG_TRAIN_H

#include "tg.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Softmax cross entropy of a vocabulary projection:
 *   t[m][v] = scale x[m] . W[v];   lse[m] = log(sum over v of e^t[m][v])
 *   loss[m] = lse[m] - t[m][targets[m]] + z_loss lse[m]^2;  0 where
 *             targets[m] == ignore_index
 *   x       : M x D, W : V x D (the nn.Linear layout), TG_IN_F16 or TG_IN_BF16
 *   targets : int64 [M]; one that is neither ignore_index nor in 0 .. V - 1
 *             makes its loss (and its gradients) NaN
 *   loss, lse : fp32 [M], each may be NULL (lse is what the gradient needs;
 *             ignored rows have one too)
 *   total   : fp32 [2] or NULL: the sum of the losses and the number of rows
 *             that are not ignored (their quotient is the mean loss)
 * Logits and sums are fp32 and are not stored: a product's tile leaves the
 * maximum and the sum of its columns.  A logit of NaN or infinity makes its
 * row's lse and loss NaN (-infinity counts as probability 0).
 * D has to be a multiple of 8, scale log2(e) (in fp32) and z_loss finite; V > 0
 * unless M == 0.
 * Offsets within a tile are 32 bits wide: 512 ldx + 2 D and 512 ldw + 2 D have
 * to be below 2^31 - 16, and for the gradient ldw at most 1398100, else
 * TG_ERR_NOT_SUPPORTED (and 0 from the queries).
 * The workspace is required when M > 0 or total is given (with M == 0 total
 * receives two zeros); its query holds for M == 0 too. */
tg_status tg_linear_xent(tg_input in, int64_t M, int64_t V, int64_t D,
                         const void *x, int64_t ldx, const void *W, int64_t ldw,
                         float scale, const int64_t *targets, int64_t ignore_index, float z_loss,
                         float *loss, float *lse, float *total,
                         void *workspace, int64_t workspace_bytes, void *stream);

int64_t tg_linear_xent_workspace_bytes(tg_input in, int64_t M, int64_t V, int64_t D);

/* Gradients of sum over m of g[m] loss[m], g[m] = grad_scale dloss[m] / count:
 *   dt[m][v] = g[m] (e^(t - lse) (1 + 2 z_loss lse) - (v == targets[m]));  0 in ignored rows
 *   dX = scale dt . W;   dW = scale dt^T . x
 *   lse   : fp32 [M], as tg_linear_xent wrote it
 *   dloss : fp32 [M], or NULL (1); not read in ignored rows
 *   total : as tg_linear_xent wrote it, or NULL: count is max(total[1], 1), or 1
 *   dX    : M x D of the input type, or NULL
 *   dW    : V x D of dw_dtype (TG_F32 or the input type), or NULL
 * Each output that is given is overwritten; with M == 0 dW is zero.  Outputs
 * must not overlap inputs or one another.  grad_scale and scale grad_scale have
 * to be finite in fp32.
 * dt is computed in pieces of the vocabulary from logits that are computed
 * again, and rounded to the input type (relative to the largest finite dloss, for
 * fp16 2^12 times that, so that small probabilities keep their digits): the
 * 16-bit operand of the two products, whose sums are fp32 over all pieces.
 * An ignored row adds zero times its x to dW: it has to hold finite values.
 *
 * The workspace is required (with an output given and V > 0); 128 MiB of it are
 * for partial sums whatever the sizes.  The rest sets the pieces: the library
 * takes as few as fit it, and adds dX in another order where that changes them.
 * workspace_bytes(piece) reports what pieces of `piece` columns need (rounded up
 * to a multiple of 256), for any ldw; piece 0 stands for the size past which
 * more gives nothing, piece 1 for the least. */
tg_status tg_linear_xent_backward(tg_input in, int64_t M, int64_t V, int64_t D,
                                  const void *x, int64_t ldx, const void *W, int64_t ldw,
                                  float scale, const int64_t *targets, int64_t ignore_index, float z_loss,
                                  const float *lse, const float *dloss, float grad_scale, const float *total,
                                  void *dX, int64_t lddx,
                                  void *dW, int64_t lddw, tg_dtype dw_dtype,
                                  void *workspace, int64_t workspace_bytes, void *stream);

int64_t tg_linear_xent_backward_workspace_bytes(tg_input in, int64_t M, int64_t V, int64_t D, int64_t piece);

/* One AdamW step over `count` tensors:
 *   g' = g min(1, max_norm / (*norm + 1e-6))        (norm NULL: g)
 *   m' = beta1 m + (1 - beta1) g';   v' = beta2 v + (1 - beta2) g'^2
 *   w' = w (1 - lr weight_decay) - lr / (1 - beta1^step) m' / (sqrt(v' / (1 - beta2^step)) + eps)
 * `tensors` is a HOST array, read before the call returns; its pointers are
 * device memory of contiguous tensors of n elements (n == 0: skipped),
 * aligned to their elements (16-byte aligned ones run faster):
 *   param     : p_dtype; receives w' (rounded); w itself where master is NULL
 *   master    : fp32 w, updated, or NULL (16-bit weights only)
 *   grad      : g_dtype
 *   exp_avg, exp_avg_sq : m and v, updated.  fp32, or with 8-bit states OCP
 *               e4m3 in blocks of 256 consecutive elements: m = scale q and
 *               sqrt(v) = scale q with a scale per block,
 *   exp_avg_scale, exp_avg_sq_scale : fp32 [ceil(n / 256)], or both NULL (fp32
 *               states).  All tensors of a call have one kind of states.
 *   Held in 8 bits, a state's scale is its block's largest finite value / 448 (0,
 *   and the block zeros, below 2^-100), its values are rounded to nearest even
 *   (one that is not finite is held as NaN), and a nonzero sqrt(v) is kept at
 *   e4m3's smallest step or above, so that no update divides by eps alone.  The
 *   update takes the new m and v before they are rounded.
 *   norm      : device fp32 [1], the gradients' norm as tg_clip_grads writes
 *               it (with max_norm infinity it leaves the gradients as they
 *               are), or NULL.  Where it is NaN or infinite the step changes
 *               nothing.
 *   step_dev, lr_dev : device int64 [1] and fp32 [1] that stand for step and lr
 *               (which are then not looked at), or NULL: for a captured step,
 *               whose graph moves them on.  step_dev has to hold 1 or more.
 * Tensors must not overlap.  All arithmetic is fp32 on fp32 constants that
 * are computed in fp64; square root and division are off by 2 units in the
 * last place at most together, also of a subnormal v.  step >= 1, betas in
 * [0, 1), eps >= 0 (below 2^-126 it counts as that; 0 makes 0 / 0 of a weight
 * whose m' and v' are 0), max_norm >= 0 (infinity: no clipping), lr and
 * weight_decay finite, else TG_ERR_INVALID_VALUE. */
typedef struct {
    void *param;
    float *master;
    const void *grad;
    void *exp_avg, *exp_avg_sq;
    float *exp_avg_scale, *exp_avg_sq_scale;
    int64_t n;
    int32_t p_dtype, g_dtype; /* tg_dtype values */
} tg_adamw_tensor;

tg_status tg_adamw(int64_t count, const tg_adamw_tensor *tensors, int64_t step,
                   double lr, double beta1, double beta2, double eps, double weight_decay,
                   const float *norm, float max_norm,
                   const int64_t *step_dev, const float *lr_dev, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* TG_TRAIN_H */
