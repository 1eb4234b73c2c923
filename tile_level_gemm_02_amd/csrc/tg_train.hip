// Entry points of the vocabulary loss (include/tg_train.h): argument checks.
// Its kernels are in the per-type translation units; tg_adamw has its own.
#include "tg_xent.hpp"

namespace tg {
tg_status xent_forward_f16(const XentCall& q);
tg_status xent_forward_bf16(const XentCall& q);
tg_status xent_backward_f16(const XentCall& q);
tg_status xent_backward_bf16(const XentCall& q);

// 32-bit offsets within a tile of an operand, as nt_eligible asks
static bool width_fits(int64_t D, int64_t ld) { return 512 * ld + 2 * D < (int64_t)kNumRecords; }

// what both calls ask of their operands
static tg_status xent_check(const XentCall& q)
{
    if (q.M == 0)
        return TG_OK;
    if (q.V == 0 || q.target == nullptr || q.ws == nullptr)
        return TG_ERR_INVALID_VALUE;
    const tg_status st[] = {check_mat(q.x, q.M, q.D, q.ldx, 2), check_mat(q.W, q.V, q.D, q.ldw, 2)};
    for (tg_status s : st)
        if (s != TG_OK)
            return s;
    if ((uintptr_t)q.target & 7u)
        return TG_ERR_MISALIGNED;
    if (q.D % 8 != 0 || !width_fits(q.D, q.ldx) || !width_fits(q.D, q.ldw))
        return TG_ERR_NOT_SUPPORTED;
    return TG_OK;
}

static bool type_ok(int in) { return in == TG_IN_F16 || in == TG_IN_BF16; }
static bool misaligned4(const void* p) { return ((uintptr_t)p & 3u) != 0; }
}  // namespace tg

using namespace tg;

extern "C" int64_t tg_linear_xent_workspace_bytes(tg_input in_arg, int64_t M, int64_t V, int64_t D)
{
    if (M < 0 || V < 0 || D < 0 || !type_ok(abi_int(in_arg)))
        return -1;
    if (!dims_fit(M, V, D) || (M > 0 && !width_fits(D, D)))
        return 0;
    return xent_fwd_layout(M, V, kFusedSkinnyRows<E_BF16>).bytes;
}

extern "C" int64_t tg_linear_xent_backward_workspace_bytes(tg_input in_arg, int64_t M, int64_t V, int64_t D, int64_t piece)
{
    if (M < 0 || V < 0 || D < 0 || piece < 0 || !type_ok(abi_int(in_arg)))
        return -1;
    if (V == 0 || !dims_fit(M, V, D) || !width_fits(D, D))
        return 0;
    const int64_t n = xent_bwd_bytes(M, V, D, piece);
    return n < 0 ? 0 : n;
}

extern "C" tg_status tg_linear_xent(tg_input in_arg, int64_t M, int64_t V, int64_t D, const void* x, int64_t ldx, const void* W,
                                    int64_t ldw, float scale, const int64_t* targets, int64_t ignore_index, float z_loss,
                                    float* loss, float* lse, float* total, void* workspace, int64_t workspace_bytes,
                                    void* stream)
{
    const int in = abi_int(in_arg);
    if (M < 0 || V < 0 || D < 0 || in < TG_IN_F16 || in > TG_IN_FP8 || !__builtin_isfinite(xent_c(scale)) ||
        !__builtin_isfinite(z_loss))
        return TG_ERR_INVALID_VALUE;
    if (in == TG_IN_FP8 || !dims_fit(M, V, D, ldx, ldw))
        return TG_ERR_NOT_SUPPORTED;
    XentCall q{};
    q.M = M;
    q.V = V;
    q.D = D;
    q.x = x;
    q.ldx = ldx;
    q.W = W;
    q.ldw = ldw;
    q.scale = scale;
    q.target = targets;
    q.ignore = ignore_index;
    q.z = z_loss;
    q.loss = loss;
    q.lse_out = lse;
    q.total_out = total;
    q.ws = workspace;
    q.ws_bytes = workspace_bytes;
    q.s = (hipStream_t)stream;
    tg_status st = xent_check(q);
    if (st == TG_OK)
        st = check_ws(workspace, workspace_bytes, M == 0 && total == nullptr ? 0 : tg_linear_xent_workspace_bytes(in_arg, M, V, D));
    if (st == TG_OK && (misaligned4(loss) || misaligned4(lse) || misaligned4(total)))
        st = TG_ERR_MISALIGNED;
    if (st != TG_OK || (M == 0 && total == nullptr))
        return st;
    if (workspace == nullptr)  // (M == 0: a workgroup of no rows writes total's zeros)
        return TG_ERR_INVALID_VALUE;
    return in == TG_IN_F16 ? xent_forward_f16(q) : xent_forward_bf16(q);
}

extern "C" tg_status tg_linear_xent_backward(tg_input in_arg, int64_t M, int64_t V, int64_t D, const void* x, int64_t ldx,
                                             const void* W, int64_t ldw, float scale, const int64_t* targets,
                                             int64_t ignore_index, float z_loss, const float* lse, const float* dloss,
                                             float grad_scale, const float* total, void* dX, int64_t lddx, void* dW,
                                             int64_t lddw, tg_dtype dw_dtype_arg, void* workspace, int64_t workspace_bytes,
                                             void* stream)
{
    const int in = abi_int(in_arg), dw_dtype = abi_int(dw_dtype_arg);
    if (M < 0 || V < 0 || D < 0 || in < TG_IN_F16 || in > TG_IN_FP8 || dw_dtype < TG_F32 || dw_dtype > TG_BF16 ||
        !__builtin_isfinite(xent_c(scale)) || !__builtin_isfinite(z_loss) || !__builtin_isfinite(grad_scale) ||
        !__builtin_isfinite((float)((double)scale * (double)grad_scale)))
        return TG_ERR_INVALID_VALUE;
    if (in == TG_IN_FP8 || (dw_dtype != TG_F32 && dw_dtype != (in == TG_IN_F16 ? TG_F16 : TG_BF16)) ||
        !dims_fit(M, V, D, ldx, ldw, lddx) || !dims_fit(lddw, 0, 0))
        return TG_ERR_NOT_SUPPORTED;
    XentCall q{};
    q.M = M;
    q.V = V;
    q.D = D;
    q.x = x;
    q.ldx = ldx;
    q.W = W;
    q.ldw = ldw;
    q.scale = scale;
    q.target = targets;
    q.ignore = ignore_index;
    q.z = z_loss;
    q.lse = lse;
    q.dloss = dloss;
    q.total = total;
    q.grad_scale = grad_scale;
    q.dX = M == 0 ? nullptr : dX;
    q.lddx = lddx;
    q.dW = dW;
    q.lddw = lddw;
    q.dw_dtype = dw_dtype;
    q.ws = workspace;
    q.ws_bytes = workspace_bytes;
    q.s = (hipStream_t)stream;
    const bool nothing = D == 0 || (q.dX == nullptr && (dW == nullptr || V == 0));
    tg_status st = M > 0 && (nothing && workspace == nullptr) ? TG_OK : xent_check(q);
    if (st == TG_OK && M > 0 && !nothing && lse == nullptr)
        st = TG_ERR_INVALID_VALUE;
    if (st == TG_OK && dX != nullptr)
        st = check_mat(dX, M, D, lddx, 2);
    if (st == TG_OK && dW != nullptr)
        st = check_mat(dW, V, D, lddw, out_bytes(dw_dtype));
    if (st == TG_OK)
        st = check_ws(workspace, workspace_bytes, nothing || workspace == nullptr ? 0 : xent_bwd_least(M, V, D, ldw));
    if (st == TG_OK && !nothing && workspace == nullptr)
        st = TG_ERR_INVALID_VALUE;
    if (st == TG_OK && (misaligned4(lse) || misaligned4(dloss) || misaligned4(total)))
        st = TG_ERR_MISALIGNED;
    if (st != TG_OK || nothing)
        return st;
    return in == TG_IN_F16 ? xent_backward_f16(q) : xent_backward_bf16(q);
}
