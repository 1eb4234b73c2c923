// Entry points of include/tg_ops.h: argument checks, and the products each
// operator runs (their kernels are in the per-type translation units).
#include "tg_fused.hpp"

namespace tg {
typedef const TileArgs& Prod;
tg_status linear_f16(Prod t, const EpiArgs& e, int y_dtype, void* ws, int64_t ws_bytes, void* stream);
tg_status linear_bf16(Prod t, const EpiArgs& e, int y_dtype, void* ws, int64_t ws_bytes, void* stream);
tg_status linear_fp8(Prod t, const EpiArgs& e, int y_dtype, void* ws, int64_t ws_bytes, void* stream);
int64_t linear_ws_bytes_f16(int64_t M, int64_t N, int64_t K);
int64_t linear_ws_bytes_bf16(int64_t M, int64_t N, int64_t K);
int64_t linear_ws_bytes_fp8(int64_t M, int64_t N, int64_t K);
tg_status glu_f16(Prod t, const EpiArgs& e, int h_dtype, void* ws, int64_t ws_bytes, void* stream);
tg_status glu_bf16(Prod t, const EpiArgs& e, int h_dtype, void* ws, int64_t ws_bytes, void* stream);
tg_status glu_fp8(Prod t, const EpiArgs& e, int h_dtype, void* ws, int64_t ws_bytes, void* stream);
int64_t glu_ws_bytes_f16(int64_t M, int64_t F, int64_t D);
int64_t glu_ws_bytes_bf16(int64_t M, int64_t F, int64_t D);
int64_t glu_ws_bytes_fp8(int64_t M, int64_t F, int64_t D);
tg_status wgrad_f16(Prod t, int c_dtype, void* ws, int64_t ws_bytes, void* stream);
tg_status wgrad_bf16(Prod t, int c_dtype, void* ws, int64_t ws_bytes, void* stream);
int64_t wgrad_ws_bytes_f16(int64_t N, int64_t K, int64_t M);
int64_t wgrad_ws_bytes_bf16(int64_t N, int64_t K, int64_t M);
tg_status xgrad_f16(Prod t, void* ws, int64_t ws_bytes, void* stream);
tg_status xgrad_bf16(Prod t, void* ws, int64_t ws_bytes, void* stream);
tg_status group_f16(const TileArgs* t, int n, int w_dtype, void* ws, int64_t ws_bytes, void* stream, bool* taken);
tg_status group_bf16(const TileArgs* t, int n, int w_dtype, void* ws, int64_t ws_bytes, void* stream, bool* taken);
int64_t group_ws_bytes_f16(const TileArgs* t, int n);
int64_t group_ws_bytes_bf16(const TileArgs* t, int n);
tg_status glu_dgu_f16(Prod t, const EpiArgs& e, void* ws, int64_t ws_bytes, void* stream);
tg_status glu_dgu_bf16(Prod t, const EpiArgs& e, void* ws, int64_t ws_bytes, void* stream);
tg_status dz_f16(const DzArgs& p, void* ws, int64_t ws_bytes, void* stream);
tg_status dz_bf16(const DzArgs& p, void* ws, int64_t ws_bytes, void* stream);

int64_t ex_workspace_bytes(int in, int64_t M, int64_t N, int64_t K, int b_layout);  // tg_ex.hip

static int64_t larger(int64_t a, int64_t b) { return a > b ? a : b; }

static int elem_bytes(int in) { return in == TG_IN_FP8 ? 1 : 2; }

static int64_t wgrad_ws(int in, int64_t N, int64_t K, int64_t M)
{
    return in == TG_IN_F16 ? wgrad_ws_bytes_f16(N, K, M) : wgrad_ws_bytes_bf16(N, K, M);
}

static int64_t linear_ws(int in, int64_t M, int64_t N, int64_t K)
{
    if (M < 0 || N < 0 || K < 0)
        return -1;
    switch (in) {
    case TG_IN_F16: return linear_ws_bytes_f16(M, N, K);
    case TG_IN_BF16: return linear_ws_bytes_bf16(M, N, K);
    case TG_IN_FP8: return linear_ws_bytes_fp8(M, N, K);
    default: return -1;
    }
}

static int64_t glu_ws(int in, int64_t M, int64_t F, int64_t D)
{
    if (M < 0 || F < 0 || D < 0)
        return -1;
    switch (in) {
    case TG_IN_F16: return glu_ws_bytes_f16(M, F, D);
    case TG_IN_BF16: return glu_ws_bytes_bf16(M, F, D);
    case TG_IN_FP8: return glu_ws_bytes_fp8(M, F, D);
    default: return -1;
    }
}

// Workspace of a backward pass's products, t[0] being dX's and t[1 .. n-1]
// weight gradients: the most of the grouped launch and of each product by
// itself (a call that leaves an output out runs them one by one).
static int64_t products_ws(int in, const TileArgs* t, int n)
{
    int64_t most = in == TG_IN_F16 ? group_ws_bytes_f16(t, n) : group_ws_bytes_bf16(t, n);
    for (int i = 0; i < n; ++i)
        most = larger(most, i == 0 ? ex_workspace_bytes(in, t[i].M, t[i].N, t[i].K, TG_ROW_MAJOR)
                                   : wgrad_ws(in, t[i].M, t[i].N, t[i].K));
    return most;
}

// A product of the workspace queries: rows as wide as its matrices
static TileArgs sizes(int64_t M, int64_t N, int64_t K, int64_t lda, int64_t ldb)
{
    TileArgs t{};
    t.M = M;
    t.N = N;
    t.K = K;
    t.lda = lda;
    t.ldb = ldb;
    return t;
}

static int64_t linear_bwd_ws(int in, int64_t M, int64_t N, int64_t K)
{
    if (M < 0 || N < 0 || K < 0 || (in != TG_IN_F16 && in != TG_IN_BF16))
        return -1;
    if (!dims_fit(M, N, K))
        return 0;
    const TileArgs t[] = {sizes(M, K, N, N, K), sizes(N, K, M, N, K)};
    return larger(products_ws(in, t, 2), dz_ws_bytes(M, N));
}

static int64_t glu_bwd_ws(int in, int64_t M, int64_t F, int64_t D)
{
    if (M < 0 || F < 0 || D < 0 || (in != TG_IN_F16 && in != TG_IN_BF16))
        return -1;
    if (!dims_fit(M, F, D) || !dims_fit(2 * F, 0, 0))
        return 0;
    const TileArgs t[] = {sizes(M, D, 2 * F, 2 * F, D), sizes(2 * F, D, M, 2 * F, D), sizes(D, F, M, D, F)};
    return larger(products_ws(in, t, 3), ex_workspace_bytes(in, M, F, D, TG_ROW_MAJOR));
}

// The products of a backward pass: t[0] is dX's (A . B with B row-major),
// t[1 .. n-1] are weight gradients (A^T . B, A stored K x M and B K x N); an
// output that was left out has C null.  All in one launch where that is
// taken, else one by one.
static tg_status products(int in, const TileArgs* t, int n, int w_dtype, void* ws, int64_t ws_bytes, void* stream)
{
    bool all = true, taken = false;
    for (int i = 0; i < n; ++i)
        all = all && t[i].C != nullptr;
    if (all) {
        const tg_status st = in == TG_IN_F16 ? group_f16(t, n, w_dtype, ws, ws_bytes, stream, &taken)
                                             : group_bf16(t, n, w_dtype, ws, ws_bytes, stream, &taken);
        if (taken || st != TG_OK)
            return st;
    }
    for (int i = 0; i < n; ++i) {
        if (t[i].C == nullptr || t[i].M == 0 || t[i].N == 0)
            continue;
        tg_status st;
        if (i == 0)
            st = in == TG_IN_F16 ? xgrad_f16(t[i], ws, ws_bytes, stream) : xgrad_bf16(t[i], ws, ws_bytes, stream);
        else
            st = in == TG_IN_F16 ? wgrad_f16(t[i], w_dtype, ws, ws_bytes, stream)
                                 : wgrad_bf16(t[i], w_dtype, ws, ws_bytes, stream);
        if (st != TG_OK)
            return st;
    }
    return TG_OK;
}

// first failing status of a list
static tg_status first_error(const tg_status* s, int n)
{
    for (int i = 0; i < n; ++i)
        if (s[i] != TG_OK)
            return s[i];
    return TG_OK;
}

static int same_dtype(int in) { return in == TG_IN_F16 ? TG_F16 : TG_BF16; }
}  // namespace tg

using namespace tg;

extern "C" int64_t tg_linear_workspace_bytes(tg_input in, int64_t M, int64_t N, int64_t K)
{
    return linear_ws(abi_int(in), M, N, K);
}

extern "C" int64_t tg_linear_backward_workspace_bytes(tg_input in, int64_t M, int64_t N, int64_t K)
{
    return linear_bwd_ws(abi_int(in), M, N, K);
}

extern "C" int64_t tg_glu_workspace_bytes(tg_input in, int64_t M, int64_t F, int64_t D)
{
    return glu_ws(abi_int(in), M, F, D);
}

extern "C" int64_t tg_glu_backward_workspace_bytes(tg_input in, int64_t M, int64_t F, int64_t D)
{
    return glu_bwd_ws(abi_int(in), M, F, D);
}

extern "C" tg_status tg_linear(tg_input in_arg, int64_t M, int64_t N, int64_t K, const void* x, int64_t ldx,
                               const void* W, int64_t ldw, const float* bias, tg_act act_arg, const void* residual,
                               int64_t ldr, float scale_x, float scale_w, void* Y, int64_t ldy, tg_dtype y_dtype_arg,
                               void* preact, int64_t ldz, void* workspace, int64_t workspace_bytes, void* stream)
{
    const int in = abi_int(in_arg), act = abi_int(act_arg), y_dtype = abi_int(y_dtype_arg);
    if (M < 0 || N < 0 || K < 0 || in < TG_IN_F16 || in > TG_IN_FP8 || !act_ok(act) || y_dtype < TG_F32 ||
        y_dtype > TG_BF16)
        return TG_ERR_INVALID_VALUE;
    if (!dims_fit(M, N, K, ldx, ldw, ldy) || !dims_fit(ldr, ldz, 0))
        return TG_ERR_NOT_SUPPORTED;
    if (in != TG_IN_FP8 && y_dtype != TG_F32 && y_dtype != same_dtype(in))
        return TG_ERR_NOT_SUPPORTED;
    if (in == TG_IN_FP8 && (!__builtin_isfinite(scale_x) || !__builtin_isfinite(scale_w)))
        return TG_ERR_INVALID_VALUE;
    const int eb = elem_bytes(in), ob = out_bytes(y_dtype);
    const tg_status st[] = {
        check_mat(x, M, N == 0 ? 0 : K, ldx, eb),
        check_mat(W, N, M == 0 ? 0 : K, ldw, eb),
        check_mat(Y, M, N, ldy, ob),
        residual == nullptr ? TG_OK : check_mat(residual, M, N, ldr, ob),
        preact == nullptr ? TG_OK : check_mat(preact, M, N, ldz, ob),
        ((uintptr_t)bias & 3u) ? TG_ERR_MISALIGNED : TG_OK,
        check_ws(workspace, workspace_bytes, workspace == nullptr ? 0 : linear_ws(in, M, N, K)),
    };
    const tg_status bad = first_error(st, sizeof st / sizeof st[0]);
    if (bad != TG_OK || M == 0 || N == 0)
        return bad;
    TileArgs t{};
    set_product(t, M, N, K, x, ldx, W, ldw, Y, ldy, in == TG_IN_FP8 ? scale_x * scale_w : 1.0f);
    EpiArgs e{};
    set_act(e, act);
    e.bias = bias;
    e.R = residual;
    e.ldr = ldr;
    e.Z = preact;
    e.ldz = ldz;
    switch (in) {
    case TG_IN_F16: return linear_f16(t, e, y_dtype, workspace, workspace_bytes, stream);
    case TG_IN_BF16: return linear_bf16(t, e, y_dtype, workspace, workspace_bytes, stream);
    default: return linear_fp8(t, e, y_dtype, workspace, workspace_bytes, stream);
    }
}

extern "C" tg_status tg_linear_backward(tg_input in_arg, int64_t M, int64_t N, int64_t K, const void* dY, int64_t lddy,
                                        const void* x, int64_t ldx, const void* W, int64_t ldw, const void* preact,
                                        int64_t ldz, tg_act act_arg, void* dZ, int64_t lddz, void* dX, int64_t lddx,
                                        void* dW, int64_t lddw, tg_dtype dw_dtype_arg, float* dbias, void* workspace,
                                        int64_t workspace_bytes, void* stream)
{
    const int in = abi_int(in_arg), act = abi_int(act_arg), dw_dtype = abi_int(dw_dtype_arg);
    if (M < 0 || N < 0 || K < 0 || in < TG_IN_F16 || in > TG_IN_FP8 || !act_ok(act) || dw_dtype < TG_F32 ||
        dw_dtype > TG_BF16)
        return TG_ERR_INVALID_VALUE;
    if (in == TG_IN_FP8 || (dw_dtype != TG_F32 && dw_dtype != same_dtype(in)))
        return TG_ERR_NOT_SUPPORTED;
    if (act == TG_ACT_NONE) {  // dZ is dY
        preact = nullptr;
        dZ = nullptr;
        ldz = lddz = 0;
    }
    if (!dims_fit(M, N, K, lddy, ldx, ldw) || !dims_fit(ldz, lddz, lddx, lddw))
        return TG_ERR_NOT_SUPPORTED;
    const tg_status st[] = {
        check_mat(dY, M, N, lddy, 2),
        dW == nullptr ? TG_OK : check_mat(x, M, N == 0 ? 0 : K, ldx, 2),
        dX == nullptr ? TG_OK : check_mat(W, N, M == 0 ? 0 : K, ldw, 2),
        act == TG_ACT_NONE ? TG_OK : check_mat(preact, M, N, ldz, 2),
        act == TG_ACT_NONE ? TG_OK : check_mat(dZ, M, N, lddz, 2),
        dX == nullptr ? TG_OK : check_mat(dX, M, K, lddx, 2),
        dW == nullptr ? TG_OK : check_mat(dW, N, K, lddw, out_bytes(dw_dtype)),
        ((uintptr_t)dbias & 3u) ? TG_ERR_MISALIGNED : TG_OK,
        check_ws(workspace, workspace_bytes, workspace == nullptr ? 0 : linear_bwd_ws(in, M, N, K)),
    };
    tg_status bad = first_error(st, sizeof st / sizeof st[0]);
    if (bad != TG_OK)
        return bad;
    if (N > 0 && (dbias != nullptr || (act != TG_ACT_NONE && M > 0))) {
        DzArgs p{};
        p.M = M;
        p.N = N;
        p.dY = dY;
        p.lddy = lddy;
        p.dZ = dZ;
        p.lddz = lddz;
        p.db = dbias;
        set_act(p.e, act);
        p.e.R = preact;
        p.e.ldr = ldz;
        bad = in == TG_IN_F16 ? dz_f16(p, workspace, workspace_bytes, stream)
                              : dz_bf16(p, workspace, workspace_bytes, stream);
        if (bad != TG_OK)
            return bad;
    }
    const void* d = act == TG_ACT_NONE ? dY : dZ;
    const int64_t ldd = act == TG_ACT_NONE ? lddy : lddz;
    TileArgs t[2] = {};
    set_product(t[0], M, K, N, d, ldd, W, ldw, dX, lddx, 1.0f);
    set_product(t[1], N, K, M, d, ldd, x, ldx, dW, lddw, 1.0f);
    return products(in, t, 2, dw_dtype, workspace, workspace_bytes, stream);
}

extern "C" tg_status tg_glu(tg_input in_arg, int64_t M, int64_t F, int64_t D, const void* x, int64_t ldx,
                            const void* W, int64_t ldw, tg_act act_arg, float scale_x, float scale_w, void* H,
                            int64_t ldh, tg_dtype h_dtype_arg, void* gate_up, int64_t ldgu, void* workspace,
                            int64_t workspace_bytes, void* stream)
{
    const int in = abi_int(in_arg), act = abi_int(act_arg), h_dtype = abi_int(h_dtype_arg);
    if (M < 0 || F < 0 || D < 0 || in < TG_IN_F16 || in > TG_IN_FP8 || !act_ok(act) || h_dtype < TG_F32 ||
        h_dtype > TG_BF16)
        return TG_ERR_INVALID_VALUE;
    if (!dims_fit(M, F, D, ldx, ldw, ldh) || !dims_fit(2 * F, ldgu, 0))
        return TG_ERR_NOT_SUPPORTED;
    if (h_dtype == TG_F32 || (in != TG_IN_FP8 && h_dtype != same_dtype(in)))
        return TG_ERR_NOT_SUPPORTED;
    if (in == TG_IN_FP8 && (!__builtin_isfinite(scale_x) || !__builtin_isfinite(scale_w)))
        return TG_ERR_INVALID_VALUE;
    const int eb = elem_bytes(in);
    const tg_status st[] = {
        check_mat(x, M, F == 0 ? 0 : D, ldx, eb),
        check_mat(W, 2 * F, M == 0 ? 0 : D, ldw, eb),
        check_mat(H, M, F, ldh, 2),
        gate_up == nullptr ? TG_OK : check_mat(gate_up, M, 2 * F, ldgu, 2),
        check_ws(workspace, workspace_bytes, workspace == nullptr ? 0 : glu_ws(in, M, F, D)),
    };
    const tg_status bad = first_error(st, sizeof st / sizeof st[0]);
    if (bad != TG_OK || M == 0 || F == 0)
        return bad;
    TileArgs t{};
    set_product(t, M, F, D, x, ldx, W, ldw, H, ldh, in == TG_IN_FP8 ? scale_x * scale_w : 1.0f);
    EpiArgs e{};
    set_act(e, act);
    e.Z = gate_up;
    e.ldz = ldgu;
    switch (in) {
    case TG_IN_F16: return glu_f16(t, e, h_dtype, workspace, workspace_bytes, stream);
    case TG_IN_BF16: return glu_bf16(t, e, h_dtype, workspace, workspace_bytes, stream);
    default: return glu_fp8(t, e, h_dtype, workspace, workspace_bytes, stream);
    }
}

extern "C" tg_status tg_glu_backward(tg_input in_arg, int64_t M, int64_t F, int64_t D, const void* dY, int64_t lddy,
                                     const void* Wd, int64_t ldwd, const void* x, int64_t ldx, const void* W,
                                     int64_t ldw, const void* gate_up, int64_t ldgu, const void* H, int64_t ldh,
                                     tg_act act_arg, void* dgate_up, int64_t lddgu, void* dX, int64_t lddx, void* dW,
                                     int64_t lddw, void* dWd, int64_t lddwd, tg_dtype dw_dtype_arg, void* workspace,
                                     int64_t workspace_bytes, void* stream)
{
    const int in = abi_int(in_arg), act = abi_int(act_arg), dw_dtype = abi_int(dw_dtype_arg);
    if (M < 0 || F < 0 || D < 0 || in < TG_IN_F16 || in > TG_IN_FP8 || !act_ok(act) || dw_dtype < TG_F32 ||
        dw_dtype > TG_BF16)
        return TG_ERR_INVALID_VALUE;
    if (in == TG_IN_FP8 || (dw_dtype != TG_F32 && dw_dtype != same_dtype(in)))
        return TG_ERR_NOT_SUPPORTED;
    if (!dims_fit(M, F, D, lddy, ldwd, ldx) || !dims_fit(2 * F, ldw, ldgu, ldh, lddgu, lddx) || !dims_fit(lddw, lddwd, 0))
        return TG_ERR_NOT_SUPPORTED;
    const int gb = out_bytes(dw_dtype);
    const tg_status st[] = {
        check_mat(dY, M, D, lddy, 2),
        check_mat(Wd, D, M == 0 ? 0 : F, ldwd, 2),
        dW == nullptr ? TG_OK : check_mat(x, M, F == 0 ? 0 : D, ldx, 2),
        dX == nullptr ? TG_OK : check_mat(W, 2 * F, M == 0 ? 0 : D, ldw, 2),
        check_mat(gate_up, M, 2 * F, ldgu, 2),
        dWd == nullptr ? TG_OK : check_mat(H, M, D == 0 ? 0 : F, ldh, 2),
        check_mat(dgate_up, M, 2 * F, lddgu, 2),
        dX == nullptr ? TG_OK : check_mat(dX, M, D, lddx, 2),
        dW == nullptr ? TG_OK : check_mat(dW, 2 * F, D, lddw, gb),
        dWd == nullptr ? TG_OK : check_mat(dWd, D, F, lddwd, gb),
        check_ws(workspace, workspace_bytes, workspace == nullptr ? 0 : glu_bwd_ws(in, M, F, D)),
    };
    tg_status bad = first_error(st, sizeof st / sizeof st[0]);
    if (bad != TG_OK)
        return bad;
    if (M > 0 && F > 0) {
        TileArgs t{};
        set_product(t, M, F, D, dY, lddy, Wd, ldwd, dgate_up, lddgu, 1.0f);
        EpiArgs e{};
        set_act(e, act);
        e.R = gate_up;
        e.ldr = ldgu;
        bad = in == TG_IN_F16 ? glu_dgu_f16(t, e, workspace, workspace_bytes, stream)
                              : glu_dgu_bf16(t, e, workspace, workspace_bytes, stream);
        if (bad != TG_OK)
            return bad;
    }
    TileArgs t[3] = {};
    set_product(t[0], M, D, 2 * F, dgate_up, lddgu, W, ldw, dX, lddx, 1.0f);
    set_product(t[1], 2 * F, D, M, dgate_up, lddgu, x, ldx, dW, lddw, 1.0f);
    set_product(t[2], D, F, M, dY, lddy, H, ldh, dWd, lddwd, 1.0f);
    return products(in, t, 3, dw_dtype, workspace, workspace_bytes, stream);
}
