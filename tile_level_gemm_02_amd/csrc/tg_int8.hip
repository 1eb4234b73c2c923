// Entry points of include/tg_int8.h, and the quantization of rows.
//
//   scale = max |x| (1 / 127);   q = round(x / scale)
//
// Bound by memory (x read, a byte per value written).  A workgroup takes a
// row; rows of up to 256 kQuantHeld pieces stay in registers between the
// maximum and the quotients, longer ones are read again (from L2).
#include "tg_int8.hpp"

namespace tg {
tg_status i8_linear_f32(const TileArgs& t, const I8Epi& e, void* ws, int64_t ws_bytes, hipStream_t s);
tg_status i8_linear_f16(const TileArgs& t, const I8Epi& e, void* ws, int64_t ws_bytes, hipStream_t s);
tg_status i8_linear_bf16(const TileArgs& t, const I8Epi& e, void* ws, int64_t ws_bytes, hipStream_t s);

constexpr int kQuantHeld = 4;  // 16-byte pieces per lane

struct QuantArgs {
    int64_t M, K;
    const void* x;
    int64_t ldx;
    int8_t* q;
    int64_t ldq;
    float* scale;
};

__device__ __forceinline__ uint32_t quant_bits(float x) { return bit_cast<uint32_t>(x) & 0x7FFFFFFFu; }

// x / scale as int8 (scale 0, NaN or infinity: 0, but for finite values over
// an infinite scale, which are 0 too)
__device__ __forceinline__ uint32_t quant_byte(float x, float scale)
{
    float r = __builtin_rintf(x / scale);
    r = r == r ? __builtin_fminf(__builtin_fmaxf(r, -127.0f), 127.0f) : 0.0f;
    r = scale == 0.0f ? 0.0f : r;
    return (uint32_t)(int)r & 0xFFu;
}

template <int O>
__device__ __forceinline__ void quant_store(int8_t* q, u32x4 v, float scale, int n)
{
    constexpr int VC = Piece<O>::N;
    uint32_t w[VC / 4];
#pragma unroll
    for (int i = 0; i < VC / 4; ++i) {
        w[i] = 0u;
#pragma unroll
        for (int e = 0; e < 4; ++e)
            w[i] |= quant_byte(piece_value<O>(v, 4 * i + e), scale) << (8 * e);
    }
    if (n == VC) {
        if constexpr (VC == 8)
            *(u32x2*)q = u32x2{w[0], w[1]};
        else
            *(uint32_t*)q = w[0];
    } else {
#pragma unroll
        for (int i = 0; i < VC; ++i)
            if (i < n)
                q[i] = (int8_t)(w[i / 4] >> (8 * (i % 4)));
    }
}

template <int O>
__global__ __launch_bounds__(256) void quantize_rows(QuantArgs p)
{
    constexpr int VC = Piece<O>::N;
    __shared__ uint32_t red[4];
    const uint32_t tid = threadIdx.x;
    const int64_t row = blockIdx.x, x0 = row * p.ldx;
    int8_t* const q = p.q + row * p.ldq;
    u32x4 held[kQuantHeld];
    uint32_t top = 0u;  // of the magnitudes' bits, whose order is the values'; NaN is above infinity
    auto piece = [&](int64_t k) __attribute__((always_inline)) -> u32x4 {
        const int64_t left = p.K - k;
        if (left <= 0)
            return u32x4{0u, 0u, 0u, 0u};
        return load_piece<O>(p.x, x0 + k, left < VC ? (int)left : VC, left >= VC);
    };
    auto raise = [&](u32x4 v) __attribute__((always_inline)) {
#pragma unroll
        for (int e = 0; e < VC; ++e) {
            const uint32_t b = quant_bits(piece_value<O>(v, e));
            top = b > top ? b : top;
        }
    };
#pragma unroll
    for (int i = 0; i < kQuantHeld; ++i)
        held[i] = piece(((int64_t)i * 256 + tid) * VC);
#pragma unroll
    for (int i = 0; i < kQuantHeld; ++i)
        raise(held[i]);
    for (int64_t k = ((int64_t)kQuantHeld * 256 + tid) * VC; k < p.K; k += 256 * VC)
        raise(piece(k));
#pragma unroll
    for (int d = 32; d > 0; d >>= 1) {
        const uint32_t o = (uint32_t)__shfl_xor((int)top, d, 64);
        top = o > top ? o : top;
    }
    if ((tid & 63u) == 0u)
        red[tid >> 6] = top;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 4; ++i)
        top = red[i] > top ? red[i] : top;
    const float scale = bit_cast<float>(top) * (1.0f / 127.0f);
    if (tid == 0u)
        p.scale[row] = scale;
    auto store = [&](int64_t k, u32x4 v) __attribute__((always_inline)) {
        const int64_t left = p.K - k;
        if (left > 0)
            quant_store<O>(q + k, v, scale, left < VC ? (int)left : VC);
    };
#pragma unroll
    for (int i = 0; i < kQuantHeld; ++i)
        store(((int64_t)i * 256 + tid) * VC, held[i]);
    for (int64_t k = ((int64_t)kQuantHeld * 256 + tid) * VC; k < p.K; k += 256 * VC)
        store(k, piece(k));
}
}  // namespace tg

using namespace tg;

extern "C" tg_status tg_quantize_i8(tg_dtype x_dtype_arg, int64_t M, int64_t K, const void* x, int64_t ldx, int8_t* q, int64_t ldq,
                                    float* scale, void* stream)
{
    const int t = abi_int(x_dtype_arg);
    if (M < 0 || K < 0 || t < TG_F32 || t > TG_BF16)
        return TG_ERR_INVALID_VALUE;
    if (!dims_fit(M, K, ldx, ldq))
        return TG_ERR_NOT_SUPPORTED;
    if (M == 0)
        return TG_OK;
    if (scale == nullptr)
        return TG_ERR_INVALID_VALUE;
    const tg_status st[] = {check_mat(x, M, K, ldx, out_bytes(t)), check_mat(q, M, K, ldq, 1),
                            ((uintptr_t)scale & 3u) ? TG_ERR_MISALIGNED : TG_OK};
    for (tg_status s : st)
        if (s != TG_OK)
            return s;
    const QuantArgs a{M, K, x, ldx, q, ldq, scale};
    hipStream_t s = (hipStream_t)stream;
    switch (t) {
    case TG_F32: hipLaunchKernelGGL(quantize_rows<O_F32>, dim3((uint32_t)M), dim3(256), 0, s, a); break;
    case TG_F16: hipLaunchKernelGGL(quantize_rows<O_F16>, dim3((uint32_t)M), dim3(256), 0, s, a); break;
    default: hipLaunchKernelGGL(quantize_rows<O_BF16>, dim3((uint32_t)M), dim3(256), 0, s, a); break;
    }
    return launched();
}

extern "C" int64_t tg_linear_i8_workspace_bytes(int64_t M, int64_t N, int64_t K)
{
    return M < 0 || N < 0 || K < 0 ? -1 : i8_ws_bytes(M, N, K);
}

extern "C" tg_status tg_linear_i8(int64_t M, int64_t N, int64_t K, const int8_t* x, int64_t ldx, const int8_t* W, int64_t ldw,
                                  const float* scale_x, const float* scale_w, const float* bias, tg_act act_arg,
                                  const void* residual, int64_t ldr, void* Y, int64_t ldy, tg_dtype y_dtype_arg, void* workspace,
                                  int64_t workspace_bytes, void* stream)
{
    const int act = abi_int(act_arg), y = abi_int(y_dtype_arg);
    if (M < 0 || N < 0 || K < 0 || !act_ok(act) || y < TG_F32 || y > TG_BF16)
        return TG_ERR_INVALID_VALUE;
    if (!dims_fit(M, N, K, ldx, ldw, ldy) || !dims_fit(ldr, 0, 0) || K % 16 != 0 || K >= 131072)
        return TG_ERR_NOT_SUPPORTED;
    const int ob = out_bytes(y);
    const bool none = M == 0 || N == 0;
    const tg_status st[] = {
        check_mat(x, M, N == 0 ? 0 : K, ldx, 1),
        check_mat(W, N, M == 0 ? 0 : K, ldw, 1),
        check_mat(Y, M, N, ldy, ob),
        residual == nullptr ? TG_OK : check_mat(residual, M, N, ldr, ob),
        !none && (scale_x == nullptr || scale_w == nullptr) ? TG_ERR_INVALID_VALUE : TG_OK,
        (((uintptr_t)bias | (uintptr_t)scale_x | (uintptr_t)scale_w) & 3u) ? TG_ERR_MISALIGNED : TG_OK,
        check_ws(workspace, workspace_bytes, workspace == nullptr ? 0 : i8_ws_bytes(M, N, K)),
    };
    for (tg_status s : st)
        if (s != TG_OK)
            return s;
    if (none)
        return TG_OK;
    TileArgs t{};
    set_product(t, M, N, K, (const uint8_t*)x, ldx, (const uint8_t*)W, ldw, Y, ldy, 1.0f);
    I8Epi e{};
    set_act(e, act);
    e.bias = bias;
    e.R = residual;
    e.ldr = ldr;
    e.sx = scale_x;
    e.sw = scale_w;
    switch (y) {
    case TG_F32: return i8_linear_f32(t, e, workspace, workspace_bytes, (hipStream_t)stream);
    case TG_F16: return i8_linear_f16(t, e, workspace, workspace_bytes, (hipStream_t)stream);
    default: return i8_linear_bf16(t, e, workspace, workspace_bytes, (hipStream_t)stream);
    }
}
