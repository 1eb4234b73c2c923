// Entry points of include/tg_int8.h, and the quantization of rows.
//
//   scale = max |x| (1 / 127);   q = round(x / scale)
//
// Bound by memory (x read, a byte per value written).  A workgroup takes a
// row; what its lanes hold in HELD pieces of 16 bytes stays in registers between
// the maximum and the quotients, the rest of a longer row is read again (from L2).
#include "tg_int8.hpp"

namespace tg {
tg_status i8_linear_f32(const TileArgs& t, const I8Epi& e, void* ws, int64_t ws_bytes, hipStream_t s);
tg_status i8_linear_f16(const TileArgs& t, const I8Epi& e, void* ws, int64_t ws_bytes, hipStream_t s);
tg_status i8_linear_bf16(const TileArgs& t, const I8Epi& e, void* ws, int64_t ws_bytes, hipStream_t s);

constexpr int64_t kQuantRows = 1 << 22;  // rows of a launch at most (a launch has less than 2^32 lanes)
constexpr int64_t kQuantFew = 512;  // rows up to which a row takes 1024 lanes
// q past this leaves the L2s before a product reads it, and is stored with the
// non-temporal hint (8192 x 10240 bf16 49.3 -> 46.5 us, its product as it was;
// 1003 x 2064 and its product, hint and none: 35.4 and 32.4)
constexpr int64_t kQuantStream = (int64_t)32 << 20;

struct QuantArgs {
    int64_t M, K;
    const void* x;
    int64_t ldx;
    int8_t* q;
    int64_t ldq;
    float* scale;
};

typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));

// A running maximum of magnitudes, held as their bits, whose order is the
// values' (NaN above infinity): two 16-bit values side by side, or an fp32 one
template <int O>
__device__ __forceinline__ uint32_t raise_top(uint32_t top, uint32_t word)
{
    if constexpr (O == O_F32) {
        const uint32_t b = word & 0x7FFFFFFFu;
        return b > top ? b : top;
    } else {
        return bit_cast<uint32_t>(__builtin_elementwise_max(bit_cast<u16x2>(word & 0x7FFF7FFFu), bit_cast<u16x2>(top)));
    }
}

// x / scale as int8 by the definition (scale 0, or a quotient of NaN: 0)
__device__ __forceinline__ uint32_t quant_byte(float x, float scale)
{
    float r = __builtin_rintf(x / scale);
    r = r == r ? __builtin_fminf(__builtin_fmaxf(r, -127.0f), 127.0f) : 0.0f;
    r = scale == 0.0f ? 0.0f : r;
    return (uint32_t)(int)r & 0xFFu;
}

// The VC values of a piece as bytes.  A division is ten instructions, and with
// one for each value the divisions bound the whole kernel (8192 x 10240 bf16 56
// us, so 49).  So a value is multiplied by the scale's reciprocal, which is off
// from the rounded quotient by three roundings of 2^-24, 2.3e-5 of 127, and
// rounded by adding 1.5 2^23, whose low byte is then the answer; only a piece
// with a value nearer than 2^-15 = 3.1e-5 to a half divides.  `inv` is 0 where
// the scale is not a number the reciprocal serves (below 2^-100, infinite or
// NaN).  FAST false: divisions at once, for rows that are all latency.
template <int O, bool FAST>
__device__ __forceinline__ void quant_words(u32x4 v, float scale, float inv, uint32_t* w)
{
    constexpr int VC = Piece<O>::N;
    constexpr float MAGIC = 12582912.0f;
    float far = 0.0f;
#pragma unroll
    for (int i = 0; i < (FAST ? VC / 4 : 0); ++i) {
        uint32_t b[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const float x = piece_value<O>(v, 4 * i + e) * inv, r = x + MAGIC;
            far = __builtin_fmaxf(far, __builtin_fabsf(x - (r - MAGIC)));
            b[e] = bit_cast<uint32_t>(r);
        }
        const uint32_t lo = __builtin_amdgcn_perm(b[1], b[0], 0x0C0C0400u), hi = __builtin_amdgcn_perm(b[3], b[2], 0x04000C0Cu);
        w[i] = lo | hi;
    }
    if (!FAST || far > 0.5f - 0x1p-15f || inv == 0.0f) {
#pragma unroll
        for (int i = 0; i < VC / 4; ++i) {
            w[i] = 0u;
#pragma unroll
            for (int e = 0; e < 4; ++e)
                w[i] |= quant_byte(piece_value<O>(v, 4 * i + e), scale) << (8 * e);
        }
    }
}

template <int O, bool FAST, bool STREAM>
__device__ __forceinline__ void quant_store(int8_t* q, u32x4 v, float scale, float inv, int n)
{
    constexpr int VC = Piece<O>::N;
    uint32_t w[VC / 4];
    quant_words<O, FAST>(v, scale, inv, w);
    if (n == VC) {
        if constexpr (STREAM && VC == 8)
            store_nt((u32x2*)q, u32x2{w[0], w[1]});
        else if constexpr (VC == 8)
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

template <int O, int T, int HELD, bool STREAM = false>
__global__ __launch_bounds__(T) void quantize_rows(QuantArgs p)
{
    constexpr int VC = Piece<O>::N;
    __shared__ uint32_t red[T / 64];
    const uint32_t tid = threadIdx.x;
    const int64_t row = blockIdx.x, x0 = row * p.ldx;
    int8_t* const q = p.q + row * p.ldq;
    u32x4 held[HELD];
    uint32_t top = 0u;
    auto piece = [&](int64_t k) __attribute__((always_inline)) -> u32x4 {
        const int64_t left = p.K - k;
        if (left <= 0)
            return u32x4{0u, 0u, 0u, 0u};
        return load_piece<O>(p.x, x0 + k, left < VC ? (int)left : VC, left >= VC);
    };
    auto raise = [&](u32x4 v) __attribute__((always_inline)) {
#pragma unroll
        for (int e = 0; e < 4; ++e)
            top = raise_top<O>(top, v[e]);
    };
#pragma unroll
    for (int i = 0; i < HELD; ++i)
        held[i] = piece(((int64_t)i * T + tid) * VC);
#pragma unroll
    for (int i = 0; i < HELD; ++i)
        raise(held[i]);
    for (int64_t k = ((int64_t)HELD * T + tid) * VC; k < p.K; k += T * VC)
        raise(piece(k));
    if constexpr (O != O_F32) {  // the larger of the two, as fp32
        const uint32_t hi = top >> 16, lo = top & 0xFFFFu;
        top = bit_cast<uint32_t>(piece_value<O>(u32x4{hi > lo ? hi : lo, 0u, 0u, 0u}, 0));
    }
#pragma unroll
    for (int d = 32; d > 0; d >>= 1) {
        const uint32_t o = (uint32_t)__shfl_xor((int)top, d, 64);
        top = o > top ? o : top;
    }
    if ((tid & 63u) == 0u)
        red[tid >> 6] = top;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < T / 64; ++i)
        top = red[i] > top ? red[i] : top;
    const float scale = bit_cast<float>(top) * (1.0f / 127.0f);
    const float inv = scale >= 0x1p-100f && scale < INFINITY ? 1.0f / scale : 0.0f;
    if (tid == 0u)
        p.scale[row] = scale;
    auto store = [&](int64_t k, u32x4 v) __attribute__((always_inline)) {
        const int64_t left = p.K - k;
        if (left > 0)
            quant_store<O, T == 256, STREAM>(q + k, v, scale, inv, left < VC ? (int)left : VC);
    };
#pragma unroll
    for (int i = 0; i < HELD; ++i)
        store(((int64_t)i * T + tid) * VC, held[i]);
    for (int64_t k = ((int64_t)HELD * T + tid) * VC; k < p.K; k += T * VC)
        store(k, piece(k));
}

// Few rows leave the chip to one workgroup each, whose latency is the call:
// 1024 lanes of one or two pieces.  More rows take 256 lanes, holding as much
// of a row as it has up to eight pieces.
template <int O>
static void quantize_launch(QuantArgs a, hipStream_t s)
{
    for (; a.M > kQuantRows; a.M -= kQuantRows) {
        QuantArgs part = a;
        part.M = kQuantRows;
        quantize_launch<O>(part, s);
        a.x = (const uint8_t*)a.x + kQuantRows * a.ldx * (O == O_F32 ? 4 : 2);
        a.q += kQuantRows * a.ldq;
        a.scale += kQuantRows;
    }
    const dim3 grid((uint32_t)a.M);
    const int64_t pieces = (a.K + Piece<O>::N - 1) / Piece<O>::N;
    if (a.M <= kQuantFew) {
        if (pieces <= 1024)
            hipLaunchKernelGGL((quantize_rows<O, 1024, 1>), grid, dim3(1024), 0, s, a);
        else
            hipLaunchKernelGGL((quantize_rows<O, 1024, 2>), grid, dim3(1024), 0, s, a);
    } else if (pieces <= 512) {
        hipLaunchKernelGGL((quantize_rows<O, 256, 2>), grid, dim3(256), 0, s, a);
    } else if (pieces <= 1024) {
        hipLaunchKernelGGL((quantize_rows<O, 256, 4>), grid, dim3(256), 0, s, a);
    } else if (a.M * a.K <= kQuantStream) {
        hipLaunchKernelGGL((quantize_rows<O, 256, 8>), grid, dim3(256), 0, s, a);
    } else {
        hipLaunchKernelGGL((quantize_rows<O, 256, 8, true>), grid, dim3(256), 0, s, a);
    }
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
    case TG_F32: quantize_launch<O_F32>(a, s); break;
    case TG_F16: quantize_launch<O_F16>(a, s); break;
    default: quantize_launch<O_BF16>(a, s); break;
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
