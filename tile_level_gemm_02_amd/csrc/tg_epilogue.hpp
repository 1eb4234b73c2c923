// Epilogues of the fused products: what a workgroup does with the fp32 tile
// it has accumulated before it stores it, and the activations they apply.
//
//   EPI_STORE   : C = alpha * acc (the plain GEMM)
//   EPI_LINEAR  : z = alpha * acc + bias[col];  C = act(z) + R;  z kept if asked
//   EPI_GLU     : the tile holds gate and up columns in alternating blocks of
//                 32 (see gemm_nt);  C = act(gate) * up;  both kept if asked
//   EPI_GLU_BWD : acc is dh, the gradient of h = act(g) * u;
//                 dg = dh * u * act'(g),  du = dh * act(g)
//
// All arithmetic is fp32, on the unrounded accumulator; each stored value is
// rounded once.  The activations:
//
//   none x;  relu max(x, 0);
//   silu      x * s(x)                        s(t) = 1 / (1 + e^-t)
//   gelu_tanh x/2 (1 + tanh(c (x + 0.044715 x^3))), c = sqrt(2/pi): with
//             (1 + tanh(a)) / 2 = s(2a) it is x * s(x (s1 + s3 x^2)) as silu
//             is (s1 = 1, s3 = 0), so both run one code path;
//   gelu      x * Phi(x), Phi(x) = erfc(-x / sqrt(2)) / 2, by Abramowitz and
//             Stegun 7.1.26: erfc(v) = t (a1 + t (a2 + ...)) e^(-v^2) with
//             t = 1 / (1 + 0.3275911 v) for v >= 0, off by at most 1.5e-7
//             (a library erf takes both of its branches in a wave of mixed
//             arguments, about three times the instructions); the derivative
//             Phi(x) + x e^(-x^2/2) / sqrt(2 pi) uses the same exponential.
//
// The paths (kinds) are told apart by a uniform branch outside the loops over
// a tile's values, so that one kernel serves every activation.
#pragma once

#include <type_traits>

#include "tg_device.hpp"

namespace tg {

enum Epi : int { EPI_STORE = 0, EPI_LINEAR = 1, EPI_GLU = 2, EPI_GLU_BWD = 3 };

// code paths of the activations
enum ActKind : int { AK_CLIP = 0, AK_SIGMOID = 1, AK_ERF = 2 };

struct EpiArgs {
    const float* bias;  // LINEAR: fp32 [N], or null
    const void* R;      // LINEAR: residual (output type), or null; GLU_BWD: [g | u]
    int64_t ldr;
    void* Z;            // LINEAR: z kept (output type), or null; GLU: [g | u] kept, or null
    int64_t ldz;
    int32_t kind;       // ActKind
    float lo, slope_lo; // AK_CLIP: values and slope at or below lo (none: lo = -inf, slope 1)
    float s1, s3;       // AK_SIGMOID
};

typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));
typedef float f32x2_t __attribute__((ext_vector_type(2)));

// ------------------------------------------------------------- activations
// 1 / (1 + e^-t): the exponential and the reciprocal to about 1 ulp each
__device__ __forceinline__ float sigmoid_f32(float t)
{
    return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(t * -1.44269504088896341f));
}

// Phi(x) and e^(-x^2/2)
__device__ __forceinline__ float normal_cdf(float x, float& e)
{
    const float v = __builtin_fabsf(x);  // (0.3275911 / sqrt(2) folded into t)
    const float t = __builtin_amdgcn_rcpf(__builtin_fmaf(0.231641888f, v, 1.0f));
    e = __builtin_amdgcn_exp2f(v * v * -0.72134752044448170f);
    float q = __builtin_fmaf(t, 1.061405429f, -1.453152027f);
    q = __builtin_fmaf(t, q, 1.421413741f);
    q = __builtin_fmaf(t, q, -0.284496736f);
    q = __builtin_fmaf(t, q, 0.254829592f);
    q = 0.5f * q * t * e;
    return x < 0.0f ? q : 1.0f - q;
}

template <int KIND>
__device__ __forceinline__ float act_value(float x, const EpiArgs& a)
{
    if constexpr (KIND == AK_CLIP) {
        return x <= a.lo ? a.lo : x;  // (NaN stays)
    } else if constexpr (KIND == AK_SIGMOID) {
        return x * sigmoid_f32(x * __builtin_fmaf(a.s3, x * x, a.s1));
    } else {
        float e;
        return x * normal_cdf(x, e);
    }
}

// act(x) and act'(x)
template <int KIND>
__device__ __forceinline__ float act_slope(float x, const EpiArgs& a, float& value)
{
    if constexpr (KIND == AK_CLIP) {
        value = x <= a.lo ? a.lo : x;
        return x <= a.lo ? a.slope_lo : 1.0f;
    } else if constexpr (KIND == AK_SIGMOID) {
        // (past |x| = 1000 the factor s (1 - s) is zero: the square is held
        // there so that it stays finite)
        const float x2 = x * x, x2f = x2 > 1e6f ? 1e6f : x2;
        const float s = sigmoid_f32(x * __builtin_fmaf(a.s3, x2f, a.s1));
        value = x * s;
        return __builtin_fmaf(value * (1.0f - s), __builtin_fmaf(3.0f * a.s3, x2f, a.s1), s);
    } else {
        float e;
        const float c = normal_cdf(x, e);
        value = x * c;
        return __builtin_fmaf(x * e, 0.39894228040143268f, c);
    }
}

// Run f(std::integral_constant<int, kind>) for the call's activation path
template <class F>
__device__ __forceinline__ void for_act_kind(int kind, F f)
{
    if (kind == AK_CLIP)
        f(std::integral_constant<int, AK_CLIP>{});
    else if (kind == AK_SIGMOID)
        f(std::integral_constant<int, AK_SIGMOID>{});
    else
        f(std::integral_constant<int, AK_ERF>{});
}

// ------------------------------------------------------ 16-byte row pieces
// Values per 16-byte piece of a row of output type O
template <int O> struct Piece { static constexpr int N = O == O_F32 ? 4 : 8; };

// two values -> one word, rounded to nearest even
template <int O>
__device__ __forceinline__ uint32_t pack2(float a, float b)
{
    if constexpr (O == O_BF16) {
        return bit_cast<uint32_t>(__builtin_convertvector(f32x2_t{a, b}, bf16x2_t));
    } else {
        return bit_cast<uint32_t>(f16x2{(_Float16)a, (_Float16)b});
    }
}

template <int O>
__device__ __forceinline__ u32x4 pack_piece(const float* v)
{
    if constexpr (O == O_F32)
        return u32x4{bit_cast<uint32_t>(v[0]), bit_cast<uint32_t>(v[1]), bit_cast<uint32_t>(v[2]),
                     bit_cast<uint32_t>(v[3])};
    else
        return u32x4{pack2<O>(v[0], v[1]), pack2<O>(v[2], v[3]), pack2<O>(v[4], v[5]), pack2<O>(v[6], v[7])};
}

// value i of a piece, in fp32
template <int O>
__device__ __forceinline__ float piece_value(u32x4 q, int i)
{
    if constexpr (O == O_F32) {
        return bit_cast<float>((uint32_t)q[i]);
    } else {
        const uint32_t w = q[i >> 1];
        if constexpr (O == O_BF16)
            return bit_cast<float>((i & 1) ? w & 0xFFFF0000u : w << 16);
        else
            return (float)bit_cast<_Float16>((uint16_t)((i & 1) ? w >> 16 : w));
    }
}

// Load and store the first n (1 .. Piece<O>::N) values of the piece at
// element `idx`; `whole`: n is the full piece and the address is 16-byte
// aligned.
template <int O>
__device__ __forceinline__ u32x4 load_piece(const void* base, int64_t idx, int n, bool whole)
{
    typedef typename OutInfo<O>::T T;
    const T* src = (const T*)base + idx;
    if (whole)
        return ldg128(src);
    uint32_t w[4] = {0u, 0u, 0u, 0u};
#pragma unroll
    for (int e = 0; e < Piece<O>::N; ++e)
        if (e < n) {
            if constexpr (O == O_F32)
                w[e] = bit_cast<uint32_t>(src[e]);
            else
                w[e >> 1] |= (uint32_t)src[e] << ((e & 1) * 16);
        }
    return u32x4{w[0], w[1], w[2], w[3]};
}

template <int O>
__device__ __forceinline__ void store_piece(void* base, int64_t idx, u32x4 q, int n, bool whole)
{
    typedef typename OutInfo<O>::T T;
    T* dst = (T*)base + idx;
    if (whole) {
        store_nt((u32x4*)dst, q);
        return;
    }
#pragma unroll
    for (int e = 0; e < Piece<O>::N; ++e)
        if (e < n) {
            if constexpr (O == O_F32)
                dst[e] = bit_cast<float>((uint32_t)q[e]);
            else
                dst[e] = (uint16_t)(q[e >> 1] >> ((e & 1) * 16));
        }
}

// one value, in the output type
template <int O>
__device__ __forceinline__ float load_value(const void* base, int64_t idx)
{
    if constexpr (O == O_F32)
        return ((const float*)base)[idx];
    else
        return piece_value<O>(u32x4{(uint32_t)((const uint16_t*)base)[idx], 0u, 0u, 0u}, 0);
}

template <int O>
__device__ __forceinline__ void store_value(void* base, int64_t idx, float v)
{
    if constexpr (O == O_F32)
        ((float*)base)[idx] = v;
    else
        ((uint16_t*)base)[idx] = (uint16_t)pack2<O>(v, 0.0f);
}

// LINEAR for one accumulated value (kernels that store value by value)
template <int O, int KIND>
__device__ __forceinline__ void linear_value(const EpiArgs& e, void* C, int64_t ldc, int64_t row, int64_t col, float z)
{
    if (e.bias != nullptr)
        z += e.bias[col];
    if (e.Z != nullptr)
        store_value<O>(e.Z, row * e.ldz + col, z);
    float y = act_value<KIND>(z, e);
    if (e.R != nullptr)
        y += load_value<O>(e.R, row * e.ldr + col);
    store_value<O>(C, row * ldc + col, y);
}

// GLU for one gate and up value; F: hidden columns
template <int O, int KIND>
__device__ __forceinline__ void glu_value(const EpiArgs& e, void* C, int64_t ldc, int64_t F, int64_t row, int64_t col,
                                          float g, float u)
{
    if (e.Z != nullptr) {
        store_value<O>(e.Z, row * e.ldz + col, g);
        store_value<O>(e.Z, row * e.ldz + F + col, u);
    }
    store_value<O>(C, row * ldc + col, act_value<KIND>(g, e) * u);
}

// GLU_BWD for one value of dh
template <int O, int KIND>
__device__ __forceinline__ void glu_bwd_value(const EpiArgs& e, void* C, int64_t ldc, int64_t F, int64_t row,
                                              int64_t col, float dh)
{
    const float g = load_value<O>(e.R, row * e.ldr + col), u = load_value<O>(e.R, row * e.ldr + F + col);
    float value;
    const float slope = act_slope<KIND>(g, e, value);
    store_value<O>(C, row * ldc + col, dh * u * slope);
    store_value<O>(C, row * ldc + F + col, dh * value);
}

}  // namespace tg
