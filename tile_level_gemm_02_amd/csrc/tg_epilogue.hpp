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
//   gelu      x * Phi(x); for x <= 0 Phi(x) = t P(t) e^(-x^2/2) with
//             t = 1 / (1 + c |x|) and a polynomial of seven terms, Phi(x) =
//             1 - Phi(-x) above.  c and P were fitted to Phi e^(x^2/2) / t, a
//             smooth function of t, by minimax over |x| <= 14: off by 0.6e-7 or by
//             1.5e-6 of Phi, whichever is less, so that the tail keeps its
//             digits (the exponent's three fp32 roundings add up to 9e-8 x^2,
//             1e-5 of the value at -10).  Fp16 1003 x 4104 x 2056 with gelu
//             44.9 us, 44.6 with a five-term fit good to 1.5e-7 absolute, 1%
//             of the value at -8.  (A library erf takes both of its branches in
//             a wave of mixed arguments, about three times the instructions.)
//             The derivative Phi(x) + x e^(-x^2/2) / sqrt(2 pi) uses the same
//             exponential.
//
// The paths (kinds) are told apart by a uniform branch outside the loops over
// a tile's values, so that one kernel serves every activation.
//
// What an epilogue costs, per round of 256 x 256 tiles at K = 4096 (4096 x
// 16384 outputs, bf16, a round of the bare product about 90 us): storing
// through fp32 rows 6 us, with a residual or with gelu and a kept
// pre-activation 13, the gated product 2, with both projections kept 10.  The
// stores themselves are hidden (all tiles writing one region: 1 us less); what
// remains is the rows' way through LDS and the operands' latency, which a
// compute unit holding one workgroup cannot overlap with another tile.
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
    const float v = __builtin_fabsf(x);
    const float t = __builtin_amdgcn_rcpf(__builtin_fmaf(0.259861737f, v, 1.0f));
    e = __builtin_amdgcn_exp2f(v * v * -0.72134752044448170f);
    float q = __builtin_fmaf(t, -0.0734351352f, 0.231094211f);
    q = __builtin_fmaf(t, q, -0.10924048f);
    q = __builtin_fmaf(t, q, 0.168300435f);
    q = __builtin_fmaf(t, q, 0.0725724027f);
    q = __builtin_fmaf(t, q, 0.107257396f);
    q = __builtin_fmaf(t, q, 0.103451163f);
    q = q * t * e;
    return x < 0.0f ? q : 1.0f - q;
}

// x^2 as the logistic argument x (s1 + s3 x^2) takes it, held at 1e6: past
// |x| = 1000 that argument is beyond +-1000 and s is 0 or 1 either way, while an
// infinite square would make silu's s3 x^2 = 0 x^2 NaN.
__device__ __forceinline__ float held_square(float x)
{
    return __builtin_fminf(x * x, 1e6f);
}

template <int KIND>
__device__ __forceinline__ float act_value(float x, const EpiArgs& a)
{
    if constexpr (KIND == AK_CLIP) {
        return x <= a.lo ? a.lo : x;  // (NaN stays)
    } else if constexpr (KIND == AK_SIGMOID) {
        return x * sigmoid_f32(x * __builtin_fmaf(a.s3, held_square(x), a.s1));
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
        // (past |x| = 1000 the factor s (1 - s) is zero too)
        const float x2 = held_square(x);
        const float s = sigmoid_f32(x * __builtin_fmaf(a.s3, x2, a.s1));
        value = x * s;
        return __builtin_fmaf(value * (1.0f - s), __builtin_fmaf(3.0f * a.s3, x2, a.s1), s);
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

// ------------------------------------------------- epilogues of a wave's tile
// A wave's WR x WC accumulator tile as quads: 4 consecutive columns of one
// row per lane.  Row block i holds RBK rows (32 or 16, the matrix
// instruction's), this lane's being row lane % RBK; its quad q covers columns
// q * 4G + 4 (lane / RBK) .. +3 with G = 64 / RBK lanes side by side.
// `get(i, q)` returns a quad, scaled; i and q are constants after unrolling.

// Round to 16 bits, stage the wave's rows in its own LDS region `ep`
// (XOR-swizzled 16-byte chunks) and store whole rows: `NQ` quads per row
// block, of columns col0 .. of an M x N matrix `dst` from row0 on, shifted by
// `shift` columns; `aligned`: 16-byte pieces of the shifted rows are aligned.
template <int O, int RBK, int WR, int HC, class Get>
__device__ __forceinline__ void store_rows16(uint8_t* ep, uint32_t lane, int64_t row0, int64_t col0, int64_t M, int64_t N,
                                             void* dst, int64_t ld, int64_t shift, bool aligned, Get get)
{
    constexpr int G = 64 / RBK, NQ = HC / (4 * G);
    constexpr int OB = HC * 2, NCH = OB / 16;
    static_assert(WR % RBK == 0 && HC % (4 * G) == 0 && (WR * NCH) % 64 == 0, "staging shape");
    const uint32_t lr = lane % RBK, lg = lane / RBK;
#pragma unroll
    for (int i = 0; i < WR / RBK; ++i) {
        const uint32_t r = i * RBK + lr;
#pragma unroll
        for (int q = 0; q < NQ; ++q) {
            const f32x4 v = get(i, q);
            const uint32_t b = (q * 4 * G + 4 * lg) * 2;  // byte of the quad in its row
            *(u32x2*)(ep + r * OB + (((b >> 4) ^ (r % NCH)) << 4) + (b & 8u)) = u32x2{pack2<O>(v[0], v[1]), pack2<O>(v[2], v[3])};
        }
    }
    __builtin_amdgcn_s_waitcnt(0xC07F);  // lgkmcnt(0): this wave's staging writes done
#pragma unroll
    for (int t = 0; t < WR * NCH / 64; ++t) {
        const uint32_t x = t * 64 + lane, r = x / NCH, c = x % NCH;
        const u32x4 q = lds128(ep, r * OB + ((c ^ (r % NCH)) << 4));
        const int64_t row = row0 + r, col = col0 + c * 8, left = N - col;
        if (row < M && left > 0)
            store_piece<O>(dst, row * ld + shift + col, q, left < 8 ? (int)left : 8, left >= 8 && aligned);
    }
}

// EPI_GLU: hidden values are formed in the accumulator layout (the gate's
// and the up projection's 32-column blocks alternate), rounded to 16 bits and
// stored by rows; the kept projections follow through the same LDS.
template <int O, int RBK, int WR, int WC, class Get>
__device__ __forceinline__ void glu_epilogue(uint8_t* ep, uint32_t lane, int64_t row0, int64_t col0, int64_t M, int64_t F,
                                             void* C, int64_t ldc, const EpiArgs& e, Get get)
{
    static_assert(O != O_F32, "16-bit hidden values");
    constexpr int G = 64 / RBK, QB = 32 / (4 * G);  // quads per 32-column block
    for_act_kind(e.kind, [&](auto kind) __attribute__((always_inline)) {
        store_rows16<O, RBK, WR, WC / 2>(ep, lane, row0, col0, M, F, C, ldc, 0, true, [&](int i, int q) __attribute__((always_inline)) {
            const f32x4 g = get(i, q / QB * 2 * QB + q % QB), u = get(i, (q / QB * 2 + 1) * QB + q % QB);
            f32x4 h;
#pragma unroll
            for (int x = 0; x < 4; ++x)
                h[x] = act_value<decltype(kind)::value>(g[x], e) * u[x];
            return h;
        });
    });
    if (e.Z != nullptr) {
        store_rows16<O, RBK, WR, WC / 2>(ep, lane, row0, col0, M, F, e.Z, e.ldz, 0, true, [&](int i, int q) __attribute__((always_inline)) {
            return get(i, q / QB * 2 * QB + q % QB);
        });
        store_rows16<O, RBK, WR, WC / 2>(ep, lane, row0, col0, M, F, e.Z, e.ldz, F, F % 8 == 0,
                                         [&](int i, int q) __attribute__((always_inline)) {
                                             return get(i, (q / QB * 2 + 1) * QB + q % QB);
                                         });
    }
}

// EPI_LINEAR, EPI_GLU_BWD and fp32 EPI_STORE: the fp32 accumulators go
// through LDS (PBY bytes of this wave's own) in passes of PR rows, and come
// back as pieces of rows: a lane handles VC consecutive columns, the same
// ones in every row, so the bias is loaded once and the other operands are
// read and written in 16-byte pieces of whole rows.  A pass's operand loads
// are issued ahead of its staging.
template <int O, int EPI, int RBK, int WR, int WC, int PBY, class Get>
__device__ __forceinline__ void rows_epilogue(uint8_t* ep, uint32_t lane, int64_t row0, int64_t col0, int64_t M, int64_t N,
                                              void* C, int64_t ldc, const EpiArgs& ea, Get get)
{
    constexpr int G = 64 / RBK, NQ = WC / (4 * G);
    constexpr int VC = Piece<O>::N;
    constexpr int LPR = WC / VC, RPT = 64 / LPR;  // lanes per row, rows per instruction
    constexpr int OB = WC * 4, NCH = OB / 16;
    constexpr int PR = PBY / OB >= WR ? WR : (PBY / OB >= WR / 2 ? WR / 2 : WR / 4);
    constexpr int NTI = PR / RPT;
    constexpr bool BWD = EPI == EPI_GLU_BWD, LIN = EPI == EPI_LINEAR;
    static_assert(PR % RBK == 0 && WR % PR == 0 && PR % RPT == 0 && 64 % LPR == 0 && PR * OB <= PBY, "staging passes");
    const uint32_t ec = lane % LPR, er = lane / LPR;
    const int64_t col = col0 + ec * VC, left = N - col;
    const int n = left >= VC ? VC : left > 0 ? (int)left : 0;
    const bool whole = n == VC, up_whole = whole && N % VC == 0;  // (BWD: the up half starts at column N)
    const void* const R = EPI == EPI_STORE ? nullptr : ea.R;
    float bias[VC];
#pragma unroll
    for (int e = 0; e < VC; ++e)
        bias[e] = LIN && ea.bias != nullptr && e < n ? ea.bias[col + e] : 0.0f;
    // (a call per pass, not a loop: the accumulator must be indexed by constants)
    auto run_pass = [&](auto pass_c) __attribute__((always_inline)) {
        constexpr int pass = decltype(pass_c)::value;
        const int64_t prow = row0 + pass * PR + er;
        u32x4 r0[NTI], r1[BWD ? NTI : 1];
        if (R != nullptr) {
#pragma unroll
            for (int t = 0; t < NTI; ++t) {
                const int64_t row = prow + t * RPT;
                r0[t] = u32x4{0u, 0u, 0u, 0u};
                if (row < M && n > 0)
                    r0[t] = load_piece<O>(R, row * ea.ldr + col, n, whole);
                if constexpr (BWD) {
                    r1[t] = u32x4{0u, 0u, 0u, 0u};
                    if (row < M && n > 0)
                        r1[t] = load_piece<O>(R, row * ea.ldr + N + col, n, up_whole);
                }
            }
        }
#pragma unroll
        for (int ii = 0; ii < PR / RBK; ++ii) {
            const uint32_t r = ii * RBK + lane % RBK;
#pragma unroll
            for (int q = 0; q < NQ; ++q) {
                const uint32_t c = q * G + lane / RBK;  // 16-byte chunk of the quad
                *(f32x4*)(ep + r * OB + ((c ^ (r % NCH)) << 4)) = get(pass * (PR / RBK) + ii, q);
            }
        }
        __builtin_amdgcn_s_waitcnt(0xC07F);  // lgkmcnt(0): this wave's staging writes done
        auto finish = [&](auto kind) __attribute__((always_inline)) {
            constexpr int KIND = decltype(kind)::value;
#pragma unroll
            for (int t = 0; t < NTI; ++t) {
                const uint32_t r = t * RPT + er;
                const int64_t row = prow + t * RPT;
                float z[VC];
#pragma unroll
                for (int h = 0; h < VC / 4; ++h) {
                    const f32x4 q = bit_cast<f32x4>(lds128(ep, r * OB + (((ec * (VC / 4) + h) ^ (r % NCH)) << 4)));
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        z[4 * h + e] = q[e];
                }
                if (row >= M || n == 0)
                    continue;
                if constexpr (BWD) {
                    float dg[VC], du[VC];
#pragma unroll
                    for (int e = 0; e < VC; ++e) {
                        float value;
                        const float slope = act_slope<KIND>(piece_value<O>(r0[t], e), ea, value);
                        dg[e] = z[e] * piece_value<O>(r1[t], e) * slope;
                        du[e] = z[e] * value;
                    }
                    store_piece<O>(C, row * ldc + col, pack_piece<O>(dg), n, whole);
                    store_piece<O>(C, row * ldc + N + col, pack_piece<O>(du), n, up_whole);
                } else if constexpr (LIN) {
#pragma unroll
                    for (int e = 0; e < VC; ++e)
                        z[e] += bias[e];
                    if (ea.Z != nullptr)
                        store_piece<O>(ea.Z, row * ea.ldz + col, pack_piece<O>(z), n, whole);
#pragma unroll
                    for (int e = 0; e < VC; ++e)
                        z[e] = act_value<KIND>(z[e], ea);
                    if (R != nullptr)
#pragma unroll
                        for (int e = 0; e < VC; ++e)
                            z[e] += piece_value<O>(r0[t], e);
                    store_piece<O>(C, row * ldc + col, pack_piece<O>(z), n, whole);
                } else {
                    store_piece<O>(C, row * ldc + col, pack_piece<O>(z), n, whole);
                }
            }
        };
        if constexpr (EPI == EPI_STORE)
            finish(std::integral_constant<int, AK_CLIP>{});
        else
            for_act_kind(ea.kind, finish);
    };
    run_pass(std::integral_constant<int, 0>{});
    if constexpr (WR / PR >= 2)
        run_pass(std::integral_constant<int, 1>{});
    if constexpr (WR / PR == 4) {
        run_pass(std::integral_constant<int, 2>{});
        run_pass(std::integral_constant<int, 3>{});
    }
}

}  // namespace tg
