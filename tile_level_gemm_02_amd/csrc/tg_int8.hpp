// Products of int8 matrices with a scale for each token and each channel
// (contract in include/tg_int8.h): their arguments, epilogue and plans.
//
//   Y = act(sx[m] sw[n] (x.W^T) + bias) + residual
//
// The sums are int32 and exact (K is held below 2^17); they are rounded to
// fp32 once, then scaled.  The kernels are those of the other products: int8
// rows have the same bytes per K step as 16-bit ones with twice the k, so the
// copies, the ring and the fragments stay as they are and only the matrix
// instruction (16x16x64, 32x32x32) and the accumulators' type differ.  Bound by
// the matrix pipe with many rows (8192 x 4096 x 10240 246 us, 2.8 POP/s, back to
// back on the same operands; behind its quantization 243 to 291, by card and
// clock; a library product of 8192^3 2.0 to 2.5 POP/s), by fills and epilogues
// around short loops (1003 x 4104 x 2064 with gelu 28 us, 10 of them with a
// single K step), and by the weight's read with few (1 x 4096 x 4096 5.3 us, 1 x
// 8192 x 8192 12.4, 5.4 TB/s).  The tile plans are fp8's; forced 64, 128, 256 x
// 128 and 256 tiles ran no faster at any of seven sizes.
#pragma once

#include "tg_fused.hpp"
#include "tg_int8.h"

namespace tg {

struct I8Epi : EpiArgs {
    const float* sx;  // [M]
    const float* sw;  // [N]
};

template <int O>
struct I8Args : TileArgs {
    I8Epi e;

    template <int RBK, int WR, int WC, int PBY, class Get>
    __device__ __forceinline__ void finish(uint8_t* ep, uint32_t lane, int64_t row0, int64_t col0, Get get) const
    {
        if constexpr (O != O_F32) {
            // without a residual everything happens in the accumulator's layout,
            // and rows go through LDS as 16 bits
            if (e.R == nullptr) {
                constexpr int G = 64 / RBK, NQ = WC / (4 * G), NB = WR / RBK;
                float sx[NB], sw[4 * NQ], bias[4 * NQ];
#pragma unroll
                for (int i = 0; i < NB; ++i) {
                    const int64_t row = row0 + i * RBK + lane % RBK;
                    sx[i] = row < M ? e.sx[row] : 0.0f;
                }
#pragma unroll
                for (int q = 0; q < NQ; ++q)
#pragma unroll
                    for (int x = 0; x < 4; ++x) {
                        const int64_t col = col0 + q * 4 * G + 4 * (lane / RBK) + x;
                        sw[4 * q + x] = col < N ? e.sw[col] : 0.0f;
                        bias[4 * q + x] = e.bias != nullptr && col < N ? e.bias[col] : 0.0f;
                    }
                for_act_kind(e.kind, [&](auto kind) __attribute__((always_inline)) {
                    store_rows16<O, RBK, WR, WC>(ep, lane, row0, col0, M, N, C, ldc, 0, true,
                                                 [&](int i, int q) __attribute__((always_inline)) {
                        f32x4 v = get(i, q);
#pragma unroll
                        for (int x = 0; x < 4; ++x)
                            v[x] = act_value<decltype(kind)::value>(v[x] * (sx[i] * sw[4 * q + x]) + bias[4 * q + x], e);
                        return v;
                    });
                });
                return;
            }
        }
        constexpr int VC = Piece<O>::N;
        const int64_t col = col0 + lane % (WC / VC) * VC, left = N - col;
        const int n = left >= VC ? VC : left > 0 ? (int)left : 0;
        float sw[VC], bias[VC];
#pragma unroll
        for (int x = 0; x < VC; ++x) {
            sw[x] = x < n ? e.sw[col + x] : 0.0f;
            bias[x] = e.bias != nullptr && x < n ? e.bias[col + x] : 0.0f;
        }
        struct Row {
            u32x4 r;
            float sx;
        };
        for_act_kind(e.kind, [&](auto kind) __attribute__((always_inline)) {
            staged_rows<VC, Row, RBK, WR, WC, PBY>(
                ep, lane, row0, get,
                [&](Row& s, int64_t row) __attribute__((always_inline)) {
                    s.r = u32x4{0u, 0u, 0u, 0u};
                    s.sx = 0.0f;
                    if (row < M) {
                        s.sx = e.sx[row];
                        if (e.R != nullptr && n > 0)
                            s.r = load_piece<O>(e.R, row * e.ldr + col, n, n == VC);
                    }
                },
                [&](const Row& s, int64_t row, float* z) __attribute__((always_inline)) {
#pragma unroll
                    for (int x = 0; x < VC; ++x)
                        z[x] = act_value<decltype(kind)::value>(z[x] * (s.sx * sw[x]) + bias[x], e);
                    if (e.R != nullptr)
#pragma unroll
                        for (int x = 0; x < VC; ++x)
                            z[x] += piece_value<O>(s.r, x);
                    if (row < M && n > 0)
                        store_piece<O>(C, row * ldc + col, pack_piece<O>(z), n, n == VC);
                });
        });
    }
};

template <int O>
struct I8SkinnyArgs : SkinnyArgs {
    I8Epi e;

    __device__ __forceinline__ void finish_quad(uint32_t, int64_t row, int64_t col, bool in, f32x4 a) const
    {
        if (!in)
            return;
        const float sx = e.sx[row];
        for_act_kind(e.kind, [&](auto kind) __attribute__((always_inline)) {
#pragma unroll
            for (int x = 0; x < 4; ++x)
                if (col + x < N) {
                    const float z = a[x] * (sx * e.sw[col + x]) + (e.bias != nullptr ? e.bias[col + x] : 0.0f);
                    float y = act_value<decltype(kind)::value>(z, e);
                    if (e.R != nullptr)
                        y += load_value<O>(e.R, row * e.ldr + col + x);
                    store_value<O>(C, row * ldc + col + x, y);
                }
        });
    }
};

// Rows up to which a call takes the skinny kernel (33 rows, N = K = 8192: 15.9
// us on the tile kernel with K split; 32 rows 14.2 here, 15.9 there)
constexpr int64_t kI8SkinnyRows = 32;

template <int O, int WAVES, int RING, int AI, int SPLIT, int CG>
void launch_i8_skinny(const I8SkinnyArgs<O>& a, int64_t blocks, int split, hipStream_t s)
{
    hipLaunchKernelGGL((skinny_gemm<E_I8, O, WAVES, AI, RING, SPLIT, CG, EPI_OWN, I8SkinnyArgs<O>>),
                       dim3((uint32_t)blocks, (uint32_t)split), dim3(64 * WAVES), 0, s, a);
}

constexpr int kI8MostRing = 4;

// Whether the few-rows kernel takes a call (a launch has less than 2^32 lanes,
// and that many workgroups four waves each)
inline bool i8_skinny(int64_t M, int64_t N, int64_t K)
{
    return M <= kI8SkinnyRows && K > 0 && fused_skinny_blocks(M, N) * 64 * 4 < (int64_t)1 << 32;
}

// Rows of x or W in a launch at most: its tiles, of 512 lanes each, are fewer
// than 2^23 then (2 M N bytes of Y fit the memory)
constexpr int64_t kI8Rows = (int64_t)1 << 30;

// Waves per workgroup and ring slots per wave of the skinny kernel.  An int8
// row is half the bytes of a 16-bit one, so eight waves get few stages each:
// four waves with a deeper ring stream faster wherever a workgroup's K is all
// that a compute unit reads (up to 256 workgroups), and what counts past that is
// how many workgroups a unit's LDS holds (three slots, and two for several
// slices of rows).  Back to back, three weights in turn, us:
//                      8 waves, 2   4 waves, 4   4 waves, 3   4 waves, 2
//    1 x  4096 x 4096      5.4          5.2          5.4          6.0
//    1 x  1024 x 4096      3.9          4.5          4.4          4.4
//   16 x  8192 x 8192     14.9         13.4         13.4         13.5
//   16 x  8200 x 8192     20.0         19.1         16.6         16.4
//   32 x  8192 x 8192     17.7         16.8         14.1         14.2
//   24 x  8200 x 8192     21.1         21.4         17.6         15.9
//   20 x 10240 x 4096       -          16.7         13.0         11.5
template <int O>
void launch_i8_rows(const I8SkinnyArgs<O>& a, int64_t blocks, int split, hipStream_t s)
{
    const bool one = a.M <= 8, wide = fused_cg(a.M, a.N) == 2;
    if (a.M > 16) {
        split > 1 ? launch_i8_skinny<O, 4, 2, 2, 2, 2>(a, blocks, split, s) : launch_i8_skinny<O, 4, 2, 2, 0, 2>(a, blocks, 1, s);
    } else if (blocks <= 128) {  // (the only ones split)
        if (split > 1)
            one ? launch_i8_skinny<O, 8, 2, 1, 2, 1>(a, blocks, split, s) : launch_i8_skinny<O, 8, 2, 2, 2, 1>(a, blocks, split, s);
        else
            one ? launch_i8_skinny<O, 8, 2, 1, 0, 1>(a, blocks, 1, s) : launch_i8_skinny<O, 8, 2, 2, 0, 1>(a, blocks, 1, s);
    } else if (blocks <= 256 && !wide) {
        one ? launch_i8_skinny<O, 4, 4, 1, 0, 1>(a, blocks, 1, s) : launch_i8_skinny<O, 4, 4, 2, 0, 1>(a, blocks, 1, s);
    } else if (wide) {
        launch_i8_skinny<O, 4, 3, 2, 0, 2>(a, blocks, 1, s);
    } else {
        one ? launch_i8_skinny<O, 4, 3, 1, 0, 1>(a, blocks, 1, s) : launch_i8_skinny<O, 4, 3, 2, 0, 1>(a, blocks, 1, s);
    }
}

inline int64_t i8_ws_bytes(int64_t M, int64_t N, int64_t K)
{
    if (M <= 0 || N <= 0 || K <= 0 || K % 16 != 0 || !dims_fit(M, N, K))
        return 0;
    if (i8_skinny(M, N, K)) {
        const int64_t blocks = fused_skinny_blocks(M, N);
        return fused_skinny_ws_bytes(M, N, blocks, fused_split<E_I8>(blocks, K));
    }
    return plan_nt<E_I8, B_KCONTIG>(M, N, K, true).ws_bytes;
}

template <int O>
tg_status i8_linear(const TileArgs& t, const I8Epi& e, void* ws, int64_t ws_bytes, hipStream_t s)
{
    if (t.M > kI8Rows || t.N > kI8Rows) {
        const int64_t ob = O == O_F32 ? 4 : 2;
        for (int64_t m0 = 0; m0 < t.M; m0 += kI8Rows)
            for (int64_t n0 = 0; n0 < t.N; n0 += kI8Rows) {
                TileArgs part = t;
                I8Epi pe = e;
                part.M = t.M - m0 < kI8Rows ? t.M - m0 : kI8Rows;
                part.N = t.N - n0 < kI8Rows ? t.N - n0 : kI8Rows;
                part.A += m0 * t.lda;
                part.B += n0 * t.ldb;
                part.C = (uint8_t*)t.C + (m0 * t.ldc + n0) * ob;
                pe.R = e.R != nullptr ? (const uint8_t*)e.R + (m0 * e.ldr + n0) * ob : nullptr;
                pe.bias = e.bias != nullptr ? e.bias + n0 : nullptr;
                pe.sx = e.sx + m0;
                pe.sw = e.sw + n0;
                const tg_status st = i8_linear<O>(part, pe, ws, ws_bytes, s);
                if (st != TG_OK)
                    return st;
            }
        return TG_OK;
    }
    if (i8_skinny(t.M, t.N, t.K) && skinny_offsets_fit(t.K, t.lda, t.ldb, kI8MostRing, fused_cg(t.M, t.N))) {
        I8SkinnyArgs<O> a{};
        a.M = t.M;
        a.N = t.N;
        a.K = t.K;
        a.A = t.A;
        a.lda = t.lda;
        a.B = t.B;
        a.ldb = t.ldb;
        a.C = t.C;
        a.ldc = t.ldc;
        a.e = e;
        const int64_t blocks = fused_skinny_blocks(a.M, a.N);
        int split = fused_split<E_I8>(blocks, a.K);
        const int64_t need = fused_skinny_ws_bytes(a.M, a.N, blocks, split);
        if (ws == nullptr || need == 0 || need > ws_bytes)
            split = 1;
        if (split > 1) {
            a.counters = (uint32_t*)ws;
            a.partials = (float*)((uint8_t*)ws + kSplitCounterBytes);
        }
        launch_i8_rows(a, blocks, split, s);
        return launched();
    }
    I8Args<O> a{};
    static_cast<TileArgs&>(a) = t;
    a.e = e;
    if (!nt_eligible<E_I8>(a))
        return TG_ERR_NOT_SUPPORTED;
    NtPlan plan = plan_nt<E_I8, B_KCONTIG>(a.M, a.N, a.K, ws != nullptr);
    if (plan.ws_bytes > ws_bytes)
        plan = plan_nt<E_I8, B_KCONTIG>(a.M, a.N, a.K, false);
    return launch_nt_plan<E_I8, O, B_KCONTIG, EPI_OWN, A_KCONTIG>(a, plan, ws, s);
}

}  // namespace tg
