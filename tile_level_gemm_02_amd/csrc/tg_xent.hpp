// The vocabulary loss and its gradient (contracts in include/tg_train.h): the
// epilogues of their products and the small kernels between them, one template
// per input type, instantiated in that type's translation units.
//
//   t = scale x.W^T,  lse = log sum_v e^t,  loss = lse - t[target] + z lse^2
//   dt = g (e^(t - lse) (1 + 2 z lse) - onehot),  dX = scale dt.W,  dW = scale dt^T.x
//
// The logits are never stored.  Forward: each wave of the product x.W^T holds
// 64 columns of its rows and leaves two numbers per row, the largest t and the
// sum of e^(t - largest) (xent_join adds them up over the vocabulary), and the
// wave that holds a row's target leaves its t.  Gradient: a piece of the
// vocabulary at a time, the same product again with dt as its epilogue,
// rounded to 16 bits, then the two products that take dt as their operand.
// All of them are bound by the matrix products: 2 M V D operations forward
// and 6 for the gradient.  Bf16 8192 x 131072 x 4096 5.9 to 6.2 ms forward by
// card, 1410 to 1490 TFLOP/s (a library product of the same size, which stores its
// logits, 1490); gradients of 4096 x 128256 x 4096 9.1 to 9.6 ms, 1340 to 1420;
// 7 x 32000 x 2048 27 us, 4.8 TB/s of the weight; 64 rows 35, 500 rows 65.  The
// forward epilogue takes 4.5 us a round of 256 tiles, 1.1 of them exponentials.  Smaller tiles (128, 256 x 128) for dt, of which two
// workgroups or a shorter epilogue would overlap, ran 8 to 50% slower at every
// size tried.
//
// Exponentials are base 2: with c = scale log2(e), e^(t - lse) is
// exp2(acc c - lse log2(e)), one multiply-add and one instruction per value.
#pragma once

#include "tg_fused.hpp"
#include "tg_train.h"

namespace tg {

constexpr int kXentCols = 64;  // columns of a wave's tile, in every tile the forward product takes

// A row of the gradient's epilogue: exp2(acc c - lse2) a - (column == target ? b : 0)
struct XentRow {
    float lse2, a, b;
    int32_t target;
};

// ------------------------------------------------------- forward epilogue
struct XentOut {
    float c, scale;
    const int64_t* target;
    f32x2_t* part;   // [slot][rows]: largest t (base 2) and sum of 2^(t - largest) over the slot's columns
    float* picked;   // [rows]: t of the target
    int64_t rows;    // of the call, of which a launch may have a part
    int64_t v0;      // first column of the launch's part of the vocabulary
};

// One value per lane reduced over the lanes that hold the same row (RBK apart:
// the other rows of 16 lanes, the other half of the wave)
template <int RBK, class F>
__device__ __forceinline__ float over_row_lanes(float v, F f)
{
    static_assert(RBK == 16 || RBK == 32, "rows of a matrix instruction");
    if constexpr (RBK == 16) {
        const auto r = __builtin_amdgcn_permlane16_swap(bit_cast<uint32_t>(v), bit_cast<uint32_t>(v), false, false);
        v = f(bit_cast<float>((uint32_t)r[0]), bit_cast<float>((uint32_t)r[1]));
    }
    const auto h = __builtin_amdgcn_permlane32_swap(bit_cast<uint32_t>(v), bit_cast<uint32_t>(v), false, false);
    return f(bit_cast<float>((uint32_t)h[0]), bit_cast<float>((uint32_t)h[1]));
}

__device__ __forceinline__ float max2(float a, float b) { return __builtin_fmaxf(a, b); }
__device__ __forceinline__ float add2(float a, float b) { return a + b; }

// reference of a sum of exponentials: 0 where there is none (all -infinity, or NaN)
__device__ __forceinline__ float reference_of(float top) { return top == -INFINITY ? 0.0f : top; }

struct XentFwdArgs : TileArgs {
    XentOut x;

    template <int RBK, int WR, int WC, int PBY, class Get>
    __device__ __forceinline__ void finish(uint8_t*, uint32_t lane, int64_t row0, int64_t col0, Get get) const
    {
        constexpr int G = 64 / RBK, NQ = WC / (4 * G);
        static_assert(WC == kXentCols, "a slot per wave");
        if (col0 >= N)
            return;
        const int64_t slot = col0 / kXentCols;
        const int left = N - col0 < WC ? (int)(N - col0) : WC;
        const int lg = (int)(lane / RBK);
        constexpr int NB = WR / RBK;
        // this row's target among the wave's columns, if it is there (the loads
        // of all rows ahead of their use)
        int at[NB];
        int64_t target[NB];
#pragma unroll
        for (int i = 0; i < NB; ++i) {
            const int64_t row = row0 + i * RBK + lane % RBK;
            target[i] = row < M ? x.target[row] : -1;
        }
#pragma unroll
        for (int i = 0; i < NB; ++i) {
            const int64_t k = target[i] - x.v0 - col0;
            at[i] = k >= 0 && k < left ? (int)k : -1;
        }
        // WHOLE: all columns are there and c is not negative, so that the largest
        // product is the one with the largest t
        auto rows = [&](auto whole) __attribute__((always_inline)) {
            constexpr bool WHOLE = decltype(whole)::value;
#pragma unroll
            for (int i = 0; i < NB; ++i) {
                const int64_t row = row0 + i * RBK + lane % RBK;
                float v[NQ * 4], top = -INFINITY;
#pragma unroll
                for (int q = 0; q < NQ; ++q) {
                    const f32x4 a = get(i, q);
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        v[4 * q + e] = WHOLE ? a[e] : a[e] * x.c;
                        if (!WHOLE && q * 4 * G + 4 * lg + e >= left)
                            v[4 * q + e] = -INFINITY;
                        top = max2(top, v[4 * q + e]);
                    }
                }
                top = over_row_lanes<RBK>(top, max2);
                top = WHOLE ? top * x.c : top;
                const float ref = reference_of(top);
                float sum = 0.0f;
#pragma unroll
                for (int k = 0; k < NQ * 4; ++k)
                    sum += __builtin_amdgcn_exp2f(WHOLE ? __builtin_fmaf(v[k], x.c, -ref) : v[k] - ref);
                sum = over_row_lanes<RBK>(sum, add2);
                if (row < M) {
                    if (lg == 0)
                        x.part[slot * x.rows + row] = f32x2_t{top, sum};
                    if (at[i] >= 0 && at[i] / 4 % G == lg) {
#pragma unroll
                        for (int q = 0; q < NQ; ++q) {
                            const f32x4 a = get(i, q);
#pragma unroll
                            for (int e = 0; e < 4; ++e)
                                if (at[i] == q * 4 * G + 4 * lg + e)
                                    x.picked[row] = a[e] * x.scale;
                        }
                    }
                }
            }
        };
        if (left == WC && x.c >= 0.0f)
            rows(std::true_type{});
        else
            rows(std::false_type{});
    }
};

// few rows: the skinny kernel, whose waves each hold 16 columns
struct XentSkinnyArgs : SkinnyArgs {
    XentOut x;

    __device__ __forceinline__ void finish_quad(uint32_t lane, int64_t row, int64_t col, bool in, f32x4 a) const
    {
        const int left = N - col < 4 ? (int)(N - col) : 4;  // (<= 0 past the last column)
        float v[4], top = -INFINITY;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            v[e] = e < left ? a[e] * x.c : -INFINITY;
            top = max2(top, v[e]);
        }
        top = over_row_lanes<16>(top, max2);
        const float ref = reference_of(top);
        float sum = 0.0f;
#pragma unroll
        for (int e = 0; e < 4; ++e)
            sum += __builtin_amdgcn_exp2f(v[e] - ref);
        sum = over_row_lanes<16>(sum, add2);
        const int64_t col16 = col & ~(int64_t)15;
        if (!in || col16 >= N)
            return;
        if (lane < 16u)
            x.part[col16 / 16 * x.rows + row] = f32x2_t{top, sum};
        const int64_t at = x.target[row] - col;
        if (at >= 0 && at < left)
            x.picked[row] = (at == 0 ? a[0] : at == 1 ? a[1] : at == 2 ? a[2] : a[3]) * x.scale;
    }
};

// ---------------------------------------------------------- joining slots
struct XentJoinArgs {
    int64_t M, V, slots;
    const f32x2_t* part;
    const float* picked;
    const int64_t* target;
    int64_t ignore;
    float z;
    float *loss, *lse, *total;
    uint32_t* counter;
    double* sums;    // [workgroups][2]: losses and counted rows
    uint32_t first;  // workgroups of the launches before
    int32_t more;    // launches follow, the last of which adds the sums
};

// Workgroups of a launch at most (of 256 lanes: a launch has less than 2^32)
constexpr int64_t kJoinGrid = 1 << 23;

__device__ __forceinline__ void join_pair(float& top, float& sum, float t, float s)
{
    const float m = max2(top, t), r = reference_of(m);
    sum = sum * __builtin_amdgcn_exp2f(top - r) + s * __builtin_amdgcn_exp2f(t - r);
    top = m;
}

// Arrivals at one word take 12 ns each, whichever workgroups make them (131072
// rows 102 us, 92 of them so).  Many workgroups therefore arrive at words on
// lines of their own, and the last at each of these at the first word.  All
// words are left zero.
constexpr uint32_t kJoinGroups = 64, kJoinMany = 256;
static_assert((kJoinGroups + 1) * 256 <= kSplitCounterBytes, "words 256 bytes apart");

__device__ __forceinline__ bool arrive(uint32_t* word, uint32_t n)
{
    if (__hip_atomic_fetch_add(word, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) != n - 1u)
        return false;
    __hip_atomic_exchange(word, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    return true;
}

// by one lane of each workgroup, whose stores are complete: true in the last
__device__ __forceinline__ bool last_arrival(uint32_t* counters)
{
    if (gridDim.x <= kJoinMany)
        return arrive(counters, gridDim.x);
    const uint32_t g = blockIdx.x % kJoinGroups, n = (gridDim.x - g + kJoinGroups - 1u) / kJoinGroups;
    return arrive(counters + 64u * (1u + g), n) && arrive(counters, kJoinGroups);
}

// The slots of R rows per workgroup, 256 / R lanes to a row, several loads
// ahead of their arithmetic; lanes and waves are added in a fixed order.  Bound
// by the slots' reads (8 bytes for every 64 columns of every row).
template <int R>
__global__ __launch_bounds__(256) void xent_join(XentJoinArgs p)
{
    constexpr int T = 256 / R, B = 8;
    __shared__ float red[2][4][R];
    __shared__ double own[2][R];
    __shared__ bool last;
    const uint32_t tid = threadIdx.x, r = tid % R, part = tid / R;
    const uint32_t group = p.first + blockIdx.x;
    const int64_t row = (int64_t)group * R + r;
    float top = -INFINITY, sum = 0.0f;
    if (row < p.M) {
        for (int64_t s0 = part; s0 < p.slots; s0 += (int64_t)T * B) {
            f32x2_t v[B];
#pragma unroll
            for (int b = 0; b < B; ++b) {
                const int64_t s = s0 + (int64_t)b * T;
                v[b] = f32x2_t{-INFINITY, 0.0f};
                if (s < p.slots)
                    v[b] = p.part[s * p.M + row];
            }
            float m = v[0][0];
#pragma unroll
            for (int b = 1; b < B; ++b)
                m = max2(m, v[b][0]);
            const float ref = reference_of(m);
            float s = 0.0f;
#pragma unroll
            for (int b = 0; b < B; ++b)
                s += v[b][1] * __builtin_amdgcn_exp2f(v[b][0] - ref);
            join_pair(top, sum, m, s);
        }
    }
    // the lanes of a wave that share a row, then the waves: first the largest,
    // then the sums relative to it
    float most = top;
#pragma unroll
    for (int d = 32; d >= R; d >>= 1)
        most = max2(most, __shfl_xor(most, d, 64));
    sum *= __builtin_amdgcn_exp2f(top - reference_of(most));
#pragma unroll
    for (int d = 32; d >= R; d >>= 1)
        sum += __shfl_xor(sum, d, 64);
    top = most;
    if (tid % 64u < (uint32_t)R) {
        red[0][tid / 64u][r] = top;
        red[1][tid / 64u][r] = sum;
    }
    __syncthreads();
    if (tid < (uint32_t)R)
#pragma unroll
        for (int k = 1; k < 4; ++k)
            join_pair(top, sum, red[0][k][r], red[1][k][r]);
    if (tid < (uint32_t)R) {
        double counted = 0.0, mine = 0.0;
        if (row < p.M) {
            const float lse = top * 0.693147180559945309f + logf(sum);
            const int64_t t = p.target[row];
            const bool counts = t != p.ignore;
            float loss = 0.0f;
            if (counts)
                loss = t < 0 || t >= p.V ? NAN : lse - p.picked[row] + p.z * lse * lse;
            if (p.lse != nullptr)
                p.lse[row] = lse;
            if (p.loss != nullptr)
                p.loss[row] = loss;
            counted = counts ? 1.0 : 0.0;
            mine = (double)loss;
        }
        own[0][r] = mine;
        own[1][r] = counted;
    }
    if (p.total == nullptr)
        return;
    // this workgroup's sums into its slot; the last to arrive adds all slots, in
    // an order that does not depend on which it is
    __syncthreads();
    if (tid == 0u) {
        double a = 0.0, b = 0.0;
        for (int k = 0; k < R; ++k) {
            a += own[0][k];
            b += own[1][k];
        }
        __hip_atomic_store(p.sums + 2 * (size_t)group, a, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        __hip_atomic_store(p.sums + 2 * (size_t)group + 1, b, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
        last = p.more == 0 && last_arrival(p.counter);
    }
    __syncthreads();
    constexpr uint32_t LANES = R == 1 ? 64u : 256u;  // (one row a workgroup: 64 slots at most)
    if (!last || tid >= LANES)
        return;
    double a = 0.0, b = 0.0;
    constexpr uint32_t AHEAD = R == 1 ? 1u : 8u;  // loads of a lane in flight
    const uint32_t groups = p.first + gridDim.x;
    for (uint32_t k0 = tid; k0 < groups; k0 += LANES * AHEAD) {
        double u[AHEAD], w[AHEAD];
#pragma unroll
        for (uint32_t i = 0; i < AHEAD; ++i) {
            const uint32_t k = k0 + i * LANES;
            u[i] = w[i] = 0.0;
            if (k < groups) {
                u[i] = __hip_atomic_load(p.sums + 2 * (size_t)k, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
                w[i] = __hip_atomic_load(p.sums + 2 * (size_t)k + 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
            }
        }
#pragma unroll
        for (uint32_t i = 0; i < AHEAD; ++i) {
            a += u[i];
            b += w[i];
        }
    }
#pragma unroll
    for (int d = 32; d > 0; d >>= 1) {
        a += __shfl_down(a, d, 64);
        b += __shfl_down(b, d, 64);
    }
    if constexpr (LANES > 64u) {
        __shared__ double waves[2][4];
        if (tid % 64u == 0u) {
            waves[0][tid / 64u] = a;
            waves[1][tid / 64u] = b;
        }
        __syncthreads();
        a = waves[0][0] + waves[0][1] + waves[0][2] + waves[0][3];
        b = waves[1][0] + waves[1][1] + waves[1][2] + waves[1][3];
    }
    if (tid == 0u) {
        p.total[0] = (float)a;
        p.total[1] = (float)b;
    }
}

// ------------------------------------------------------ gradient epilogues
// dt of a piece of the vocabulary, rounded to 16 bits; columns from N up to
// the next multiple of 8 are written as zeros, since the product dt.W reads
// whole 16-byte chunks of dt's rows.
template <int O>
struct XentGradArgs : TileArgs {
    const XentRow* rows;
    float c;
    int64_t v0;  // first column of the piece

    template <int RBK, int WR, int WC, int PBY, class Get>
    __device__ __forceinline__ void finish(uint8_t* ep, uint32_t lane, int64_t row0, int64_t col0, Get get) const
    {
        constexpr int G = 64 / RBK, NB = WR / RBK;
        const int64_t padded = (N + 7) / 8 * 8;
        if (col0 >= padded)
            return;
        const int lg4 = 4 * (int)(lane / RBK);
        const int left = N - col0 < WC ? (int)(N - col0) : WC;
        XentRow r[NB];
        int at[NB], here = 0;
        bool none[NB];  // (NaN is not equal to 0)
#pragma unroll
        for (int i = 0; i < NB; ++i) {
            const int64_t row = row0 + i * RBK + lane % RBK;
            r[i] = XentRow{0.0f, 0.0f, 0.0f, -1};
            if (row < M)
                r[i] = rows[row];
        }
#pragma unroll
        for (int i = 0; i < NB; ++i) {
            const int64_t k = (int64_t)r[i].target - v0 - col0;
            at[i] = k >= 0 && k < left ? (int)k : -1;
            here |= at[i] >= 0;
            none[i] = r[i].a == 0.0f && r[i].b == 0.0f;
        }
        // most tiles hold no row's target (64 columns of a vocabulary), and most
        // are whole: those run a multiply-add, an exponential, a product and a
        // selection a value (an ignored row's dt is zero whatever its logits)
        auto store = [&](auto plain) __attribute__((always_inline)) {
            store_rows16<O, RBK, WR, WC>(ep, lane, row0, col0, M, padded, C, ldc, 0, true,
                                         [&](int i, int q) __attribute__((always_inline)) {
                const f32x4 v = get(i, q);
                f32x4 d;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    d[e] = __builtin_amdgcn_exp2f(__builtin_fmaf(v[e], c, -r[i].lse2)) * r[i].a;
                    d[e] = none[i] ? 0.0f : d[e];
                    if constexpr (!decltype(plain)::value) {
                        const int col = q * 4 * G + lg4 + e;
                        d[e] = col == at[i] ? d[e] - r[i].b : d[e];  // (never of an ignored row: it has no target)
                        d[e] = col >= left ? 0.0f : d[e];
                    }
                }
                return d;
            });
        };
        if (left == WC && __builtin_amdgcn_ballot_w64(here != 0) == 0)
            store(std::true_type{});
        else
            store(std::false_type{});
    }
};

// The products that take dt: C = factor (acc + R), the factor in device memory,
// R the fp32 sums over the pieces before (or null).  O_F32 without a factor
// keeps such sums.
template <int O>
struct XentProdArgs : TileArgs {
    const float* factor;  // null: 1
    const float* R;
    int64_t ldr;

    template <int RBK, int WR, int WC, int PBY, class Get>
    __device__ __forceinline__ void finish(uint8_t* ep, uint32_t lane, int64_t row0, int64_t col0, Get get) const
    {
        const float f = factor != nullptr ? *factor : 1.0f;
        if constexpr (O != O_F32) {
            if (R == nullptr) {
                store_rows16<O, RBK, WR, WC>(ep, lane, row0, col0, M, N, C, ldc, 0, true,
                                             [&](int i, int q) __attribute__((always_inline)) { return get(i, q) * f; });
                return;
            }
        }
        constexpr int VC = Piece<O>::N;
        const int64_t col = col0 + lane % (WC / VC) * VC, left = N - col;
        const int n = left >= VC ? VC : left > 0 ? (int)left : 0;
        struct Sums {
            u32x4 q[VC / 4];
        };
        staged_rows<VC, Sums, RBK, WR, WC, PBY>(
            ep, lane, row0, get,
            [&](Sums& s, int64_t row) __attribute__((always_inline)) {
#pragma unroll
                for (int h = 0; h < VC / 4; ++h) {
                    const int m = n - 4 * h < 4 ? n - 4 * h : 4;
                    s.q[h] = u32x4{0u, 0u, 0u, 0u};
                    if (R != nullptr && row < M && m > 0)
                        s.q[h] = load_piece<O_F32>(R, row * ldr + col + 4 * h, m, m == 4);
                }
            },
            [&](const Sums& s, int64_t row, float* z) __attribute__((always_inline)) {
#pragma unroll
                for (int e = 0; e < VC; ++e)
                    z[e] = (z[e] + piece_value<O_F32>(s.q[e / 4], e % 4)) * f;
                if (row < M && n > 0)
                    store_piece<O>(C, row * ldc + col, pack_piece<O>(z), n, n == VC);
            });
    }
};

// dX's product with its K, a piece of the vocabulary, split over workgroups:
// it has few tiles and a long K
struct XentPartArgs : TileArgs, KeepsPartials {
    template <int RBK, int WR, int WC, int PBY, class Get>
    __device__ __forceinline__ void finish(uint8_t*, uint32_t, int64_t, int64_t, Get) const {}  // (not reached)
};

struct XentAddArgs {
    int64_t M, N;
    uint32_t tiles_n, splits;
    const float* partials;
    const float* factor;  // null: 1
    const float* R;       // the pieces before, or null
    int64_t ldr;
    void* C;
    int64_t ldc;
};

// C = factor (sum of the splits' partial tiles, in order, + R): a lane takes
// four values, a workgroup 16 rows of a tile's 256 columns
template <int O>
__global__ __launch_bounds__(256) void xent_add_partials(XentAddArgs p)
{
    const uint32_t lane = threadIdx.x & 63u, wn = threadIdx.x >> 6, i = blockIdx.x % 8u, wm = blockIdx.x / 8u % 2u, tile = blockIdx.x / 16u;
    const int64_t row = (int64_t)(tile / p.tiles_n) * 256 + wm * 128 + i * 16 + lane % 16u;
    const int64_t col0 = (int64_t)(tile % p.tiles_n) * 256 + wn * 64 + 4 * (lane / 16u);
    if (row >= p.M)
        return;
    const float f = p.factor != nullptr ? *p.factor : 1.0f;
    const float* const share = p.partials + ((size_t)tile * p.splits * 8 + wm * 4 + wn) * 8192 + (i * 4 * 64 + lane) * 4;
    f32x4 sum[4];
#pragma unroll
    for (int j = 0; j < 4; ++j)
        sum[j] = *(const f32x4*)(share + j * 256);
    for (uint32_t s = 1; s < p.splits; ++s)
#pragma unroll
        for (int j = 0; j < 4; ++j)
            sum[j] += *(const f32x4*)(share + (size_t)s * 65536 + j * 256);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const int64_t col = col0 + 16 * j, left = p.N - col;
        if (left <= 0)
            continue;
        const int n = left < 4 ? (int)left : 4;
        if (p.R != nullptr) {
            const u32x4 r = load_piece<O_F32>(p.R, row * p.ldr + col, n, n == 4);
#pragma unroll
            for (int e = 0; e < 4; ++e)
                sum[j][e] += piece_value<O_F32>(r, e);
        }
        sum[j] *= f;
        if constexpr (O == O_F32) {
            store_piece<O_F32>(p.C, row * p.ldc + col, bit_cast<u32x4>(sum[j]), n, n == 4);
        } else if (n == 4) {
            *(u32x2*)((uint16_t*)p.C + row * p.ldc + col) = u32x2{pack2<O>(sum[j][0], sum[j][1]), pack2<O>(sum[j][2], sum[j][3])};
        } else {
            for (int e = 0; e < n; ++e)
                store_value<O>(p.C, row * p.ldc + col + e, sum[j][e]);
        }
    }
}

// --------------------------------------------------------- gradient's rows
struct XentRowsArgs {
    int64_t M, V;
    const int64_t* target;
    int64_t ignore;
    float z, scale, grad_scale, lift;  // lift: 2^12 for fp16, 1 for bf16
    const float *lse, *dloss, *total;
    const float* most;  // the largest row factors (xent_most), or null: 1
    int32_t most_n;     // how many
    XentRow* rows;
    float* factor;
};

constexpr int kXentMost = 32;  // workgroups of xent_most at most: a lane of xent_rows' waves for each

// The largest finite factor of the rows that count, one for each workgroup (an
// infinite one's row is lost, the others keep their scale); a lane has four rows'
// loads in flight (131072 rows in one workgroup, a row at a time: 130 us)
template <int = 0>
__global__ __launch_bounds__(1024) void xent_most(XentRowsArgs p, float* out)
{
    __shared__ float red[16];
    const uint32_t tid = threadIdx.x;
    const int64_t step = (int64_t)gridDim.x * 1024;
    float most = 0.0f;
    for (int64_t i0 = (int64_t)blockIdx.x * 1024 + tid; i0 < p.M; i0 += 4 * step) {
        float b[4], lse[4];
        bool counts[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const int64_t i = i0 + u * step;
            b[u] = 1.0f;
            lse[u] = 0.0f;
            counts[u] = false;
            if (i < p.M) {
                counts[u] = p.target[i] != p.ignore;
                if (p.dloss != nullptr)
                    b[u] = __builtin_fabsf(p.dloss[i]);
                lse[u] = p.lse[i];
            }
        }
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const float f = max2(b[u], b[u] * __builtin_fabsf(1.0f + 2.0f * p.z * lse[u]));
            if (counts[u] && f < INFINITY)
                most = max2(most, f);
        }
    }
#pragma unroll
    for (int d = 32; d > 0; d >>= 1)
        most = max2(most, __shfl_xor(most, d, 64));
    if ((tid & 63u) == 0u)
        red[tid >> 6] = most;
    __syncthreads();
#pragma unroll
    for (int k = 0; k < 16; ++k)
        most = max2(most, red[k]);
    if (tid == 0u)
        out[blockIdx.x] = most;
}

// Each row's numbers relative to a power of two at or above the largest; what
// that (and `lift`) divides out returns in the products' factor.
template <int = 0>
__global__ __launch_bounds__(256) void xent_rows(XentRowsArgs p)
{
    // 2^e >= most, within fp32's normal numbers (none at all: 1)
    int e = 0;
    float most = 1.0f;
    if (p.most != nullptr) {
        const int lane = (int)(threadIdx.x % 64u);
        most = lane < p.most_n ? p.most[lane] : 0.0f;
#pragma unroll
        for (int d = kXentMost; d > 0; d >>= 1)
            most = max2(most, __shfl_xor(most, d, 64));
    }
    if (most > 0.0f && most != 1.0f) {
        (void)frexpf(most, &e);
        e = e < -100 ? -100 : e;
    }
    const float down = ldexpf(1.0f, -e) * p.lift;  // (e <= 128, lift <= 2^12: a normal number or a subnormal 2^-128)
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (i == 0) {
        const float count = p.total != nullptr ? max2(p.total[1], 1.0f) : 1.0f;
        *p.factor = (float)((double)p.scale * (double)p.grad_scale * ldexp(1.0, e) / ((double)p.lift * (double)count));
    }
    if (i >= p.M)
        return;
    const int64_t t = p.target[i];
    XentRow r{0.0f, 0.0f, 0.0f, -1};
    if (t != p.ignore) {
        const bool known = t >= 0 && t < p.V;
        const float lse = p.lse[i];
        r.lse2 = lse * 1.44269504088896341f;
        r.b = known ? (p.dloss != nullptr ? p.dloss[i] * down : down) : NAN;
        r.a = r.b * (1.0f + 2.0f * p.z * lse);
        r.target = known ? (int32_t)t : -1;
    }
    p.rows[i] = r;
}

// --------------------------------------------------------------- host side
inline int64_t up(int64_t n, int64_t to) { return (n + to - 1) / to * to; }

// forward: the skinny kernel's rows, as for tg_linear (a launch has less than 2^32 lanes)
template <int E>
bool xent_skinny(int64_t M, int64_t D, int64_t ldx, int64_t ldw, int64_t V)
{
    return M <= kFusedSkinnyRows<E> && D > 0 && fused_skinny_blocks(M, V) * 64 * SkinnyCfg::WAVES < (int64_t)1 << 32 &&
           skinny_offsets_fit(D, ldx, ldw, SkinnyCfg::RING, fused_cg(M, V));
}

struct XentFwd {
    int64_t slots, part, picked, sums, bytes;  // offsets and bytes in the workspace
    int join_rows;
};

// rows per workgroup of xent_join: one where there are few, which then take 256 lanes each
inline int xent_join_rows(int64_t M) { return M <= 64 ? 1 : 16; }

// (slots of 16 columns for few rows, whichever kernel then takes them)
inline XentFwd xent_fwd_layout(int64_t M, int64_t V, int64_t few)
{
    XentFwd f{};
    const int64_t cols = M <= few ? 16 : kXentCols;
    f.slots = (V + cols - 1) / cols;
    f.join_rows = xent_join_rows(M);
    f.part = kSplitCounterBytes;
    f.picked = up(f.part + f.slots * M * 8, 256);
    f.sums = up(f.picked + M * 4, 256);
    // (a slot of the sums without rows as well: their workgroup writes the total)
    f.bytes = up(f.sums + (M == 0 ? 1 : (M + f.join_rows - 1) / f.join_rows) * 16, 256);
    return f;
}

struct XentCall {
    int64_t M, V, D;
    const void* x;
    int64_t ldx;
    const void* W;
    int64_t ldw;
    float scale;
    const int64_t* target;
    int64_t ignore;
    float z;
    // forward
    float *loss, *lse_out, *total_out;
    // gradient
    const float *lse, *dloss, *total;
    float grad_scale;
    void* dX;
    int64_t lddx;
    void* dW;
    int64_t lddw;
    int dw_dtype;
    void* ws;
    int64_t ws_bytes;
    hipStream_t s;
};

inline float xent_c(float scale) { return (float)((double)scale * 1.4426950408889634074); }

template <int E, int AI, int CG>
void launch_xent_skinny(const XentSkinnyArgs& a, int64_t blocks, hipStream_t s)
{
    typedef SkinnyCfg G;
    hipLaunchKernelGGL((skinny_gemm<E, O_F32, G::WAVES, AI, G::RING, 0, CG, EPI_OWN, XentSkinnyArgs>), dim3((uint32_t)blocks),
                       dim3(64 * G::WAVES), 0, s, a);
}

// A part of the forward product, of up to kXentTiles tiles
template <int E>
tg_status xent_logits(XentFwdArgs a, hipStream_t s)
{
    // tiles whose waves hold 64 columns: no 64 x 64 ones
    const NtPlan p = plan_nt<E, B_KCONTIG>(a.M, a.N, a.K, false);
    if (p.tile == 256 && p.tn == 128)
        return launch_nt<E, O_F32, 256, 128, B_KCONTIG, kWideNH, EPI_OWN, A_KCONTIG>(a, 1, s);
    if (p.tile == 256 && p.tail == kTailNone)
        return launch_nt<E, O_F32, 256, 256, B_KCONTIG, 5, EPI_OWN, A_KCONTIG>(a, 1, s);
    if (p.tile == 256) {
        XentFwdArgs b = a;
        const int64_t rest = n_tiles<256, 256>(a.M, a.N) - p.dp;
        a.dp = (uint32_t)p.dp;
        const tg_status st = launch_nt<E, O_F32, 256, 256, B_KCONTIG, 5, EPI_OWN, A_KCONTIG>(a, 1, s, p.dp);
        if (st != TG_OK)
            return st;
        b.sub256 = (uint32_t)p.dp + 1u;
        return p.tail == kTailWide ? launch_nt<E, O_F32, 256, 128, B_KCONTIG, kWideNH, EPI_OWN, A_KCONTIG>(b, 1, s, 2 * rest)
                                   : launch_nt<E, O_F32, 128, 128, B_KCONTIG, 8, EPI_OWN, A_KCONTIG>(b, 1, s, 4 * rest);
    }
    if (n_tiles<128, 128>(a.M, a.N) <= 256)
        return launch_nt<E, O_F32, 128, 128, B_KCONTIG, 8, EPI_OWN, A_KCONTIG>(a, 1, s);
    return launch_nt<E, O_F32, 128, 128, B_KCONTIG, 4, EPI_OWN, A_KCONTIG>(a, 1, s);
}

// Tiles of 512 lanes in a launch (which has less than 2^32) of the forward
// product, and columns: past 2^39 logits it goes in parts
constexpr int64_t kXentTiles = (1 << 23) - 1, kXentWide = (int64_t)1 << 30;

template <int E>
tg_status xent_forward(const XentCall& q)
{
    const XentFwd f = xent_fwd_layout(q.M, q.V, kFusedSkinnyRows<E>);
    uint8_t* const ws = (uint8_t*)q.ws;
    XentOut o{xent_c(q.scale), q.scale, q.target, (f32x2_t*)(ws + f.part), (float*)(ws + f.picked), q.M, 0};
    int64_t slots = f.slots;
    if (q.M == 0) {
        // (only the total, of no rows)
    } else if (xent_skinny<E>(q.M, q.D, q.ldx, q.ldw, q.V)) {
        XentSkinnyArgs a{};
        a.M = q.M;
        a.N = q.V;
        a.K = q.D;
        a.A = (const uint8_t*)q.x;
        a.lda = q.ldx;
        a.B = (const uint8_t*)q.W;
        a.ldb = q.ldw;
        a.x = o;
        const int64_t blocks = fused_skinny_blocks(q.M, q.V);
        if (q.M <= 8)
            launch_xent_skinny<E, 1, 1>(a, blocks, q.s);
        else if (fused_cg(q.M, q.V) == 1)
            launch_xent_skinny<E, 2, 1>(a, blocks, q.s);
        else
            launch_xent_skinny<E, 2, 2>(a, blocks, q.s);
    } else {
        slots = (q.V + kXentCols - 1) / kXentCols;
        const int64_t wide = q.V < kXentWide ? q.V : kXentWide, high = kXentTiles / ((wide + 255) / 256) * 256;
        for (int64_t v0 = 0; v0 < q.V; v0 += wide)
            for (int64_t r0 = 0; r0 < q.M; r0 += high) {
                XentFwdArgs a{};
                set_product(a, q.M - r0 < high ? q.M - r0 : high, q.V - v0 < wide ? q.V - v0 : wide, q.D, (const uint8_t*)q.x + 2 * r0 * q.ldx, q.ldx,
                            (const uint8_t*)q.W + 2 * v0 * q.ldw, q.ldw, nullptr, 0, 1.0f);
                a.x = o;
                a.x.target += r0;
                a.x.part += v0 / kXentCols * q.M + r0;
                a.x.picked += r0;
                a.x.v0 = v0;
                a.group_m = 4;
                a.splits = 1;
                if (!nt_eligible<E>(a))
                    return TG_ERR_NOT_SUPPORTED;
                const tg_status st = xent_logits<E>(a, q.s);
                if (st != TG_OK)
                    return st;
            }
    }
    XentJoinArgs j{};
    j.M = q.M;
    j.V = q.V;
    j.slots = slots;
    j.part = o.part;
    j.picked = o.picked;
    j.target = q.target;
    j.ignore = q.ignore;
    j.z = q.z;
    j.loss = q.loss;
    j.lse = q.lse_out;
    j.total = q.total_out;
    j.counter = (uint32_t*)ws;
    j.sums = (double*)(ws + f.sums);
    const int64_t groups = q.M == 0 ? 1 : (q.M + f.join_rows - 1) / f.join_rows;
    for (int64_t first = 0; first < groups; first += kJoinGrid) {
        const uint32_t grid = (uint32_t)(groups - first < kJoinGrid ? groups - first : kJoinGrid);
        j.first = (uint32_t)first;
        j.more = first + grid < groups;
        if (f.join_rows == 1)
            hipLaunchKernelGGL(xent_join<1>, dim3(grid), dim3(256), 0, q.s, j);
        else
            hipLaunchKernelGGL(xent_join<16>, dim3(grid), dim3(256), 0, q.s, j);
    }
    return launched();
}

// Columns of a piece: as many as dt holds in kXentPieceBytes, kXentPiece with
// many rows (each piece reads and writes dX's fp32 sums), and a piece's rows of
// W lie within one buffer descriptor (as nt_eligible_nrow asks).  From 256 MiB to
// 1 GiB the gradients take the same time within 1% (4096 x 128256 x 4096; 4% at
// 8192 x 131072 x 1024), 128 MiB costs 1 to 13% and 64 MiB 2 to 30.
constexpr int64_t kXentPieceBytes = (int64_t)512 << 20, kXentPiece = 8192;

inline int64_t xent_most_piece(int64_t M, int64_t V, int64_t ldw)
{
    int64_t most = kXentPieceBytes / (2 * (M < 1 ? 1 : M)) / 256 * 256;
    most = most < kXentPiece ? kXentPiece : most;
    const int64_t fits = ((int64_t)kNumRecords - 1024) / (2 * (ldw < 1 ? 1 : ldw)) - 512;
    if (most > 131072)
        most = 131072;
    if (most > fits / 256 * 256)
        most = fits / 256 * 256;
    if (most > up(V, 256))
        most = up(V, 256);
    return most;
}

// Pieces of equal size (multiples of 256, the last one the rest) of at most `most` columns
inline int64_t xent_even(int64_t V, int64_t most)
{
    const int64_t pieces = (V + most - 1) / most;
    return up((V + pieces - 1) / pieces, 256);
}

// Splits of dX's product (K columns of the vocabulary) over workgroups that
// keep their partial tiles, or 1: the other plans.  In cycles of a compute unit,
// a step of the 256 tile takes about 2450, a round of workgroups 12000 besides,
// and adding the partial tiles 10000 and their way out and back at 2500 bytes a
// cycle.  Up to 128 rows half the tile is idle, and below 4096 tile steps the
// second launch costs more than the split saves.  Gradients of x alone, M x V x D
// bf16, us, other plans -> split: 777 x 32003 x 1032 188 -> 152, 2048 x 50000 x
// 2048 825 -> 705, 512 x 100000 x 4096 868 -> 735, 4096 x 32000 x 1024 564 -> 491,
// 300 x 100000 x 768 203 -> 191; but 128 x 100000 x 4096 392 -> 408, 100 x 32000 x
// 1024 42 -> 59, 700 x 10000 x 256 30 -> 42, 4000 x 5000 x 512 68 -> 75.
inline int64_t xent_dx_splits(int64_t M, int64_t D, int64_t K)
{
    const int64_t tiles = n_tiles<256, 256>(M, D), steps = (K + 63) / 64;
    int64_t best_s = 1;
    double best = 0.0;
    if (M <= 128 || tiles * steps < 4096)
        return 1;
    for (int64_t s = 1; tiles * s <= 512 && steps / s >= 8; ++s) {
        const double rounds = (double)((tiles * s + 255) / 256);
        const double cost = rounds * ((double)steps / s * 2450.0 + 12000.0) + (s > 1 ? 10000.0 + (double)s * M * D * 8.0 / 2500.0 : 0.0);
        if (best == 0.0 || cost < best) {
            best = cost;
            best_s = s;
        }
    }
    return best_s;
}

// partial tiles of any split plan: two rounds of 256 x 256 fp32
constexpr int64_t kXentSplitBytes = (int64_t)128 << 20;

struct XentBwd {
    int64_t piece, pieces, ldz;
    int64_t rows, factor, sums, dz, bytes;  // offsets and bytes in the workspace
};

inline XentBwd xent_bwd_layout(int64_t M, int64_t V, int64_t D, int64_t piece)
{
    XentBwd b{};
    b.piece = piece;
    b.pieces = (V + piece - 1) / piece;
    b.ldz = piece;
    b.rows = kSplitCounterBytes + kXentSplitBytes;
    b.factor = up(b.rows + M * (int64_t)sizeof(XentRow), 256);
    b.sums = b.factor + 256;
    b.dz = up(b.sums + (b.pieces > 1 ? M * up(D, 4) * 4 : 0), 256);
    b.bytes = b.dz + M * b.ldz * 2;
    return b;
}

// The layout with the fewest pieces that `ws_bytes` hold; bytes 0 if none does
inline XentBwd xent_bwd_plan(int64_t M, int64_t V, int64_t D, int64_t most, int64_t ws_bytes)
{
    int64_t last = 0;
    for (int64_t k = (V + most - 1) / most; k <= (V + 255) / 256; ++k) {
        const int64_t piece = up((V + k - 1) / k, 256);
        if (piece == last || piece > most)
            continue;
        last = piece;
        const XentBwd b = xent_bwd_layout(M, V, D, piece);
        if (b.bytes <= ws_bytes)
            return b;
        if (piece == 256)
            break;
    }
    return XentBwd{};
}

// Bytes of pieces of `piece` columns, with room for dX's sums also where they
// make one piece: rows of W far apart may ask for several (xent_most_piece)
inline int64_t xent_bwd_bytes(int64_t M, int64_t V, int64_t D, int64_t piece)
{
    const int64_t most = xent_most_piece(M, V, D);
    if (most < 256)
        return -1;
    const XentBwd b = xent_bwd_layout(M, V, D, piece == 0 || piece > most ? xent_even(V, most) : up(piece, 256));
    return b.bytes + (b.pieces == 1 && V > 256 ? up(M * up(D, 4) * 4, 256) : 0);
}

// The least that a call takes: one piece needs no sums, and may take less than several
inline int64_t xent_bwd_least(int64_t M, int64_t V, int64_t D, int64_t ldw)
{
    const int64_t most = xent_most_piece(M, V, ldw), bytes = xent_bwd_layout(M, V, D, 256).bytes;
    if (up(V, 256) > most)
        return bytes;
    const int64_t whole = xent_bwd_layout(M, V, D, up(V, 256)).bytes;
    return whole < bytes ? whole : bytes;
}

// dt of a piece
template <int E>
tg_status xent_dz(const TileArgs& t, const XentRow* rows, float c, int64_t v0, hipStream_t s)
{
    XentGradArgs<OutOf<E>::O> a{};
    static_cast<TileArgs&>(a) = t;
    a.rows = rows;
    a.c = c;
    a.v0 = v0;
    if (!nt_eligible<E>(a))
        return TG_ERR_NOT_SUPPORTED;
    return launch_nt_plan<E, OutOf<E>::O, B_KCONTIG, EPI_OWN, A_KCONTIG>(a, plan_nt<E, B_KCONTIG>(a.M, a.N, a.K, false), nullptr, s);
}

// A product that takes dt (which may end inside a 16-byte chunk: the rest of
// it is zeros, or feeds rows that are not stored)
template <int E, int O, int AL>
tg_status xent_product(const TileArgs& t, const float* factor, const float* R, int64_t ldr, void* ws, hipStream_t s)
{
    XentProdArgs<O> a{};
    static_cast<TileArgs&>(a) = t;
    a.factor = factor;
    a.R = R;
    a.ldr = ldr;
    return launch_nt_plan<E, O, B_NCONTIG, EPI_OWN, AL>(a, plan_nt<E, B_NCONTIG>(a.M, a.N, a.K, true), ws, s);
}

template <int E, int O>
tg_status xent_dx(const TileArgs& t, const float* factor, const float* R, int64_t ldr, void* ws, hipStream_t s)
{
    const int64_t splits = xent_dx_splits(t.M, t.N, t.K);
    if (splits == 1)
        return xent_product<E, O, A_KCONTIG>(t, factor, R, ldr, ws, s);
    XentPartArgs a{};
    static_cast<TileArgs&>(a) = t;
    a.group_m = 4;
    a.splits = (uint32_t)splits;
    a.partials = (float*)((uint8_t*)ws + kSplitCounterBytes);
    const tg_status st = launch_nt<E, O_F32, 256, 256, B_NCONTIG, 5, EPI_OWN, A_KCONTIG>(a, (int)splits, s);
    if (st != TG_OK)
        return st;
    const uint32_t tiles_n = (uint32_t)((t.N + 255) / 256);
    const XentAddArgs p{t.M, t.N, tiles_n, (uint32_t)splits, a.partials, factor, R, ldr, t.C, t.ldc};
    hipLaunchKernelGGL(xent_add_partials<O>, dim3((uint32_t)(n_tiles<256, 256>(t.M, t.N) * 16)), dim3(256), 0, s, p);
    return launched();
}

// (defined in the translation units of their kernels)
template <int E> tg_status xent_xgrad(const TileArgs& t, bool last, const float* factor, const float* R, int64_t ldr, void* ws, hipStream_t s);
template <int E> tg_status xent_wgrad(const TileArgs& t, int dtype, const float* factor, void* ws, hipStream_t s);
template <> tg_status xent_xgrad<E_F16>(const TileArgs&, bool, const float*, const float*, int64_t, void*, hipStream_t);
template <> tg_status xent_xgrad<E_BF16>(const TileArgs&, bool, const float*, const float*, int64_t, void*, hipStream_t);
template <> tg_status xent_wgrad<E_F16>(const TileArgs&, int, const float*, void*, hipStream_t);
template <> tg_status xent_wgrad<E_BF16>(const TileArgs&, int, const float*, void*, hipStream_t);

template <int E>
tg_status xent_backward(const XentCall& q)
{
    const int64_t most = xent_most_piece(q.M, q.V, q.ldw);
    if (most < 256)
        return TG_ERR_NOT_SUPPORTED;
    const XentBwd b = xent_bwd_plan(q.M, q.V, q.D, most, q.ws_bytes);
    if (b.bytes == 0)
        return TG_ERR_INVALID_VALUE;
    uint8_t* const ws = (uint8_t*)q.ws;
    XentRow* const rows = (XentRow*)(ws + b.rows);
    float* const factor = (float*)(ws + b.factor);
    float* const sums = (float*)(ws + b.sums);
    const int64_t lds = up(q.D, 4);
    XentRowsArgs r{q.M, q.V, q.target, q.ignore, q.z, q.scale, q.grad_scale, E == E_F16 ? 4096.0f : 1.0f, q.lse, q.dloss, q.total, nullptr, 0, rows, factor};
    // factors of the rows' own are taken relative to the largest; 1 + 2 z lse is
    // near enough to 1 for bf16's range
    if (q.dloss != nullptr || (E == E_F16 && q.z != 0.0f)) {
        const int64_t groups = (q.M + 1023) / 1024;
        r.most_n = (int32_t)(groups > kXentMost ? kXentMost : groups + (groups == 0));
        hipLaunchKernelGGL(xent_most<>, dim3((uint32_t)r.most_n), dim3(1024), 0, q.s, r, factor + 1);
        r.most = factor + 1;
    }
    hipLaunchKernelGGL(xent_rows<>, dim3((uint32_t)((q.M + 255) / 256 + (q.M == 0))), dim3(256), 0, q.s, r);
    tg_status st = launched();
    for (int64_t i = 0; i < b.pieces && st == TG_OK; ++i) {
        const int64_t v0 = i * b.piece, n = q.V - v0 < b.piece ? q.V - v0 : b.piece;
        const uint8_t* const Wp = (const uint8_t*)q.W + v0 * q.ldw * 2;
        void* const dz = ws + b.dz;
        if (q.M > 0) {
            TileArgs t{};
            set_product(t, q.M, n, q.D, q.x, q.ldx, Wp, q.ldw, dz, b.ldz, 1.0f);
            st = xent_dz<E>(t, rows, xent_c(q.scale), v0, q.s);
            if (st == TG_OK && q.dX != nullptr) {
                const bool last = i == b.pieces - 1;
                set_product(t, q.M, q.D, n, dz, b.ldz, Wp, q.ldw, last ? q.dX : sums, last ? q.lddx : lds, 1.0f);
                st = xent_xgrad<E>(t, last, last ? factor : nullptr, i > 0 ? sums : nullptr, lds, q.ws, q.s);
            }
        }
        if (st == TG_OK && q.dW != nullptr) {
            TileArgs t{};
            set_product(t, n, q.D, q.M, dz, b.ldz, q.x, q.ldx, (uint8_t*)q.dW + v0 * q.lddw * out_bytes(q.dw_dtype), q.lddw, 1.0f);
            st = xent_wgrad<E>(t, q.dw_dtype, factor, q.ws, q.s);
        }
    }
    return st;
}

}  // namespace tg
