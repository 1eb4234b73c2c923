// Host side of the fused products (contracts in include/tg_ops.h): argument
// checks, plans and launches, one template per operator and input type, each
// instantiated in that type's translation unit.
#pragma once

#include <math.h>

#include "tg_host.hpp"
#include "tg_ops.h"

namespace tg {

// The NT tile plans and the skinny kernel's splits are those of the plain
// GEMM of the same product; workspaces follow tg_gemm_ex's contract.

inline bool act_ok(int act) { return act >= TG_ACT_NONE && act <= TG_ACT_SILU; }

inline void set_act(EpiArgs& e, int act)
{
    e.lo = -INFINITY;
    e.slope_lo = 1.0f;
    e.s1 = 1.0f;
    e.s3 = 0.0f;
    switch (act) {
    case TG_ACT_RELU: e.lo = 0.0f; e.slope_lo = 0.0f;  // fall through
    case TG_ACT_NONE: e.kind = AK_CLIP; break;
    case TG_ACT_GELU: e.kind = AK_ERF; break;
    case TG_ACT_GELU_TANH:  // 2 sqrt(2/pi) and 0.044715 of it
        e.s1 = 1.5957691216057308f;
        e.s3 = 0.071354816272600245f;  // fall through
    default: e.kind = AK_SIGMOID; break;
    }
}

// A matrix argument of rows x cols elements; empty ones are not looked at.
inline tg_status check_mat(const void* p, int64_t rows, int64_t cols, int64_t ld, int elem_bytes)
{
    if (rows == 0 || cols == 0)
        return TG_OK;
    if (p == nullptr || ld < cols)
        return TG_ERR_INVALID_VALUE;
    if (!aligned16(p) || ((ld * elem_bytes) & 15))
        return TG_ERR_MISALIGNED;
    return TG_OK;
}

// The workspace argument of a fused call that could use `need` bytes.
inline tg_status check_ws(const void* ws, int64_t ws_bytes, int64_t need)
{
    if (ws_bytes < 0 || (ws == nullptr && ws_bytes != 0))
        return TG_ERR_INVALID_VALUE;
    if (ws != nullptr) {
        if (((uintptr_t)ws & 255u) != 0)
            return TG_ERR_MISALIGNED;
        if (ws_bytes < need)
            return TG_ERR_INVALID_VALUE;
    }
    return TG_OK;
}

template <int E> struct OutOf { static constexpr int O = E == E_F16 ? O_F16 : O_BF16; };

inline void set_product(TileArgs& a, int64_t M, int64_t N, int64_t K, const void* A, int64_t lda, const void* B,
                        int64_t ldb, void* C, int64_t ldc, float alpha)
{
    a.M = M;
    a.N = N;
    a.K = K;
    a.A = (const uint8_t*)A;
    a.lda = lda;
    a.B = (const uint8_t*)B;
    a.ldb = ldb;
    a.C = C;
    a.ldc = ldc;
    a.alpha = alpha;
}

// The NT kernel with both operands as k rows (a transposed A): whole 16-byte
// chunks along M and N; offsets span one K step of rows, so K is free.
template <int E>
inline bool nt_eligible_tn(const TileArgs& a)
{
    constexpr int EB = ElemInfo<E>::bytes, CE = 16 / EB, KE = 128 / EB;
    const int64_t lim = (int64_t)kNumRecords;
    return a.M % CE == 0 && a.N % CE == 0 && KE * a.lda * EB + 512 < lim && KE * a.ldb * EB + 512 < lim;
}

// One product on the NT kernel where its element grid allows, else on the
// generic tile kernel (64 x 128 tiles; for EPI_GLU 64 hidden columns).
template <int E, int O, int BL, int EPI, int AL, class P>
tg_status launch_fused(P& a, void* ws, int64_t ws_bytes, hipStream_t s)
{
    const int64_t Nt = EPI == EPI_GLU ? 2 * a.N : a.N;
    bool nt;
    if constexpr (AL == A_MCONTIG)
        nt = nt_eligible_tn<E>(a);
    else
        nt = nt_takes<E, BL>(a);
    if (nt) {
        NtPlan plan = plan_nt<E, BL>(a.M, Nt, a.K, ws != nullptr);
        if (plan.ws_bytes > ws_bytes)
            plan = plan_nt<E, BL>(a.M, Nt, a.K, false);
        return launch_nt_plan<E, O, BL, EPI, AL>(a, plan, ws, s);
    }
    const int64_t tiles = n_tiles<64, 128>(a.M, Nt);
    if (tiles > 0x7FFFFFFF)
        return TG_ERR_NOT_SUPPORTED;
    a.group_m = 4;
    hipLaunchKernelGGL((tile_gemm<E, BL, O, 64, 128, false, EPI, AL, P>), dim3((uint32_t)tiles), dim3(kThreads), 0, s,
                       a);
    return launched();
}

// skinny_split, by the bytes of K that a workgroup streams
template <int E>
inline int fused_split(int64_t blocks, int64_t K)
{
    return skinny_split(blocks, K * ElemInfo<E>::bytes / 2, false);
}

template <int E, int O, int AI, int SPLIT, int CG, int EPI>
void launch_skinny_epi(const FusedSkinnyArgs& sa, int64_t blocks, int split, hipStream_t s)
{
    typedef SkinnyCfg G;
    hipLaunchKernelGGL((skinny_gemm<E, O, G::WAVES, AI, G::RING, SPLIT, CG, EPI, FusedSkinnyArgs>),
                       dim3((uint32_t)blocks, (uint32_t)split), dim3(64 * G::WAVES), 0, s, sa);
}

// Rows up to which a call takes the skinny kernel.  fp8's second slice of 16
// rows runs slower there than the tile kernel with K split (32 rows,
// N = 8192, K = 4096: 14.8 us against 12.1; one slice, N = K = 8192: 13.5
// against 20.5).
template <int E>
constexpr int64_t kFusedSkinnyRows = E == E_FP8 ? 16 : kSkSliceMaxMSplit;

// 16-column groups per workgroup: two with several slices of rows, and for
// 9 to 16 rows where that leaves a workgroup for every compute unit, since
// each workgroup copies its rows of x over all of K (bf16 N = K = 8192: 16
// rows 26.9 -> 25.8 us, but 1 row 24.3 -> 24.9).
inline int fused_cg(int64_t M, int64_t N) { return M > 16 || (M > 8 && N > 32 * 255) ? 2 : 1; }

inline int64_t fused_skinny_blocks(int64_t M, int64_t N)
{
    const int64_t cols = 16 * fused_cg(M, N);
    const int64_t nblk = (N + cols - 1) / cols, slices = (M + 15) / 16;
    return slices == 1 ? nblk : (nblk + 7) / 8 * 8 * slices;
}

inline int64_t fused_skinny_ws_bytes(int64_t M, int64_t N, int64_t blocks, int split)
{
    const int64_t groups = fused_cg(M, N);
    if (split <= 1 || blocks * groups * 16 > kSplitMaxCounters)  // (kCounterStride words each)
        return 0;
    return kSplitCounterBytes + blocks * groups * split * 1024;
}

template <int E, int O, int SPLIT>
void launch_skinny_fused(const FusedSkinnyArgs& sa, int64_t blocks, int split, hipStream_t s)
{
    if (sa.M <= 8)
        launch_skinny_epi<E, O, 1, SPLIT, 1, EPI_LINEAR>(sa, blocks, split, s);
    else if (fused_cg(sa.M, sa.N) == 1)
        launch_skinny_epi<E, O, 2, SPLIT, 1, EPI_LINEAR>(sa, blocks, split, s);
    else
        launch_skinny_epi<E, O, 2, SPLIT, 2, EPI_LINEAR>(sa, blocks, split, s);
}

template <int E, int O, int SPLIT>
void launch_skinny_glu(const FusedSkinnyArgs& sa, int64_t blocks, int split, hipStream_t s)
{
    if (sa.M <= 8)
        launch_skinny_epi<E, O, 1, SPLIT, 2, EPI_GLU>(sa, blocks, split, s);
    else
        launch_skinny_epi<E, O, 2, SPLIT, 2, EPI_GLU>(sa, blocks, split, s);
}

// ------------------------------------------------------------------ linear
template <int E>
int64_t linear_ws_bytes(int64_t M, int64_t N, int64_t K)
{
    if (M <= 0 || N <= 0 || K <= 0 || !dims_fit(M, N, K))
        return 0;
    if (M <= kFusedSkinnyRows<E>) {
        const int64_t blocks = fused_skinny_blocks(M, N);
        return fused_skinny_ws_bytes(M, N, blocks, fused_split<E>(blocks, K));
    }
    return K % (16 / ElemInfo<E>::bytes) == 0 ? plan_nt<E, B_KCONTIG>(M, N, K, true).ws_bytes : 0;
}

template <int E, int O>
tg_status linear_out(FusedArgs& a, void* ws, int64_t ws_bytes, hipStream_t s)
{
    if (a.M <= kFusedSkinnyRows<E> && a.K > 0 &&
        skinny_offsets_fit(a.K, a.lda, a.ldb, SkinnyCfg::RING, fused_cg(a.M, a.N))) {
        FusedSkinnyArgs sa{};
        sa.M = a.M;
        sa.N = a.N;
        sa.K = a.K;
        sa.A = a.A;
        sa.lda = a.lda;
        sa.B = a.B;
        sa.ldb = a.ldb;
        sa.C = a.C;
        sa.ldc = a.ldc;
        sa.e = a.e;
        sa.alpha = a.alpha;
        const int64_t blocks = fused_skinny_blocks(a.M, a.N);
        if (blocks > 0x7FFFFFFF)
            return TG_ERR_NOT_SUPPORTED;
        int split = fused_split<E>(blocks, a.K);
        const int64_t need = fused_skinny_ws_bytes(a.M, a.N, blocks, split);
        if (ws == nullptr || need == 0 || need > ws_bytes)
            split = 1;
        if (split > 1) {
            sa.counters = (uint32_t*)ws;
            sa.partials = (float*)((uint8_t*)ws + kSplitCounterBytes);
            launch_skinny_fused<E, O, 2>(sa, blocks, split, s);
        } else {
            launch_skinny_fused<E, O, 0>(sa, blocks, 1, s);
        }
        return launched();
    }
    return launch_fused<E, O, B_KCONTIG, EPI_LINEAR, A_KCONTIG>(a, ws, ws_bytes, s);
}

template <int E>
tg_status linear_typed(const TileArgs& t, const EpiArgs& e, int y_dtype, void* ws, int64_t ws_bytes, void* stream)
{
    FusedArgs a{};
    static_cast<TileArgs&>(a) = t;
    a.e = e;
    hipStream_t s = (hipStream_t)stream;
    if (y_dtype == TG_F32)
        return linear_out<E, O_F32>(a, ws, ws_bytes, s);
    if constexpr (E != E_BF16)
        if (y_dtype == TG_F16)
            return linear_out<E, O_F16>(a, ws, ws_bytes, s);
    if constexpr (E != E_F16)
        if (y_dtype == TG_BF16)
            return linear_out<E, O_BF16>(a, ws, ws_bytes, s);
    return TG_ERR_NOT_SUPPORTED;
}

// --------------------------------------------------------------------- glu
// The skinny kernel's launch for EPI_GLU: 16 hidden columns per workgroup.
inline int64_t glu_skinny_blocks(int64_t M, int64_t F)
{
    const int64_t nblk = (F + 15) / 16, slices = (M + 15) / 16;
    return slices == 1 ? nblk : (nblk + 7) / 8 * 8 * slices;
}

inline int64_t glu_skinny_ws_bytes(int64_t blocks, int split)
{
    return split <= 1 || blocks * 16 > kSplitMaxCounters ? 0 : kSplitCounterBytes + blocks * split * 2048;
}

template <int E>
int64_t glu_ws_bytes(int64_t M, int64_t F, int64_t D)
{
    if (M <= 0 || F <= 0 || D <= 0 || !dims_fit(M, F, D) || !dims_fit(2 * F, 0, 0))
        return 0;
    if (M <= kFusedSkinnyRows<E>) {
        const int64_t blocks = glu_skinny_blocks(M, F);
        return glu_skinny_ws_bytes(blocks, fused_split<E>(blocks, D));
    }
    return D % (16 / ElemInfo<E>::bytes) == 0 ? plan_nt<E, B_KCONTIG>(M, 2 * F, D, true).ws_bytes : 0;
}

template <int E, int O>
tg_status glu_out(FusedArgs& a, void* ws, int64_t ws_bytes, hipStream_t s)
{
    if (a.M <= kFusedSkinnyRows<E> && a.K > 0 && skinny_offsets_fit(a.K, a.lda, a.ldb, SkinnyCfg::RING, 1)) {
        FusedSkinnyArgs sa{};
        sa.M = a.M;
        sa.N = a.N;
        sa.K = a.K;
        sa.A = a.A;
        sa.lda = a.lda;
        sa.B = a.B;
        sa.ldb = a.ldb;
        sa.C = a.C;
        sa.ldc = a.ldc;
        sa.e = a.e;
        sa.alpha = a.alpha;
        const int64_t blocks = glu_skinny_blocks(a.M, a.N);
        if (blocks > 0x7FFFFFFF)
            return TG_ERR_NOT_SUPPORTED;
        int split = fused_split<E>(blocks, a.K);
        const int64_t need = glu_skinny_ws_bytes(blocks, split);
        if (ws == nullptr || need == 0 || need > ws_bytes)
            split = 1;
        if (split > 1) {
            sa.counters = (uint32_t*)ws;
            sa.partials = (float*)((uint8_t*)ws + kSplitCounterBytes);
            launch_skinny_glu<E, O, 2>(sa, blocks, split, s);
        } else {
            launch_skinny_glu<E, O, 0>(sa, blocks, 1, s);
        }
        return launched();
    }
    return launch_fused<E, O, B_KCONTIG, EPI_GLU, A_KCONTIG>(a, ws, ws_bytes, s);
}

template <int E>
tg_status glu_typed(const TileArgs& t, const EpiArgs& e, int h_dtype, void* ws, int64_t ws_bytes, void* stream)
{
    FusedArgs a{};
    static_cast<TileArgs&>(a) = t;
    a.e = e;
    hipStream_t s = (hipStream_t)stream;
    if constexpr (E != E_BF16)
        if (h_dtype == TG_F16)
            return glu_out<E, O_F16>(a, ws, ws_bytes, s);
    if constexpr (E != E_F16)
        if (h_dtype == TG_BF16)
            return glu_out<E, O_BF16>(a, ws, ws_bytes, s);
    return TG_ERR_NOT_SUPPORTED;
}

// --------------------------------------------------------------- gradients
// dW = A^T . B with A stored K x M and B stored K x N (the reduction runs
// over their rows): the weight gradient, in fp32 or the inputs' type.
template <int E>
tg_status wgrad_typed(const TileArgs& t, int c_dtype, void* ws, int64_t ws_bytes, void* stream)
{
    FxArgs a{};
    static_cast<TileArgs&>(a) = t;
    hipStream_t s = (hipStream_t)stream;
    if (c_dtype == TG_F32)
        return launch_fused<E, O_F32, B_NCONTIG, EPI_STORE, A_MCONTIG>(a, ws, ws_bytes, s);
    return launch_fused<E, OutOf<E>::O, B_NCONTIG, EPI_STORE, A_MCONTIG>(a, ws, ws_bytes, s);
}

// dX = dZ . W with W as it is stored (row-major in this product)
template <int E>
tg_status xgrad_typed(const TileArgs& t, void* ws, int64_t ws_bytes, void* stream)
{
    FxArgs a{};
    static_cast<TileArgs&>(a) = t;
    return launch_fused<E, OutOf<E>::O, B_NCONTIG, EPI_STORE, A_KCONTIG>(a, ws, ws_bytes, (hipStream_t)stream);
}

// The products of a backward pass in one launch.  dX = dZ . W (A K-contiguous)
// and one or two weight gradients (A M-contiguous) do not depend on one
// another; a small pass's products fill the chip badly one by one and each
// pays a launch, a ring fill and an epilogue.  Workgroups 0 .. end[0]-1 run
// product 0, then those of products 1 and 2.  Tiles are 128 x 128 with four
// ring slots: 64 KiB, so two workgroups share a compute unit and fill each
// other's waits.  K splits only into parts of at least kGroupSteps steps (with
// parts of 8 the partial tiles cost more than the split saved).  Whole passes,
// one by one -> grouped: gated 509 x 2728 x 1024 fp16 59 -> 44 us,
// 724 x 2048 x 1024 bf16 64 -> 49, 6000 x 1000 x 600 fp16 127 -> 94; linear
// 777 x 2056 x 1032 fp16 38 -> 31, 2048^3 bf16 52 -> 47, 1000 x 6000 x 1000
// 72 -> 60.
struct GroupArgs {
    TileArgs a[3];
    uint32_t end[3];
};

constexpr int kGroupTile = 128, kGroupNH = 4, kGroupSteps = 16, kGroupPartials = 1000;
static_assert(kGroupPartials / 2 * 4 <= kSplitMaxCounters, "a counter per wave of every split tile");

template <int E, int OW>
__global__ __launch_bounds__(256, 2) void gemm_group(GroupArgs g)
{
    constexpr int T = kGroupTile, RB = NtStaging<E>::RB;
    __shared__ __attribute__((aligned(1024))) uint8_t lds[nt_lds_bytes<T, T, RB, kGroupNH>()];
    const uint32_t bid = blockIdx.x;
    if (bid < g.end[0]) {
        gemm_nt_body<E, OutOf<E>::O, T, T, RB, kGroupNH, 2, 2, B_NCONTIG, EPI_STORE, A_KCONTIG, TileArgs>(g.a[0], bid, g.end[0], lds);
    } else {
        const uint32_t i = bid < g.end[1] ? 1u : 2u, first = g.end[i - 1u];
        gemm_nt_body<E, OW, T, T, RB, kGroupNH, 2, 2, B_NCONTIG, EPI_STORE, A_MCONTIG, TileArgs>(g.a[i], bid - first, g.end[i] - first, lds);
    }
}

// Split counts of the group's products, and the workspace they need: K split
// so that no workgroup runs much longer than the whole group's share, within
// 1000 partial tiles (62.5 MiB).  Split tiles are then 500 at most, and their
// arrival counters, side by side as the plain GEMM's (kCounterStride), 2000 of
// kSplitMaxCounters.
struct GroupPlan {
    int64_t tiles[3], ws_bytes;
    int splits[3];
};

template <int E>
GroupPlan plan_group(const TileArgs* t, int n, bool allow_split)
{
    constexpr int KE = 64;
    GroupPlan p{};
    int64_t work = 0;
    for (int i = 0; i < n; ++i) {
        p.tiles[i] = n_tiles<kGroupTile, kGroupTile>(t[i].M, t[i].N);
        p.splits[i] = 1;
        work += p.tiles[i] * ((t[i].K + KE - 1) / KE);
    }
    // 512 workgroups run at once; at least kGroupSteps steps each
    int64_t share = (work + 511) / 512;
    share = share < kGroupSteps ? kGroupSteps : share;
    int64_t partials = 0;
    for (int i = 0; i < n; ++i) {
        const int64_t kt = (t[i].K + KE - 1) / KE;
        int64_t s = allow_split ? kt / share : 1;
        s = s > 8 ? 8 : s;
        while (s > 1 && partials + p.tiles[i] * s > kGroupPartials)
            --s;
        if (s > 1) {
            p.splits[i] = (int)s;
            partials += p.tiles[i] * s;
        }
    }
    p.ws_bytes = partials == 0 ? 0 : kSplitCounterBytes + partials * kGroupTile * kGroupTile * 4;
    return p;
}

// Whether a group takes these products: all on the NT kernel's grid, at most
// kGroupWork tile steps together (128 for each of the 512 workgroups that run
// at once), none that fills half the chip with tiles of 256 over 32 steps or
// more, and no weight gradient that by itself makes enough whole rounds of
// 256 tiles of 256 (whole_rounds).  Grouped against one by one:
// 1024 x 6144 x 1536 (18 K steps) 67 -> 64 us, 200 x 4096 x 2048 31 -> 26,
// gated 128 x 4096 x 2048 48 -> 41, 1504 x 4000 x 1504 (45 K) 191 -> 158,
// 96 x 9000 x 3600 207 -> 145; what stays out: 4096^3 (131 K) 260 -> 309,
// 7000 x 2048 x 1536 126 -> 135, for which the 256 tile's fewer bytes per
// operation win.
constexpr int64_t kGroupWork = 65536;

// Rounds of whole 256 tiles from which a weight gradient of `steps` K steps
// keeps its pass out of the group: it leaves no unit idle for the others to
// fill.  A single step (up to 64 rows) is all epilogue, which the larger tile
// does better: one round in a linear pass, two in a gated one, whose three
// products have more to share.  Bf16, one by one against grouped:
// 64 x 8192 x 8192 72 against 80 us, 16 x 16384 x 4096 65 / 75, 64 x 8192 x
// 4096 42 / 45, 64 x 8192 x 2048 27 / 30, gated 16 x 8192 x 4096 109 / 117,
// 64 x 4096 x 4096 59 / 63, but (one round) 64 x 4096 x 2048 43 / 38.  Two
// steps: 128 x 8192 x 8192 (four rounds) level, 128 x 16384 x 4096 95 / 82,
// gated 96 x 8192 x 8192 (eight) 241 / 262.  More: 256 x 8192 x 8192 113 / 118,
// 160 x 4096 x 28672 158 / 185, gated 256 x 8192 x 4096 181 / 192, but (two
// rounds) 256 x 8192 x 4096 63 / 60.  A short last round makes up for it in
// the group's favour at every size (64 x 8192 x 9000 127 / 106, 64 x 6000 x
// 6000 66 / 50, gated 64 x 7168 x 5120 135 / 125), and so do widths of a gated
// block off the 64 grid, whose dh and dX run edge loops (64 x 8184 x 4096
// 133 / 126, 8 x 8192 x 4088 131 / 122; linear 64 x 8184 x 8192 75 / 84).
inline int64_t whole_rounds(int64_t steps, int n)
{
    return steps == 1 ? n - 1 : steps == 2 ? 8 : 4;
}

template <int E>
bool group_takes(const TileArgs* t, int n)
{
    int64_t work = 0;
    for (int i = 0; i < n; ++i) {
        if (t[i].M <= 0 || t[i].N <= 0 || t[i].K <= 0)
            return false;
        if (!(i == 0 ? nt_eligible_nrow<E>(t[i]) : nt_eligible_tn<E>(t[i])))
            return false;
        const int64_t tiles = n_tiles<kGroupTile, kGroupTile>(t[i].M, t[i].N), steps = (t[i].K + 63) / 64;
        if (tiles > kGroupWork || steps > kGroupWork)
            return false;
        const int64_t tiles256 = n_tiles<256, 256>(t[i].M, t[i].N);
        if (steps >= 32 && tiles256 >= 128)
            return false;
        if (i > 0 && tiles256 % 256 == 0 && tiles256 >= 256 * whole_rounds(steps, n) &&
            (n == 2 || (t[0].K % 64 == 0 && t[0].N % 64 == 0)))
            return false;
        work += tiles * steps;
    }
    return work <= kGroupWork;
}

// t[0] is dX's product, t[1 .. n-1] are weight gradients of type w_dtype.
template <int E>
tg_status group_typed(const TileArgs* t, int n, int w_dtype, void* ws, int64_t ws_bytes, void* stream, bool* taken)
{
    *taken = group_takes<E>(t, n);
    if (!*taken)
        return TG_OK;
    GroupPlan p = plan_group<E>(t, n, ws != nullptr);
    if (p.ws_bytes > ws_bytes)
        p = plan_group<E>(t, n, false);
    GroupArgs g{};
    int64_t end = 0, counters = 0, partials = 0;
    for (int i = 0; i < 3; ++i) {
        if (i < n) {
            g.a[i] = t[i];
            g.a[i].group_m = 4;
            g.a[i].splits = (uint32_t)p.splits[i];
            if (p.splits[i] > 1) {
                g.a[i].counters = (uint32_t*)ws + counters;
                g.a[i].partials = (float*)((uint8_t*)ws + kSplitCounterBytes) + partials * kGroupTile * kGroupTile;
                counters += p.tiles[i] * 4;
                partials += p.tiles[i] * p.splits[i];
            }
            end += p.tiles[i] * p.splits[i];
        }
        g.end[i] = (uint32_t)end;
    }
    if (end > 0x7FFFFFFF)
        return TG_ERR_NOT_SUPPORTED;
    hipStream_t s = (hipStream_t)stream;
    if (w_dtype == TG_F32)
        hipLaunchKernelGGL((gemm_group<E, O_F32>), dim3((uint32_t)end), dim3(256), 0, s, g);
    else
        hipLaunchKernelGGL((gemm_group<E, OutOf<E>::O>), dim3((uint32_t)end), dim3(256), 0, s, g);
    return launched();
}

template <int E>
int64_t group_ws_bytes(const TileArgs* t, int n)
{
    return group_takes<E>(t, n) ? plan_group<E>(t, n, true).ws_bytes : 0;
}

template <int E>
int64_t wgrad_ws_bytes(int64_t N, int64_t K, int64_t M)
{
    if (M <= 0 || N <= 0 || K <= 0 || !dims_fit(M, N, K) || N % 8 != 0 || K % 8 != 0)
        return 0;
    return plan_nt<E, B_NCONTIG>(N, K, M, true).ws_bytes;
}

// dh = dY . Wd with the gated block's gradient in its epilogue
template <int E>
tg_status glu_dgu_typed(const TileArgs& t, const EpiArgs& e, void* ws, int64_t ws_bytes, void* stream)
{
    FusedArgs a{};
    static_cast<TileArgs&>(a) = t;
    a.e = e;
    return launch_fused<E, OutOf<E>::O, B_NCONTIG, EPI_GLU_BWD, A_KCONTIG>(a, ws, ws_bytes, (hipStream_t)stream);
}

// dz = dy * act'(z), rounded to the inputs' type, and its column sums (of the
// unrounded products, in fp32): 256 columns and a range of rows per
// workgroup of 8 x 32 lanes, 8 consecutive columns per lane.  Bound by its
// reads and its write: 4096 x 4096 bf16 without an activation 12 us, with gelu
// (three times the bytes) 28, 3.6 TB/s.  The row ranges' partial sums meet in the workspace
// and the last arrival adds them in range order, so that results do not
// depend on the order of arrival.
constexpr int kDzSplits = 64;

struct DzArgs {
    int64_t M, N;
    const void* dY;
    int64_t lddy;
    void* dZ;  // null: not written (no activation)
    int64_t lddz;
    float* db;  // null: no sums
    uint32_t* counters;  // one per 256 columns, cstride words apart
    uint32_t cstride;
    float* partials;
    EpiArgs e;  // R, ldr: z, or null (no activation)
};

template <int O>
__global__ __launch_bounds__(256) void dz_colsum(DzArgs p)
{
    __shared__ float red[8][256];
    __shared__ bool last;
    const uint32_t tid = threadIdx.x, lane = tid & 63u, c8 = tid & 31u, rg = tid >> 5;
    const int64_t col = (int64_t)blockIdx.x * 256 + c8 * 8, left = p.N - col;
    const int n = left >= 8 ? 8 : left > 0 ? (int)left : 0;
    const int64_t r0 = p.M * blockIdx.y / gridDim.y, r1 = p.M * (blockIdx.y + 1) / gridDim.y;
    float sum[8];
#pragma unroll
    for (int e = 0; e < 8; ++e)
        sum[e] = 0.0f;
    // Rows in batches of B per thread, all of a batch's loads ahead of its
    // arithmetic (one row at a time waited for memory in every row: 24 us at
    // 4096 x 4096 without an activation, against 11).
    if (n > 0)
        for_act_kind(p.e.kind, [&](auto kind) __attribute__((always_inline)) {
            constexpr int KIND = decltype(kind)::value, B = 8;
            auto rows = [&](auto whole_c) __attribute__((always_inline)) {
                constexpr bool whole = decltype(whole_c)::value;
                for (int64_t rb = r0 + rg; rb < r1; rb += 8 * B) {
                    u32x4 dy[B], z[B];
#pragma unroll
                    for (int b = 0; b < B; ++b) {
                        const int64_t r = rb + 8 * b;
                        dy[b] = z[b] = u32x4{0u, 0u, 0u, 0u};
                        if (r < r1) {
                            dy[b] = load_piece<O>(p.dY, r * p.lddy + col, n, whole);
                            if (p.e.R != nullptr)
                                z[b] = load_piece<O>(p.e.R, r * p.e.ldr + col, n, whole);
                        }
                    }
#pragma unroll
                    for (int b = 0; b < B; ++b) {
                        const int64_t r = rb + 8 * b;
                        float d[8];
#pragma unroll
                        for (int e = 0; e < 8; ++e)
                            d[e] = piece_value<O>(dy[b], e);
                        if (p.e.R != nullptr) {
#pragma unroll
                            for (int e = 0; e < 8; ++e) {
                                float value;
                                d[e] *= act_slope<KIND>(piece_value<O>(z[b], e), p.e, value);
                            }
                        }
                        if (p.dZ != nullptr && r < r1) {
                            const u32x4 q = pack_piece<O>(d);
                            if (whole)
                                *(u32x4*)((uint16_t*)p.dZ + r * p.lddz + col) = q;  // (read again soon: not streamed)
                            else
                                store_piece<O>(p.dZ, r * p.lddz + col, q, n, false);
                        }
#pragma unroll
                        for (int e = 0; e < 8; ++e)
                            sum[e] += d[e];  // (rows past the range add zero)
                    }
                }
            };
            if (n == 8)
                rows(std::true_type{});
            else
                rows(std::false_type{});
        });
    if (p.db == nullptr)
        return;
#pragma unroll
    for (int e = 0; e < 8; ++e)
        red[rg][c8 * 8 + e] = sum[e];
    __syncthreads();
    // thread t adds the row groups of column t
    float s = red[0][tid];
#pragma unroll
    for (int g = 1; g < 8; ++g)
        s += red[g][tid];
    const uint32_t S = gridDim.y;
    const int64_t c = (int64_t)blockIdx.x * 256 + tid;
    if (S > 1u) {
        // The range's sums into its slot; the last workgroup of these columns
        // adds the slots, each wave every fourth one, all of a wave's loads
        // ahead of its adds (one wave adding 64 slots in turn took 15 us).
        __syncthreads();
        red[0][tid] = s;
        __syncthreads();
        float* const slot0 = p.partials + (size_t)blockIdx.x * S * 256;
        if (tid < 64u) {
            splitk_store(slot0 + (size_t)blockIdx.y * 256, 0, 0, lane, *(const f32x4*)&red[0][4 * lane]);
            const bool l = splitk_last(p.counters + blockIdx.x * p.cstride, S, lane);
            if (lane == 0u)
                last = l;
        }
        __syncthreads();
        if (!last)
            return;
        const uint32_t w = tid >> 6;
        f32x4 v[kDzSplits / 4];
#pragma unroll
        for (uint32_t q = 0; q < kDzSplits / 4; ++q) {
            v[q] = f32x4{0.f, 0.f, 0.f, 0.f};
            if (4 * q + w < S)
                v[q] = splitk_load(slot0 + (size_t)(4 * q + w) * 256, 0, 0, lane);
        }
#pragma unroll
        for (uint32_t q = 1; q < kDzSplits / 4; ++q)
            v[0] += v[q];
        *(f32x4*)&red[w][4 * lane] = v[0];
        __syncthreads();
        s = (red[0][tid] + red[1][tid]) + (red[2][tid] + red[3][tid]);
    }
    if (c < p.N)
        p.db[c] = s;
}

// Row ranges of dz_colsum: about four workgroups per compute unit, each of at
// least 32 rows, kDzSplits at most; one where the partial sums have no
// workspace.
inline int64_t dz_splits(int64_t M, int64_t N)
{
    const int64_t blocks = (N + 255) / 256, most = (M + 31) / 32;
    int64_t s = 1024 / blocks;
    if (s > kDzSplits)
        s = kDzSplits;
    if (s > most)
        s = most;
    return s < 1 ? 1 : s;
}

inline int64_t dz_ws_bytes(int64_t M, int64_t N)
{
    if (M <= 0 || N <= 0 || !dims_fit(M, N, 0))
        return 0;
    const int64_t blocks = (N + 255) / 256, s = dz_splits(M, N);
    return s <= 1 || blocks > kSplitMaxCounters ? 0 : kSplitCounterBytes + blocks * s * 1024;
}

template <int E>
tg_status dz_typed(DzArgs p, void* ws, int64_t ws_bytes, void* stream)
{
    const int64_t blocks = (p.N + 255) / 256;
    int64_t splits = dz_splits(p.M, p.N);
    if (p.db != nullptr && splits > 1) {
        if (ws == nullptr || dz_ws_bytes(p.M, p.N) == 0 || dz_ws_bytes(p.M, p.N) > ws_bytes) {
            splits = 1;
        } else {
            // (a line each while they fit: see kCounterStride)
            p.counters = (uint32_t*)ws;
            p.cstride = blocks * 32 <= kSplitMaxCounters ? 32u : 1u;
            p.partials = (float*)((uint8_t*)ws + kSplitCounterBytes);
        }
    }
    hipLaunchKernelGGL((dz_colsum<OutOf<E>::O>), dim3((uint32_t)blocks, (uint32_t)splits), dim3(256), 0,
                       (hipStream_t)stream, p);
    return launched();
}

}  // namespace tg
