// The 256 x 256 tile of the feed-forward operators' products, for 16-bit
// inputs (A: M x K rows, or its transpose, K x M rows; B: N x K rows, or K x N
// rows; any fused epilogue) and int8 (N x K rows: the same bytes, twice the k).  The staging, the ring of LDS half-stages, the
// tile walk and the K split are gemm_nt's; what differs is the matrix
// instruction and the loop around it.
//
// A sustained product is bound by the socket's power: at the cap the clock
// falls from 2.4 to about 1.6 GHz, so that energy per operation is what
// counts.  With operands in registers alone (256 workgroups of 8 waves, random
// bf16 data, 0.3 s), v_mfma_f32_16x16x32 sustains 2055 TFLOP/s and
// v_mfma_f32_32x32x16, which gemm_nt uses, 1830: per operation the former
// moves half the accumulator bytes.  So this kernel takes the former.
//
// A wave computes 128 x 64 of the tile as 8 x 4 blocks of 16 x 16.  One K step
// of 64 is four units of 16 MFMAs: rows 0-63 and 64-127 of the wave's A over
// k 0-31, then both over k 32-63.  A unit's fragments are read from LDS while
// the unit before it multiplies, so the fragments in registers are two halves
// of A (4 each) and two k ranges of B (4 each): 64 registers beside the 128 of
// the accumulator, where double-buffering whole sub-steps would take 96.
// The one barrier per step sits before the last unit.
#pragma once

#include "tg_gemm_nt.hpp"

namespace tg {

// arguments of a plain product on this path (P of EPI_STORE)
struct FxArgs : TileArgs {
    static constexpr EpiArgs e{};
};

// Arguments whose K split leaves its partial tiles in the workspace for a
// kernel of its own to add (with many splits the last arrival's adding, one
// compute unit for a whole tile, would take longer than the product).
// Workgroup (tile, split) writes f32x4 number b 64 + lane of wave w at
// ((tile S + split) 8 + w) 8192 floats: rows 16 (b / 4) + lane % 16 and columns
// 16 (b % 4) + 4 (lane / 16) .. +3 of the wave's 128 x 64.
struct KeepsPartials {};

template <int E, int O, int NH, int AL, int BL, int EPI, class P>
__global__ __launch_bounds__(512) void gemm_fx(P p)
{
    static_assert(ElemInfo<E>::bytes == 2 || (E == E_I8 && AL == A_KCONTIG && BL == B_KCONTIG), "16-bit inputs, or rows of int8");
    constexpr bool GLU = EPI == EPI_GLU;
    constexpr int BM = 256, BN = 256, WM = 2, WN = 4, NW = 8;
    constexpr int BNO = GLU ? BN / 2 : BN;  // output columns per tile
    constexpr int EB = ElemInfo<E>::bytes, CE = 16 / EB, RB = 128, KE = RB / EB, CH = 8;
    constexpr int AI = 4, BI = 4;  // copy instructions per wave and half-stage
    constexpr uint32_t HALF = 256 * RB;
    constexpr int LDS_BYTES = NH * (int)HALF;
    static_assert(NH >= 4 && LDS_BYTES <= 160 * 1024, "LDS");
    constexpr bool NA = AL == A_MCONTIG, NB = BL == B_NCONTIG;
    static_assert(!NA || NB, "a transposed A comes with a row-major B");
    static_assert(!GLU || !NB, "gate and up rows");
    // k-row operands: 512 bytes (32 chunks) per k row, two rows per copy
    // instruction; physical chunk of logical chunk c of row k is c ^ swk(k).
    // Half a wave of a transposing read takes 32 bytes of each of the rows
    // k .. k+3 and k+8 .. k+11: eight chunk pairs, each in its own banks.
    auto swk = [](uint32_t k) __attribute__((always_inline)) -> uint32_t { return 4u * (k % 4u) + 2u * ((k / 8u) % 2u); };
    auto slot_of = [](int64_t h) __attribute__((always_inline)) -> uint32_t { return (uint32_t)h % (uint32_t)NH * HALF; };

    __shared__ __attribute__((aligned(1024))) uint8_t lds[LDS_BYTES];

    const uint32_t tid = threadIdx.x, lane = tid & 63u;
    const uint32_t wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int64_t M = p.M, N = p.N, K = p.K;
    const uint32_t tiles_m = (uint32_t)((M + BM - 1) / BM);
    const uint32_t tiles_n = (uint32_t)((N + BNO - 1) / BNO);
    // whole tiles, K split over S workgroups per tile, or whole tiles first
    // and only the last round's split: as gemm_nt
    uint32_t S = p.splits > 1u ? p.splits : 1u;
    uint32_t tmi, tni, ks = 0u, stile = 0u;
    if (p.dp == 0u) {
        tile_split_coords(blockIdx.x, gridDim.x, tiles_m, tiles_n, S, p.group_m, tmi, tni, ks);
        stile = tmi * tiles_n + tni;
    } else if (blockIdx.x < p.dp) {
        tile_coords(blockIdx.x, p.dp, tiles_m, tiles_n, p.group_m, tmi, tni);
        S = 1u;
    } else {
        const uint32_t R = tiles_m * tiles_n - p.dp;
        const uint32_t idx = xcd_remap(blockIdx.x - p.dp, gridDim.x - p.dp);
        ks = idx / R;
        stile = idx - ks * R;
        group_walk(p.dp + stile, tiles_m, tiles_n, p.group_m, tmi, tni);
    }
    const int64_t m0 = (int64_t)tmi * BM, n0 = (int64_t)tni * BNO;
    const uint32_t ldab = (uint32_t)(p.lda * EB), ldbb = (uint32_t)(p.ldb * EB);
    const int32_t rows_a = (int32_t)(M - m0 < BM ? M - m0 : BM);
    const int32_t rows_b = (int32_t)(N - n0 < BNO ? N - n0 : BNO);
    const int64_t KT = (K + KE - 1) / KE;
    const int64_t kt0 = KT * ks / S, NK = KT * (ks + 1) / S - kt0;

    // ---- copies.  Half-stage h is A of step h / 2 for even h, B for odd h; a
    // wave fills 4 KiB of it in four instructions of 1 KiB.
    // K-contiguous: 8 rows of 128 bytes per instruction, physical chunk
    // lane % 8 of row r holding logical chunk (lane % 8) ^ ((r / 2) % 8).
    // GLU: staged rows in blocks of 32, one per wave, of the gate (even waves)
    // or the up projection, of hidden columns 32 (wave / 2) .. +31 of the tile.
    // k rows: 2 rows of 512 bytes per instruction, 8 per wave.
    const i32x4_t ra = make_rsrc(NA ? p.A + m0 * EB : p.A + m0 * (int64_t)ldab);
    const i32x4_t rb = make_rsrc(NB ? p.B + n0 * EB : p.B + (GLU && (wave & 1u) ? N + n0 : n0) * (int64_t)ldbb);
    const uint32_t arow = wave * 32u, brow = GLU ? (wave >> 1) * 32u : wave * 32u;
    const uint32_t lrow8 = lane / 8u, lrow2 = lane / 32u;
    // this lane's logical chunk in even (q = 0) and odd copy instructions
    auto kchunk = [&](uint32_t q) __attribute__((always_inline)) -> uint32_t { return (lane % 8u) ^ ((4u * q + lrow8 / 2u) % 8u); };
    auto rchunk = [&](uint32_t q) __attribute__((always_inline)) -> uint32_t { return (lane % 32u) ^ swk(wave * 8u + 2u * q + lrow2); };
    auto krow_off = [&](uint32_t q, uint32_t ld, int64_t left) __attribute__((always_inline)) -> uint32_t {
        const uint32_t c = rchunk(q);
        return (lrow2 * ld + c * 16u) | ((int64_t)c * CE < left ? 0u : kOutOfRange);
    };
    const uint32_t va0 = NA ? krow_off(0u, ldab, M - m0) : (arow + lrow8) * ldab + kchunk(0u) * 16u;
    const uint32_t va1 = NA ? krow_off(1u, ldab, M - m0) : (arow + lrow8) * ldab + kchunk(1u) * 16u;
    const uint32_t vb0 = NB ? krow_off(0u, ldbb, N - n0) : (brow + lrow8) * ldbb + kchunk(0u) * 16u;
    const uint32_t vb1 = NB ? krow_off(1u, ldbb, N - n0) : (brow + lrow8) * ldbb + kchunk(1u) * 16u;
    const uint32_t lds0 = __builtin_amdgcn_readfirstlane(lds_addr(lds)) + wave * 4096u;
    // LEAN (kernels with an epilogue of their own): the copies' row checks are in
    // an offset per copy instruction of a K-contiguous half-stage, out of range
    // where the row is past the last one (8 registers; base and distance took 4),
    // and the loop runs without any check until the copies reach the end of K.
    // The other kernels compare their copies' rows with the tile's on edge tiles,
    // in every tile where K ends inside a step, all along the loop: 48 us a round
    // of 256 fp16 tiles at K = 1544, where this takes 45, and 4% less with none
    // at all to check (4096 x 128256 x 4096 3118 -> 3004 us).
    constexpr bool LEAN = EPI == EPI_OWN;
    uint32_t oa[4], ob[4];
    if constexpr (LEAN) {
#pragma unroll
        for (uint32_t q = 0; q < 4; ++q) {
            const uint32_t r = 8u * q + lrow8;
            oa[q] = (arow + r) * ldab + kchunk(q & 1u) * 16u;
            oa[q] |= (int32_t)(arow + r) < rows_a ? 0u : kOutOfRange;
            ob[q] = (brow + r) * ldbb + kchunk(q & 1u) * 16u;
            ob[q] |= (int32_t)(brow + r) < rows_b ? 0u : kOutOfRange;
        }
    }
    // offsets of a half-stage's even and odd copies; a step past the last one
    // and, on edge tiles, chunks past K read out of range (zeros)
    auto half_offs = [&](auto edge, int64_t h, uint32_t& o0, uint32_t& o1) __attribute__((always_inline)) {
        const int64_t kt = h >> 1;
        const bool b = h & 1;
        o0 = b ? vb0 : va0;
        o1 = b ? vb1 : va1;
        if constexpr (decltype(edge)::value) {
            if (!(b ? NB : NA)) {
                const int64_t left = K - (kt0 + kt) * KE;
                const uint32_t most = left >= KE ? (uint32_t)KE : (uint32_t)left;
                o0 |= kchunk(0u) * CE < most ? 0u : kOutOfRange;
                o1 |= kchunk(1u) * CE < most ? 0u : kOutOfRange;
            }
        }
        const uint32_t past = kt < NK ? 0u : kOutOfRange;
        o0 |= past;
        o1 |= past;
    };
    // with both operands as k rows the base moves with the step (as gemm_nt)
    auto half_src = [&](int64_t h) __attribute__((always_inline)) {
        if constexpr (NA) {
            const int64_t k0 = (kt0 + (h >> 1)) * KE;
            return make_rsrc_moving((h & 1) ? p.B + n0 * EB + k0 * (int64_t)ldbb : p.A + m0 * EB + k0 * (int64_t)ldab);
        } else {
            return 0;
        }
    };
    auto copy_half = [&](auto edge, int64_t h, int q, uint32_t o0, uint32_t o1, auto src) __attribute__((always_inline)) {
        const int64_t kt = kt0 + (h >> 1);
        const bool b = h & 1;
        uint32_t v = (q & 1) ? o1 : o0;
        const uint32_t dst = lds0 + slot_of(h) + (uint32_t)q * 1024u;
        if (b ? NB : NA) {
            const uint32_t kr = wave * 8u + 2u * (uint32_t)q;
            if constexpr (decltype(edge)::value)
                v |= kt * KE + kr + lrow2 < K ? 0u : kOutOfRange;
            if constexpr (NA)
                load_lds_1k_at(src, dst, v, kr * (b ? ldbb : ldab));
            else
                load_lds_1k_at(rb, dst, v, ((uint32_t)kt * KE + kr) * ldbb);
            return;
        }
        if constexpr (decltype(edge)::value)
            v |= (int32_t)((b ? brow : arow) + 8u * (uint32_t)q + lrow8) < (b ? rows_b : rows_a) ? 0u : kOutOfRange;
        load_lds_1k_at(b ? rb : ra, dst, v, (uint32_t)kt * RB + 8u * (uint32_t)q * (b ? ldbb : ldab));
    };

    // copy instruction q of half-stage h; `tail`: its step may be past the last
    // one or hold the end of K
    auto copy_lean = [&](auto tail, int64_t h, int q, auto src) __attribute__((always_inline)) {
        const int64_t kt = kt0 + (h >> 1);
        const bool b = h & 1;
        const uint32_t dst = lds0 + slot_of(h) + (uint32_t)q * 1024u;
        const uint32_t past = decltype(tail)::value && (h >> 1) >= NK ? kOutOfRange : 0u;
        if (b ? NB : NA) {
            const uint32_t kr = wave * 8u + 2u * (uint32_t)q;
            uint32_t v = b ? ((q & 1) ? vb1 : vb0) : ((q & 1) ? va1 : va0);
            if constexpr (decltype(tail)::value)
                v |= past | (kt * KE + kr + lrow2 < K ? 0u : kOutOfRange);
            if constexpr (NA)
                load_lds_1k_at(src, dst, v, kr * (b ? ldbb : ldab));
            else
                load_lds_1k_at(rb, dst, v, ((uint32_t)kt * KE + kr) * ldbb);
            return;
        }
        uint32_t v = b ? ob[q] : oa[q];
        if constexpr (decltype(tail)::value)
            v |= past | ((int64_t)(kchunk(q & 1) * CE) < K - kt * KE ? 0u : kOutOfRange);
        load_lds_1k_at(b ? rb : ra, dst, v, (uint32_t)kt * RB);
    };

    auto copy = [&](auto edge, int64_t h, int q, uint32_t o0, uint32_t o1, auto src) __attribute__((always_inline)) {
        if constexpr (LEAN)
            copy_lean(edge, h, q, src);
        else
            copy_half(edge, h, q, o0, o1, src);
    };

    // ---- fragments of 16 rows and 32 k: lane l holds row l % 16, k range
    // 8 (l / 16) .. +7 (the k order inside an instruction does not matter as
    // long as both operands agree)
    const uint32_t wm = wave / WN, wn = wave % WN;
    const uint32_t l16 = lane % 16u, lgrp = lane / 16u;
    u32x4 fa[2][4], fb[2][4];
    // 16 rows from row `row` of a K-contiguous stage, k sub-step s
    auto frag_k = [&](const uint8_t* st, uint32_t row, int s) __attribute__((always_inline)) -> u32x4 {
        return lds128(st, (row + l16) * RB + (((4u * (uint32_t)s + lgrp) ^ ((l16 / 2u) % 8u)) << 4));
    };
    // 16 columns from `col` of a k-row stage: two transposing reads of 4 k
    // rows; in each 16-lane group source lane 4e + a addresses row e, columns
    // 4a .. 4a+3, and lane 4a + j receives column 4a + j of the four rows
    auto frag_r = [&](const uint8_t* st, uint32_t col, int s) __attribute__((always_inline)) -> u32x4 {
        const uint32_t c = col + 4u * (l16 % 4u);
        uint32_t w[4];
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            const uint32_t k = 32u * (uint32_t)s + 8u * lgrp + 4u * (uint32_t)r + l16 / 4u;
            const uint32_t off = k * 512u + (((c / CE) ^ swk(k)) << 4) + (c % CE) * EB;
            const auto v = __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) short4_t*)(lds_u8_t)(st + off));
            w[2 * r] = (uint32_t)(uint16_t)v[0] | ((uint32_t)(uint16_t)v[1] << 16);
            w[2 * r + 1] = (uint32_t)(uint16_t)v[2] | ((uint32_t)(uint16_t)v[3] << 16);
        }
        return u32x4{w[0], w[1], w[2], w[3]};
    };
    // rows h*64 + 16i of the wave's A, and columns 16j of its B, of step kt
    auto read_a = [&](int64_t kt, int s, int h, int i) __attribute__((always_inline)) {
        const uint8_t* st = lds + slot_of(2 * kt);
        const uint32_t row = wm * 128u + (uint32_t)(h * 64 + i * 16);
        fa[h][i] = NA ? frag_r(st, row, s) : frag_k(st, row, s);
    };
    auto read_b = [&](int64_t kt, int s, int j) __attribute__((always_inline)) {
        const uint8_t* st = lds + slot_of(2 * kt + 1);
        const uint32_t row = wn * 64u + (uint32_t)j * 16u;
        fb[s][j] = NB ? frag_r(st, row, s) : frag_k(st, row, s);
    };

    // acc[i][j], operands swapped: lane l holds row 16i + l % 16, columns
    // 16j + 4 (l / 16) .. +3 of the wave's tile
    f32x4 acc[8][4];
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j)
            acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};

    // A unit: rows h of A against k sub-step s, with NR fragment reads over
    // its first half and NQ copies over all of it between the MFMAs.  In snake
    // order (each MFMA shares an operand with the one before it): with
    // operands in registers alone 2088 TFLOP/s against 2045 row by row and
    // 1990 with none shared.
    auto unit = [&](int h, int s, auto nr, auto rd, auto nq, auto cp) __attribute__((always_inline)) {
        constexpr int NR = decltype(nr)::value, NQ = decltype(nq)::value;
#pragma unroll
        for (int t = 0; t < 16; ++t) {
            const int i = t / 4, j = (i & 1) ? 3 - t % 4 : t % 4;
            acc[h * 4 + i][j] = Mfma16<E>::run(fb[s][j], fa[h][i], acc[h * 4 + i][j]);
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int r = 0; r < NR; ++r)
                if (r * 8 / NR == t)
                    rd(r);
            if constexpr (NQ > 0) {
#pragma unroll
                for (int q = 0; q < NQ; ++q)
                    if (q * 16 / NQ == t)
                        cp(q);
            }
            __builtin_amdgcn_sched_barrier(0);
        }
    };
    constexpr std::integral_constant<int, 4> n4c{};
    constexpr std::integral_constant<int, 6> n6c{};
    constexpr std::integral_constant<int, 8> n8c{};

    // One K step.  Entering, fa[0] and fb[0] hold its first unit.  The last
    // barrier freed two half-stages: one (2(kt-1)+NH) was copied in the unit
    // behind it, the other, 2kt+NH-1, is copied in this step's first units.
    // Five slots: that one holds A rows of step kt+2, needed in two barriers'
    // time, so its four copies are spread over the three units before the
    // barrier; the B rows behind it get a whole step to land.  Four slots: it
    // holds B rows of step kt+1, needed at this step's barrier, and goes out
    // at once.  8192 x 4096 x 10240 with a residual 578 -> 565 us with five,
    // gated 4096 x 10240 x 4096 532 -> 516 (interleaved, snake order included).
    // (LEAN: `edge` is copy_lean's `tail`)
    auto step = [&](auto edge, int64_t kt) __attribute__((always_inline)) {
        uint32_t p0 = 0u, p1 = 0u, r0 = 0u, r1 = 0u;
        if constexpr (!LEAN) {
            half_offs(edge, 2 * kt + NH - 1, p0, p1);
            half_offs(edge, 2 * kt + NH, r0, r1);
        }
        const auto psrc = half_src(2 * kt + NH - 1), rsrc = half_src(2 * kt + NH);
        constexpr bool SPREAD = NH % 2 == 1;
        auto early = [&](int q0) __attribute__((always_inline)) {
            return [&, q0](int q) __attribute__((always_inline)) { copy(edge, 2 * kt + NH - 1, q0 + q, p0, p1, psrc); };
        };
        unit(0, 0, n6c,
             [&](int r) __attribute__((always_inline)) {
                 if (r < 4)
                     read_a(kt, 0, 1, r);
                 else
                     read_b(kt, 1, r - 4);
             },
             std::integral_constant<int, SPREAD ? 1 : 4>{}, early(0));
        unit(1, 0, n6c,
             [&](int r) __attribute__((always_inline)) {
                 if (r == 0)
                     read_a(kt, 1, 0, 0);
                 else if (r < 3)
                     read_b(kt, 1, r + 1);
                 else
                     read_a(kt, 1, 0, r - 2);
             },
             std::integral_constant<int, SPREAD ? 1 : 0>{}, early(1));
        unit(0, 1, n4c, [&](int r) __attribute__((always_inline)) { read_a(kt, 1, 1, r); },
             std::integral_constant<int, SPREAD ? 2 : 0>{}, early(2));
        __builtin_amdgcn_sched_barrier(0);
        // copies of step kt+1 landed: those of half-stages 2kt+4 .. 2kt+NH-1 may be in flight
        wait_copies<4 * (NH - 4)>();
        __syncthreads();
        __builtin_amdgcn_sched_barrier(0);
        // (after the last step the reads are stale and unused)
        unit(1, 1, n8c,
             [&](int r) __attribute__((always_inline)) {
                 if (r == 0)
                     read_a(kt + 1, 0, 0, 0);
                 else if (r < 5)
                     read_b(kt + 1, 0, r - 1);
                 else
                     read_a(kt + 1, 0, 0, r - 4);
             },
             n4c, [&](int q) __attribute__((always_inline)) { copy(edge, 2 * kt + NH, q, r0, r1, rsrc); });
    };
    auto run_lean = [&]() __attribute__((always_inline)) {
#pragma unroll
        for (int h = 0; h < NH - 1; ++h) {
            const auto src = half_src(h);
#pragma unroll
            for (int q = 0; q < 4; ++q)
                copy_lean(std::true_type{}, h, q, src);
        }
        wait_copies<4 * (NH - 3)>();  // step 0 landed
        __syncthreads();
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            read_a(0, 0, 0, r);
            read_b(0, 0, r);
        }
        // step kt copies for steps up to kt + 2
        const int64_t inside = K / KE - kt0, whole = (inside < NK ? inside : NK) - 2;
        int64_t kt = 0;
        for (; kt < whole; ++kt)
            step(std::false_type{}, kt);
        for (; kt < NK; ++kt)
            step(std::true_type{}, kt);
        wait_copies<0>();
    };
    auto run = [&](auto edge) __attribute__((always_inline)) {
#pragma unroll
        for (int h = 0; h < NH - 1; ++h) {
            uint32_t o0, o1;
            half_offs(edge, h, o0, o1);
            const auto src = half_src(h);
#pragma unroll
            for (int q = 0; q < 4; ++q)
                copy_half(edge, h, q, o0, o1, src);
        }
        wait_copies<4 * (NH - 3)>();  // step 0 landed
        __syncthreads();
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            read_a(0, 0, 0, r);
            read_b(0, 0, r);
        }
        for (int64_t kt = 0; kt < NK; ++kt)
            step(edge, kt);
        wait_copies<0>();  // copies past the last step (zeros) must land before LDS is reused
    };
    if (NK > 0) {
        if constexpr (LEAN)
            run_lean();
        else if (rows_a == BM && rows_b == BNO && K % KE == 0)  // full tiles, no K tail
            run(std::false_type{});
        else
            run(std::true_type{});
    }
    mfma_drain();
    if constexpr (std::is_base_of<KeepsPartials, P>::value) {
        float* const share = p.partials + (((size_t)stile * S + ks) * NW + wave) * 8192;
#pragma unroll
        for (int b = 0; b < 32; ++b)
            if (m0 + wm * 128 + b / 4 * 16 < M)  // (rows past the last are not read)
                *(f32x4*)(share + (b * 64 + lane) * 4) = acc[b / 4][b % 4];
        return;
    }
    __syncthreads();  // the epilogue reuses the stage buffers

    // ---- K split: as gemm_nt's for tiles of many blocks (the own share is
    // read back with the others, eight quads at a time)
    if (S > 1u) {
        constexpr int SHARE = 32 * 256;  // floats of a wave's share: 32 quads per lane
        float* const share0 = p.partials + ((size_t)stile * S * NW + wave) * SHARE;
        auto slot = [&](uint32_t q) __attribute__((always_inline)) { return share0 + (size_t)q * NW * SHARE; };
#pragma unroll
        for (int b = 0; b < 32; ++b)
            splitk_store(slot(ks), b / 4, b % 4, lane, acc[b / 4][b % 4]);
        if (!splitk_last(p.counters + ((size_t)stile * NW + wave) * kCounterStride<P, TileArgs>, S, lane))
            return;
        for (uint32_t q = ks == 0u ? 1u : 0u; q < S; ++q) {
            const float* src = slot(q);
#pragma unroll
            for (int b0 = 0; b0 < 32; b0 += 8) {
                f32x4 v[8];
#pragma unroll
                for (int b = 0; b < 8; ++b)
                    v[b] = splitk_load(src, (b0 + b) / 4, b % 4, lane);
#pragma unroll
                for (int b = 0; b < 8; ++b)
                    acc[(b0 + b) / 4][b % 4] = q == 0u ? v[b] : acc_add<E>(acc[(b0 + b) / 4][b % 4], v[b]);
            }
        }
    }

    // ---- epilogue
    const int64_t row0 = m0 + wm * 128, col0 = n0 + wn * (BNO / WN);
    auto quad = [&](int i, int q) __attribute__((always_inline)) -> f32x4 { return acc_value<E>(acc[i][q]); };
    uint8_t* const ep = lds + wave * (LDS_BYTES / NW);
    if constexpr (EPI == EPI_OWN)
        p.template finish<16, 128, 64, LDS_BYTES / NW>(ep, lane, row0, col0, quad);
    else if constexpr (GLU)
        glu_epilogue<O, 16, 128, 64>(ep, lane, row0, col0, M, N, p.C, p.ldc, p.e, quad);
    else if constexpr (EPI == EPI_STORE && O != O_F32)
        store_rows16<O, 16, 128, 64>(ep, lane, row0, col0, M, N, p.C, p.ldc, 0, true, quad);
    else
        rows_epilogue<O, EPI, 16, 128, 64, LDS_BYTES / NW>(ep, lane, row0, col0, M, N, p.C, p.ldc, p.e, quad);
}

}  // namespace tg
