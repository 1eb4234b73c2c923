// tg_adamw: one AdamW step over many tensors (contract in include/tg_train.h).
//
//   m' = b1 m + (1 - b1) g;   v' = b2 v + (1 - b2) g^2
//   w' = w (1 - lr wd) - lr / (1 - b1^t) m' / (sqrt(v' / (1 - b2^t)) + eps)
//
// Bound by memory: every value is read once and written once (fp32 28 bytes a
// value, bf16 weights and gradients with 8-bit states 10).  Tensors of one
// combination of types share launches of up to kAdamTensors, whose
// descriptors travel in the kernel arguments; a workgroup takes a chunk.  A
// lane takes V consecutive values, 4 or 8, so that 64 or 32 lanes hold a block
// of 8-bit states and its largest value is a reduction between lanes.
//
// 300 M bf16 weights with fp32 masters and states 1410 us, 6.0 TB/s; 400 M
// with 8-bit states 670 us, 6.0 TB/s (a large copy moves 4.7); 9 fp32 tensors
// of 60 K values 6.6 us, three times a launch that reads one row.  Buffers off
// 16 bytes go a byte at a time: the 300 M, one element off, 6.1 ms.  What got
// it there: 2048 workgroups that walk the chunks with 32 bytes of each fp32
// buffer per lane 2456 and 978 us; one run of whole lines per instruction 1632
// and 865; a workgroup for each chunk 1500 and 685; chunks of one unit 1400
// with fp32 buffers (two units of 8 values 685, one 692).  Without the non-
// temporal hint on large loads +3 and +5%, on the stores +4 and +7%.
#include <math.h>

#include "tg_abi.hpp"
#include "tg_epilogue.hpp"
#include "tg_train.h"

namespace tg {

constexpr int kAdamTensors = 48;       // descriptors per launch (under 4 KiB of kernel arguments)
constexpr int64_t kAdamGrid = 1 << 23;  // workgroups of a launch at most
static_assert(kAdamGrid * 256 <= 0x7FFFFFFF + (int64_t)1, "a launch has less than 2^32 lanes");
constexpr int kAdamBlock = 256;        // elements per scale of 8-bit states
constexpr float kE4m3Max = 448.0f, kE4m3Step = 0.001953125f;  // largest and smallest positive value
constexpr float kAdamTiny = 7.888609052210118e-31f;           // 2^-100

// Values per lane and unit, units per chunk, of a combination of types: see adamw_step
constexpr int adam_values(bool narrow) { return narrow ? 8 : 4; }
constexpr int adam_units(bool narrow) { return narrow ? 2 : 1; }
constexpr int64_t adam_chunk(bool narrow) { return 256 * adam_values(narrow) * adam_units(narrow); }

struct AdamHyper {
    float b1, omb1, b2, omb2;  // omb: 1 - b
    float decay, step_size, root, eps;
    double lr, wd, beta1, beta2;  // where step or lr are in device memory
    const int64_t* step_dev;
    const float* lr_dev;
    int64_t step;
    const float* norm;
    float max_norm;
};

struct AdamArgs {
    void* p[kAdamTensors];
    float* w[kAdamTensors];
    const void* g[kAdamTensors];
    void* m[kAdamTensors];
    void* v[kAdamTensors];
    float* sm[kAdamTensors];
    float* sv[kAdamTensors];
    int64_t n[kAdamTensors];
    uint32_t first[kAdamTensors + 1];  // first chunk of each tensor; [count]: all
    uint8_t aligned[kAdamTensors];     // every pointer on 16 bytes
    int32_t count;
    AdamHyper h;
};
static_assert(sizeof(AdamArgs) <= 4096, "kernel arguments");

// beta^t by squaring
__host__ __device__ inline double beta_power(double beta, int64_t t)
{
    double r = 1.0;
    for (; t > 0; t >>= 1) {
        if (t & 1)
            r *= beta;
        beta *= beta;
    }
    return r;
}

__host__ __device__ inline void adam_constants(AdamHyper& h, int64_t step, double lr)
{
    h.decay = (float)(1.0 - lr * h.wd);
    h.step_size = (float)(lr / (1.0 - beta_power(h.beta1, step)));
    h.root = (float)(1.0 / __builtin_sqrt(1.0 - beta_power(h.beta2, step)));
}

// W words of a lane from byte `at` on, `left` bytes of them there; whole: all
// are, on a boundary of their size.  STREAM: with the non-temporal hint.
template <int W, bool STREAM>
__device__ __forceinline__ void load_words(const void* base, int64_t at, int left, bool whole, uint32_t* q)
{
    typedef uint32_t vec __attribute__((ext_vector_type(W)));
    const uint8_t* src = (const uint8_t*)base + at;
    if (whole) {
        vec v;
        if constexpr (STREAM)
            v = __builtin_nontemporal_load((const vec*)src);
        else
            v = *(const vec*)src;
#pragma unroll
        for (int i = 0; i < W; ++i)
            q[i] = v[i];
        return;
    }
#pragma unroll
    for (int i = 0; i < W; ++i)
        q[i] = 0u;
#pragma unroll
    for (int i = 0; i < 4 * W; ++i)
        if (i < left)
            q[i / 4] |= (uint32_t)src[i] << (8 * (i % 4));
}

template <int W>
__device__ __forceinline__ void store_words(void* base, int64_t at, int left, bool whole, const uint32_t* q)
{
    typedef uint32_t vec __attribute__((ext_vector_type(W)));
    uint8_t* dst = (uint8_t*)base + at;
    if (whole) {
        vec v;
#pragma unroll
        for (int i = 0; i < W; ++i)
            v[i] = q[i];
        store_nt((vec*)dst, v);
        return;
    }
#pragma unroll
    for (int i = 0; i < 4 * W; ++i)
        if (i < left)
            dst[i] = (uint8_t)(q[i / 4] >> (8 * (i % 4)));
}

template <int O> struct AdamBytes { static constexpr int N = O == O_F32 ? 4 : 2; };

// value i of words of type O, and V values as such words
template <int O>
__device__ __forceinline__ float word_value(const uint32_t* q, int i)
{
    if constexpr (O == O_F32)
        return bit_cast<float>(q[i]);
    else
        return piece_value<O>(u32x4{q[i >> 1], 0u, 0u, 0u}, i & 1);
}

template <int O, int V>
__device__ __forceinline__ void to_words(const float* v, uint32_t* q)
{
#pragma unroll
    for (int i = 0; i < V * AdamBytes<O>::N / 4; ++i) {
        if constexpr (O == O_F32)
            q[i] = bit_cast<uint32_t>(v[i]);
        else
            q[i] = pack2<O>(v[2 * i], v[2 * i + 1]);
    }
}

template <int V>
__device__ __forceinline__ void from_e4m3(const uint32_t* q, float scale, float* v)
{
#pragma unroll
    for (int i = 0; i < V / 4; ++i) {
        const auto lo = __builtin_amdgcn_cvt_pk_f32_fp8((int)q[i], false);
        const auto hi = __builtin_amdgcn_cvt_pk_f32_fp8((int)q[i], true);
        v[4 * i] = lo[0] * scale;
        v[4 * i + 1] = lo[1] * scale;
        v[4 * i + 2] = hi[0] * scale;
        v[4 * i + 3] = hi[1] * scale;
    }
}

// largest of the 32 or 64 lanes that hold a block, in each of them
template <int LANES>
__device__ __forceinline__ float lanes_max(float v)
{
    // within a row of 16 lanes: rotated by 8, 4, 2, 1
#define TG_ROW_MAX(ctrl) \
    v = __builtin_fmaxf(v, bit_cast<float>(__builtin_amdgcn_mov_dpp(bit_cast<int>(v), ctrl, 0xF, 0xF, true)))
    TG_ROW_MAX(0x128);
    TG_ROW_MAX(0x124);
    TG_ROW_MAX(0x122);
    TG_ROW_MAX(0x121);
#undef TG_ROW_MAX
    // then with the row beside it, and the other half of the wave
    const auto r = __builtin_amdgcn_permlane16_swap(bit_cast<uint32_t>(v), bit_cast<uint32_t>(v), false, false);
    v = __builtin_fmaxf(bit_cast<float>((uint32_t)r[0]), bit_cast<float>((uint32_t)r[1]));
    if constexpr (LANES == 64) {
        const auto h = __builtin_amdgcn_permlane32_swap(bit_cast<uint32_t>(v), bit_cast<uint32_t>(v), false, false);
        v = __builtin_fmaxf(bit_cast<float>((uint32_t)h[0]), bit_cast<float>((uint32_t)h[1]));
    }
    return v;
}

// A block's values as e4m3 and a scale; LIFT: positive ones stay positive.  The
// scale is that of the finite values: an infinite one would leave the others as
// 0 of an infinite scale, NaN to the next step.  It becomes NaN, which e4m3 has
// and which stays its own.
template <int V, bool LIFT>
__device__ __forceinline__ void to_e4m3(float* v, uint32_t* q, float& scale)
{
    auto largest = [&]() __attribute__((always_inline)) -> float {
        float top = 0.0f;
#pragma unroll
        for (int i = 0; i < V; ++i)
            top = __builtin_fmaxf(top, LIFT ? v[i] : __builtin_fabsf(v[i]));
        return lanes_max<kAdamBlock / V>(top);
    };
    float top = largest();
    if (__builtin_amdgcn_ballot_w64(top == INFINITY) != 0) {  // (the whole wave: its lanes exchange their largest)
#pragma unroll
        for (int i = 0; i < V; ++i)
            v[i] = __builtin_fabsf(v[i]) == INFINITY ? NAN : v[i];
        top = largest();
    }
    top = top < kAdamTiny ? 0.0f : top;
    const float inv = top > 0.0f ? kE4m3Max / top : 0.0f;
    scale = top * (1.0f / kE4m3Max);
#pragma unroll
    for (int i = 0; i < V / 4; ++i) {
        float s[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            s[e] = v[4 * i + e] * inv;
            if (LIFT)
                s[e] = s[e] > 0.0f ? __builtin_fmaxf(s[e], kE4m3Step) : s[e];
        }
        int w = __builtin_amdgcn_cvt_pk_fp8_f32(s[0], s[1], 0, false);
        w = __builtin_amdgcn_cvt_pk_fp8_f32(s[2], s[3], w, true);
        q[i] = (uint32_t)w;
    }
}

__device__ __forceinline__ int adam_tensor(const AdamArgs& p, uint32_t c)
{
    int lo = 0, hi = p.count;  // first[lo] <= c < first[hi]
    while (hi - lo > 1) {
        const int mid = (lo + hi) / 2;
        if (p.first[mid] <= c)
            lo = mid;
        else
            hi = mid;
    }
    return lo;
}

// P: type of the weights, G: of the gradients; MASTER: fp32 weights beside
// them; EIGHT: 8-bit states.  A unit is V consecutive values of a lane, V such
// that the widest of the buffers takes 16 bytes (and the others less): every
// load and store of a wave covers one run of whole lines.
template <int P, int G, bool MASTER, bool EIGHT, bool STREAM>
__global__ __launch_bounds__(256) void adamw_step(AdamArgs a)
{
    static_assert(!MASTER || P != O_F32, "masters of 16-bit weights");
    constexpr int WT = MASTER ? (int)O_F32 : P;
    constexpr bool NARROW = WT != O_F32 && G != O_F32 && EIGHT;  // nothing of 32 bits
    constexpr int V = adam_values(NARROW), UNITS = adam_units(NARROW);
    constexpr int PW = V * AdamBytes<P>::N / 4, GW = V * AdamBytes<G>::N / 4, WW = V * AdamBytes<WT>::N / 4, SW = EIGHT ? V / 4 : V;
    AdamHyper h = a.h;
    float coef = 1.0f;
    if (h.norm != nullptr) {
        const float norm = *h.norm, d = norm + 1e-6f;
        if (!(__builtin_fabsf(norm) < INFINITY))
            return;
        coef = d <= h.max_norm ? 1.0f : h.max_norm / d;
    }
    if (h.step_dev != nullptr || h.lr_dev != nullptr)
        adam_constants(h, h.step_dev != nullptr ? *h.step_dev : h.step, h.lr_dev != nullptr ? (double)*h.lr_dev : h.lr);
    const uint32_t chunks = a.first[a.count], tid = threadIdx.x;
    for (uint32_t c = blockIdx.x; c < chunks; c += gridDim.x) {
        const int t = adam_tensor(a, c);
        const int64_t c0 = (int64_t)(c - a.first[t]) * adam_chunk(NARROW) + tid * V, n = a.n[t];
        const bool aligned = a.aligned[t] != 0;
        uint32_t gq[UNITS][GW], wq[UNITS][WW], mq[UNITS][SW], vq[UNITS][SW];
        float sm[UNITS], sv[UNITS];
        auto values_left = [&](int u) __attribute__((always_inline)) -> int {
            const int64_t rest = n - (c0 + (int64_t)u * 256 * V);
            return rest >= V ? V : rest > 0 ? (int)rest : 0;
        };
#pragma unroll
        for (int u = 0; u < UNITS; ++u) {
            const int64_t e = c0 + (int64_t)u * 256 * V;
            const int left = values_left(u);
            const bool whole = aligned && left == V;
            if (left > 0) {
                constexpr int S = EIGHT ? 1 : 4;
                load_words<GW, STREAM>(a.g[t], e * AdamBytes<G>::N, left * AdamBytes<G>::N, whole, gq[u]);
                load_words<WW, STREAM>(MASTER ? (const void*)a.w[t] : a.p[t], e * AdamBytes<WT>::N, left * AdamBytes<WT>::N, whole, wq[u]);
                load_words<SW, STREAM>(a.m[t], e * S, left * S, whole, mq[u]);
                load_words<SW, STREAM>(a.v[t], e * S, left * S, whole, vq[u]);
                if constexpr (EIGHT) {
                    sm[u] = a.sm[t][e / kAdamBlock];
                    sv[u] = a.sv[t][e / kAdamBlock];
                }
            }
        }
#pragma unroll
        for (int u = 0; u < UNITS; ++u) {
            const int64_t e = c0 + (int64_t)u * 256 * V;
            const int left = values_left(u);
            const bool whole = aligned && left == V;
            float w[V], m[V], v[V], r[V];
#pragma unroll
            for (int i = 0; i < V; ++i)
                m[i] = r[i] = 0.0f;
            if (left > 0) {
                if constexpr (EIGHT) {
                    from_e4m3<V>(mq[u], sm[u], m);
                    from_e4m3<V>(vq[u], sv[u], v);
                }
                float least = INFINITY;
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    const float g = word_value<G>(gq[u], i) * coef;
                    const float m0 = EIGHT ? m[i] : bit_cast<float>(mq[u][EIGHT ? 0 : i]);
                    const float v0 = EIGHT ? v[i] * v[i] : bit_cast<float>(vq[u][EIGHT ? 0 : i]);
                    m[i] = m0 * h.b1 + g * h.omb1;
                    v[i] = v0 * h.b2 + g * h.omb2 * g;
                    r[i] = __builtin_amdgcn_sqrtf(v[i]);
                    least = __builtin_fminf(least, v[i]);
                }
                // the instruction takes a subnormal number, whose root is 2^-75 to 2^-63, for 0
                // (a selection for each value made the step with 8-bit states 1% slower)
                if (__builtin_amdgcn_ballot_w64(least < 0x1p-126f) != 0) {
#pragma unroll
                    for (int i = 0; i < V; ++i)
                        r[i] = v[i] < 0x1p-126f ? __builtin_amdgcn_sqrtf(v[i] * 0x1p64f) * 0x1p-32f : r[i];
                }
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    const float w0 = word_value<WT>(wq[u], i);
                    w[i] = w0 * h.decay - m[i] * __builtin_amdgcn_rcpf(r[i] * h.root + h.eps) * h.step_size;
                }
                uint32_t q[V];
                to_words<P, V>(w, q);
                store_words<PW>(a.p[t], e * AdamBytes<P>::N, left * AdamBytes<P>::N, whole, q);
                if constexpr (MASTER) {
                    to_words<O_F32, V>(w, q);
                    store_words<V>(a.w[t], e * 4, left * 4, whole, q);
                }
            }
            if constexpr (EIGHT) {
                // (values past the tensor's end stay out of the block's largest; every lane of the block takes part)
#pragma unroll
                for (int i = 0; i < V; ++i)
                    if (i >= left)
                        m[i] = r[i] = 0.0f;
                uint32_t qm[V / 4], qv[V / 4];
                float nm, nv;
                to_e4m3<V, false>(m, qm, nm);
                to_e4m3<V, true>(r, qv, nv);
                if (left > 0) {
                    store_words<V / 4>(a.m[t], e, left, whole, qm);
                    store_words<V / 4>(a.v[t], e, left, whole, qv);
                    if (e % kAdamBlock == 0) {
                        a.sm[t][e / kAdamBlock] = nm;
                        a.sv[t][e / kAdamBlock] = nv;
                    }
                }
            } else if (left > 0) {
                uint32_t q[V];
                to_words<O_F32, V>(m, q);
                store_words<V>(a.m[t], e * 4, left * 4, whole, q);
                to_words<O_F32, V>(v, q);
                store_words<V>(a.v[t], e * 4, left * 4, whole, q);
            }
        }
    }
}

template <int P, int G, bool MASTER, bool EIGHT>
static void adam_launch(const AdamArgs& a, uint32_t grid, bool stream, hipStream_t s)
{
    if (stream)
        hipLaunchKernelGGL((adamw_step<P, G, MASTER, EIGHT, true>), dim3(grid), dim3(256), 0, s, a);
    else
        hipLaunchKernelGGL((adamw_step<P, G, MASTER, EIGHT, false>), dim3(grid), dim3(256), 0, s, a);
}

template <int P, int G>
static void adam_launch_pg(bool master, bool eight, const AdamArgs& a, uint32_t grid, bool stream, hipStream_t s)
{
    if (master && P != O_F32)
        eight ? adam_launch<P, G, P != O_F32, true>(a, grid, stream, s) : adam_launch<P, G, P != O_F32, false>(a, grid, stream, s);
    else
        eight ? adam_launch<P, G, false, true>(a, grid, stream, s) : adam_launch<P, G, false, false>(a, grid, stream, s);
}

template <int P>
static void adam_launch_p(int g, bool master, bool eight, const AdamArgs& a, uint32_t grid, bool stream, hipStream_t s)
{
    switch (g) {
    case TG_F32: adam_launch_pg<P, O_F32>(master, eight, a, grid, stream, s); break;
    case TG_F16: adam_launch_pg<P, O_F16>(master, eight, a, grid, stream, s); break;
    default: adam_launch_pg<P, O_BF16>(master, eight, a, grid, stream, s); break;
    }
}

static bool dtype_ok(int t) { return t == TG_F32 || t == TG_F16 || t == TG_BF16; }
static uintptr_t elem_mask(int t) { return t == TG_F32 ? 3u : 1u; }
}  // namespace tg

using namespace tg;

extern "C" tg_status tg_adamw(int64_t count, const tg_adamw_tensor* tensors, int64_t step, double lr, double beta1, double beta2,
                              double eps, double weight_decay, const float* norm, float max_norm, const int64_t* step_dev,
                              const float* lr_dev, void* stream)
{
    if (count < 0 || (count > 0 && tensors == nullptr) || (step_dev == nullptr && step < 1) ||
        (lr_dev == nullptr && !__builtin_isfinite(lr)) || !(beta1 >= 0.0 && beta1 < 1.0) || !(beta2 >= 0.0 && beta2 < 1.0) ||
        !(eps >= 0.0) || __builtin_isinf(eps) || !__builtin_isfinite(weight_decay) || !(max_norm >= 0.0f))
        return TG_ERR_INVALID_VALUE;
    if (((uintptr_t)norm & 3u) || ((uintptr_t)lr_dev & 3u) || ((uintptr_t)step_dev & 7u))
        return TG_ERR_MISALIGNED;
    int64_t bytes = 0;
    bool eight = false, fp32 = false;
    for (int64_t i = 0; i < count; ++i) {
        const tg_adamw_tensor& t = tensors[i];
        if (t.n < 0 || !dtype_ok(t.p_dtype) || !dtype_ok(t.g_dtype))
            return TG_ERR_INVALID_VALUE;
        if (t.n == 0)
            continue;
        if (t.param == nullptr || t.grad == nullptr || t.exp_avg == nullptr || t.exp_avg_sq == nullptr ||
            (t.exp_avg_scale == nullptr) != (t.exp_avg_sq_scale == nullptr) || (t.master != nullptr && t.p_dtype == TG_F32))
            return TG_ERR_INVALID_VALUE;
        const bool e = t.exp_avg_scale != nullptr;
        (e ? eight : fp32) = true;
        const uintptr_t states = e ? 0u : 3u;
        if (((uintptr_t)t.param & elem_mask(t.p_dtype)) || ((uintptr_t)t.grad & elem_mask(t.g_dtype)) || ((uintptr_t)t.master & 3u) ||
            ((uintptr_t)t.exp_avg & states) || ((uintptr_t)t.exp_avg_sq & states) || ((uintptr_t)t.exp_avg_scale & 3u) ||
            ((uintptr_t)t.exp_avg_sq_scale & 3u))
            return TG_ERR_MISALIGNED;
        if (t.n > (int64_t)1 << 40)
            return TG_ERR_NOT_SUPPORTED;
        bytes += t.n * ((t.p_dtype == TG_F32 ? 4 : 2) + (t.g_dtype == TG_F32 ? 4 : 2) + (t.master != nullptr ? 4 : 0) + (e ? 2 : 8));
    }
    if (eight && fp32)
        return TG_ERR_INVALID_VALUE;

    AdamArgs a;
    AdamHyper& h = a.h;
    h.b1 = (float)beta1;
    h.omb1 = (float)(1.0 - beta1);
    h.b2 = (float)beta2;
    h.omb2 = (float)(1.0 - beta2);
    // (the reciprocal instruction takes a subnormal eps for 0, and 0 / 0 of a weight without gradients for NaN)
    h.eps = eps > 0.0 && eps < 0x1p-126 ? 0x1p-126f : (float)eps;
    h.lr = lr;
    h.wd = weight_decay;
    h.beta1 = beta1;
    h.beta2 = beta2;
    h.step = step;
    h.step_dev = step_dev;
    h.lr_dev = lr_dev;
    h.norm = norm;
    h.max_norm = max_norm;
    h.decay = h.step_size = h.root = 0.0f;
    if (step_dev == nullptr && lr_dev == nullptr)
        adam_constants(h, step, lr);
    // one combination of types after another, up to kAdamTensors tensors a launch
    for (int kind = 0; kind < 18; ++kind) {  // (masters of fp32 weights: none)
        const int p = kind / 6, g = kind / 2 % 3;
        const bool master = kind % 2 != 0;
        const int64_t chunk = adam_chunk(eight && p != TG_F32 && g != TG_F32 && !master);
        for (int64_t i = 0; i < count;) {
            int64_t chunks = 0;
            a.count = 0;
            for (; i < count && a.count < kAdamTensors; ++i) {
                const tg_adamw_tensor& t = tensors[i];
                if (t.n == 0 || t.p_dtype != p || t.g_dtype != g || (t.master != nullptr) != master)
                    continue;
                const int64_t c = (t.n + chunk - 1) / chunk;
                if (chunks + c > 0x7FFFFFFF)  // (a chunk's number and a grid more fit in 32 bits)
                    break;
                const int k = a.count++;
                a.p[k] = t.param;
                a.w[k] = t.master;
                a.g[k] = t.grad;
                a.m[k] = t.exp_avg;
                a.v[k] = t.exp_avg_sq;
                a.sm[k] = t.exp_avg_scale;
                a.sv[k] = t.exp_avg_sq_scale;
                a.n[k] = t.n;
                a.first[k] = (uint32_t)chunks;
                a.aligned[k] = (((uintptr_t)t.param | (uintptr_t)t.master | (uintptr_t)t.grad | (uintptr_t)t.exp_avg |
                                 (uintptr_t)t.exp_avg_sq) & 15u) == 0;
                chunks += c;
            }
            if (a.count == 0)
                continue;
            a.first[a.count] = (uint32_t)chunks;
            const uint32_t grid = (uint32_t)(chunks < kAdamGrid ? chunks : kAdamGrid);
            // (what exceeds the 256 MB Infinity Cache is read with the non-temporal hint)
            const bool streamed = bytes > (int64_t)256 << 20;
            switch (p) {
            case TG_F32: adam_launch_p<O_F32>(g, master, eight, a, grid, streamed, (hipStream_t)stream); break;
            case TG_F16: adam_launch_p<O_F16>(g, master, eight, a, grid, streamed, (hipStream_t)stream); break;
            default: adam_launch_p<O_BF16>(g, master, eight, a, grid, streamed, (hipStream_t)stream); break;
            }
            if (hipGetLastError() != hipSuccess)
                return TG_ERR_LAUNCH;
        }
    }
    return TG_OK;
}
