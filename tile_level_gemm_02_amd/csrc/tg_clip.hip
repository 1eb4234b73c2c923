// tg_clip_grads: the global gradient norm over many tensors, and clipping
// (contract in include/tg_ops.h).
//
//   norm = sqrt(sum g^2);   out = g * min(1, max_norm / (norm + eps))
//
// Two passes over the gradients, each one launch per kMaxTensors tensors: the
// tensors' descriptors travel in the kernel arguments, and workgroups walk
// the tensors' chunks of kChunk elements.  Both are bound by memory: the sum
// reads every value once, the scaling reads it again and writes it.  The
// scaling walks the chunks in the opposite order, so that what the sum read
// last is found in the 256 MB Infinity Cache; where the gradients exceed that
// cache it reads with the non-temporal hint (56 tensors of 400 M values,
// 0.8 GB: 447 -> 430 us; 8 M values 25.8 us without it, 27.0 with).  430 us
// for 0.8 GB read twice and written once is 5.6 TB/s; a large copy moves 4.7.
// A small call is its two launches: 9 tensors of 60 K values take 9.3 us.
// Squares and sums are fp64
// (exact for the squares of all three types' values up to the sum's own
// rounding; a large fp32 gradient's square leaves fp32's range).  Each
// workgroup's partial sum goes to a slot of its own and the last workgroup to
// arrive adds the slots in order: the norm does not depend on the order of
// arrival.
#include <math.h>

#include "tg_abi.hpp"
#include "tg_epilogue.hpp"
#include "tg_ops.h"

namespace tg {

constexpr int kMaxTensors = 96;       // descriptors per launch (under 4 KiB of kernel arguments)
constexpr int64_t kChunk = 8192;      // elements per chunk
constexpr int64_t kClipGrid = 2048;   // workgroups of a launch: 8 per compute unit
constexpr int64_t kClipSlots = 16384; // partial sums of a call
constexpr int64_t kClipCounterBytes = 65536;

struct ClipArgs {
    const void* in[kMaxTensors];
    void* out[kMaxTensors];
    int64_t n[kMaxTensors];
    uint32_t first[kMaxTensors + 1];  // first chunk of each tensor; [count]: all
    uint8_t type[kMaxTensors];        // Out, + 4 where both pointers are 16-byte aligned
    int32_t count;
    uint32_t slot0, slots;            // this launch's first slot; slots of the whole call
    uint32_t* counter;
    double* total;                    // sum of squares
    double* partials;
    float* norm;
    float max_norm, eps;
};

__device__ __forceinline__ int tensor_of_chunk(const ClipArgs& p, uint32_t c)
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

// f(first element, elements) over a chunk of `n` elements of type O, in
// pieces of 16 bytes (whole) or one element at a time
template <int O, bool WHOLE, class F>
__device__ __forceinline__ void over_chunk(int64_t e0, int64_t n, F f)
{
    constexpr int V = Piece<O>::N;
    const uint32_t tid = threadIdx.x;
    if constexpr (WHOLE) {
        if (n == kChunk) {
#pragma unroll
            for (int i = 0; i < (int)kChunk / (256 * V); ++i)
                f(std::true_type{}, e0 + ((int64_t)i * 256 + tid) * V);
            return;
        }
        const int64_t pieces = n / V;
        for (int64_t i = tid; i < pieces; i += 256)
            f(std::true_type{}, e0 + i * V);
        for (int64_t i = pieces * V + tid; i < n; i += 256)
            f(std::false_type{}, e0 + i);
    } else {
        for (int64_t i = tid; i < n; i += 256)
            f(std::false_type{}, e0 + i);
    }
}

// the four ways a tensor is walked
template <class F>
__device__ __forceinline__ void for_tensor_type(uint32_t type, F f)
{
    switch (type) {
    case O_F32: f(std::integral_constant<int, O_F32>{}, std::false_type{}); break;
    case O_F16: f(std::integral_constant<int, O_F16>{}, std::false_type{}); break;
    case O_BF16: f(std::integral_constant<int, O_BF16>{}, std::false_type{}); break;
    case O_F32 + 4: f(std::integral_constant<int, O_F32>{}, std::true_type{}); break;
    case O_F16 + 4: f(std::integral_constant<int, O_F16>{}, std::true_type{}); break;
    default: f(std::integral_constant<int, O_BF16>{}, std::true_type{}); break;
    }
}

// sum over the workgroup, in a fixed order; in thread 0
__device__ __forceinline__ double group_sum(double v, double* lds4)
{
#pragma unroll
    for (int d = 32; d > 0; d >>= 1)
        v += __shfl_down(v, d, 64);
    if ((threadIdx.x & 63u) == 0u)
        lds4[threadIdx.x >> 6] = v;
    __syncthreads();
    return lds4[0] + lds4[1] + lds4[2] + lds4[3];
}

__global__ __launch_bounds__(256) void clip_sum(ClipArgs p)
{
    __shared__ double lds4[4];
    __shared__ uint32_t arrived;
    double s0 = 0.0, s1 = 0.0;
    const uint32_t chunks = p.first[p.count];
    for (uint32_t c = blockIdx.x; c < chunks; c += gridDim.x) {
        const int t = tensor_of_chunk(p, c);
        const int64_t e0 = (int64_t)(c - p.first[t]) * kChunk;
        const int64_t n = p.n[t] - e0 < kChunk ? p.n[t] - e0 : kChunk;
        const void* g = p.in[t];
        for_tensor_type(p.type[t], [&](auto o, auto whole) __attribute__((always_inline)) {
            constexpr int O = decltype(o)::value;
            over_chunk<O, decltype(whole)::value>(e0, n, [&](auto piece, int64_t e) __attribute__((always_inline)) {
                if constexpr (decltype(piece)::value) {
                    const u32x4 q = ldg128((const typename OutInfo<O>::T*)g + e);
#pragma unroll
                    for (int i = 0; i < Piece<O>::N; i += 2) {
                        const double a = (double)piece_value<O>(q, i), b = (double)piece_value<O>(q, i + 1);
                        s0 = __builtin_fma(a, a, s0);
                        s1 = __builtin_fma(b, b, s1);
                    }
                } else {
                    const double a = (double)load_value<O>(g, e);
                    s0 = __builtin_fma(a, a, s0);
                }
            });
        });
    }
    const double s = group_sum(s0 + s1, lds4);
    // the slot's store has completed before the workgroup counts itself in;
    // stores and loads of slots are device-scope (see splitk_last)
    if (threadIdx.x == 0u) {
        __hip_atomic_store(p.partials + p.slot0 + blockIdx.x, s, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
        arrived = __hip_atomic_fetch_add(p.counter, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    }
    __syncthreads();
    if (arrived != p.slots - 1u)
        return;
    double v = 0.0;
    for (uint32_t i = threadIdx.x; i < p.slots; i += 256u)
        v += __hip_atomic_load(p.partials + i, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    v = group_sum(v, lds4);
    if (threadIdx.x == 0u) {
        __hip_atomic_exchange(p.counter, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        *p.total = v;
        if (p.norm != nullptr)
            *p.norm = (float)__builtin_sqrt(v);
    }
}

// STREAM: the gradients are read with the non-temporal hint (a template
// parameter: the compiler folds a branch between the two loads into one
// without the hint)
template <bool STREAM>
__global__ __launch_bounds__(256) void clip_scale(ClipArgs p)
{
    const double d = __builtin_sqrt(*p.total) + (double)p.eps;
    // (compared first: 0 / 0 and inf / inf clip nothing; a NaN norm fails the
    // comparison and stays)
    const float coef = d <= (double)p.max_norm ? 1.0f : (float)((double)p.max_norm / d);
    const uint32_t chunks = p.first[p.count];
    for (uint32_t i = blockIdx.x; i < chunks; i += gridDim.x) {
        const uint32_t ch = chunks - 1u - i;
        const int t = tensor_of_chunk(p, ch);
        const int64_t e0 = (int64_t)(ch - p.first[t]) * kChunk;
        const int64_t n = p.n[t] - e0 < kChunk ? p.n[t] - e0 : kChunk;
        const void* g = p.in[t];
        void* out = p.out[t];
        if (coef == 1.0f && g == out)
            continue;
        for_tensor_type(p.type[t], [&](auto o, auto whole) __attribute__((always_inline)) {
            constexpr int O = decltype(o)::value;
            over_chunk<O, decltype(whole)::value>(e0, n, [&](auto piece, int64_t e) __attribute__((always_inline)) {
                if constexpr (decltype(piece)::value) {
                    const u32x4* src = (const u32x4*)((const typename OutInfo<O>::T*)g + e);
                    u32x4 q;
                    if constexpr (STREAM)
                        q = __builtin_nontemporal_load(src);
                    else
                        q = *src;
                    float v[Piece<O>::N];
#pragma unroll
                    for (int j = 0; j < Piece<O>::N; ++j)
                        v[j] = piece_value<O>(q, j) * coef;
                    store_nt((u32x4*)((typename OutInfo<O>::T*)out + e), pack_piece<O>(v));
                } else {
                    store_value<O>(out, e, load_value<O>(g, e) * coef);
                }
            });
        });
    }
}

}  // namespace tg

using namespace tg;

extern "C" int64_t tg_clip_grads_workspace_bytes(int64_t count)
{
    return count < 0 ? -1 : count == 0 ? 0 : kClipCounterBytes + 256 + kClipSlots * 8;
}

extern "C" tg_status tg_clip_grads(int64_t count, const void* const* grads, void* const* outs, const int64_t* sizes,
                                   const int32_t* dtypes, float max_norm, float eps, float* norm, void* workspace,
                                   int64_t workspace_bytes, void* stream)
{
    if (count < 0 || !(max_norm >= 0.0f) || !(eps >= 0.0f) || __builtin_isinf(eps) || workspace_bytes < 0)
        return TG_ERR_INVALID_VALUE;
    if (count > 0 && (grads == nullptr || outs == nullptr || sizes == nullptr || dtypes == nullptr))
        return TG_ERR_INVALID_VALUE;
    if (count > kMaxTensors * kClipSlots)
        return TG_ERR_NOT_SUPPORTED;
    for (int64_t i = 0; i < count; ++i) {
        if (sizes[i] < 0 || (dtypes[i] != TG_F32 && dtypes[i] != TG_F16 && dtypes[i] != TG_BF16))
            return TG_ERR_INVALID_VALUE;
        if (sizes[i] == 0)
            continue;
        if (grads[i] == nullptr || outs[i] == nullptr)
            return TG_ERR_INVALID_VALUE;
        const uintptr_t mask = dtypes[i] == TG_F32 ? 3u : 1u;
        if (((uintptr_t)grads[i] & mask) || ((uintptr_t)outs[i] & mask))
            return TG_ERR_MISALIGNED;
        if (sizes[i] > (int64_t)1 << 40)
            return TG_ERR_NOT_SUPPORTED;
    }
    if ((uintptr_t)norm & 3u)
        return TG_ERR_MISALIGNED;
    if (count == 0 && norm == nullptr)
        return TG_OK;
    if (workspace == nullptr || workspace_bytes < tg_clip_grads_workspace_bytes(1))
        return TG_ERR_INVALID_VALUE;
    if ((uintptr_t)workspace & 255u)
        return TG_ERR_MISALIGNED;

    // launches of up to kMaxTensors non-empty tensors; one with none where all
    // are empty (the norm is still written)
    hipStream_t s = (hipStream_t)stream;
    int64_t full = 0, bytes = 0;
    for (int64_t i = 0; i < count; ++i) {
        full += sizes[i] > 0;
        bytes += sizes[i] * (dtypes[i] == TG_F32 ? 4 : 2);
    }
    const int64_t launches = full == 0 ? 1 : (full + kMaxTensors - 1) / kMaxTensors;
    int64_t most = kClipSlots / launches;
    if (most > kClipGrid)
        most = kClipGrid;
    ClipArgs p;
    p.counter = (uint32_t*)workspace;
    p.total = (double*)((uint8_t*)workspace + kClipCounterBytes);
    p.partials = (double*)((uint8_t*)workspace + kClipCounterBytes + 256);
    p.norm = norm;
    p.max_norm = max_norm;
    p.eps = eps;
    // fill the descriptors from tensor i on; returns the next tensor
    auto fill = [&](int64_t i, int64_t* grid) -> int64_t {
        int64_t chunks = 0;
        p.count = 0;
        for (; i < count && p.count < kMaxTensors; ++i) {
            if (sizes[i] == 0)
                continue;
            const int64_t c = (sizes[i] + kChunk - 1) / kChunk;
            if (chunks + c > 0xFFFFFFFF)
                break;
            const int t = p.count++;
            p.in[t] = grads[i];
            p.out[t] = outs[i];
            p.n[t] = sizes[i];
            p.first[t] = (uint32_t)chunks;
            p.type[t] = (uint8_t)(dtypes[i] + ((((uintptr_t)grads[i] | (uintptr_t)outs[i]) & 15u) ? 0 : 4));
            chunks += c;
        }
        p.first[p.count] = (uint32_t)chunks;
        *grid = chunks < 1 ? 1 : chunks < most ? chunks : most;
        return i;
    };
    // slots of the whole call, then the sums, then the scaling
    int64_t grid = 0, slots = 0;
    for (int64_t i = 0, first = 1; first || i < count; first = 0) {
        i = fill(i, &grid);
        if (p.count > 0 || first)
            slots += grid;
    }
    if (slots > kClipSlots)
        return TG_ERR_NOT_SUPPORTED;
    p.slots = (uint32_t)slots;
    p.slot0 = 0;
    for (int64_t i = 0, first = 1; first || i < count; first = 0) {
        i = fill(i, &grid);
        if (p.count == 0 && !first)
            continue;
        hipLaunchKernelGGL(clip_sum, dim3((uint32_t)grid), dim3(256), 0, s, p);
        if (hipGetLastError() != hipSuccess)
            return TG_ERR_LAUNCH;
        p.slot0 += (uint32_t)grid;
    }
    for (int64_t i = 0; i < count;) {
        i = fill(i, &grid);
        if (p.count == 0)
            continue;
        if (bytes > (int64_t)256 << 20)
            hipLaunchKernelGGL(clip_scale<true>, dim3((uint32_t)grid), dim3(256), 0, s, p);
        else
            hipLaunchKernelGGL(clip_scale<false>, dim3((uint32_t)grid), dim3(256), 0, s, p);
        if (hipGetLastError() != hipSuccess)
            return TG_ERR_LAUNCH;
    }
    return TG_OK;
}
