// Host side of the feed-forward entry points under AddressSanitizer and
// UndefinedBehaviorSanitizer: calls that fail validation, empty problems and
// workspace queries up to INT64_MAX.  No call here launches anything.
#include <limits.h>
#include <math.h>
#include <stdio.h>
#include <stdlib.h>

#include "tg_ops.h"

static int failures = 0;

static void expect(tg_status got, tg_status want, const char* what)
{
    if (got != want) {
        printf("%s: got %d, want %d\n", what, (int)got, (int)want);
        ++failures;
    }
}

int main(void)
{
    void* const A = (void*)0x10000;
    void* const W = (void*)(1 << 20);
    const int64_t sizes[] = {INT64_MIN, -1, 0, 1, 7, 8, 16, 17, 33, 255, 256, 1000, 4096, 100000, 0x7FFFFFFF, 0x80000000LL,
                             INT64_MAX / 4, INT64_MAX / 2 + 1, INT64_MAX};
    const int n = sizeof sizes / sizeof sizes[0];
    for (int in = -1; in <= 3; ++in)
        for (int a = 0; a < n; ++a)
            for (int b = 0; b < n; ++b)
                for (int c = 0; c < n; ++c) {
                    const int64_t M = sizes[a], N = sizes[b], K = sizes[c];
                    const bool bad = M < 0 || N < 0 || K < 0, any = in >= 0 && in <= 2, half = in == 0 || in == 1;
                    const int64_t q[] = {tg_linear_workspace_bytes((tg_input)in, M, N, K), tg_glu_workspace_bytes((tg_input)in, M, N, K),
                                         tg_linear_backward_workspace_bytes((tg_input)in, M, N, K),
                                         tg_glu_backward_workspace_bytes((tg_input)in, M, N, K)};
                    for (int i = 0; i < 4; ++i) {
                        const bool known = !bad && (i < 2 ? any : half);
                        if (known ? (q[i] < 0 || q[i] > (64 << 20) + (64 << 10)) : q[i] != -1) {
                            printf("query %d of %d, %lld x %lld x %lld: %lld\n", i, in, (long long)M, (long long)N, (long long)K,
                                   (long long)q[i]);
                            ++failures;
                        }
                    }
                    // sizes that no call takes: refused before anything is formed from them
                    if (any && (bad || M > 0x7FFFFFFF || N > 0x7FFFFFFF || K > 0x7FFFFFFF)) {
                        const tg_status want = bad ? TG_ERR_INVALID_VALUE : TG_ERR_NOT_SUPPORTED;
                        const tg_dtype o = in == 0 ? TG_F16 : TG_BF16;
                        expect(tg_linear((tg_input)in, M, N, K, A, K, A, K, NULL, TG_ACT_NONE, NULL, 0, 1.f, 1.f, A, N, o, NULL, 0, NULL, 0, NULL), want, "tg_linear");
                        expect(tg_glu((tg_input)in, M, N, K, A, K, A, K, TG_ACT_SILU, 1.f, 1.f, A, N, o, NULL, 0, NULL, 0, NULL), want, "tg_glu");
                        if (half) {
                            expect(tg_linear_backward((tg_input)in, M, N, K, A, N, A, K, A, K, A, N, TG_ACT_GELU, A, N, A, K, A, K, o, NULL, NULL, 0, NULL), want, "tg_linear_backward");
                            expect(tg_glu_backward((tg_input)in, M, N, K, A, K, A, N, A, K, A, K, A, N, A, N, TG_ACT_SILU, A, N, A, K, A, K, A, N, o, NULL, 0, NULL), want, "tg_glu_backward");
                        }
                    }
                }
    const void* g[3] = {A, A, A};
    void* o[3] = {A, A, A};
    int64_t sz[3] = {4, 0, 4};
    int32_t ty[3] = {0, 1, 2};
    const int64_t need = tg_clip_grads_workspace_bytes(3);
    if (need <= 0 || tg_clip_grads_workspace_bytes(-1) != -1 || tg_clip_grads_workspace_bytes(0) != 0)
        ++failures;
    expect(tg_clip_grads(-1, g, o, sz, ty, 1.f, 0.f, NULL, W, need, NULL), TG_ERR_INVALID_VALUE, "count");
    expect(tg_clip_grads(3, g, o, sz, ty, NAN, 0.f, NULL, W, need, NULL), TG_ERR_INVALID_VALUE, "max_norm");
    expect(tg_clip_grads(3, g, o, sz, ty, 1.f, 0.f, NULL, NULL, 0, NULL), TG_ERR_INVALID_VALUE, "workspace");
    expect(tg_clip_grads(INT64_MAX, g, o, sz, ty, 1.f, 0.f, NULL, W, need, NULL), TG_ERR_NOT_SUPPORTED, "count");
    sz[2] = INT64_MAX;
    expect(tg_clip_grads(3, g, o, sz, ty, 1.f, 0.f, NULL, W, need, NULL), TG_ERR_NOT_SUPPORTED, "size");
    sz[2] = -1;
    expect(tg_clip_grads(3, g, o, sz, ty, 1.f, 0.f, NULL, W, need, NULL), TG_ERR_INVALID_VALUE, "size");
    expect(tg_clip_grads(0, NULL, NULL, NULL, NULL, 1.f, 0.f, NULL, NULL, 0, NULL), TG_OK, "empty");
    expect(tg_linear((tg_input)99, 1, 1, 1, A, 8, A, 8, NULL, (tg_act)0, NULL, 0, 1.f, 1.f, A, 8, TG_BF16, NULL, 0, NULL, 0, NULL), TG_ERR_INVALID_VALUE, "input");
    expect(tg_glu(TG_IN_BF16, 1, 8, 8, A, 8, A, 8, (tg_act)INT_MIN, 1.f, 1.f, A, 8, TG_BF16, NULL, 0, NULL, 0, NULL), TG_ERR_INVALID_VALUE, "act");
    expect(tg_linear(TG_IN_FP8, 0, 8, 8, NULL, 16, NULL, 16, NULL, TG_ACT_RELU, NULL, 0, 1.f, 1.f, NULL, 8, TG_F32, NULL, 0, NULL, 0, NULL), TG_OK, "empty");
    if (failures == 0)
        printf("ok\n");
    return failures != 0;
}
