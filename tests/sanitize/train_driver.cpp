// Host side of the training operators' and the int8 layers' entry points under
// AddressSanitizer and UndefinedBehaviorSanitizer: calls that fail validation,
// empty problems and workspace queries up to INT64_MAX.  No call here launches
// anything.
#include <limits.h>
#include <math.h>
#include <stdio.h>
#include <stdlib.h>

#include "tg_int8.h"
#include "tg_train.h"

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
    const int64_t* const T = (const int64_t*)A;
    float* const F = (float*)A;
    const int8_t* const Q = (const int8_t*)A;
    const int64_t sizes[] = {INT64_MIN, -1, 0, 1, 7, 8, 16, 17, 33, 255, 256, 1000, 4096, 100000, 4000000, 0x7FFFFFFF, 0x80000000LL,
                             INT64_MAX / 4, INT64_MAX / 2 + 1, INT64_MAX};
    const int n = sizeof sizes / sizeof sizes[0];
    for (int in = -1; in <= 3; ++in)
        for (int a = 0; a < n; ++a)
            for (int b = 0; b < n; ++b)
                for (int c = 0; c < n; ++c) {
                    const int64_t M = sizes[a], N = sizes[b], K = sizes[c];
                    const bool bad = M < 0 || N < 0 || K < 0, half = in == 0 || in == 1;
                    const bool large = M > 0x7FFFFFFF || N > 0x7FFFFFFF || K > 0x7FFFFFFF;
                    const int64_t q[] = {tg_linear_xent_workspace_bytes((tg_input)in, M, N, K),
                                         tg_linear_xent_backward_workspace_bytes((tg_input)in, M, N, K, 0),
                                         tg_linear_xent_backward_workspace_bytes((tg_input)in, M, N, K, 1),
                                         tg_linear_xent_backward_workspace_bytes((tg_input)in, M, N, K, INT64_MAX)};
                    for (int i = 0; i < 4; ++i)
                        if (bad || !half ? q[i] != -1 : q[i] < 0) {
                            printf("query %d of %d, %lld x %lld x %lld: %lld\n", i, in, (long long)M, (long long)N, (long long)K, (long long)q[i]);
                            ++failures;
                        }
                    const int64_t w = tg_linear_i8_workspace_bytes(M, N, K);
                    if (bad ? w != -1 : w < 0 || w > (64 << 20) + (64 << 10)) {
                        printf("int8 query %lld x %lld x %lld: %lld\n", (long long)M, (long long)N, (long long)K, (long long)w);
                        ++failures;
                    }
                    if (bad || large) {
                        const tg_status want = bad ? TG_ERR_INVALID_VALUE : TG_ERR_NOT_SUPPORTED;
                        expect(tg_linear_i8(M, N, K, Q, K, Q, K, F, F, NULL, TG_ACT_NONE, NULL, 0, A, N, TG_BF16, NULL, 0, NULL), want, "tg_linear_i8");
                        if (bad ? (M < 0 || K < 0) : (M > 0x7FFFFFFF || K > 0x7FFFFFFF))
                            expect(tg_quantize_i8(TG_F32, M, K, A, K, (int8_t*)A, K, F, NULL), want, "tg_quantize_i8");
                        if (half) {
                            expect(tg_linear_xent((tg_input)in, M, N, K, A, K, A, K, 1.f, T, -100, 0.f, F, F, F, W, INT64_MAX, NULL), want, "tg_linear_xent");
                            expect(tg_linear_xent_backward((tg_input)in, M, N, K, A, K, A, K, 1.f, T, -100, 0.f, F, F, 1.f, F, A, K, A, K, TG_F32, W, INT64_MAX, NULL),
                                   want, "tg_linear_xent_backward");
                        }
                    }
                }
    // sizes that are taken, workspaces that do not hold them
    const int64_t least = tg_linear_xent_backward_workspace_bytes(TG_IN_BF16, 1000, 0x7FFFFFFF, 64, 1);
    expect(tg_linear_xent_backward(TG_IN_BF16, 1000, 0x7FFFFFFF, 64, A, 64, A, 64, 1.f, T, -100, 0.f, F, F, 1.f, F, A, 64, A, 64, TG_F32, W, least - 1, NULL),
           TG_ERR_INVALID_VALUE, "workspace");
    tg_adamw_tensor t[2] = {};
    t[1].param = t[1].exp_avg = t[1].exp_avg_sq = A;
    t[1].grad = A;
    expect(tg_adamw(2, t, 1, 1e-3, 0.9, 0.99, 1e-8, 0.1, NULL, INFINITY, NULL, NULL, NULL), TG_OK, "empty tensors");
    expect(tg_adamw(0, NULL, INT64_MAX, 1e-3, 0.9, 0.99, 1e-8, 0.1, NULL, 1.f, NULL, NULL, NULL), TG_OK, "no tensors");
    expect(tg_adamw(INT64_MIN, t, 1, 1e-3, 0.9, 0.99, 1e-8, 0.1, NULL, 1.f, NULL, NULL, NULL), TG_ERR_INVALID_VALUE, "count");
    expect(tg_adamw(2, t, 0, 1e-3, 0.9, 0.99, 1e-8, 0.1, NULL, 1.f, NULL, NULL, NULL), TG_ERR_INVALID_VALUE, "step");
    t[1].n = INT64_MAX;
    expect(tg_adamw(2, t, 1, 1e-3, 0.9, 0.99, 1e-8, 0.1, NULL, 1.f, NULL, NULL, NULL), TG_ERR_NOT_SUPPORTED, "size");
    t[1].n = INT64_MIN;
    expect(tg_adamw(2, t, 1, 1e-3, 0.9, 0.99, 1e-8, 0.1, NULL, 1.f, NULL, NULL, NULL), TG_ERR_INVALID_VALUE, "size");
    t[1].n = 4;
    t[1].p_dtype = INT_MIN;
    expect(tg_adamw(2, t, 1, 1e-3, 0.9, 0.99, 1e-8, 0.1, NULL, 1.f, NULL, NULL, NULL), TG_ERR_INVALID_VALUE, "type");
    expect(tg_linear_i8(8, 8, 16, Q, 16, Q, 16, F, F, NULL, (tg_act)INT_MAX, NULL, 0, A, 8, TG_BF16, NULL, 0, NULL), TG_ERR_INVALID_VALUE, "act");
    expect(tg_quantize_i8((tg_dtype)99, 8, 16, A, 16, (int8_t*)A, 16, F, NULL), TG_ERR_INVALID_VALUE, "dtype");
    if (failures == 0)
        printf("ok\n");
    return failures != 0;
}
