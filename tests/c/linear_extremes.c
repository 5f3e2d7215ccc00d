/* Every entry point of include/hkg_linear.h called with extreme and invalid sizes and
 * pitches on a host without a GPU, as ops_extremes.c does for hkg_ops.h.  Prints "LINEAR
 * EXTREMES OK" and exits 0 on success. */
#include <inttypes.h>
#include <stdint.h>
#include <stdio.h>

#include "hkg_linear.h"

static long calls, failures;

static void expect(int rc, const char *what, int64_t a, int64_t b, int64_t c, int64_t ld)
{
    ++calls;
    if (rc > HKG_OK || rc < HKG_ERR_WORKSPACE || rc == HKG_ERR_LAUNCH) {
        fprintf(stderr, "FAIL %s %" PRId64 " %" PRId64 " %" PRId64 " ld %" PRId64 ": %d\n", what, a, b, c, ld, rc);
        ++failures;
    }
}

static void expect_bytes(int64_t n, const char *what, int64_t a, int64_t b, int64_t c)
{
    ++calls;
    if (n < 0 && n != HKG_ERR_SHAPE && n != HKG_ERR_SIZE) {
        fprintf(stderr, "FAIL %s %" PRId64 " %" PRId64 " %" PRId64 ": %" PRId64 "\n", what, a, b, c, n);
        ++failures;
    }
}

static const int64_t kVals[] = {INT64_MIN, -8, 0, 1, 8, 24, 4096, 65528, ((int64_t)1 << 22) - 16, ((int64_t)1 << 22) - 8,
                                (int64_t)1 << 22, ((int64_t)1 << 31) - 8, ((int64_t)1 << 31) - 1, (int64_t)1 << 31,
                                (int64_t)1 << 56, INT64_MAX - 7, INT64_MAX};
#define NV ((int)(sizeof(kVals) / sizeof(kVals[0])))

/* aligned addresses that are never read, far apart */
#define P(i) ((void *)(uintptr_t)((uint64_t)(i) << 44))

int main(void)
{
    const float ps[] = {0.0f, 0.1f, 1.0f, -1.0f, 2.0f};
    for (int i = 0; i < NV; ++i)
        for (int j = 0; j < NV; ++j)
            for (int l = 0; l < NV; ++l)
                for (int t = -1; t < 4; ++t) {
                    const int64_t R = kVals[i], C = kVals[j], ld = kVals[l];
                    const hkg_dropout_opts d = {ps[(i + j + l) % 5], UINT64_MAX, (uint64_t)ld, 0};
                    expect(hkg_dropout(R, C, P(1), t, ld, &d, 0, 0, P(2), t, 0, 0), "dropout x", R, C, 0, ld);
                    expect(hkg_dropout(R, C, P(1), t, 0, &d, P(3), ld, P(2), HKG_T_F32, 0, 0), "dropout r", R, C, 0, ld);
                    expect(hkg_dropout(R, C, P(1), t, 0, 0, P(2), ld, P(2), t, ld, 0), "dropout out", R, C, 0, ld);
                }
    for (int i = 0; i < NV; ++i)
        for (int j = 0; j < NV; ++j)
            for (int k = 0; k < NV; ++k) {
                const int64_t M = kVals[i], N = kVals[j], K = kVals[k];
                expect_bytes(hkg_linear_workspace_bytes(M, N, K), "linear bytes", M, N, K);
                expect_bytes(hkg_linear_backward_workspace_bytes(M, N, K), "backward bytes", M, N, K);
                for (int l = 0; l < NV; ++l) {
                    const int64_t ld = kVals[l];
                    hkg_epilogue e = {P(4), HKG_T_F32, 1 + l % 4, P(5), 0, P(6), 0, {0.5f, 1, 2, 0}};
                    expect(hkg_linear(M, N, K, 2 * (l % 2), P(1), ld, P(2), 0, 0, P(3), HKG_T_F32, 0, P(7), INT64_MAX, 0), "linear x",
                           M, N, K, ld);
                    expect(hkg_linear(M, N, K, 0, P(1), 0, P(2), ld, &e, P(3), 0, 0, P(7), INT64_MAX, 0), "linear W", M, N, K, ld);
                    e.ldr = ld;
                    expect(hkg_linear(M, N, K, 0, P(1), 0, P(2), 0, &e, P(5), 0, ld, P(7), INT64_MAX, 0), "linear y", M, N, K, ld);
                    e.ldz = ld;
                    expect(hkg_linear(M, N, K, 2, P(1), 0, P(2), 0, &e, P(3), 2, 0, P(7), 0, 0), "linear z", M, N, K, ld);
                    expect(hkg_linear_backward(M, N, K, 0, P(1), l % 2, ld, P(2), 0, P(3), 0, P(4), 0, 2, &e.dropout, P(5), 0, P(6), 0,
                                               (float *)P(7), P(8), INT64_MAX, 0),
                           "backward dy", M, N, K, ld);
                    expect(hkg_linear_backward(M, N, K, 2, P(1), 2, 0, P(2), ld, P(3), ld, P(4), ld, 3, 0, P(5), ld, P(6), ld, 0, P(8),
                                               INT64_MAX, 0),
                           "backward", M, N, K, ld);
                }
            }
    printf("%ld calls, %ld failures\n", calls, failures);
    if (failures)
        return 1;
    printf("LINEAR EXTREMES OK\n");
    return 0;
}
