/* Every entry point of include/hkg_ops.h called with extreme and invalid sizes and
 * pitches on a host without a GPU: each call returns a documented status before any
 * device work.  Built with the library's host code under AddressSanitizer and
 * UndefinedBehaviorSanitizer, so a signed overflow in a check ends the run.  Prints
 * "OPS EXTREMES OK" and exits 0 on success. */
#include <inttypes.h>
#include <stdint.h>
#include <stdio.h>

#include "hkg_ops.h"

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
    if (n < HKG_ERR_WORKSPACE || (n < 0 && n != HKG_ERR_SHAPE && n != HKG_ERR_SIZE)) {
        fprintf(stderr, "FAIL %s %" PRId64 " %" PRId64 " %" PRId64 ": %" PRId64 "\n", what, a, b, c, n);
        ++failures;
    }
}

static const int64_t kVals[] = {INT64_MIN, -1, 0, 1, 16, 33, 10241, ((int64_t)1 << 22) - 96, ((int64_t)1 << 23) - 33,
                                (int64_t)1 << 23, ((int64_t)1 << 29) - 128, ((int64_t)1 << 31) - 1, (int64_t)1 << 31,
                                (int64_t)1 << 56, INT64_MAX - 15, INT64_MAX};
#define NV ((int)(sizeof(kVals) / sizeof(kVals[0])))

/* aligned addresses that are never read, far apart */
#define P(i) ((void *)(uintptr_t)((uint64_t)(i) << 44))

int main(void)
{
    for (int i = 0; i < NV; ++i)
        for (int j = 0; j < NV; ++j)
            for (int t = 0; t < 2; ++t)
                for (int l = 0; l < NV; ++l) {
                    const int64_t R = kVals[i], K = kVals[j], ld = kVals[l];
                    expect_bytes(hkg_mxfp4_code_bytes(R, K), "code bytes", R, K, 0);
                    expect(hkg_mxfp4_quantize(0, R, K, P(1), t, ld, P(2), P(3), 0), "quantize", R, K, 0, ld);
                    expect(hkg_mxfp4_quantize_both(0, 1, R, K, P(1), t, ld, P(2), P(3), P(4), P(5), 0), "both", R, K, 0, ld);
                    expect(hkg_mxfp4_dequantize(1, R, K, P(1), P(2), P(3), t, ld, 0), "dequantize", R, K, 0, ld);
                    expect_bytes(hkg_orthogonalize_workspace_bytes(R, K), "orth bytes", R, K, 0);
                    expect(hkg_orthogonalize(R, K, P(1), t, ld, 5, 3.4f, -4.8f, 2.0f, 1e-7f, P(2), 0, P(3), INT64_MAX, 0),
                           "orthogonalize", R, K, 0, ld);
                    expect(hkg_orthogonalize(R, K, P(1), t, 0, 5, 3.4f, -4.8f, 2.0f, 1e-7f, P(2), ld, P(3), INT64_MAX, 0),
                           "orthogonalize out", R, K, 0, ld);
                }
    for (int i = 0; i < NV; ++i)
        for (int j = 0; j < NV; ++j)
            for (int k = 0; k < NV; ++k)
                for (int l = 0; l < NV; ++l) {
                    const int64_t M = kVals[i], N = kVals[j], K = kVals[k], ld = kVals[l];
                    expect_bytes(hkg_linear_mxfp4_workspace_bytes(M, N, K), "linear bytes", M, N, K);
                    expect_bytes(hkg_linear_mxfp4_backward_workspace_bytes(M, N, K), "backward bytes", M, N, K);
                    expect(hkg_gemm_mxfp4(M, N, K, P(1), P(2), P(3), P(4), P(5), P(6), ld, 0), "gemm", M, N, K, ld);
                    expect(hkg_linear_mxfp4(M, N, K, P(1), 1, ld, P(2), P(3), P(4), 0, P(5), INT64_MAX, 0), "linear x", M, N, K, ld);
                    expect(hkg_linear_mxfp4(M, N, K, P(1), 0, 0, P(2), P(3), P(4), ld, P(5), INT64_MAX, 0), "linear y", M, N, K, ld);
                    for (int w = 0; w < 3; ++w) {
                        /* both gradients, dw alone, dx alone: the pitch of an absent one means nothing */
                        void *dx = w == 1 ? 0 : P(6), *dw = w == 2 ? 0 : P(7);
                        expect(hkg_linear_mxfp4_backward(M, N, K, P(1), 1, 0, P(2), P(3), P(4), P(5), dx, ld, dw, 0, P(8),
                                                         INT64_MAX, 0), "backward dx", M, N, K, ld);
                        expect(hkg_linear_mxfp4_backward(M, N, K, P(1), 0, ld, P(2), P(3), P(4), P(5), dx, 0, dw, ld, P(8),
                                                         INT64_MAX, 0), "backward dw", M, N, K, ld);
                    }
                }
    if (failures)
        return 1;
    printf("OPS EXTREMES OK (%ld calls)\n", calls);
    return 0;
}
