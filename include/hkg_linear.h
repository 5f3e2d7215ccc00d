/*
 * hkg_linear.h -- C ABI of the 16-bit linear layer: a product with bias,
 * activation, dropout and residual in its epilogue, its gradients, and dropout
 * by itself.  Same library and conventions as hkg.h and hkg_ops.h: device
 * pointers owned by the caller, every argument checked before the first HIP
 * call, work enqueued on `stream` and never waited for, HKG_OK or a negative
 * hkg_status returned, intermediate results in a workspace of the caller's.
 *
 * Element types: HKG_T_BF16, HKG_T_F16, and HKG_T_F32 where it is named.  Row
 * pitches (ldx, ...) count elements, 0 = dense.  x and W are operands of the
 * matrix cores: K a multiple of 8 (HKG_ERR_SHAPE), bases and pitches multiples
 * of 16 bytes (HKG_ERR_ALIGN), 256 rows below 2 GiB (HKG_ERR_SIZE), as in
 * hkg_gemm_bf16.  All other matrices need no alignment beyond their element's.
 */
#ifndef HKG_LINEAR_H
#define HKG_LINEAR_H

#include <stdint.h>

#include "hkg_ops.h"

#ifdef __cplusplus
extern "C" {
#endif

enum { HKG_T_F16 = 2 };

/*
 * act(z); its slope act'(z) at 0 is 0 for relu, 1/2 for the others.
 *   HKG_ACT_RELU       max(z, 0)
 *   HKG_ACT_GELU       z Phi(z), Phi the normal distribution function
 *   HKG_ACT_GELU_TANH  z / 2 (1 + tanh(sqrt(2 / pi) (z + 0.044715 z^3)))
 *   HKG_ACT_SILU       z / (1 + exp(-z))
 * Evaluated within 2^-20 of the value for a y in fp32, and within 2^-15 of it for one
 * of 16 bits, which is then rounded by up to 2^-8 (bf16) or 2^-11 (fp16); a value below
 * 2^-116 in magnitude may become 0.  Slopes within 2^-19.  At -infinity all but
 * HKG_ACT_NONE are 0, with slope 0; a NaN stays one.
 */
enum {
    HKG_ACT_NONE = 0,
    HKG_ACT_RELU = 1,
    HKG_ACT_GELU = 2,
    HKG_ACT_GELU_TANH = 3,
    HKG_ACT_SILU = 4
};

/*
 * Dropout D of a matrix, its mask computed where it is used and never stored.
 * With q = round(65536 p) / 65536, an element is dropped, and becomes 0 whatever
 * it was, with probability q; a kept one is multiplied by 1 / (1 - q).  (16-bit
 * numbers: eight decisions from one call of the generator, which takes longer
 * than anything else an element needs.  p = 0.1 is 6554 / 65536 = 0.100006.)
 *
 * The generator is Philox-4x32 with 10 rounds (Salmon, Moraes, Dror, Shaw:
 * "Parallel random numbers: as easy as 1, 2, 3", 2011).  Key: seed (low word,
 * high word).  Counter: (column / 8, row, offset's low word, offset's high
 * word).  Its four words are eight 16-bit numbers, low halves first, those of
 * columns 8 c .. 8 c + 7 of the row; an element is dropped where its number is
 * below 65536 q.  The mask depends on seed, offset, row and column alone, so
 * hkg_linear, hkg_linear_backward and hkg_dropout agree on it; calls that shall
 * be independent take different offsets.
 *   p     0 .. 1 (HKG_ERR_OPTS); 0: no dropout, and nothing else is read
 *   rng   NULL, or a device pointer, 8-byte aligned, to {seed, offset}, read when
 *         the kernels run and used instead of the fields: a captured graph takes
 *         other masks when they are changed between its replays
 */
typedef struct {
    float p;
    uint64_t seed, offset;
    const uint64_t *rng;
} hkg_dropout_opts;

/* Dropout: out = residual + D(x), on a matrix [rows][cols]; of dy without a
 * residual it is its own backward pass.
 *   x         bf16, fp16 or fp32 (x_type), rows ldx elements apart (0 = cols)
 *   residual  NULL, or of out's type, rows ldr elements apart
 *   out       x's type or fp32 (out_type; HKG_ERR_OPTS else), rows ldo elements
 *             apart; may be x (of out's type) or residual itself, with that
 *             one's pitch, else must overlap neither (HKG_ERR_OVERLAP)
 * rows and cols below 2^31 (HKG_ERR_SIZE).
 */
int hkg_dropout(int64_t rows, int64_t cols, const void *x, int32_t x_type, int64_t ldx,
                const hkg_dropout_opts *dropout, const void *residual, int64_t ldr, void *out,
                int32_t out_type, int64_t ldo, void *stream);

/* What a product's results pass through on their way out. */
typedef struct {
    const void *bias;        /* NULL, or [N] of bias_type                        */
    int32_t bias_type;       /* the operands' type, or HKG_T_F32                 */
    int32_t activation;      /* HKG_ACT_*                                        */
    const void *residual;    /* NULL, or [M][N] of y's type                      */
    int64_t ldr;
    void *z;                 /* NULL, or [M][N] of the operands' type: receives z */
    int64_t ldz;
    hkg_dropout_opts dropout;
} hkg_epilogue;

/*
 * Linear layer:  z = x W^T + bias,  y = residual + D(act(z)).
 *   type      of x [M][K] and W [N][K]: HKG_T_BF16 or HKG_T_F16
 *   epilogue  NULL: y = x W^T
 *   y         [M][N] of `type` or fp32 (y_type), rows ldy elements apart; may be
 *             the residual itself (the same pitch), else must not overlap it
 * 2^24 tiles of 128 x 128 results, and M or N of 2^31, are refused (HKG_ERR_SIZE).
 * Sums and everything after them are fp32; y and z are each rounded once (z is
 * rounded to be kept, act takes it unrounded).  K == 0 is z = bias.
 */
int64_t hkg_linear_workspace_bytes(int64_t M, int64_t N, int64_t K);
int hkg_linear(int64_t M, int64_t N, int64_t K, int32_t type, const void *x, int64_t ldx,
               const void *W, int64_t ldw, const hkg_epilogue *epilogue, void *y, int32_t y_type,
               int64_t ldy, void *workspace, int64_t workspace_bytes, void *stream);

/*
 * Its gradients, from dy and the z that the forward pass kept:
 *   dz = D(dy) act'(z),  dx = dz W,  dw = dz^T x,  dbias = sums of dz over rows
 * (the residual's gradient is dy itself).  The operands of the two products are of
 * `type`, so dz is rounded to it for them; dbias sums dz unrounded, in a fixed order.
 * fp16 holds no number beyond 65504: a larger dz, dx or dw (or y or z of the forward
 * pass) becomes infinity, and dz below 2^-25 zero, so a loss is scaled to suit it.
 *   dy          [M][N] of `type` or fp32 (dy_type), rows lddy elements apart
 *   z           of `type`; unused, and may be NULL, with HKG_ACT_NONE
 *   dropout     NULL: none
 *   dx, dw      [M][K] and [N][K] of `type`; dbias [N] fp32.  Any may be NULL;
 *               W may be NULL with dx, x with dw.  Which of them are asked for does not
 *               change the others' bits
 * M, N and K below 2^22 - 8, and together 2^23 tiles of 64 x 64 of the three matrices
 * (HKG_ERR_SIZE).
 */
int64_t hkg_linear_backward_workspace_bytes(int64_t M, int64_t N, int64_t K);
int hkg_linear_backward(int64_t M, int64_t N, int64_t K, int32_t type, const void *dy,
                        int32_t dy_type, int64_t lddy, const void *x, int64_t ldx, const void *W,
                        int64_t ldw, const void *z, int64_t ldz, int32_t activation,
                        const hkg_dropout_opts *dropout, void *dx, int64_t lddx, void *dw,
                        int64_t lddw, float *dbias, void *workspace, int64_t workspace_bytes,
                        void *stream);

#ifdef __cplusplus
}
#endif
#endif
