/*
 * hkg_ops.h -- C ABI of the operators around the GEMM of hkg.h: the MXFP4
 * linear layer (quantisation, product, few-token form, gradients) and the
 * orthogonalised weight update.  Same library, same conventions: device
 * pointers owned by the caller, every argument checked before the first HIP
 * call, work enqueued on `stream` and never waited for, HKG_OK or a negative
 * hkg_status returned.  Intermediate results live in a workspace that the
 * caller passes (16-byte aligned, at least the bytes the matching
 * *_workspace_bytes function returns, used until the stream has passed the
 * call, its contents undefined before and after).
 *
 * MXFP4 (OCP Microscaling Formats v1.0).  A matrix of `rows` rows of K values:
 *   codes   [rows][Kp/2] bytes, Kp = K rounded up to a multiple of 32: e2m1
 *           codes (sign, 2-bit exponent, 1-bit mantissa: 0, 0.5, 1, 1.5, 2, 3,
 *           4, 6), element k in bits 4 (k & 1) .. +3 of byte k / 2, zeros past
 *           K; 16-byte aligned
 *   scales  one E8M0 byte per 32 consecutive k of a row, in the packed order
 *           of hkg_mx_pack_scales(operand, rows, Kp) -- the order is the same
 *           for MXFP8 and MXFP4, so that function also packs the scales of
 *           MXFP4 weights that come from elsewhere;
 *           hkg_mx_packed_scale_bytes(rows, Kp) bytes, 16-byte aligned
 * K may be any number >= 0; sizes are limited as for MXFP8 (HKG_ERR_SIZE).
 *
 * Element types of x, values, gradients: HKG_T_BF16 or HKG_T_F32.  Row pitches
 * (ldx, ldc, ...) count elements, 0 = dense; rows need no alignment beyond
 * their element's (16-byte aligned rows are read and written faster).
 */
#ifndef HKG_OPS_H
#define HKG_OPS_H

#include <stdint.h>

#include "hkg.h"

#ifdef __cplusplus
extern "C" {
#endif

enum { HKG_T_BF16 = 0, HKG_T_F32 = 1 };

/* Bytes of the codes of a [rows][K] matrix: rows * (K rounded up to 32) / 2.
 * HKG_ERR_SHAPE for negative sizes, HKG_ERR_SIZE beyond the limits above. */
int64_t hkg_mxfp4_code_bytes(int64_t rows, int64_t K);

/*
 * Quantise x [rows][K] to MXFP4 along K.  For a block with largest magnitude
 * amax > 0 the scale is 2^s, s = max(floor(log2 amax) - 2, -127), and an
 * element's code is x / 2^s rounded to the nearest e2m1 value (ties to the
 * even code, magnitudes above 6 to 6).  A block of zeros has scale 1, a block
 * that holds a NaN or an infinity the NaN scale 0xFF and codes 0.  The packed
 * scales of rows past `rows` and blocks past Kp / 32 are 1.
 *   x        bf16 or fp32 (x_type), rows ldx elements apart
 *   operand  which GEMM operand the scales are packed for (HKG_MX_OPERAND_*)
 * codes and packed must not overlap x or each other (HKG_ERR_OVERLAP).
 */
int hkg_mxfp4_quantize(int32_t operand, int64_t rows, int64_t K, const void *x, int32_t x_type,
                       int64_t ldx, void *codes, void *packed, void *stream);

/*
 * The same, and in the same pass over x the MXFP4 form of x^T: a matrix of K
 * rows of `rows` values (codes_t, packed_t for operand_t), with blocks of 32
 * consecutive rows of x.  What a training step needs: an activation or weight
 * enters the forward product along K and a gradient's along its rows.
 */
int hkg_mxfp4_quantize_both(int32_t operand, int32_t operand_t, int64_t rows, int64_t K,
                            const void *x, int32_t x_type, int64_t ldx, void *codes, void *packed,
                            void *codes_t, void *packed_t, void *stream);

/*
 * The values an MXFP4 matrix stands for: values [rows][Kp] in bf16 or fp32
 * (v_type), rows ldv elements apart (0 = Kp; ldv >= Kp).  Exact in either type
 * for scales up to 2^125 (code 252, the largest that the quantiser gives); with
 * codes 253 and 254 magnitudes from 2^128 on are infinity.  A block with scale
 * 0xFF gives NaN.
 */
int hkg_mxfp4_dequantize(int32_t operand, int64_t rows, int64_t K, const void *codes,
                         const void *packed, void *values, int32_t v_type, int64_t ldv,
                         void *stream);

/*
 * MXFP4 GEMM: C[M][N] = bf16(A[M][K] * B[N][K]^T), fp32 accumulation.
 *   A, B   codes, SA, SB their packed scales (operand A resp. B)
 *   C      bf16, rows ldc elements apart (0 = N), 16-byte aligned base
 *   C_f32  NULL, or the fp32 accumulator, same pitch
 * K == 0 writes zeros, M == 0 or N == 0 is a no-op.  Outputs must not overlap
 * inputs or each other.
 */
int hkg_gemm_mxfp4(int64_t M, int64_t N, int64_t K, const void *A, const void *B, const void *SA,
                   const void *SB, void *C, float *C_f32, int64_t ldc, void *stream);

/*
 * A linear layer with MXFP4 weights: y[M][N] = bf16(Q(x)[M][K] * W[N][K]^T),
 * Q the quantisation above.  The same result as hkg_mxfp4_quantize followed by
 * hkg_gemm_mxfp4 up to the order of the fp32 sums; up to 16 rows of
 * K <= 10240 x is quantised inside the product (one launch, no workspace used).
 *   x  bf16 or fp32 (x_type), W / SW codes and packed scales (operand B)
 *   y  bf16, rows ldy elements apart (0 = N)
 */
int64_t hkg_linear_mxfp4_workspace_bytes(int64_t M, int64_t N, int64_t K);
int hkg_linear_mxfp4(int64_t M, int64_t N, int64_t K, const void *x, int32_t x_type, int64_t ldx,
                     const void *W, const void *SW, void *y, int64_t ldy, void *workspace,
                     int64_t workspace_bytes, void *stream);

/*
 * Its gradients, with the rounding of Q passed straight through:
 *   dx[M][K] = bf16(Q(dy)[M][N] * Wt[K][N]^T)
 *   dw[N][K] = bf16(Q(dy^T)[N][M] * Xt[K][M]^T)
 * where Wt and Xt are the MXFP4 forms of W^T [K][N] and x^T [K][M] (codes_t,
 * packed_t of hkg_mxfp4_quantize_both for operand B).  dy is read once.
 *   dy  bf16 or fp32 (dy_type), rows lddy elements apart (0 = N)
 *   dx, dw  bf16, 16-byte aligned, rows lddx / lddw elements apart (0 = K); either
 *           may be NULL (then its operands may be too)
 */
int64_t hkg_linear_mxfp4_backward_workspace_bytes(int64_t M, int64_t N, int64_t K);
int hkg_linear_mxfp4_backward(int64_t M, int64_t N, int64_t K, const void *dy, int32_t dy_type,
                              int64_t lddy, const void *Wt, const void *SWt, const void *Xt,
                              const void *SXt, void *dx, int64_t lddx, void *dw, int64_t lddw,
                              void *workspace, int64_t workspace_bytes, void *stream);

/*
 * The orthogonalised direction of an update (the Muon optimiser's step):
 * X = G / (|G|_F + eps), then `steps` times
 *   A = X X^T,  X <- a X + (b A + c A A) X
 * on G, or on G^T where G has more rows than columns, and out = X (bf16).  The
 * odd polynomial drives every singular value of X towards 1 while its singular
 * vectors stay.
 *   G    [rows][cols] bf16 or fp32 (g_type), rows ldg elements apart (0 = cols)
 *   out  [rows][cols] bf16, rows ldo elements apart (0 = cols); may be G itself
 *        when both are bf16 with one pitch, else must not overlap it
 *   steps 0 .. 64; eps >= 0 (a zero matrix stays zero)
 * X is held in fp32, as are the diagonals of A and of b A + c A A.  The products'
 * operands (X, and both matrices off their diagonals) are fp16, 11-bit significands,
 * their sums fp32.  A result is within 2^-8 of the exact iteration's norm, bf16's
 * largest rounding of one value, whatever the rank and the spectrum of G; 0.0017 to
 * 0.0019 of the norm for most, of which its own rounding to bf16 makes 0.0017.  This holds
 * for up to about 7 steps with a = 3.4: a step multiplies what lies outside G's singular
 * directions, fp32's rounding included, by a.  The polynomial must keep the singular
 * values of X below 15 (beyond that fp16 overflows to infinity), as the usual
 * coefficients (3.4445, -4.7750, 2.0315) do.  A NaN or an infinity in G makes every
 * element of out NaN.
 */
int64_t hkg_orthogonalize_workspace_bytes(int64_t rows, int64_t cols);
int hkg_orthogonalize(int64_t rows, int64_t cols, const void *G, int32_t g_type, int64_t ldg,
                      int32_t steps, float a, float b, float c, float eps, void *out, int64_t ldo,
                      void *workspace, int64_t workspace_bytes, void *stream);

#ifdef __cplusplus
}
#endif
#endif
