// orth_kernels.h -- launch interface between hkg_orthogonalize (orth_api.cpp) and
// its gfx950 kernels (orth_kernels.hip).  Internal to libhkg; all argument checks
// are done by the caller.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "ops_kernels.h"

namespace hkg {

// X, and its fp16 form for the products, are held times this (the step's two
// symmetric matrices as they are).
constexpr int kOrthScaleLog2 = 12;
constexpr float kOrthScale = 1 << kOrthScaleLog2;

// X in fp32 [mp][np] (multiples of 64): 16 x 32 blocks of 512 values, the blocks of 16
// rows one after the other.  Column c of row r of a block lies at 256 ((c >> 2) & 1) +
// 4 (16 (c >> 3) + r) + (c & 3): lane 16 q + x of a product's results holds row x,
// columns 8 q .. + 7, so a wave reads and writes a block as two whole KiB.
constexpr int kOrthBlock = 512;
struct OrthState {
    float *x;
    int64_t pitch;       // values of 16 rows
    int blocks;          // 32-column blocks of a row
};

struct OrthInput {
    const void *G;       // [rows][cols], rows ldg elements apart
    int64_t ldg;
    int rows, cols;
};

// C = A B^T, fp16: A [M][K], B [N][K], rows of K elements (a multiple of 64).  low: the
// rows of both hold K elements more, l (X less its fp16 form, in fp16), and C = A B^T +
// A Bl^T + Al B^T (32 x 32 blocks of a symmetric product without D only).
struct OrthProduct {
    const void *A, *B;
    int M, N, K;
    bool low;
};

// What becomes of acc = A B^T.
//   a symmetric product (a triangle of tiles), off the diagonal
//       v_ij = gamma acc + (beta + gamma (r_i + r_j)) D_ij,
//     on it v_ii = beta r_i + gamma (acc + r_i^2), which goes to diag in fp32 and
//     leaves a zero in the matrix: with D and r the off-diagonal part and the diagonal
//     of a symmetric S, and A = B = D, that is beta S + gamma S S.  D null: gamma acc.
//   an update (state.x set), with d_i = d[i] and h the fp16 form of x,
//       x <- v = acc + a x + d_i (h + t_i (x - h)), t_i = min(1, (d_i / (0.6 a))^2),
//     or, the last one, gamma v as bf16.
// Stored to straight [M] and / or transposed [N] (either null); for a triangle both are
// the same symmetric matrix.
struct OrthEpilogue {
    float gamma, beta;
    const _Float16 *D;   // [M], rows ldd elements apart, cols_d of each read
    int64_t ldd;
    int cols_d;
    const float *r;      // [cols_d]
    float *diag;         // [cols_s]
    OrthState state;
    float a;
    const float *d;      // [rows_d]
    int rows_d;
    uint16_t *straight;  // rows lds apart, cols_s columns of each are stored
    int64_t lds;
    int cols_s;
    uint16_t *transposed;
    int64_t ldt;
    int cols_t;
    int low;             // l too, so many elements behind h in straight (32 x 32 blocks only), or 0
    int last;            // the result: bf16, else fp16
};

int orth_norm_parts();   // doubles that launch_orth_norm writes
hipError_t launch_orth_norm(ElemType t, const OrthInput &p, double *partial, hipStream_t stream);
// G / (|G| + eps) to `state` (X, the transpose of G where it has more rows than
// columns), and times 2^12 as fp16 to straight [rows] and transposed [cols]; or to out
// as bf16 (state.x null).  low: l too, so many elements behind the fp16 form in the rows
// of X's own orientation, or 0.
hipError_t launch_orth_convert(ElemType t, const OrthInput &p, const double *partial, float eps, const OrthState &state,
                               void *straight, int ps, void *transposed, int pt, int low, uint16_t *out, int64_t ldo,
                               hipStream_t stream);
hipError_t launch_orth_product(int tile, const TileOrder &order, bool triangle, const OrthProduct &p,
                               const OrthEpilogue &e, hipStream_t stream);

}  // namespace hkg
