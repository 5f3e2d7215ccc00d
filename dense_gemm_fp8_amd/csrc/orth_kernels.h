// orth_kernels.h -- launch interface between hkg_orthogonalize (orth_api.cpp) and
// its gfx950 kernels (orth_kernels.hip).  Internal to libhkg; all argument checks
// are done by the caller.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "ops_kernels.h"

namespace hkg {

// X is held as fp16 times this (the step's two symmetric matrices as they are).
constexpr int kOrthScaleLog2 = 12;
constexpr float kOrthScale = 1 << kOrthScaleLog2;

struct OrthInput {
    const void *G;       // [rows][cols], rows ldg elements apart
    int64_t ldg;
    int rows, cols;
};

// C = A B^T, fp16: A [M][K], B [N][K], rows of K elements (a multiple of 64).
struct OrthProduct {
    const void *A, *B;
    int M, N, K;
};

// v = alpha (A B^T) + beta D + diag I, to straight [M] and / or transposed [N] (either
// null).  With a triangle of tiles both are the same symmetric matrix.
struct OrthEpilogue {
    float alpha, beta, diag;
    const _Float16 *D;   // [M], rows ldd elements apart, cols_d of each read, or null
    int64_t ldd;
    int cols_d;
    uint16_t *straight;  // rows lds apart, cols_s columns of each are stored
    int64_t lds;
    int cols_s;
    uint16_t *transposed;
    int64_t ldt;
    int cols_t;
    int bf16;            // stored as bf16 (the result), else fp16
};

int orth_norm_parts();   // doubles that launch_orth_norm writes
hipError_t launch_orth_norm(ElemType t, const OrthInput &p, double *partial, hipStream_t stream);
hipError_t launch_orth_convert(ElemType t, const OrthInput &p, const double *partial, float eps, void *straight, int ps,
                               void *transposed, int pt, uint16_t *out, int64_t ldo, hipStream_t stream);
hipError_t launch_orth_product(int tile, const TileOrder &order, bool triangle, const OrthProduct &p,
                               const OrthEpilogue &e, hipStream_t stream);

}  // namespace hkg
