// ops_kernels.h -- launch interface between the operators' entry points
// (ops_api.cpp) and their gfx950 kernels (mxfp4_kernels.hip, mxfp4_gemm.hip).  Internal to
// libhkg; all argument checks are done by the caller.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace hkg {

enum ElemType { kElemBf16 = 0, kElemF32 = 1 };

// One quantisation pass over x [rows][K] (rows ldx elements apart).  codes_t
// null: along K only.
struct QuantParams {
    const void *x;
    int64_t ldx;
    int rows, K;
    int operand, operand_t;
    uint8_t *codes, *packed;       // [rows][Kp/2], packed scales
    uint8_t *codes_t, *packed_t;   // [K][Rp/2], packed scales of the transposed form
};
hipError_t launch_mx4_quantize(ElemType t, const QuantParams &p, hipStream_t stream);

struct DequantParams {
    const uint8_t *codes, *packed;
    void *values;
    int64_t ldv;
    int rows, kp;                  // kp: K rounded up to 32
    int operand;
};
hipError_t launch_mx4_dequantize(ElemType t, const DequantParams &p, hipStream_t stream);

// C[M][N] = A B^T of MXFP4 operands, kb = bytes of an operand row (Kp / 2).
struct Mx4GemmParams {
    const uint8_t *A, *B;          // codes; A null: quantise x inside the product
    const uint8_t *SA, *SB;        // packed scales
    const void *x;                 // [M][K] values (A null)
    int64_t ldx;
    uint16_t *C;                   // bf16
    float *C_f32;                  // or null
    int64_t ldc;
    int M, N, K, kb;
};
// K = 0: C and C_f32 are zeros, whatever the operands.
hipError_t launch_mx4_zero(const Mx4GemmParams &p, hipStream_t stream);
// K > 0 from here on.
hipError_t launch_mx4_few_rows(ElemType xt, const Mx4GemmParams &p, hipStream_t stream);
// Two products in one launch (both A's are codes).
hipError_t launch_mx4_few_rows2(const Mx4GemmParams &p, const Mx4GemmParams &p2, hipStream_t stream);

// A grid of Gm x Gn tiles and the order its workgroups walk it in (remap.h).
struct TileOrder {
    int Gm, Gn, W, C;
};
// The same product on tile x tile output tiles (256 or 128); A is codes.
hipError_t launch_mx4_tiles(int tile, const TileOrder &order, const Mx4GemmParams &p, hipStream_t stream);
// Two products in one launch, the first one's tiles first.
hipError_t launch_mx4_tiles2(int tile, const TileOrder &order, const Mx4GemmParams &p, const TileOrder &order2,
                             const Mx4GemmParams &p2, hipStream_t stream);

}  // namespace hkg
