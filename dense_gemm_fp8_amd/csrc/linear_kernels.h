// linear_kernels.h -- launch interface between the entry points of hkg_linear.h
// (linear_api.cpp) and their gfx950 kernels (linear_kernels.hip; tiles and products
// split along K: linear_gemm.hip).  Internal to libhkg; all argument checks are done by the
// caller.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace hkg {

enum Activation { kActNone = 0, kActRelu = 1, kActGelu = 2, kActGeluTanh = 3, kActSilu = 4 };

struct DropoutParams {
    uint32_t below;                // 65536 q: numbers below it drop; 0: no dropout
    float scale;                   // 1 / (1 - q)
    uint64_t seed, offset;
    const uint64_t *rng;           // device {seed, offset} instead, or null
};

struct DropoutCall {
    const void *x, *residual;      // residual may be null
    void *out;
    int64_t ldx, ldr, ldo;
    int rows, cols;
    DropoutParams drop;
};
// x_bits, out_bits: 16 or 32; f16: the 16-bit type is fp16, else bf16
hipError_t launch_dropout(bool f16, int x_bits, int out_bits, const DropoutCall &p, hipStream_t stream);

// y[M][N] = residual + D(act(A B^T + bias)), A [M][K] and B [N][K] of a 16-bit type; or,
// transposed, A [K][M] and B [K][N] (tiles only).
struct LinearParams {
    const uint16_t *A, *B;
    bool tr_a, tr_b;
    int64_t lda, ldb;
    int M, N, K;
    const void *bias, *residual;   // may be null
    void *y, *z;                   // z may be null
    int64_t ldr, ldy, ldz;
    int bias_f32, y_f32;           // else of the 16-bit type
    int act;
    DropoutParams drop;
    int row0, col0;                // place of [0][0] in the whole result, for dropout; col0 % 8 == 0
};
// Rows m .. m + rows - 1 and columns n .. n + cols - 1 of a product.
inline LinearParams linear_part(const LinearParams &p, int64_t m, int64_t rows, int64_t n, int64_t cols)
{
    LinearParams q = p;
    const int64_t e = p.y_f32 ? 4 : 2;
    q.M = (int)rows;
    q.N = (int)cols;
    q.row0 = p.row0 + (int)m;
    q.col0 = p.col0 + (int)n;
    q.A = p.A + m * (p.tr_a ? 1 : p.lda);
    q.B = p.B + n * (p.tr_b ? 1 : p.ldb);
    q.bias = p.bias ? static_cast<const char *>(p.bias) + n * (p.bias_f32 ? 4 : 2) : nullptr;
    q.residual = p.residual ? static_cast<const char *>(p.residual) + (m * p.ldr + n) * e : nullptr;
    q.y = static_cast<char *>(p.y) + (m * p.ldy + n) * e;
    q.z = p.z ? static_cast<char *>(p.z) + (m * p.ldz + n) * 2 : nullptr;
    return q;
}
// A grid of Gm x Gn tiles of edge `tile` (256, 192 or 128; transposed operands: 256 or 128)
// and its order (remap.h).
struct TileGrid {
    int tile, Gm, Gn, W, C;
};
// K > 0.  A transposed operand's K is p.K; beside one, an operand that is not has rows of K
// rounded up to 8 elements, zeros past K.
hipError_t launch_linear_tiles(bool f16, const TileGrid &g, const LinearParams &p, hipStream_t stream);
// The same on 128-tiles with K over `splits` workgroups a tile, `steps` K steps of 64 each
// (the last one the rest, at least one), whose sums go to `parts` (linear_parts_bytes) and
// are joined, in order, by a second kernel.
inline int64_t linear_parts_bytes(int64_t M, int64_t N, int64_t splits)
{
    return splits * ((M + 127) / 128) * ((N + 127) / 128) * 128 * 128 * 4;
}
hipError_t launch_linear_split(bool f16, const TileGrid &g, int splits, int steps, float *parts, const LinearParams &p,
                               hipStream_t stream);
// The kernel for few rows: workgroups of 16 mb rows x 16 nb columns, and about what 64 k take,
// in ns, for each 256 workgroups.  The smallest blocks whose grid still is one workgroup for
// each compute unit, since what bounds it is how much each unit has in flight; one column
// block and long runs always for up to 16 rows.  Replayed graphs over weights in turn, us, for
// mb, nb and the 32-k steps of a run = 122 / 114: 1 x 4096 x 4096 11.5 / 7.6, 1 x 14336 x 4096
// 26.0 / 23.3, 16 x 8192 x 8192 33.6 / 28.6; 222 / 212: 32 x 4096 x 4096 13.9 / 10.3, 32 x 14336 x
// 4096 29.2 / 32.7; 422 / 412: 64 x 4096 x 4096 16.7 / 13.5, 64 x 8192 x 8192 39.0 / 46.0.
struct RowsGrid {
    int mb, nb, step_ns;
    int64_t blocks(int64_t M, int64_t N) const { return (M + 16 * mb - 1) / (16 * mb) * ((N + 16 * nb - 1) / (16 * nb)); }
};
inline RowsGrid rows_grid(int64_t M, int64_t N)
{
    constexpr RowsGrid one = {1, 1, 130}, small = {2, 1, 130}, wide = {2, 2, 200}, tall = {4, 1, 180}, large = {4, 2, 240};
    if (M <= 16)
        return one;
    if (small.blocks(M, N) <= 256)
        return small;
    if (M <= 32)
        return wide;
    return tall.blocks(M, N) <= 256 ? tall : large;
}
hipError_t launch_linear_few_rows(bool f16, const LinearParams &p, hipStream_t stream);

// Two products (either may have M = 0) in blocks of grid `g`, 16 rows as 32, and unless dbias
// is null launch_linear_bias_sum, in one launch (of at most 2^22 workgroups).
hipError_t launch_linear_few_rows2(bool f16, const RowsGrid &g, const LinearParams &p, const LinearParams &p2, const float *sums, int groups, int N,
                                   float *dbias, hipStream_t stream);

// What the gradients' products read, formed in one pass (any output may be null):
//   dz  [M][Np] and dzt [N][Mp]   dz and its transpose, zeros past N and M
//   wt  [K][Np], xt [K][Mp]       the transposes of W [N][K] and x [M][K]
//   sums [ceil(M / 64)][N]        fp32 column sums of 64 rows of dz each
// Np, Mp: N and M rounded up to 8.
struct PrepareParams {
    const void *dy, *z, *x, *W;
    int64_t lddy, ldz, ldx, ldw;
    uint16_t *dz, *dzt, *wt, *xt;
    float *sums;
    int M, N, K;
    int dy_f32, act;
    DropoutParams drop;
};
hipError_t launch_linear_prepare(bool f16, const PrepareParams &p, hipStream_t stream);
// dbias[N] = the sum of `groups` rows of sums
hipError_t launch_linear_bias_sum(const float *sums, int groups, int N, float *dbias, hipStream_t stream);

}  // namespace hkg
