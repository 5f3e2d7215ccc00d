// mxfp4_gemm.hip -- the tiled MXFP4 product for gfx950 (tile16.h's loop with a
// bf16 epilogue).  Bound by the matrix cores at the clock the power cap leaves
// them: 16384 x 14336 x 4096 takes 442 to 472 us by the card, 4350 TFLOPS at 1.95 GHz on
// the best; a K step's 128 instructions take 2445 cycles back to back and 2630 to 2830 in
// the loop, and about a fifth of a tile's time is its first loads and its epilogue;
// 16384^3 reaches 4930 TFLOPS.  The fp32 copy leaves as single elements, which doubles
// the time (2048 x 4096 x 4096 25 and 49 us, 16384 x 14336 x 4096 456 and 940).
// 256-tiles read 2 x 128 bytes of operands per 2 x 256 x 256 x 256 operations; a
// 128-tile twice that, but four times as many of them fill a small grid: 1111 x
// 2777 x 1184 8.8 us.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "ops_kernels.h"
#include "tile16.h"

namespace hkg {
namespace {

template <int kT>
__device__ __forceinline__ void mx4_tile(const TileOperands &o, const Mx4GemmParams &p, int block, char *smem)
{
    using Loop = TileLoop<F4, kT>;
    int tm, tn;
    remap_tile(block, o.Gm, o.Gn, o.W, o.C, tm, tn);
    f32x4_t acc[Loop::kB][Loop::kB];
#pragma unroll
    for (int i = 0; i < Loop::kB; ++i)
#pragma unroll
        for (int j = 0; j < Loop::kB; ++j)
            acc[i][j] = f32x4_t{0.f, 0.f, 0.f, 0.f};
    Loop loop;
    loop.init(o, smem, tm, tn);
    loop.run(acc, o.nk);
    settle(acc);
    // a lane owns row 16 i + x of block row i and, per pair of blocks, 8 consecutive columns
    constexpr int kB = Loop::kB;
    const int x = loop.lane & 15, q = loop.lane >> 4;
    const int row0 = tm * kT + loop.a_rows / kStepBytes, col0 = tn * kT + loop.b_rows / kStepBytes;
    barrier();   // every wave has read its last fragments
    const Stage<kB> st(smem, loop.wave);
    const int64_t at = row0 * p.ldc + col0;
    const StageOut<kB> out(p.C, at, p.ldc, p.M - row0, p.N - col0, p.N);
#pragma unroll
    for (int i = 0; i < kB; ++i) {
        settle_row(acc, i);
#pragma unroll
        for (int h = 0; h < kB / 2; ++h) {
            const f32x4_t lo = acc[i][2 * h], hi = acc[i][2 * h + 1];
            *st.unit(16 * i + x, 4 * h + q) = u32x4_t{pack2_bf16(lo[0], lo[1]), pack2_bf16(lo[2], lo[3]),
                                                      pack2_bf16(hi[0], hi[1]), pack2_bf16(hi[2], hi[3])};
        }
        if (i > 0)
            out.rows16(st, loop.lane, 16 * (i - 1));   // while the next rows are converted
    }
    out.rows16(st, loop.lane, 16 * (kB - 1));
    out.odd_rows(st, loop.lane);
    if (!p.C_f32)
        return;
#pragma unroll
    for (int i = 0; i < kB; ++i)
#pragma unroll
        for (int j = 0; j < kB; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int r = 16 * i + x, c = 32 * (j >> 1) + 8 * q + 4 * (j & 1) + e;
                if (row0 + r < p.M && col0 + c < p.N)
                    p.C_f32[at + r * p.ldc + c] = acc[i][j][e];
            }
}

template <int kT>
__global__ __launch_bounds__(256, kT == 128 ? 2 : 1) void mx4_tile_kernel(const TileOperands o, const Mx4GemmParams p)
{
    __shared__ __attribute__((aligned(1024))) char smem[TileLoop<F4, kT>::kLds];
    mx4_tile<kT>(o, p, blockIdx.x, smem);
}

// Two products: the first `first` workgroups (a multiple of 8: both orders count on the
// workgroups of one b mod 8 sharing an XCD) are product 0's tiles, padded, the rest product 1's.
struct TilePair {
    TileOperands o[2];
    Mx4GemmParams p[2];
    int first;
};
template <int kT>
__global__ __launch_bounds__(256, kT == 128 ? 2 : 1) void mx4_tile_pair_kernel(const TilePair t)
{
    __shared__ __attribute__((aligned(1024))) char smem[TileLoop<F4, kT>::kLds];
    const int which = (int)blockIdx.x >= t.first, block = blockIdx.x - (which ? t.first : 0);
    const TileOperands o = t.o[which];
    if (block < o.Gm * o.Gn)
        mx4_tile<kT>(o, t.p[which], block, smem);
}

}  // namespace

static TileOperands operands(const TileOrder &order, const Mx4GemmParams &p)
{
    TileOperands o = {};
    o.A = p.A;
    o.B = p.B;
    o.pitch_a = o.pitch_b = o.kb = p.kb;
    o.rows_a = p.M;
    o.rows_b = p.N;
    o.Gm = order.Gm;
    o.Gn = order.Gn;
    o.W = order.W;
    o.C = order.C;
    o.nk = (p.kb + kStepBytes - 1) / kStepBytes;
    o.SA = p.SA;
    o.SB = p.SB;
    const int64_t steps = (p.kb + 63) / 64;
    o.sa_bytes = (int)((p.M + 127) / 128 * steps * kMxStepScales);
    o.sb_bytes = (int)((p.N + 127) / 128 * steps * kMxStepScales);
    return o;
}

hipError_t launch_mx4_tiles2(int tile, const TileOrder &order, const Mx4GemmParams &p, const TileOrder &order2,
                             const Mx4GemmParams &p2, hipStream_t stream)
{
    TilePair t = {{operands(order, p), operands(order2, p2)}, {p, p2}, (order.Gm * order.Gn + 7) / 8 * 8};
    const dim3 grid((unsigned)t.first + (unsigned)order2.Gm * (unsigned)order2.Gn), block(256);
    if (tile == 256)
        hipLaunchKernelGGL(mx4_tile_pair_kernel<256>, grid, block, 0, stream, t);
    else if (tile == 128)
        hipLaunchKernelGGL(mx4_tile_pair_kernel<128>, grid, block, 0, stream, t);
    else
        return hipErrorInvalidValue;
    return hipGetLastError();
}

hipError_t launch_mx4_tiles(int tile, const TileOrder &order, const Mx4GemmParams &p, hipStream_t stream)
{
    const TileOperands o = operands(order, p);
    const dim3 grid((unsigned)order.Gm * (unsigned)order.Gn), block(256);
    if (tile == 256)
        hipLaunchKernelGGL(mx4_tile_kernel<256>, grid, block, 0, stream, o, p);
    else if (tile == 128)
        hipLaunchKernelGGL(mx4_tile_kernel<128>, grid, block, 0, stream, o, p);
    else
        return hipErrorInvalidValue;
    return hipGetLastError();
}

}  // namespace hkg
