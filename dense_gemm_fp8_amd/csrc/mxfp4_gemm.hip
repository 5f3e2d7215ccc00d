// mxfp4_gemm.hip -- the tiled MXFP4 product for gfx950 (tile16.h's loop with a
// bf16 epilogue).
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "ops_kernels.h"
#include "tile16.h"

namespace hkg {
namespace {

template <int kT>
__global__ __launch_bounds__(256, kT == 128 ? 2 : 1) void mx4_tile_kernel(const TileOperands o, const Mx4GemmParams p)
{
    using Loop = TileLoop<F4, kT>;
    __shared__ __attribute__((aligned(1024))) char smem[Loop::kLds];
    int tm, tn;
    remap_tile(blockIdx.x, o.Gm, o.Gn, o.W, o.C, tm, tn);
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
#pragma unroll
    for (int i = 0; i < kB; ++i) {
        settle_row(acc, i);
#pragma unroll
        for (int h = 0; h < kB / 2; ++h) {
            const f32x4_t lo = acc[i][2 * h], hi = acc[i][2 * h + 1];
            *st.unit(16 * i + x, 4 * h + q) = u32x4_t{pack2_bf16(lo[0], lo[1]), pack2_bf16(lo[2], lo[3]),
                                                      pack2_bf16(hi[0], hi[1]), pack2_bf16(hi[2], hi[3])};
        }
    }
    const int64_t at = row0 * p.ldc + col0;
    store_stage(st, loop.lane, p.C + at, p.ldc, p.M - row0, p.N - col0, ((p.N | p.ldc) & 7) == 0 && p.ldc < (1 << 22));
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

}  // namespace

hipError_t launch_mx4_tiles(int tile, const TileOrder &order, const Mx4GemmParams &p, hipStream_t stream)
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
