// mxfp4_gemm.hip -- the tiled MXFP4 product for gfx950 (tile16.h's loop with a
// bf16 epilogue).
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "ops_kernels.h"
#include "tile16.h"

namespace hkg {
namespace {

// Rows row_off .. of tile (tm, tn) from one wave's blocks: a lane owns row 16 i + x
// and, per pair of column blocks, 8 consecutive columns.  Whole tiles store 16 bytes
// through one buffer resource, edge tiles check rows and columns.
template <int kT, int kB>
__device__ __forceinline__ void store_bf16(const Mx4GemmParams &p, int tm, int tn, int row_off, int col_off, int lane,
                                           f32x4_t (&acc)[kB][kB])
{
    const int x = lane & 15, q = lane >> 4;
    const int64_t row0 = (int64_t)tm * kT + row_off, col0 = (int64_t)tn * kT + col_off;
    const bool vec = ((p.N | p.ldc) & 7) == 0;
    const bool inside = (int64_t)(tm + 1) * kT <= p.M && (int64_t)(tn + 1) * kT <= p.N && vec;
    if (inside && !p.C_f32 && (uint64_t)32 * kB * (uint64_t)p.ldc < (uint64_t(1) << 32)) {
        const __amdgpu_buffer_rsrc_t rc = buffer_of(p.C + row0 * p.ldc + col0, (uint32_t)(32 * kB) * (uint32_t)p.ldc);
        const int voff = (x * (int)p.ldc + 8 * q) * 2;
#pragma unroll
        for (int i = 0; i < kB; ++i) {
            const int soff = __builtin_amdgcn_readfirstlane((int)((uint32_t)(32 * i) * (uint32_t)p.ldc));
            settle_row(acc, i);
#pragma unroll
            for (int h = 0; h < kB / 2; ++h) {
                const f32x4_t lo = acc[i][2 * h], hi = acc[i][2 * h + 1];
                const u32x4_t v = {pack2_bf16(lo[0], lo[1]), pack2_bf16(lo[2], lo[3]), pack2_bf16(hi[0], hi[1]),
                                   pack2_bf16(hi[2], hi[3])};
                __builtin_amdgcn_raw_buffer_store_b128(v, rc, voff + 64 * h, soff, 0);
            }
        }
        return;
    }
#pragma unroll
    for (int i = 0; i < kB; ++i) {
        const int64_t m = row0 + 16 * i + x;
        settle_row(acc, i);
        if (m >= p.M)
            continue;
#pragma unroll
        for (int h = 0; h < kB / 2; ++h) {
            const f32x4_t lo = acc[i][2 * h], hi = acc[i][2 * h + 1];
            const float v[8] = {lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
            const u32x4_t w = {pack2_bf16(v[0], v[1]), pack2_bf16(v[2], v[3]), pack2_bf16(v[4], v[5]),
                               pack2_bf16(v[6], v[7])};
            const int64_t n = col0 + 32 * h + 8 * q, at = m * p.ldc + n;
            if (vec && n < p.N) {
                *reinterpret_cast<u32x4_t *>(p.C + at) = w;
                if (p.C_f32) {
                    *reinterpret_cast<f32x4_t *>(p.C_f32 + at) = lo;
                    *reinterpret_cast<f32x4_t *>(p.C_f32 + at + 4) = hi;
                }
            } else if (!vec) {
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    if (n + e < p.N) {
                        p.C[at + e] = (uint16_t)(w[e >> 1] >> (16 * (e & 1)));
                        if (p.C_f32)
                            p.C_f32[at + e] = v[e];
                    }
                }
            }
        }
    }
}

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
    store_bf16<kT>(p, tm, tn, loop.a_rows / kStepBytes, loop.b_rows / kStepBytes, loop.lane, acc);
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
