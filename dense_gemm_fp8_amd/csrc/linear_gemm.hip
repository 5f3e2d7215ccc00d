// linear_gemm.hip -- the tiled product of the 16-bit linear layer for gfx950: tile16.h's
// loop, and an epilogue that applies bias, activation, dropout and residual in fp32.
//
// The accumulators go to LDS as they are, and come back as runs of a row: a lane then
// holds 8 consecutive columns, so z, the residual and y are whole lines of their rows,
// one call of the generator serves a lane's 8 elements, and the code that handles 8
// elements stands in a loop instead of once for each of a lane's 256 accumulators.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "epilogue.h"
#include "linear_kernels.h"
#include "tile16.h"

namespace hkg {
namespace {

// A wave's quarter of fp32 results in LDS, kRows rows at a time.
template <int kB>
struct F32Stage {
    static constexpr int kSide = 16 * kB, kUnits = 4 * kB;             // 16-byte units of a row
    static constexpr int kPasses = kB == 4 ? 1 : 2, kBlocks = kB / kPasses, kRows = 16 * kBlocks;
    static constexpr int kBytes = kRows * kSide * 4;
    static constexpr int kLanes = kSide / 8;                           // lanes of a row on the way back
    static constexpr int kTurn = kB == 6 ? 3 : 4;                      // groups of a lane in a turn
    static constexpr int kTurnRows = 64 * kTurn / kLanes, kTurns = kRows / kTurnRows;
    static_assert(64 * kTurn % kLanes == 0 && kRows % kTurnRows == 0, "whole turns");
    // Where unit u of a row is: permuted so that 16 lanes with one unit of 16 rows, and 16
    // lanes with every other unit of one or two rows, meet different slots of the 256-byte
    // bank line.
    __device__ __forceinline__ static int place(int row, int u)
    {
        const int at = kB == 8 ? u ^ (row & 15) ^ (u >> 4) : kB == 6 ? u ^ ((row >> 1) & 7) : u ^ (row & 15);
        return (row * kUnits + at) * 16;
    }
};

// Raw residual values of 8 columns, 16 or 32 bits each.
struct Raw8 {
    u32x4_t a, b;
};

template <class T, class Mma, int kT>
__device__ __forceinline__ void linear_tile(const TileOperands &o, const LinearParams &p, int block, char *smem)
{
    using Loop = TileLoop<Mma, kT>;
    constexpr int kB = Loop::kB;
    using St = F32Stage<kB>;
    static_assert(4 * St::kBytes <= Loop::kLds, "the stage fits");
    int tm, tn;
    remap_tile(block, o.Gm, o.Gn, o.W, o.C, tm, tn);
    f32x4_t acc[kB][kB];
#pragma unroll
    for (int i = 0; i < kB; ++i)
#pragma unroll
        for (int j = 0; j < kB; ++j)
            acc[i][j] = f32x4_t{0.f, 0.f, 0.f, 0.f};
    Loop loop;
    loop.init(o, smem, tm, tn);
    loop.run(acc, o.nk);
    settle(acc);
    const int lane = loop.lane, x = lane & 15, q = lane >> 4;
    const int row0 = tm * kT + loop.a_rows / kStepBytes, col0 = tn * kT + loop.b_rows / kStepBytes;
    const int ye = p.y_f32 ? 4 : 2;
    // group u of a turn: 8 columns of one row
    int lrow[St::kTurn], col[St::kTurn], n[St::kTurn];
    float bias[St::kTurn][8];
#pragma unroll
    for (int u = 0; u < St::kTurn; ++u) {
        lrow[u] = (64 * u + lane) / St::kLanes;
        col[u] = col0 + 8 * ((64 * u + lane) % St::kLanes);
        n[u] = p.N - col[u];
        if (!p.bias) {
#pragma unroll
            for (int e = 0; e < 8; ++e)
                bias[u][e] = 0.0f;
        } else if (p.bias_f32) {
            load8_32(element_at(p.bias, col[u], 4), n[u], bias[u]);
        } else {
            load8_16<T>(element_at(p.bias, col[u], 2), n[u], bias[u]);
        }
    }
    const Key key(p.drop);
    char *const mine = smem + loop.wave * St::kBytes;
    barrier();   // every wave has read its last fragments
#pragma unroll
    for (int pass = 0; pass < St::kPasses; ++pass) {
        const int top = row0 + pass * St::kRows;
#pragma unroll
        for (int b = 0; b < St::kBlocks; ++b) {
            const int i = pass * St::kBlocks + b;
            settle_row(acc, i);
#pragma unroll
            for (int j = 0; j < kB; ++j)   // columns 32 (j / 2) + 8 q + 4 (j % 2) ..
                *reinterpret_cast<f32x4_t *>(mine + St::place(16 * b + x, 8 * (j >> 1) + 2 * q + (j & 1))) = acc[i][j];
        }
        lanes_in_step();
        auto fetch = [&](int turn, int u) __attribute__((always_inline)) {
            Raw8 r = {{0u, 0u, 0u, 0u}, {0u, 0u, 0u, 0u}};
            const int row = top + turn * St::kTurnRows + lrow[u];
            const int m = hold_v(n[u]);   // else the comparisons below are kept in registers for the whole loop
            if (!p.residual || turn >= St::kTurns || row >= p.M || m <= 0)
                return r;
            const char *const from = element_at(p.residual, row * p.ldr + col[u], ye);
            if (m >= 8) {
                r.a = load16(from);
                if (p.y_f32)
                    r.b = load16(from + 16);
            } else {
#pragma unroll
                for (int e = 0; e < 7; ++e)
                    if (e < m) {
                        if (p.y_f32)
                            (e < 4 ? r.a : r.b)[e & 3] = reinterpret_cast<const uint32_t *>(from)[e];
                        else
                            r.a[e >> 1] |= (uint32_t)reinterpret_cast<const uint16_t *>(from)[e] << (16 * (e & 1));
                    }
            }
            return r;
        };
        Raw8 next[St::kTurn];
#pragma unroll
        for (int u = 0; u < St::kTurn; ++u)
            next[u] = fetch(0, u);
        for (int turn = 0; turn < St::kTurns; ++turn) {
            float v[St::kTurn][8];
            Raw8 now[St::kTurn];
#pragma unroll
            for (int u = 0; u < St::kTurn; ++u) {
                const int r = turn * St::kTurnRows + lrow[u], first = (col[u] - col0) >> 2;
                const f32x4_t lo = *reinterpret_cast<const f32x4_t *>(mine + St::place(r, first));
                const f32x4_t hi = *reinterpret_cast<const f32x4_t *>(mine + St::place(r, first + 1));
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    v[u][e] = lo[e] + bias[u][e];
                    v[u][4 + e] = hi[e] + bias[u][4 + e];
                }
                now[u] = next[u];
            }
#pragma unroll
            for (int u = 0; u < St::kTurn; ++u)
                next[u] = fetch(turn + 1, u);
            if (p.z)
#pragma unroll
                for (int u = 0; u < St::kTurn; ++u) {
                    const int row = top + turn * St::kTurnRows + lrow[u];
                    if (row < p.M)
                        store8_16<T>(element_at(p.z, row * p.ldz + col[u], 2), hold_v(n[u]), v[u]);
                }
            with_activation(p.act, [&](auto a) __attribute__((always_inline)) {
#pragma unroll
                for (int u = 0; u < St::kTurn; ++u)
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        v[u][e] = act_of<decltype(a)::value>(v[u][e]);
            });
            if (p.drop.below > 0)
#pragma unroll
                for (int u = 0; u < St::kTurn; ++u)
                    drop8(p.drop, key.numbers(p.row0 + top + turn * St::kTurnRows + lrow[u], (p.col0 + col[u]) >> 3), v[u]);
#pragma unroll
            for (int u = 0; u < St::kTurn; ++u) {
                const int row = top + turn * St::kTurnRows + lrow[u];
                if (row >= p.M)
                    continue;
                const int m = hold_v(n[u]);
                char *const to = element_at(p.y, row * p.ldy + col[u], ye);
                if (p.y_f32) {
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const uint32_t a = now[u].a[e], b = now[u].b[e];
                        v[u][e] += __builtin_bit_cast(float, a);
                        v[u][4 + e] += __builtin_bit_cast(float, b);
                    }
                    store8_32(to, m, v[u]);
                } else {
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        v[u][2 * e] += T::low(now[u].a[e]);
                        v[u][2 * e + 1] += T::high(now[u].a[e]);
                    }
                    store8_16<T>(to, m, v[u]);
                }
            }
        }
        lanes_in_step();   // the next pass overwrites these rows
    }
}

template <class T, class Mma, int kT>
__global__ __launch_bounds__(256, kT == 128 ? 2 : 1) void linear_tile_kernel(const TileOperands o, const LinearParams p)
{
    __shared__ __attribute__((aligned(1024))) char smem[TileLoop<Mma, kT>::kLds];
    linear_tile<T, Mma, kT>(o, p, blockIdx.x, smem);
}

TileOperands operands(const TileGrid &g, const LinearParams &p)
{
    TileOperands o = {};
    o.A = p.A;
    o.B = p.B;
    o.pitch_a = (int)(2 * p.lda);
    o.pitch_b = (int)(2 * p.ldb);
    o.kb = 2 * p.K;
    o.rows_a = p.M;
    o.rows_b = p.N;
    o.Gm = g.Gm;
    o.Gn = g.Gn;
    o.W = g.W;
    o.C = g.C;
    o.nk = (o.kb + kStepBytes - 1) / kStepBytes;
    return o;
}

template <class T, class Mma>
hipError_t tiles_of(const TileGrid &g, const LinearParams &p, hipStream_t stream)
{
    const TileOperands o = operands(g, p);
    const dim3 grid((unsigned)g.Gm * (unsigned)g.Gn), block(256);
    if (g.tile == 256)
        hipLaunchKernelGGL((linear_tile_kernel<T, Mma, 256>), grid, block, 0, stream, o, p);
    else if (g.tile == 192)
        hipLaunchKernelGGL((linear_tile_kernel<T, Mma, 192>), grid, block, 0, stream, o, p);
    else
        hipLaunchKernelGGL((linear_tile_kernel<T, Mma, 128>), grid, block, 0, stream, o, p);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_linear_tiles(bool f16, const TileGrid &g, const LinearParams &p, hipStream_t stream)
{
    return f16 ? tiles_of<TypeF16, F16Masked>(g, p, stream) : tiles_of<TypeBf16, Bf16Masked>(g, p, stream);
}

}  // namespace hkg
