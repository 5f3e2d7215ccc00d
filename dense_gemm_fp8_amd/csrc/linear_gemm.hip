// linear_gemm.hip -- the tiled product of the 16-bit linear layer for gfx950: tile16.h's
// loop, and an epilogue that applies bias, activation, dropout and residual in fp32.
//
// The accumulators go to LDS as they are, and come back as runs of a row: a lane then
// holds 8 consecutive columns, so z, the residual and y are whole lines of their rows,
// one call of the generator serves a lane's 8 elements, and the code that handles 8
// elements stands in a loop instead of once for each of a lane's 256 accumulators.
//
// Bound by the matrix cores at the power-capped clock: 8192 x 4096 x 14336 with bias,
// residual and dropout 633-680 us (1.42-1.52 PFLOPS), the cores busy 82 % of the launch.
// With 64 K steps a tile instead of 224 the epilogue counts: 16384 x 14336 x 4096 with bias,
// gelu_tanh and z 1395-1614 us, busy 73 %, a tenth of it the epilogue (60 cycles of vector
// instructions an element, two stores), beside which nothing runs: a 256-tile's ring of 160
// KB of LDS leaves one workgroup a compute unit.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "epilogue.h"
#include "linear_kernels.h"
#include "tile16.h"

namespace hkg {
namespace {

// A wave's quarter of fp32 results in LDS, kRows rows at a time.
// (kRB blocks of rows, kB of columns)
template <int kRB, int kB>
struct F32Stage {
    static constexpr int kSide = 16 * kB, kUnits = 4 * kB;             // 16-byte units of a row
    static constexpr int kPasses = kRB <= 4 ? 1 : 2, kBlocks = kRB / kPasses, kRows = 16 * kBlocks;
    static constexpr int kBytes = kRows * kSide * 4;
    static constexpr int kLanes = kSide / 8;                           // lanes of a row on the way back
    // groups of a lane in a turn: what the registers hold, of which 128-tiles have 256
    static constexpr int kTurn = kB == 6 ? 3 : kB == 4 && kRB == 4 ? 2 : 4;
    static constexpr int kTurnRows = 64 * kTurn / kLanes, kTurns = kRows / kTurnRows;
    static constexpr bool kAligned = 64 % kLanes == 0;                 // a lane's groups share their columns
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

// Four accumulators to LDS: from the AGPRs of 256 and 192 tiles without a detour through
// VGPRs, for which the compiler takes two instructions an element.  The caller sees to it
// that the matrix instructions are done.
template <int kB, int kOffset>
__device__ __forceinline__ void acc_to_lds(int at, const f32x4_t &v)
{
    if constexpr (kB >= 6)
        asm volatile("ds_write_b128 %0, %1 offset:%2" ::"v"(at), "a"(v), "n"(kOffset) : "memory");
    else
        asm volatile("ds_write_b128 %0, %1 offset:%2" ::"v"(at), "v"(v), "n"(kOffset) : "memory");
}

// The rows of one matrix that a lane goes through: an address per group, moved on by
// whole turns.
template <int kRB, int kB>
struct RowPtr {
    using St = F32Stage<kRB, kB>;
    char *at[St::kAligned ? 1 : St::kTurn];
    int64_t row;                                             // bytes from row to row
    __device__ __forceinline__ void init(const void *base, int64_t ld, int bytes, int row0, int col, int lane)
    {
        row = ld * bytes;
#pragma unroll
        for (int u = 0; u < (St::kAligned ? 1 : St::kTurn); ++u)
            at[u] = static_cast<char *>(const_cast<void *>(base)) + (row0 + (64 * u + lane) / St::kLanes) * row +
                    (int64_t)(col + 8 * ((64 * u + lane) % St::kLanes)) * bytes;
    }
    __device__ __forceinline__ char *get(int u) const { return St::kAligned ? at[0] + u * (64 / St::kLanes) * row : at[u]; }
    __device__ __forceinline__ void next()
    {
#pragma unroll
        for (int u = 0; u < (St::kAligned ? 1 : St::kTurn); ++u)
            at[u] += St::kTurnRows * row;
    }
};

// Results leave with the hint that nothing reads them soon: a round of 256-tiles writes 33
// MB or more at once, which else drives the operands' panels out of the L2s (16384 x 14336
// x 4096 with bias, gelu_tanh and z 1440 us so, 1366 with it).
//
// From accumulators to results: the quarter's rows in passes of what LDS holds, a pass in
// turns of kTurn groups of 8 columns a lane.  kWhole: the quarter lies inside the matrix.
// kTrB: B is transposed, whose blocks are 16 consecutive columns, and the product is one of
// the gradients', whose results go out as they are in 16 bits.
template <class T, int kRB, int kB, bool kWhole, bool kTrB>
struct Epilogue {
    using St = F32Stage<kRB, kB>;
    const LinearParams &p;
    char *const mine;
    const int lane, row0, col0;
    int col[St::kTurn];
    float bias[St::kTurn][8];
    RowPtr<kRB, kB> y, z, r;
    Raw8 next[St::kTurn];

    __device__ __forceinline__ int columns(int u) const { return kWhole ? 8 : hold_v(p.N - col[u]); }   // (held: else the
    // comparisons with it stay in registers for the whole loop)

    __device__ __forceinline__ Epilogue(const LinearParams &params, char *lds, int l, int r0, int c0)
        : p(params), mine(lds), lane(l), row0(r0), col0(c0)
    {
#pragma unroll
        for (int u = 0; u < St::kTurn; ++u)
            col[u] = col0 + 8 * ((64 * u + lane) % St::kLanes);
        y.init(p.y, p.ldy, !kTrB && p.y_f32 ? 4 : 2, row0, col0, lane);
        if (!kTrB && p.z)
            z.init(p.z, p.ldz, 2, row0, col0, lane);
        if (!kTrB && p.residual)
            r.init(p.residual, p.ldr, p.y_f32 ? 4 : 2, row0, col0, lane);
        if (!kTrB && p.bias)
#pragma unroll
            for (int u = 0; u < St::kTurn; ++u) {
                if (St::kAligned && u > 0) {
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        bias[u][e] = bias[0][e];
                } else if (p.bias_f32) {
                    load8_32(element_at(p.bias, col[u], 4), columns(u), bias[u]);
                } else {
                    load8_16<T>(element_at(p.bias, col[u], 2), columns(u), bias[u]);
                }
            }
    }
    // Row of group u of a turn, from the quarter's first.
    __device__ __forceinline__ int row_of(int turn, int u) const { return turn * St::kTurnRows + (64 * u + lane) / St::kLanes; }
    __device__ __forceinline__ bool inside(int turn, int u) const { return kWhole || row0 + row_of(turn, u) < p.M; }

    // The residual's values of a turn, and on to the next.
    __device__ __forceinline__ void fetch(int turn)
    {
        if (kTrB || !p.residual || turn >= St::kPasses * St::kTurns)
            return;
#pragma unroll
        for (int u = 0; u < St::kTurn; ++u)
            next[u] = load_raw8(r.get(u), inside(turn, u) ? columns(u) : 0, p.y_f32);
        r.next();
    }
    // One turn, whose rows start `local` rows into what LDS holds.
    __device__ __forceinline__ void one(const Key &key, int turn, int local)
    {
        float v[St::kTurn][8];
#pragma unroll
        for (int u = 0; u < St::kTurn; ++u) {
            const int rl = local + (64 * u + lane) / St::kLanes, first = (col[u] - col0) >> 2;
            const f32x4_t lo = *reinterpret_cast<const f32x4_t *>(mine + St::place(rl, first));
            const f32x4_t hi = *reinterpret_cast<const f32x4_t *>(mine + St::place(rl, first + 1));
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                v[u][e] = lo[e];
                v[u][4 + e] = hi[e];
            }
        }
        Raw8 now[St::kTurn];
#pragma unroll
        for (int u = 0; u < St::kTurn; ++u)
            now[u] = next[u];
        fetch(turn + 1);
        if (!kTrB && p.bias)
#pragma unroll
            for (int u = 0; u < St::kTurn; ++u)
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    v[u][e] += bias[u][e];
        if (!kTrB && p.z) {
#pragma unroll
            for (int u = 0; u < St::kTurn; ++u)
                if (inside(turn, u))
                    store8_16<T, true>(z.get(u), columns(u), v[u]);
            z.next();
        }
        if constexpr (!kTrB)
            with_evaluation(p.act, p.y_f32, [&](auto a, auto wide) __attribute__((always_inline)) {
    #pragma unroll
                for (int u = 0; u < St::kTurn; ++u)
    #pragma unroll
                    for (int e = 0; e < 8; ++e)
                        v[u][e] = act_of<decltype(a)::value, decltype(wide)::value>(v[u][e]);
            });
        if (!kTrB && p.drop.below > 0)
#pragma unroll
            for (int u = 0; u < St::kTurn; ++u)
                drop8(p.drop, key.numbers(p.row0 + row0 + row_of(turn, u), (p.col0 + col[u]) >> 3), v[u]);
        if (!kTrB && p.y_f32) {
            if (!kTrB && p.residual)
#pragma unroll
                for (int u = 0; u < St::kTurn; ++u)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const uint32_t a = now[u].a[e], b = now[u].b[e];
                        v[u][e] += __builtin_bit_cast(float, a);
                        v[u][4 + e] += __builtin_bit_cast(float, b);
                    }
            // back to where they came from, and out in whole lines: a lane's 32 bytes would be
            // two stores of half lines (16384 x 14336 x 4096 with a residual 1540 us so, 1488
            // with the hint that nothing reads them soon)
#pragma unroll
            for (int u = 0; u < St::kTurn; ++u) {
                const int rl = local + (64 * u + lane) / St::kLanes, first = (col[u] - col0) >> 2;
                *reinterpret_cast<f32x4_t *>(mine + St::place(rl, first)) = f32x4_t{v[u][0], v[u][1], v[u][2], v[u][3]};
                *reinterpret_cast<f32x4_t *>(mine + St::place(rl, first + 1)) = f32x4_t{v[u][4], v[u][5], v[u][6], v[u][7]};
            }
            lanes_in_step();
#pragma unroll
            for (int u = 0; u < St::kTurn; ++u) {
                const int rl = local + (64 * u + lane) / St::kLanes, i = (64 * u + lane) % St::kLanes;
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    const int unit = half * St::kLanes + i, m = kWhole ? 4 : hold_v(p.N - col0 - 4 * unit);
                    const u32x4_t w = *reinterpret_cast<const u32x4_t *>(mine + St::place(rl, unit));
                    char *const to = y.get(u) + 16 * (half * St::kLanes - i);
                    if (!inside(turn, u))
                        continue;
                    if (m >= 4)
                        store16<true>(to, w);
                    else
                        store_tail32(to, m, Raw8{w, {0u, 0u, 0u, 0u}});
                }
            }
        } else {
            if (!kTrB && p.residual)
#pragma unroll
                for (int u = 0; u < St::kTurn; ++u)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        v[u][2 * e] += T::low(now[u].a[e]);
                        v[u][2 * e + 1] += T::high(now[u].a[e]);
                    }
#pragma unroll
            for (int u = 0; u < St::kTurn; ++u)
                if (inside(turn, u))
                    store8_16<T, true>(y.get(u), columns(u), v[u]);
        }
        y.next();
    }
    __device__ __forceinline__ void run(f32x4_t (&acc)[kRB][kB])
    {
        const Key key(p.drop);
        const int x = lane & 15, q = lane >> 4;
        int to[kB];                                          // LDS address of the lane's unit of column block j
#pragma unroll
        for (int j = 0; j < kB; ++j)                         // columns 32 (j / 2) + 8 q + 4 (j % 2) .., or 16 j + 4 q ..
            to[j] = (int)(uintptr_t)(__attribute__((address_space(3))) char *)mine +
                    St::place(x, kTrB ? 4 * j + q : 8 * (j >> 1) + 2 * q + (j & 1));
        fetch(0);
        for (int pass = 0; pass < St::kPasses; ++pass) {
            slots<St::kPasses>([&](auto which) __attribute__((always_inline)) {
                if (pass == decltype(which)::value)
                    slots<St::kBlocks>([&](auto b) __attribute__((always_inline)) {
                        constexpr int k = decltype(b)::value;
#pragma unroll
                        for (int j = 0; j < kB; ++j)
                            acc_to_lds<kB, 16 * k * St::kUnits * 16>(to[j], acc[decltype(which)::value * St::kBlocks + k][j]);
                    });
            });
            lanes_in_step();
            for (int turn = 0; turn < St::kTurns; ++turn)
                one(key, pass * St::kTurns + turn, turn * St::kTurnRows);
            lanes_in_step();                                 // the next pass overwrites these rows
        }
    }
};

// The rows from row0 on, columns from col0 on.
template <class T, bool kTrB, int kRB, int kB>
__device__ __forceinline__ void finish(const LinearParams &p, char *lds, int lane, int row0, int col0, f32x4_t (&acc)[kRB][kB])
{
    if (row0 + 16 * kRB <= p.M && col0 + 16 * kB <= p.N)
        Epilogue<T, kRB, kB, true, kTrB>(p, lds, lane, row0, col0).run(acc);
    else
        Epilogue<T, kRB, kB, false, kTrB>(p, lds, lane, row0, col0).run(acc);
}
// The last matrix instructions' results are there, for what reads them in assembly.
__device__ __forceinline__ void results_ready() { asm volatile("s_nop 15\n\ts_nop 15" ::: "memory"); }

template <int kB>
__device__ __forceinline__ void clear(f32x4_t (&acc)[kB][kB])
{
#pragma unroll
    for (int i = 0; i < kB; ++i)
#pragma unroll
        for (int j = 0; j < kB; ++j)
            acc[i][j] = f32x4_t{0.f, 0.f, 0.f, 0.f};
}

template <class T, class Mma, int kT, bool kTrA, bool kTrB>
__global__ __launch_bounds__(256, kT == 128 ? 2 : 1) void linear_tile_kernel(const TransposableOperands o, const LinearParams p)
{
    using Loop = TileLoop<Mma, kT, kTrA, kTrB>;
    constexpr int kB = Loop::kB;
    static_assert(4 * F32Stage<kB, kB>::kBytes <= Loop::kLds, "the stage fits");
    __shared__ __attribute__((aligned(1024))) char smem[Loop::kLds];
    int tm, tn;
    remap_tile(blockIdx.x, o.Gm, o.Gn, o.W, o.C, tm, tn);
    f32x4_t acc[kB][kB];
    clear(acc);
    Loop loop;
    loop.init(o, smem, tm, tn);
    loop.run(acc, o.nk);
    settle(acc);
    results_ready();
    const int row0 = tm * kT + loop.a_rows / kStepBytes, col0 = tn * kT + loop.b_rows / kStepBytes;
    barrier();   // every wave has read its last fragments
    finish<T, kTrB>(p, smem + loop.wave * F32Stage<kB, kB>::kBytes, loop.lane, row0, col0, acc);
}

// ---- 128-tiles with K over two groups of waves -------------------------------------------
// For grids of at most one tile a compute unit: four waves alone wait for their loads most of
// the time (0.6 us a K step, of which the matrix instructions take 0.25).  Eight waves, each
// group of four with half of K and a ring of its own; then wave w of group 0 gets the sums of
// rows 0 .. 31 of its quarter, wave w of group 1 those of rows 32 .. 63.
template <bool kTrA, bool kTrB>
__device__ __forceinline__ TransposableOperands part_of(const TransposableOperands &all, int first, int steps)   // of K
{
    TransposableOperands o = all;
    o.A = static_cast<const char *>(o.A) + (int64_t)first * (kTrA ? 64 * (int64_t)o.pitch_a : kStepBytes);
    o.B = static_cast<const char *>(o.B) + (int64_t)first * (kTrB ? 64 * (int64_t)o.pitch_b : kStepBytes);
    o.kb = max(min(steps * kStepBytes, all.kb - first * kStepBytes), 0);
    o.kt = max(min(steps * 64, all.kt - first * 64), 0);
    return o;
}
constexpr int kGroupLds = TileLoop<Bf16Masked, 128>::kLds;

template <class Mma, bool kTrA, bool kTrB>
struct TwoGroups {
    using Loop = TileLoop<Mma, 128, kTrA, kTrB>;
    Loop loop;
    int group;
    f32x4_t sum[2][4];

    // K steps k0 .. k0 + steps - 1 (of all.nk) of tile (tm, tn), half of them a group
    __device__ __forceinline__ void run(const TransposableOperands &all, char *smem, int tm, int tn, int k0, int steps)
    {
        group = __builtin_amdgcn_readfirstlane(threadIdx.x >> 8);
        const int each = (steps + 1) / 2, first = k0 + group * each, mine = group == 0 ? each : steps - each;
        f32x4_t acc[4][4];
        clear(acc);
        // both groups go through `each` steps, which share their barriers; past its part a
        // group's operands are zeros
        loop.init(part_of<kTrA, kTrB>(all, first, mine), smem + group * kGroupLds, tm, tn, (threadIdx.x >> 6) & 3);
        loop.run(acc, each);
        settle(acc);
        barrier();                                   // every wave has read its last fragments
        // a wave's other half to its partner: KiB (w, i, j), lane by lane
        char *const at = smem + loop.lane * 16;
        const int to = (loop.wave * 2 + (1 - group)) * 8, from = (loop.wave * 2 + group) * 8;
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                *reinterpret_cast<f32x4_t *>(at + (to + 4 * i + j) * 1024) = group == 0 ? acc[2 + i][j] : acc[i][j];
                sum[i][j] = group == 0 ? acc[i][j] : acc[2 + i][j];
            }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const f32x4_t v = *reinterpret_cast<const f32x4_t *>(at + (from + 4 * i + j) * 1024);
                sum[i][j] = group == 0 ? sum[i][j] + v : v + sum[i][j];
            }
        __syncthreads();                             // the LDS is free again
    }
};

template <class T, class Mma, bool kTrA, bool kTrB>
__global__ __launch_bounds__(512, 1) void linear_tile2_kernel(const TransposableOperands o, const LinearParams p)
{
    __shared__ __attribute__((aligned(1024))) char smem[2 * kGroupLds];
    int tm, tn;
    remap_tile(blockIdx.x, o.Gm, o.Gn, o.W, o.C, tm, tn);
    TwoGroups<Mma, kTrA, kTrB> g;
    g.run(o, smem, tm, tn, 0, o.nk);
    const int row0 = tm * 128 + g.loop.a_rows / kStepBytes + 32 * g.group, col0 = tn * 128 + g.loop.b_rows / kStepBytes;
    finish<T, kTrB>(p, smem + (4 * g.group + g.loop.wave) * F32Stage<2, 4>::kBytes, g.loop.lane, row0, col0, g.sum);
}

// ---- K over several workgroups ----------------------------------------------------------
// For grids of 128-tiles that would leave compute units idle.  Part s of a tile has K steps
// steps s .. and writes its sums in an order of its own, whole KiB a store: of a wave's
// quarter, 16 x 32 blocks (i, h), of a block the units of columns 4 (j & 1) .. in turn, of
// those lane 16 q + x's four columns 8 q + 4 (j & 1) .. of row x.
constexpr int kPartQuarter = 64 * 64;   // floats

template <bool kTrB, int kRB>
__device__ __forceinline__ void store_part(float *to, int lane, int first, const f32x4_t (&acc)[kRB][4])
{
    const int x = lane & 15, q = lane >> 4;
#pragma unroll
    for (int i = 0; i < kRB; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            // transposed B: unit 4 j + q of 4 columns instead of 8 (j / 2) + 2 q + j % 2
            const int jj = kTrB ? 2 * (j >> 1) + (q & 1) : j, qq = kTrB ? 2 * (j & 1) + (q >> 1) : q;
            *reinterpret_cast<f32x4_t *>(to + (((first + i) * 4 + jj) * 64 + 16 * qq + x) * 4) = acc[i][j];
        }
}

// kTwo: two groups of waves, as above.
template <class Mma, bool kTrA, bool kTrB, bool kTwo>
__global__ __launch_bounds__(kTwo ? 512 : 256, kTwo ? 1 : 2) void linear_part_kernel(const TransposableOperands all, int steps, float *parts)
{
    __shared__ __attribute__((aligned(1024))) char smem[kTwo ? 2 * kGroupLds : kGroupLds];
    const int tiles = all.Gm * all.Gn, split = blockIdx.x / tiles, block = blockIdx.x % tiles, k0 = split * steps;
    int tm, tn;
    remap_tile(block, all.Gm, all.Gn, all.W, all.C, tm, tn);
    float *const to = parts + ((int64_t)split * tiles + (int64_t)tm * all.Gn + tn) * (4 * kPartQuarter);
    if constexpr (kTwo) {
        TwoGroups<Mma, kTrA, kTrB> g;
        g.run(all, smem, tm, tn, k0, min(steps, all.nk - k0));
        store_part<kTrB>(to + g.loop.wave * kPartQuarter, g.loop.lane, 2 * g.group, g.sum);
    } else {
        TileLoop<Mma, 128, kTrA, kTrB> loop;
        f32x4_t acc[4][4];
        clear(acc);
        loop.init(part_of<kTrA, kTrB>(all, k0, steps), smem, tm, tn);
        loop.run(acc, min(steps, all.nk - k0));
        settle(acc);
        store_part<kTrB>(to + loop.wave * kPartQuarter, loop.lane, 0, acc);
    }
}

// A wave joins one 16 x 32 block: a lane has 8 columns of a row.
template <class T>
__global__ __launch_bounds__(256) void linear_join_kernel(const LinearParams p, int Gn, int tiles, int splits, const float *parts)
{
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, x = lane & 15, q = lane >> 4;
    const int unit = 4 * blockIdx.x + wave;                  // of tiles x 4 quarters x 8 blocks
    const int tile = unit >> 5, quarter = (unit >> 3) & 3, i = (unit >> 1) & 3, h = unit & 1;
    const int row = 128 * (tile / Gn) + 64 * (quarter >> 1) + 16 * i + x, col = 128 * (tile % Gn) + 64 * (quarter & 1) + 32 * h + 8 * q;
    const int n = row < p.M ? p.N - col : 0;
    const float *from = parts + (int64_t)tile * (4 * kPartQuarter) + quarter * kPartQuarter + ((i * 4 + 2 * h) * 64 + lane) * 4;
    const int64_t stride = (int64_t)tiles * (4 * kPartQuarter);
    if (n <= 0)
        return;
    const int ye = p.y_f32 ? 4 : 2;
    float r[8];
    if (p.residual) {
        if (p.y_f32)
            load8_32(element_at(p.residual, row * p.ldr + col, 4), n, r);
        else
            load8_16<T>(element_at(p.residual, row * p.ldr + col, 2), n, r);
    }
    f32x4_t lo = {0.f, 0.f, 0.f, 0.f}, hi = lo;
    int s = 0;
    for (; s + 4 <= splits; s += 4) {
        f32x4_t a[4], b[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            a[k] = *reinterpret_cast<const f32x4_t *>(from + (s + k) * stride);
            b[k] = *reinterpret_cast<const f32x4_t *>(from + (s + k) * stride + 256);
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            lo += a[k];
            hi += b[k];
        }
    }
    for (; s < splits; ++s) {
        lo += *reinterpret_cast<const f32x4_t *>(from + s * stride);
        hi += *reinterpret_cast<const f32x4_t *>(from + s * stride + 256);
    }
    float v[8] = {lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
    if (p.bias) {
        float b[8];
        if (p.bias_f32)
            load8_32(element_at(p.bias, col, 4), n, b);
        else
            load8_16<T>(element_at(p.bias, col, 2), n, b);
#pragma unroll
        for (int e = 0; e < 8; ++e)
            v[e] += b[e];
    }
    if (p.z)
        store8_16<T>(element_at(p.z, row * p.ldz + col, 2), n, v);
    act8(p.act, p.y_f32, v);
    if (p.drop.below > 0)
        drop8(p.drop, Key(p.drop).numbers(p.row0 + row, (p.col0 + col) >> 3), v);
    if (p.residual)
#pragma unroll
        for (int e = 0; e < 8; ++e)
            v[e] += r[e];
    char *const to = element_at(p.y, row * p.ldy + col, ye);
    if (p.y_f32)
        store8_32(to, n, v);
    else
        store8_16<T>(to, n, v);
}

TransposableOperands operands(const TileGrid &g, const LinearParams &p)
{
    TransposableOperands o = {};
    o.A = p.A;
    o.B = p.B;
    o.pitch_a = (int)(2 * p.lda);
    o.pitch_b = (int)(2 * p.ldb);
    o.kb = 2 * ((p.K + 7) & ~7);
    o.kt = p.K;
    o.rows_a = p.M;
    o.rows_b = p.N;
    o.Gm = g.Gm;
    o.Gn = g.Gn;
    o.W = g.W;
    o.C = g.C;
    o.nk = (o.kb + kStepBytes - 1) / kStepBytes;
    return o;
}

// K steps from which two groups of waves gain more than their exchange costs, in replayed graphs
// (us, one group / two).  1000 x 4096: 8 steps 9.5 / 9.4, 12 11.3 / 11.3, 16 13.0 / 13.1, 24 18.4 /
// 17.3, 64 38.5 / 33.2; 1000 x 2000: 8 10.0 / 9.2, 16 12.5 / 11.5, 64 26.6 / 26.7.  Operands with K
// along their columns gain later, a gradient dx of 1000 x 4096: 4 steps 10.1 / 11.3, 8 12.4 / 13.4,
// 12 14.8 / 16.2, 16 17.8 / 18.1, 24 22.8 / 23.0, 32 27.3 / 26.3; dw of 1000 x 4096: 8 13.2 / 14.0, 16
// 19.5 / 19.4, 32 28.8 / 27.8.
constexpr int kTwoFrom = 12;

template <class T, class Mma, bool kTrA, bool kTrB>
hipError_t tiles_of(const TileGrid &g, const LinearParams &p, hipStream_t stream)
{
    const TransposableOperands o = operands(g, p);
    const dim3 grid((unsigned)g.Gm * (unsigned)g.Gn), block(256);
    if (g.tile == 256)
        hipLaunchKernelGGL((linear_tile_kernel<T, Mma, 256, kTrA, kTrB>), grid, block, 0, stream, o, p);
    else if (g.tile == 128 && g.Gm * g.Gn <= 256 && o.nk >= kTwoFrom)
        hipLaunchKernelGGL((linear_tile2_kernel<T, Mma, kTrA, kTrB>), grid, dim3(512), 0, stream, o, p);
    else if (g.tile == 128)
        hipLaunchKernelGGL((linear_tile_kernel<T, Mma, 128, kTrA, kTrB>), grid, block, 0, stream, o, p);
    else if constexpr (!kTrA && !kTrB)
        hipLaunchKernelGGL((linear_tile_kernel<T, Mma, 192, false, false>), grid, block, 0, stream, o, p);
    else
        return hipErrorInvalidValue;
    return hipGetLastError();
}
template <class T, class Mma>
hipError_t tiles_as(const TileGrid &g, const LinearParams &p, hipStream_t stream)
{
    return p.tr_a ? tiles_of<T, Mma, true, true>(g, p, stream)
         : p.tr_b ? tiles_of<T, Mma, false, true>(g, p, stream)
                  : tiles_of<T, Mma, false, false>(g, p, stream);
}

// Parts of many steps by two groups of waves: 128 x 8192 x 8192 in 4 parts of 32 steps 40.4 us
// against 36.9, 512 x 4096 x 14336 in 2 of 112 82.9 against 76.3; of 8 steps (128 x 4096 x 4096
// in 8) 16.9 against 18.4.  1024 x 1024 in 4 parts with operands that the caches hold (one group /
// two): 16 steps 22.0 / 23.8, 32 31.8 / 34-38, 48 37.2 / 36.7, 64 45.0 / 42.3, 128 77.2 / 70.1; a
// gradient dx, with dz's pass: 32 39.2 / 43.1, 48 47.2 / 45.6, 64 57.2 / 55.6, 128 100 / 93.5; dw 32
// 39.2 / 41.8, 48 47.5 / 47.1, 64 57.9 / 56.5, 96 80 / 78, 128 101 / 103.
template <class Mma, bool kTrA, bool kTrB>
void part_launch(unsigned blocks, const TransposableOperands &o, int steps, float *parts, hipStream_t stream)
{
    if (steps >= (kTrB ? 64 : 32))
        hipLaunchKernelGGL((linear_part_kernel<Mma, kTrA, kTrB, true>), dim3(blocks), dim3(512), 0, stream, o, steps, parts);
    else
        hipLaunchKernelGGL((linear_part_kernel<Mma, kTrA, kTrB, false>), dim3(blocks), dim3(256), 0, stream, o, steps, parts);
}

template <class T, class Mma>
hipError_t split_of(const TileGrid &g, int splits, int steps, float *parts, const LinearParams &p, hipStream_t stream)
{
    const TransposableOperands o = operands(g, p);
    const int tiles = g.Gm * g.Gn;
    const unsigned blocks = (unsigned)tiles * (unsigned)splits;
    if (p.tr_a)
        part_launch<Mma, true, true>(blocks, o, steps, parts, stream);
    else if (p.tr_b)
        part_launch<Mma, false, true>(blocks, o, steps, parts, stream);
    else
        part_launch<Mma, false, false>(blocks, o, steps, parts, stream);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess)
        return e;
    hipLaunchKernelGGL(linear_join_kernel<T>, dim3(8u * (unsigned)tiles), dim3(256), 0, stream, p, g.Gn, tiles, splits, parts);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_linear_tiles(bool f16, const TileGrid &g, const LinearParams &p, hipStream_t stream)
{
    return f16 ? tiles_as<TypeF16, F16Masked>(g, p, stream) : tiles_as<TypeBf16, Bf16Masked>(g, p, stream);
}

hipError_t launch_linear_split(bool f16, const TileGrid &g, int splits, int steps, float *parts, const LinearParams &p,
                               hipStream_t stream)
{
    return f16 ? split_of<TypeF16, F16Masked>(g, splits, steps, parts, p, stream)
               : split_of<TypeBf16, Bf16Masked>(g, splits, steps, parts, p, stream);
}

}  // namespace hkg
