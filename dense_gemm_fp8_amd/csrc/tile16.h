// tile16.h -- the tiled product loop of the operators' kernels: C = A B^T for
// operands whose matrix-instruction fragment is 16 bytes a lane, MXFP4 (32 e2m1
// elements with a block scale), fp16 and bf16 (8 elements).
//
// One workgroup of 4 waves computes a kT x kT tile (kT = 256, 192 or 128), wave
// w the quarter (w >> 1, w & 1): kB x kB blocks of 16 x 16, kB = kT / 32.  The K
// loop is the 4-wave interleave that the GEMM of gemm_kernels.hip uses, with the
// same LDS ring and slot order; it stands apart because that file's code is what
// the committed counters were measured on, and because these operands need block
// scales per half step, and epilogues of their own.
//
// A K step is 128 bytes of every row.  LDS: A ring of 2 panels, B ring of 3, a
// panel kT rows x 128 bytes (160 KiB at kT = 256).  Half h of a step runs the
// kB^2 matrix instructions on bytes 64 h .. 64 h + 63 of each row:
//   half 0 of step t: loads B(t+2); reads the fragments of half 1 from LDS
//   barrier:          loads of step t+1 have landed, reads of A(t) are back
//   half 1 of step t: loads A(t+2) over A(t); reads half 0 of step t+1
// Each load and read sits after a fixed matrix instruction (sched_barrier after
// every one), so a wave -- the only one on its SIMD at kT = 256 -- keeps the
// matrix core fed while they issue.
//
// A row's eight 16-byte chunks of a panel are stored permuted, chunk c in slot c ^
// swz(r): the 16 rows that a fragment read touches then fall into 16 different
// 16-byte slots of the 256-byte bank line.  The permutation is applied to the
// address each lane loads from, since a load to LDS writes lane l's bytes at l * 16.
// The 16 x 16 instruction: 32 x 32 ones take 16.2 cycles instead of 19.0 for the same
// work back to back and raise the cores' share of busy cycles (fp16 192-tiles 69 to 75
// %), but the power-capped clock falls by more (1.82 to 1.56 GHz): 16384 x 14336 x
// 4096 e2m1 465 to 504 us, measured both ways.
// B's rows are handed to the matrix instruction in the order 32 (j >> 1) + 4 (j & 1)
// + (x & 3) + 8 (x >> 2), as its first operand, so that a lane's results for two
// blocks are 8 consecutive columns of one row of C.
//
// Transposed operands (kTrA, kTrB; 16-bit types, kT = 256 or 128): an operand may also be
// held with K along its rows, [K][rows], as the gradients' products meet x, W and dz.  A
// panel is then 64 rows of K by 2 kT bytes, loaded as it lies, and a fragment is two
// ds_read_b64_tr_b16: of 16 lanes, lane 4 r + c addresses 4 columns of row r, and lane i
// receives column i of the four rows.  B's blocks are 16 consecutive columns then.  A
// row's 16-byte chunks are permuted by an even number, 2 ((k & 3) + 4 (k >> 3 & 1)): the
// 8 rows x 32 bytes that half a wave reads at once fill the 256-byte bank line.  Every step
// has a buffer of its own, so that an operand's offsets may pass 32 bits; rows past K read
// as zeros, being past its range.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>
#include <utility>

#include "mx4.h"
#include "remap.h"

namespace hkg {

constexpr int kStepBytes = 128;                  // one K step of one row
constexpr int kLoadBytes = 1024;                 // one wave-wide load to LDS: 8 rows

typedef _Float16 f16x8_t __attribute__((ext_vector_type(8)));
typedef _Float16 f16x2_t __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));

// Slot permutations: A's fragment reads vary row bits 1, 2, 3 within 16 lanes
// (rows 16 i + x), B's bits 1, 3, 4; two rows share a bank line.
__device__ __forceinline__ int swz_a(int r)
{
    return ((r >> 1) & 1) | (((r >> 3) & 1) << 1) | (((r >> 2) & 1) << 2);
}
__device__ __forceinline__ int swz_b(int r)
{
    return ((r >> 1) & 1) | (((r >> 3) & 1) << 1) | (((r >> 4) & 1) << 2);
}

template <int N>
__device__ __forceinline__ void wait_loads()
{
    asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
}
__device__ __forceinline__ void wait_lds() { asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory"); }
__device__ __forceinline__ void barrier() { asm volatile("s_barrier" ::: "memory"); }
// Between LDS accesses of a wave's own lanes: the hardware keeps them in order, and this
// keeps the compiler from moving one lane's read over another lane's write.  No
// instruction of its own.
__device__ __forceinline__ void lanes_in_step()
{
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

// Empty asm statements that keep a value where it is formed: `hold_v` stops the
// compiler from folding a panel offset into one precomputed address per read,
// `hold_s` keeps scalar bookkeeping in its slot of the loop (plain arithmetic
// drifts and bunches up, which delays the next matrix instruction).
__device__ __forceinline__ int hold_v(int x)
{
    asm volatile("" : "+v"(x));
    return x;
}
__device__ __forceinline__ int hold_s(int x)
{
    asm volatile("" : "+s"(x));
    return x;
}
__device__ __forceinline__ uint32_t copy_v(uint32_t x)
{
    uint32_t y;
    asm volatile("v_mov_b32 %0, %1" : "=v"(y) : "v"(x));
    return y;
}
__device__ __forceinline__ int copy_s(int x)
{
    int y;
    asm volatile("s_mov_b32 %0, %1" : "=s"(y) : "s"(x));
    return y;
}

// From a panel's first row to the last of its `rows` rows' kb bytes: what lies
// past them reads as zeros.
__device__ __forceinline__ uint32_t panel_range(int rows, int pitch, int kb)
{
    return rows > 0 ? (uint32_t)(rows - 1) * (uint32_t)pitch + (uint32_t)kb : 0u;
}

template <class F, int... kN>
__device__ __forceinline__ void slots_seq(F &&f, std::integer_sequence<int, kN...>)
{
    (f(std::integral_constant<int, kN>{}), ...);
}
template <int kN, class F>
__device__ __forceinline__ void slots(F &&f)   // f(0) .. f(kN - 1), the number a constant in each
{
    slots_seq(f, std::make_integer_sequence<int, kN>{});
}

// Operands of one launch.
struct TileOperands {
    const void *A, *B;           // rows pitch_a / pitch_b bytes apart, kb bytes of K each
    int pitch_a, pitch_b, kb;
    int rows_a, rows_b;          // rows that exist (M, N)
    int Gm, Gn, W, C;            // tile grid and its order (remap.h)
    int nk;                      // K steps, ceil(kb / 128)
    int triangle;                // symmetric result: only tiles tm <= tn (grid order W, C unused)
    const void *SA, *SB;         // MXFP4: packed scales and their sizes in bytes
    int sa_bytes, sb_bytes;
};
// And where an operand may be transposed.
struct TransposableOperands : TileOperands {
    int kt;                      // rows of a transposed operand: K itself, where kb is rounded up
};

// The scales a wave needs for one K step: [half][word], byte i & 3 of word i >> 2
// for block i (kB = 8), byte i of word 0 (kB = 4).
template <int kB>
struct StepScales {
    uint32_t a[2][kB == 8 ? 2 : 1], b[2][kB == 8 ? 2 : 1];
};

// kScaled: block scales; kMasked: rows may end inside a K step (at whole 16-byte chunks).
struct F16 {
    static constexpr bool kScaled = false, kMasked = false;
    template <int kI, int kJ, int kB>
    __device__ __forceinline__ static f32x4_t mma(const u32x4_t &b, const u32x4_t &a, const f32x4_t &c,
                                                  const StepScales<kB> &, int)
    {
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8_t, b),
                                                      __builtin_bit_cast(f16x8_t, a), c, 0, 0, 0);
    }
};
struct F16Masked : F16 {
    static constexpr bool kMasked = true;
};
struct Bf16Masked {
    static constexpr bool kScaled = false, kMasked = true;
    template <int kI, int kJ, int kB>
    __device__ __forceinline__ static f32x4_t mma(const u32x4_t &b, const u32x4_t &a, const f32x4_t &c,
                                                  const StepScales<kB> &, int)
    {
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, b),
                                                       __builtin_bit_cast(bf16x8_t, a), c, 0, 0, 0);
    }
};
struct F4 {
    static constexpr bool kScaled = true, kMasked = true;
    template <int kI, int kJ, int kB>
    __device__ __forceinline__ static f32x4_t mma(const u32x4_t &b, const u32x4_t &a, const f32x4_t &c,
                                                  const StepScales<kB> &s, int half)
    {
        return mma_f4<kJ & 3, kI & 3>(b, a, c, s.b[half][kJ >> 2], s.a[half][kI >> 2]);
    }
};

// When each load, read and piece of bookkeeping issues: after matrix instruction
// number .. of a half (kB^2 of them).  A's loads (half 1) go early: their panel is
// free once the barrier is past, and they have to land before the next one.
template <int kB>
struct Plan16 {
    static constexpr int kMfmas = kB * kB;
    __device__ static constexpr int load(int h, int v)
    {
        return kB == 8   ? (h == 0 ? 8 * v + 4 : 6 * v + 1)
               : kB == 6 ? (h == 0 ? 6 * v + 3 : 4 * v + 1)
                         : (h == 0 ? 4 * v + 1 : 2 * v + 1);
    }
    __device__ static constexpr int read(int r) { return kB == 8 ? 3 * r : 2 * r; }
    static constexpr int kBaseA = kB == 8 ? 50 : kB == 6 ? 24 : 9;
    static constexpr int kBaseB = kB == 8 ? 53 : kB == 6 ? 26 : 11;
    static constexpr int kRing = kB == 8 ? 55 : kB == 6 ? 28 : 12;   // three slots from here
    static constexpr int kTail = kB == 8 ? 61 : kB == 6 ? 34 : 15;   // after the half's last load
    static constexpr int kMask = kB == 8 ? 47 : kB == 6 ? 22 : 7;
};
template <int kB>
constexpr bool plan_ok()
{
    using P = Plan16<kB>;
    bool ok = P::read(2 * kB - 1) < P::kMfmas && P::kRing + 2 < P::kTail && P::kTail < P::kMfmas &&
              P::load(0, kB - 1) < P::kMfmas && P::load(1, kB - 1) < P::kTail;
    return ok && P::kBaseA < P::kMfmas && P::kBaseB < P::kMfmas && P::kMask < P::kMfmas;
}
static_assert(plan_ok<8>() && plan_ok<6>() && plan_ok<4>(), "slot plans");

// Runs the K loop of tile (tm, tn) into acc; smem: 5 panels, nk at least 1 (its first
// loads, and those of the scales, are not guarded).  On return every load
// of this wave has landed; other waves may still be reading their last fragments.
template <class Mma, int kT, bool kTrA = false, bool kTrB = false>
struct TileLoop {
    static_assert((!kTrA && !kTrB) || kT == 256 || kT == 128, "transposed panels");
    static constexpr int kB = kT / 32;
    static constexpr int kPanel = kT * kStepBytes;
    static constexpr int kRingB = 2 * kPanel;
    static constexpr int kLds = 5 * kPanel;
    using Plan = Plan16<kB>;

    struct Frags {
        u32x4_t a[2][kB], b[2][kB];   // [half][block]
    };

    __amdgpu_buffer_rsrc_t ra, rb, rsa, rsb;
    char *smem;
    int wave, lane;
    int w_load;                    // LDS bytes of its first row group in a panel
    int a_rows, b_rows;            // LDS bytes of its rows in a panel
    int voff_a, voff_b;            // lane's load offset: its row and permuted chunk
    int cb_a, cb_b;                // byte of that chunk in a K step
    int pitch_a, pitch_b, kb;
    int la[2], lb[2];              // lane's fragment offset, per half
    int voff_ta[2], voff_tb[2];    // transposed: lane's load offset for even and odd v
    int ta[kB], tb[kB];            // and its fragment offset for each block
    int s_off_a, s_off_b, s_last;  // lane's scale byte; offset of the last 128-k step's scales

    __device__ __forceinline__ static constexpr int blk_a(int i) { return 16 * i * kStepBytes; }
    __device__ __forceinline__ static constexpr int blk_b(int j) { return (32 * (j >> 1) + 4 * (j & 1)) * kStepBytes; }

    // Transposed panels: rows of 2 kT bytes, kChunks 16-byte chunks; a wave-wide load is
    // kLoadK rows, and the waves' loads v are 4 kLoadK rows apart.
    static constexpr int kRowT = 2 * kT, kChunks = kRowT / 16, kLoadK = kLoadBytes / kRowT;
    __device__ __forceinline__ static int swz_t(int k) { return 2 * ((k & 3) | ((k >> 1) & 4)); }
    // buffer_of()'s words.
    __device__ __forceinline__ static i32x4_t resource(const char *base, uint32_t bytes)
    {
        const uint64_t at = reinterpret_cast<uint64_t>(base);
        return i32x4_t{(int)(uint32_t)at, (int)(uint32_t)(at >> 32), (int)bytes, 0x00020000};
    }
    // A transposed operand's columns of this tile (`rows` of the product's rows or columns).
    struct Columns {
        const char *base;
        int pitch, width, kt;                    // width: bytes, whole 16-byte chunks
        // The buffer of K step t.
        __device__ __forceinline__ i32x4_t step(int t) const
        {
            const int left = min(kt - 64 * t, 64);
            return resource(base + (int64_t)t * 64 * pitch, left > 0 ? panel_range(left, pitch, width) : 0u);
        }
    };
    Columns cols_a, cols_b;
    i32x4_t plain_a;                             // ra, beside a transposed B
    __device__ __forceinline__ Columns init_t(const void *base, int pitch, int rows, int kt, int tile, int half,
                                              int (&voff)[2], int (&t)[kB]) const
    {
        const int k = kLoadK * wave + lane / kChunks;
#pragma unroll
        for (int odd = 0; odd < 2; ++odd)   // rows 4 kLoadK apart: of 256-tiles bit 3 of k follows v
            voff[odd] = k * pitch + 16 * ((lane % kChunks) ^ swz_t(k + (kT == 256 ? 8 * odd : 0)));
        const int q = lane >> 4, r = (lane >> 2) & 3, c = lane & 3;
#pragma unroll
        for (int j = 0; j < kB; ++j)
            t[j] = (8 * q + r) * kRowT + 16 * (((kChunks / 2 * half + 2 * j) ^ swz_t(8 * q + r)) + (c >> 1)) + 8 * (c & 1);
        return Columns{static_cast<const char *>(base) + (int64_t)tile * kRowT, pitch, (2 * min(kT, rows - tile * kT) + 15) & ~15, kt};
    }
    template <class Operands>
    __device__ __forceinline__ void init(const Operands &p, char *lds, int tm, int tn, int of = threadIdx.x >> 6)
    {
        smem = lds;
        lane = threadIdx.x & 63;
        wave = __builtin_amdgcn_readfirstlane(of);   // of the four that share the tile
        w_load = wave * kLoadBytes;
        a_rows = (kT / 2) * (wave >> 1) * kStepBytes;
        b_rows = (kT / 2) * (wave & 1) * kStepBytes;
        pitch_a = p.pitch_a;
        pitch_b = p.pitch_b;
        kb = p.kb;
        if constexpr (kTrA)
            cols_a = init_t(p.A, pitch_a, p.rows_a, p.kt, tm, wave >> 1, voff_ta, ta);
        else
            ra = buffer_of(static_cast<const char *>(p.A) + (int64_t)tm * kT * pitch_a,
                           panel_range(min(kT, p.rows_a - tm * kT), pitch_a, kb));
        if constexpr (kTrB && !kTrA)
            plain_a = resource(static_cast<const char *>(p.A) + (int64_t)tm * kT * pitch_a,
                               panel_range(min(kT, p.rows_a - tm * kT), pitch_a, kb));
        if constexpr (kTrB)
            cols_b = init_t(p.B, pitch_b, p.rows_b, p.kt, tn, wave & 1, voff_tb, tb);
        else
            rb = buffer_of(static_cast<const char *>(p.B) + (int64_t)tn * kT * pitch_b,
                           panel_range(min(kT, p.rows_b - tn * kT), pitch_b, kb));
        // row groups u = wave + 4 v: row bits 3, 4 are the wave's for all its loads
        const int r8 = lane >> 3;
        cb_a = ((lane & 7) ^ swz_a(r8 | (wave << 3))) << 4;
        cb_b = ((lane & 7) ^ swz_b(r8 | (wave << 3))) << 4;
        voff_a = (8 * wave + r8) * pitch_a + cb_a;
        voff_b = (8 * wave + r8) * pitch_b + cb_b;
        const int x = lane & 15, q = lane >> 4, xb = (x & 3) + 8 * (x >> 2);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            la[h] = x * kStepBytes + (((4 * h + q) ^ swz_a(x)) << 4);
            lb[h] = xb * kStepBytes + (((4 * h + q) ^ swz_b(xb)) << 4);
        }
        if constexpr (Mma::kScaled) {
            // packed groups of 128 rows, n128 steps of 512 bytes each; a 128-row
            // tile's waves use bytes 0..3 or 4..7 of a lane's 8
            const int n128 = (kb + 63) / 64, span = n128 * kMxStepScales;
            const int ga = kT == 256 ? 2 * tm + (wave >> 1) : tm;
            const int gb = kT == 256 ? 2 * tn + (wave & 1) : tn;
            rsa = buffer_of(static_cast<const char *>(p.SA) + (int64_t)ga * span,
                            (int64_t)ga * span < p.sa_bytes ? span : 0);
            rsb = buffer_of(static_cast<const char *>(p.SB) + (int64_t)gb * span,
                            (int64_t)gb * span < p.sb_bytes ? span : 0);
            s_off_a = lane * 8 + (kT == 256 ? 0 : 4 * (wave >> 1));
            s_off_b = lane * 8 + (kT == 256 ? 0 : 4 * (wave & 1));
            s_last = span - kMxStepScales;
        }
    }

    // Rows 8 (wave + 4 v) .. + 7 of a panel; lds_off: the panel's place in its
    // ring, counted from the wave's first row group.
    __device__ __forceinline__ void load8rows(__amdgpu_buffer_rsrc_t rs, int lds_off, int v, int voff, int soff,
                                              int pitch) const
    {
        __builtin_amdgcn_raw_ptr_buffer_load_lds(
            rs, (__attribute__((address_space(3))) void *)(smem + lds_off + 4 * v * kLoadBytes), 16, voff,
            soff + 32 * v * pitch, 0, 0);
    }
    // Loads beside transposed operands are in assembly, which writes no register: the
    // compiler else waits for all loads to LDS before each ds_read_b64_tr_b16 (a gradient of
    // 8192 x 14336 x 4096 2600 us instead of 650), where the loop waits for those that it
    // needs.  M0 holds a load's LDS address, a wait state before it at least; nothing else
    // in these kernels writes it, which the load's statement cannot say: tests/test_linear_m0.py
    // reads it off the listing.
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"
    __device__ __forceinline__ void set_m0(int lds_off, int v) const
    {
        const int base = (int)(uintptr_t)(__attribute__((address_space(3))) char *)smem + lds_off;
        asm volatile("s_add_u32 m0, %0, %1" ::"s"(base), "s"(4 * v * kLoadBytes) : "memory", "m0", "scc");
    }
    __device__ __forceinline__ void load_m0(const i32x4_t &rs, int voff, int soff) const
    {
        asm volatile("buffer_load_dwordx4 %0, %1, %2 offen lds" ::"v"(voff), "s"(rs), "s"(soff) : "memory");
    }
#pragma clang diagnostic pop
    __device__ __forceinline__ void first_m0(int lds_off, int v) const   // before the loop
    {
        if constexpr (kTrB) {
            set_m0(lds_off, v);
            asm volatile("s_nop 0" ::: "memory");
        }
    }
    // Load v of a panel.  Transposed: loads v are 4 kLoadK rows apart in step t+2's buffer,
    // and set_m0 came before.
    __device__ __forceinline__ void load_a(int lds_off, int v, int voff, int soff, const i32x4_t &step) const
    {
        if constexpr (kTrA)
            load_m0(step, voff_ta[v & 1], 4 * kLoadK * v * pitch_a);
        else if constexpr (kTrB)
            load_m0(plain_a, voff, soff + 32 * v * pitch_a);
        else
            load8rows(ra, lds_off, v, voff, soff, pitch_a);
    }
    __device__ __forceinline__ void load_b(int lds_off, int v, int voff, int soff, const i32x4_t &step) const
    {
        if constexpr (kTrB)
            load_m0(step, voff_tb[v & 1], 4 * kLoadK * v * pitch_b);
        else
            load8rows(rb, lds_off, v, voff, soff, pitch_b);
    }
    // The fragment of a block for half h: its place `at` in the panel from `base` on.
    template <bool kTr>
    __device__ __forceinline__ u32x4_t fragment(int base, int blk, int at, int h) const
    {
        if constexpr (kTr) {
            typedef short s16x4 __attribute__((ext_vector_type(4)));
            const u32x2_t lo = __builtin_bit_cast(u32x2_t, __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                (__attribute__((address_space(3))) s16x4 *)(smem + (at + base) + 32 * h * kRowT)));
            const u32x2_t hi = __builtin_bit_cast(u32x2_t, __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                (__attribute__((address_space(3))) s16x4 *)(smem + (at + base) + (32 * h + 4) * kRowT)));
            return u32x4_t{lo[0], lo[1], hi[0], hi[1]};
        } else {
            return *reinterpret_cast<const u32x4_t *>(smem + blk + base);
        }
    }
    // What the reads of a panel (wave's first row group at `panel` of its ring) start from:
    // the lane's offset for half h, or for transposed panels the panel itself.
    template <bool kTr>
    __device__ __forceinline__ int read_base(const int (&l)[2], int h, int to_rows, int panel) const
    {
        if constexpr (kTr)
            return hold_s(panel - w_load);
        else
            return hold_v(l[h] + hold_s(to_rows + panel));
    }
    // Lane offset in a K step that starts `at` bytes into the rows: a chunk past
    // the rows' end reads zeros (kb is whole chunks).
    __device__ __forceinline__ int masked(int voff, int cb, int at) const
    {
        return at + cb < kb ? voff : kPastEnd;
    }

    // Scales of K step t.  The last K step may hold one 128-k step only; its second
    // half then takes the first half's scales, never another group's: the elements
    // there are zeros, and zero times a NaN scale of another row would be NaN.
    __device__ __forceinline__ void scales(StepScales<kB> &s, int s0, int s1) const
    {
        if constexpr (kB == 8) {
            const u32x2_t a0 = __builtin_amdgcn_raw_buffer_load_b64(rsa, s_off_a, s0, 0);
            const u32x2_t b0 = __builtin_amdgcn_raw_buffer_load_b64(rsb, s_off_b, s0, 0);
            const u32x2_t a1 = __builtin_amdgcn_raw_buffer_load_b64(rsa, s_off_a, s1, 0);
            const u32x2_t b1 = __builtin_amdgcn_raw_buffer_load_b64(rsb, s_off_b, s1, 0);
#pragma unroll
            for (int w = 0; w < 2; ++w) {
                s.a[0][w] = a0[w];
                s.b[0][w] = b0[w];
                s.a[1][w] = a1[w];
                s.b[1][w] = b1[w];
            }
        } else {
            s.a[0][0] = __builtin_amdgcn_raw_buffer_load_b32(rsa, s_off_a, s0, 0);
            s.b[0][0] = __builtin_amdgcn_raw_buffer_load_b32(rsb, s_off_b, s0, 0);
            s.a[1][0] = __builtin_amdgcn_raw_buffer_load_b32(rsa, s_off_a, s1, 0);
            s.b[1][0] = __builtin_amdgcn_raw_buffer_load_b32(rsb, s_off_b, s1, 0);
        }
    }

    // One half: its matrix instructions, after each of which load(v), the reads of
    // the other half's fragments (from LDS offsets ba, bb) and hook(n) may follow.
    // (to: where the loads go, a wave's first row group in its panel)
    template <int kH, class Load, class Hook>
    __device__ __forceinline__ void half(Frags &f, f32x4_t (&acc)[kB][kB], const StepScales<kB> &sc, int ba, int bb, int to,
                                         Load &&load, Hook &&hook) const
    {
        slots<Plan::kMfmas>([&](auto slot) __attribute__((always_inline)) {
            constexpr int n = decltype(slot)::value, i = n / kB, j = n % kB;
            if constexpr (kTrB) {
#pragma unroll
                for (int v = 0; v < kB; ++v)
                    if (Plan::load(kH, v) == n) {
                        set_m0(to, v);
                        __builtin_amdgcn_sched_barrier(0);
                    }
            }
            acc[i][j] = Mma::template mma<i, j, kB>(f.b[kH][j], f.a[kH][i], acc[i][j], sc, kH);
            if constexpr (kTrB)
                __builtin_amdgcn_sched_barrier(0);   // the instruction between M0 and the load
#pragma unroll
            for (int v = 0; v < kB; ++v)
                if (Plan::load(kH, v) == n)
                    load(v);
#pragma unroll
            for (int r = 0; r < 2 * kB; ++r) {
                if (Plan::read(r) != n)
                    continue;
                if (r < kB)
                    f.b[1 - kH][r] = fragment<kTrB>(bb, blk_b(r), tb[r], 1 - kH);
                else
                    f.a[1 - kH][r - kB] = fragment<kTrA>(ba, blk_a(r - kB), ta[r - kB], 1 - kH);
            }
            hook(slot);
            __builtin_amdgcn_sched_barrier(0);
        });
    }

    __device__ __forceinline__ void run(f32x4_t (&acc)[kB][kB], int nk)
    {
        constexpr int kHi = kB == 8;             // the last scale word
        constexpr bool kMasked = Mma::kMasked;
        StepScales<kB> sc = {};
        if constexpr (Mma::kScaled)
            scales(sc, 0, min(kMxStepScales, s_last));   // first: the wait below covers it
        // steps 0 and 1 (step 1 may be absent: what it loads is not used)
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            const int va = kMasked ? masked(voff_a, cb_a, s * kStepBytes) : voff_a;
            const int vb = kMasked ? masked(voff_b, cb_b, s * kStepBytes) : voff_b;
#pragma unroll
            for (int v = 0; v < kB; ++v) {
                first_m0(w_load + s * kPanel, v);
                load_a(w_load + s * kPanel, v, va, s * kStepBytes, kTrA ? cols_a.step(s) : i32x4_t{});
            }
#pragma unroll
            for (int v = 0; v < kB; ++v) {
                first_m0(w_load + kRingB + s * kPanel, v);
                load_b(w_load + kRingB + s * kPanel, v, vb, s * kStepBytes, kTrB ? cols_b.step(s) : i32x4_t{});
            }
        }
        wait_loads<2 * kB>();
        barrier();
        Frags f;
        {
            const int ba = kTrA ? 0 : hold_v(la[0] + a_rows), bb = kTrB ? kRingB : hold_v(lb[0] + kRingB + b_rows);
#pragma unroll
            for (int j = 0; j < kB; ++j)
                f.b[0][j] = fragment<kTrB>(bb, blk_b(j), tb[j], 0);
#pragma unroll
            for (int i = 0; i < kB; ++i)
                f.a[0][i] = fragment<kTrA>(ba, blk_a(i), ta[i], 0);
        }
        // Nothing is on its way from LDS when the loop begins: the compiler, which orders
        // the reads above as it likes, else waits at the loop's head for every read in
        // flight, the next half's among them, in all of the steps.
        __builtin_amdgcn_sched_barrier(0);
        __builtin_amdgcn_s_waitcnt(0xC07F);          // lgkmcnt(0)
        __builtin_amdgcn_sched_barrier(0);
        // LDS offsets of the wave's first row group in A(t), A(t+1), B(t), B(t+1),
        // B(t+2), and of its fragments' rows from there; K bytes of step t+2
        int pa = w_load, pa1 = pa + kPanel, pb = w_load + kRingB, pb1 = pb + kPanel, pb2 = pb1 + kPanel;
        const int fa = a_rows - w_load, fb = b_rows - w_load;
        int so = 2 * kStepBytes;
        int s_next = 2 * kMxStepScales;              // scales of step t+1
        int vb = kMasked ? masked(voff_b, cb_b, so) : voff_b;
        int ba0 = kTrA ? pa - w_load : hold_v(la[1] + fa + pa), bb0 = kTrB ? pb - w_load : hold_v(lb[1] + fb + pb);   // half 1 of step t
        for (int t = 0; t < nk; ++t) {
            StepScales<kB> next = {};
            int va = voff_a, vb_next = voff_b, ba1 = 0, bb1 = 0;
            int npa = 0, npa1 = 0, nso = 0, npb = 0, npb1 = 0, npb2 = 0;
            i32x4_t na = {}, nb = {};                    // transposed: step t+2's buffers
            if constexpr (kTrB)
                nb = cols_b.step(t + 2);
            __builtin_amdgcn_sched_barrier(0);
            half<0>(
                f, acc, sc, ba0, bb0, pb2,
                [&](int v) {
                    pb2 = hold_s(pb2);
                    if constexpr (!kTrB)
                        so = hold_s(so);
                    load_b(pb2, v, vb, so, nb);
                },
                [&](auto slot) __attribute__((always_inline)) {
                    constexpr int n = decltype(slot)::value;
                    if constexpr (Mma::kScaled && n == 0) {
                        // ahead of B's loads, which the wait below leaves in flight
                        s_next = hold_s(s_next);
                        scales(next, min(s_next, s_last), min(s_next + kMxStepScales, s_last));
                    }
                    if constexpr (n == Plan::kBaseA) {
                        pa1 = hold_s(pa1);
                        ba1 = read_base<kTrA>(la, 0, fa, pa1);
                    }
                    if constexpr (n == Plan::kBaseB) {
                        pb1 = hold_s(pb1);
                        bb1 = read_base<kTrB>(lb, 0, fb, pb1);
                    }
                    if constexpr (kTrA && n == Plan::kMask)
                        na = cols_a.step(t + 2);
                    if constexpr (kMasked && !kTrA && n == Plan::kMask) {
                        so = hold_s(so);
                        va = hold_v(masked(voff_a, cb_a, so));
                    }
                });
            wait_lds();
            wait_loads<kB>();                        // step t+1 and its scales; B(t+2) in flight
            barrier();
            half<1>(
                f, acc, sc, ba1, bb1, pa,
                [&](int v) {
                    pa = hold_s(pa);
                    if constexpr (!kTrA)
                        so = hold_s(so);
                    load_a(pa, v, va, so, na);
                },
                [&](auto slot) __attribute__((always_inline)) {
                    constexpr int n = decltype(slot)::value;
                    if constexpr (n == Plan::kBaseA) {
                        pa1 = hold_s(pa1);
                        ba0 = read_base<kTrA>(la, 1, fa, pa1);
                    }
                    if constexpr (n == Plan::kBaseB) {
                        pb1 = hold_s(pb1);
                        bb0 = read_base<kTrB>(lb, 1, fb, pb1);
                    }
                    // the next step's scales move over those no instruction needs any
                    // more (half 0's, and half 1's of A blocks 0..3 after 32 of 64):
                    // left to the compiler, the moves bunch at the loop's end and
                    // push accumulators out of their registers
                    if constexpr (Mma::kScaled && n == 5)
                        sc.b[0][0] = copy_v(next.b[0][0]);
                    if constexpr (Mma::kScaled && n == 8)
                        sc.a[0][0] = copy_v(next.a[0][0]);
                    if constexpr (Mma::kScaled && kB == 8 && n == 14)
                        sc.b[0][kHi] = copy_v(next.b[0][kHi]);
                    if constexpr (Mma::kScaled && kB == 8 && n == 17)
                        sc.a[0][kHi] = copy_v(next.a[0][kHi]);
                    if constexpr (Mma::kScaled && kB == 8 && n == 40)
                        sc.a[1][0] = copy_v(next.a[1][0]);
                    if constexpr (n == Plan::kRing)
                        npb = copy_s(pb1);
                    if constexpr (n == Plan::kRing + 1)
                        npb1 = copy_s(pb2);
                    if constexpr (n == Plan::kRing + 2)
                        npb2 = copy_s(pb);
                    if constexpr (kMasked && !kTrB && n == Plan::kMask) {
                        so = hold_s(so);
                        vb_next = hold_v(masked(voff_b, cb_b, hold_s(so + kStepBytes)));
                    }
                    if constexpr (n == Plan::kTail) {
                        npa = copy_s(pa1);
                        npa1 = copy_s(pa);
                        nso = hold_s(hold_s(so) + kStepBytes);
                        if constexpr (Mma::kScaled)
                            s_next = hold_s(hold_s(s_next) + 2 * kMxStepScales);
                    }
                });
            pa = npa;
            pa1 = npa1;
            so = nso;
            pb = npb;
            pb1 = npb1;
            pb2 = npb2;
            vb = vb_next;
            if constexpr (Mma::kScaled) {
                sc.b[1][0] = next.b[1][0];
                sc.b[1][kHi] = next.b[1][kHi];
                sc.a[1][kHi] = next.a[1][kHi];
            }
        }
        wait_loads<0>();
    }
};

// The accumulators leave the loop in fixed registers, whatever the epilogue does
// with them (else its needs feed back into the loop's assignment; and a matrix
// instruction must not move under the epilogue's lane masks): AGPRs for 256 and
// 192 tiles, VGPRs for 128 tiles.
template <int kB>
__device__ __forceinline__ void settle(f32x4_t (&acc)[kB][kB])
{
#pragma unroll
    for (int i = 0; i < kB; ++i)
#pragma unroll
        for (int j = 0; j < kB; ++j) {
            if constexpr (kB >= 6)
                asm volatile("" : "+a"(acc[i][j]));
            else
                asm volatile("" : "+v"(acc[i][j]));
        }
}
// Row i's blocks, so that an epilogue copies one row out of the AGPRs at a time.
template <int kB>
__device__ __forceinline__ void settle_row(f32x4_t (&acc)[kB][kB], int i)
{
    if constexpr (kB >= 6) {
#pragma unroll
        for (int j = 0; j < kB; ++j)
            asm volatile("" : "+a"(acc[i][j]));
    }
}

// A wave's quarter of 16-bit results in LDS, so that stores go out as whole runs of
// a row: straight from the accumulators, neighbouring lanes hold neighbouring rows
// and every lane's 16 bytes are a request of their own (64 cycles a store; 32 stores
// a wave took 8500 of a 256-tile's 57000 cycles at K = 4096 e2m1).  The units
// of a row are permuted (place) so that 16 lanes with one unit of 16 rows, with 16
// neighbouring units, or with one element of every eighth row meet different banks.
template <int kB>
struct Stage {
    static constexpr int kSide = 16 * kB;
    static constexpr int kPitch = kB == 4 ? 64 : 128;   // elements: a power of two of units
    static constexpr int kUnits = kSide / 8;
    uint16_t *base;

    __device__ __forceinline__ Stage(char *smem, int wave) : base(reinterpret_cast<uint16_t *>(smem) + wave * kSide * kPitch) {}
    __device__ __forceinline__ static int place(int row, int unit)
    {
        return row * kPitch + 8 * (unit ^ (kPitch == 128 ? (row ^ (row >> 3)) & 15 : ((row >> 1) ^ (row >> 4)) & 7));
    }
    __device__ __forceinline__ u32x4_t *unit(int row, int u) const
    {
        return reinterpret_cast<u32x4_t *>(base + place(row, u));
    }
};

// Where a staged quarter goes: `to`, rows ld elements apart, of which rows x cols exist.
// Rows that start 16-byte aligned and hold whole units leave 16 at a time (rows16), as
// soon as they are staged, 16 lanes (8 or 12 for smaller tiles) to a row; others at the
// end (odd_rows), neighbouring lanes writing neighbouring elements (1111 x 2777 x 1184
// e2m1: 8.8 us, against 12.2 with a unit's elements stored one after the other by one
// lane).
template <int kB>
struct StageOut {
    using St = Stage<kB>;
    uint16_t *to;
    int64_t ld;
    int rows, cols;
    bool units;
    __amdgpu_buffer_rsrc_t rs;

    __device__ __forceinline__ StageOut(uint16_t *base, int64_t at, int64_t pitch, int r, int c, int width)
        : to(base + at), ld(pitch), rows(min(r, St::kSide)), cols(c)
    {
        units = ((reinterpret_cast<uintptr_t>(base) | (uintptr_t)(2 * pitch) | (uintptr_t)(2 * width)) & 15) == 0 &&
                pitch < (1 << 22);
        rs = buffer_of(to, units && rows > 0 ? (uint32_t)rows * (uint32_t)(2 * ld) : 0u);
    }
    __device__ __forceinline__ void rows16(const St &st, int lane, int r0) const
    {
        if (!units)
            return;
        lanes_in_step();
#pragma unroll
        for (int k = 0; k < 16 * St::kUnits / 64; ++k) {
            const int at = 64 * k + lane, row = r0 + at / St::kUnits, u = at % St::kUnits;
            __builtin_amdgcn_raw_buffer_store_b128(*st.unit(row, u), rs,
                                                   8 * u < cols ? (int)(2 * (row * ld + 8 * u)) : kPastEnd, 0, 0);
        }
    }
    __device__ __forceinline__ void odd_rows(const St &st, int lane) const
    {
        if (units)
            return;
        lanes_in_step();
        for (int row = 0; row < rows; ++row)
            for (int c = lane; c < min(cols, St::kSide); c += 64)
                to[row * ld + c] = st.base[St::place(row, c >> 3) + (c & 7)];
    }
};

// The tile of workgroup b of a triangle of Gm x Gm tiles, tm <= tn: consecutive
// workgroups of an XCD (b mod 8 equal) take neighbouring tiles of one column, so
// that its L2 holds that column's panel and a run of row panels.
__device__ __forceinline__ void triangle_tile(int b, int G, int &tm, int &tn)
{
    const int total = G * (G + 1) / 2, per = total / kNumXcd, whole = per * kNumXcd;
    const int id = b < whole ? (b % kNumXcd) * per + b / kNumXcd : b;
    // column tn holds tiles tn (tn + 1) / 2 .. + tn
    // (a scalar again: buffers are made from the tile's place)
    int c = __builtin_amdgcn_readfirstlane((int)((sqrtf(8.0f * (float)id + 1.0f) - 1.0f) * 0.5f));
    while ((c + 1) * (c + 2) / 2 <= id)
        ++c;
    while (c * (c + 1) / 2 > id)
        --c;
    tn = c;
    tm = id - c * (c + 1) / 2;
}

}  // namespace hkg
