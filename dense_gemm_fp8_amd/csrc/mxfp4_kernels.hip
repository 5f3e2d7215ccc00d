// mxfp4_kernels.hip -- gfx950 kernels of the MXFP4 linear layer: quantisation
// (along rows, and of the transpose in the same pass), its inverse, and the
// product of few rows.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "mx4.h"
#include "ops_kernels.h"

namespace hkg {
namespace {

// ---- quantisation -----------------------------------------------------------
// One workgroup takes a 128 x 128 tile: one packed group of one packed step
// along K, and at the same time one group (of columns) of one step (of rows) of
// the transpose, so both forms' 512 scale bytes of the tile are whole runs.
// Along K: a lane holds 8 consecutive elements, a quad of lanes one block, so a
// wave reads 4 rows of 256 or 512 bytes at once and two DPP steps give a
// block's largest magnitude.  Along rows: the tile is staged in LDS, a wave
// takes 32 of its rows and a lane 2 columns, one after the other.  Bound by its
// bytes: both forms of 14336 x 4096 fp32 (235 MB read, 62 written) in 60 us, 5.0 TB/s,
// of 8192 x 14336 bf16 (235 and 125) in 88 us, 4.1 TB/s, with buffers that change from
// call to call; a 2 GiB copy reaches 4.9.  On the same buffers again, part of which the
// last-level cache holds, 53 and 84 us.
constexpr int kQTile = 128;

template <int kElem, bool kBoth>
__global__ __launch_bounds__(256) void mx4_quantize_kernel(const QuantParams p)
{
    __shared__ uint32_t sc[kMxStepScales / 4];
    __shared__ uint32_t sct[kBoth ? kMxStepScales / 4 : 1];
    // bf16 pairs (2 columns a word) or fp32 values of the tile
    __shared__ uint32_t tile[kBoth ? kQTile * (kElem == 0 ? kQTile / 2 : kQTile) : 1];
    const int nk = (p.K + kMxStep - 1) / kMxStep, nr = (p.rows + kMxStep - 1) / kMxStep;
    const int g = blockIdx.x / nk, t = blockIdx.x % nk;
    const int kp = (p.K + kMxBlock - 1) / kMxBlock * kMxBlock;
    const int rp = (p.rows + kMxBlock - 1) / kMxBlock * kMxBlock;
    const bool vec = (((reinterpret_cast<uintptr_t>(p.x)) | (uintptr_t)(p.ldx * (kElem == 0 ? 2 : 4))) & 15) == 0;
    if (threadIdx.x < kMxStepScales / 4) {
        sc[threadIdx.x] = 0x7f7f7f7fu;
        if constexpr (kBoth)
            sct[threadIdx.x] = 0x7f7f7f7fu;
    }
    __syncthreads();
    const int c8 = threadIdx.x & 15, r0 = threadIdx.x >> 4;   // 8-column group, row of 16
    const int k = kQTile * t + 8 * c8;
    Vec8<kElem> v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i)
        v[i] = load8<kElem>(p.x, p.ldx, kQTile * g + r0 + 16 * i, p.rows, k, p.K, vec);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int rl = r0 + 16 * i, row = kQTile * g + rl;
        const uint32_t code = scale_code(quad_max(v[i].amax_bits()));
        const uint32_t q = code == kScaleNan ? 0u : v[i].codes(scale_operand(code));
        if (row < p.rows && k < kp) {
            *reinterpret_cast<uint32_t *>(p.codes + (int64_t)row * (kp / 2) + k / 2) = q;
            if ((threadIdx.x & 3) == 0)
                reinterpret_cast<uint8_t *>(sc)[scale_byte(p.operand, rl, c8 >> 2)] = (uint8_t)code;
        }
        if constexpr (kBoth) {
            constexpr int kW = kElem == 0 ? 4 : 8;
#pragma unroll
            for (int w = 0; w < kW; ++w)
                tile[rl * (16 * kW) + c8 * kW + w] = v[i].w[w];
        }
    }
    __syncthreads();
    if (threadIdx.x < kMxStepScales / 4)
        reinterpret_cast<uint32_t *>(p.packed + ((int64_t)g * nk + t) * kMxStepScales)[threadIdx.x] =
            sc[threadIdx.x];
    if constexpr (kBoth) {
        // wave w: rows 32 w .. +31 of the tile; lane: columns 2 l, 2 l + 1
        const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
        const int row0 = kQTile * g + 32 * w;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int cl = 2 * lane + h, col = kQTile * t + cl;
            uint32_t m = 0;
            float f[32];
#pragma unroll
            for (int i = 0; i < 32; ++i) {
                uint32_t b;
                if constexpr (kElem == 0) {
                    const uint32_t two = tile[(32 * w + i) * 64 + lane];
                    b = h == 0 ? two << 16 : two & 0xffff0000u;
                } else {
                    b = tile[(32 * w + i) * 128 + cl];
                }
                f[i] = __builtin_bit_cast(float, b);
                m = max_u32(m, b & 0x7fffffffu);
            }
            const uint32_t code = scale_code(m);
            const float s = scale_operand(code);
            u32x4_t q;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                uint32_t r = 0;
                r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, f[8 * i], f[8 * i + 1], s, 0);
                r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, f[8 * i + 2], f[8 * i + 3], s, 1);
                r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, f[8 * i + 4], f[8 * i + 5], s, 2);
                r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, f[8 * i + 6], f[8 * i + 7], s, 3);
                q[i] = code == kScaleNan ? 0u : r;
            }
            if (col < p.K && row0 < rp) {
                *reinterpret_cast<u32x4_t *>(p.codes_t + (int64_t)col * (rp / 2) + row0 / 2) = q;
                reinterpret_cast<uint8_t *>(sct)[scale_byte(p.operand_t, cl, w)] = (uint8_t)code;
            }
        }
        __syncthreads();
        if (threadIdx.x < kMxStepScales / 4)
            reinterpret_cast<uint32_t *>(p.packed_t + ((int64_t)t * nr + g) * kMxStepScales)[threadIdx.x] =
                sct[threadIdx.x];
    }
}

// ---- the values of an MXFP4 matrix ------------------------------------------
// A lane turns one word of codes (8 elements) into 16 or 32 bytes.  Bound by its
// bytes: 14336 x 4096 to bf16 (31 MB read, 117 written) in 37 us, 4.0 TB/s, to fp32 (31
// and 235) in 63 us, 4.2 TB/s, with buffers that change from call to call; 24 and 51 us
// on the same ones again, which the last-level cache holds or nearly holds.
template <int kElem>
__global__ __launch_bounds__(256) void mx4_dequantize_kernel(const DequantParams p)
{
    const int words = p.kp / 8, nk = (p.kp + kMxStep - 1) / kMxStep;
    const int cols = (words + 63) / 64;           // workgroups per 4 rows
    const int w = blockIdx.x % cols * 64 + (threadIdx.x & 63);
    if (w >= words)
        return;
    const int64_t stride = gridDim.x / cols * 4;
    for (int64_t row = blockIdx.x / cols * 4 + (threadIdx.x >> 6); row < p.rows; row += stride) {
        const uint32_t q = *reinterpret_cast<const uint32_t *>(p.codes + row * (p.kp / 2) + 4 * w);
        const int blk = w >> 2;
        const uint32_t code = p.packed[((int64_t)(row >> 7) * nk + (blk >> 2)) * kMxStepScales +
                                       scale_byte(p.operand, (int)row & 127, blk & 3)];
        const float s = scale_operand(code);
        const bool nan = code == kScaleNan;
        const int64_t at = row * p.ldv + 8 * w;
        const bool vec = ((reinterpret_cast<uintptr_t>(p.values) | (uintptr_t)(p.ldv * (kElem == 0 ? 2 : 4))) & 15) == 0;
        if constexpr (kElem == 0) {
            u32x4_t o;
            o[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(q, s, 0));
            o[1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(q, s, 1));
            o[2] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(q, s, 2));
            o[3] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(q, s, 3));
#pragma unroll
            for (int i = 0; i < 4; ++i)
                o[i] = nan ? 0x7fc07fc0u : o[i];
            uint16_t *d = static_cast<uint16_t *>(p.values) + at;
            if (vec)
                *reinterpret_cast<u32x4_t *>(d) = o;
            else
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    d[i] = (uint16_t)(o[i >> 1] >> (16 * (i & 1)));
        } else {
            typedef float f32x2 __attribute__((ext_vector_type(2)));
            uint32_t o[8];
            const f32x2 a = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q, s, 0);
            const f32x2 b = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q, s, 1);
            const f32x2 c = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q, s, 2);
            const f32x2 e = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q, s, 3);
            const float f[8] = {a[0], a[1], b[0], b[1], c[0], c[1], e[0], e[1]};
#pragma unroll
            for (int i = 0; i < 8; ++i)
                o[i] = nan ? 0x7fc00000u : __builtin_bit_cast(uint32_t, f[i]);
            uint32_t *d = static_cast<uint32_t *>(p.values) + at;
            if (vec) {
                *reinterpret_cast<u32x4_t *>(d) = u32x4_t{o[0], o[1], o[2], o[3]};
                *reinterpret_cast<u32x4_t *>(d + 4) = u32x4_t{o[4], o[5], o[6], o[7]};
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    d[i] = o[i];
            }
        }
    }
}

// ---- the product of few rows ------------------------------------------------
// What bounds it is reading B once, so each wave streams its own part of K and keeps
// a whole run of loads in flight.  One workgroup computes 16 kMb rows (of A or x) x 32
// columns (rows of B); its 8 waves take runs of kS 128-k steps in turn:
//   wait for the run in LDS, take its fragments into registers, send the next run's
//   loads into the same LDS, and multiply while they fly;
// the waves' sums are joined in LDS at the end, in a fixed order.  The detour through
// LDS is what makes the loads whole lines: a lane of a fragment holds 16 bytes of a row
// of its own, and loaded straight into registers every lane is a request of its own
// (16 x 8192 x 8192: 15.4 us so, x among them, against 11.4 through LDS).  x with rows that
// are not 16-byte aligned, or K not a multiple of 32, does go straight to registers, element
// by element: 1 x 14336 x 4096 18.5 us against 10.5, 16 x 8192 x 8192 47.6 against 11.8.
// B is the matrix instruction's first operand: fragments 2 j and 2 j + 1 of a packed
// group then give a lane 8 consecutive columns of one row of C.  kXt: -1 A is codes, 0
// / 1 x is bf16 / fp32 and each lane quantises the one block that its fragment holds (16
// q + x holds row x, block q), so the quantised activations never leave the registers.
constexpr int kFewWaves = 8;

// kXt: see above.  kMb: 16-row blocks of A.  kS: steps of a run -- two where a compute
// unit gets one workgroup, so that enough is in flight, else one, so that several
// workgroups share it.
template <int kXt, int kMb, int kS>
struct FewRows {
    static_assert(kXt < 0 || kMb == 1, "x is quantised for 16 rows");
    static constexpr int kElem = kXt == 1 ? 4 : 2;
    static constexpr int kRow = 64 * kS;                        // bytes of a row of codes in a run
    static constexpr int kXRow = 128 * kElem;                   // bytes of a row of x in a step
    static constexpr int kBBytes = 32 * kRow;
    static constexpr int kABytes = kXt < 0 ? 16 * kMb * kRow : kS * 16 * kXRow;
    static constexpr int kWave = kBBytes + kABytes;             // LDS bytes of one wave
    static constexpr int kSums = kFewWaves * 64 * 9 * 4;
    static constexpr int kLds = kFewWaves * kWave > kSums ? kFewWaves * kWave : kSums;

    // Places of a row's 16-byte chunks in LDS, permuted so that the 16 rows of a
    // fragment, which differ in bits 0, 1 and 3, 4 (B, interleaved) or 0..3 (A, x),
    // fall into different 16-byte slots of the 256-byte bank line.
    __device__ __forceinline__ static int b_chunk(int row, int c)
    {
        return kS == 2 ? c ^ (((row >> 1) & 1) | (((row >> 3) & 3) << 1)) : c ^ ((row >> 3) & 3);
    }
    __device__ __forceinline__ static int a_chunk(int row, int c)
    {
        return kS == 2 ? c ^ ((row >> 1) & 7) : c ^ ((row >> 2) & 3);
    }
    __device__ __forceinline__ static int x_chunk(int row, int c) { return c ^ (row & 15); }
};

template <int kXt, int kMb, int kS>
__device__ __forceinline__ void mx4_few_rows(const Mx4GemmParams &p, int block, char *smem)
{
    using G = FewRows<kXt, kMb, kS>;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int x = lane & 15, q = lane >> 4;
    const int gn = (p.N + 31) / 32;
    const int n0 = 32 * (block % gn), m0 = 16 * kMb * (block / gn);
    const int nk = (p.kb + 63) / 64;              // 128-k steps
    const int g = n0 >> 7, j = (n0 >> 5) & 3;     // B's packed group, pair of fragments in it
    const uint32_t span = (uint32_t)nk * kMxStepScales;
    char *const lb = smem + wave * G::kWave, *const la = lb + G::kBBytes;
    const int rows = min(16 * kMb, p.M - m0);
    // buffers over the workgroup's rows: rows past the matrix read zeros
    const __amdgpu_buffer_rsrc_t rb = buffer_of(p.B + (int64_t)n0 * p.kb, (uint32_t)min(32, p.N - n0) * (uint32_t)p.kb);
    const __amdgpu_buffer_rsrc_t rsb = buffer_of(p.SB + (int64_t)g * span, span);
    __amdgpu_buffer_rsrc_t ra, rsa;
    // x in whole aligned blocks, its 16 rows within one buffer: else element by element
    const bool whole = kXt >= 0 && (p.K & 31) == 0 && p.ldx < (1 << 24) &&
                       ((reinterpret_cast<uintptr_t>(p.x) | (uintptr_t)(p.ldx * G::kElem)) & 15) == 0;
    if constexpr (kXt < 0) {
        ra = buffer_of(p.A + (int64_t)m0 * p.kb, (uint32_t)rows * (uint32_t)p.kb);
        rsa = buffer_of(p.SA + (int64_t)(m0 >> 7) * span, span);   // 16 kMb rows from m0 lie in one group
    } else {
        ra = buffer_of(static_cast<const char *>(p.x) + m0 * p.ldx * G::kElem,
                       whole ? (uint32_t)((rows - 1) * p.ldx + p.K) * G::kElem : 0u);
    }
    auto to_lds = [&](__amdgpu_buffer_rsrc_t rs, char *to, int voff) {
        __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, (__attribute__((address_space(3))) void *)to, 16, voff, 0, 0, 0);
    };
    uint32_t sb[kS], sa[kS];
    // the loads of run r (steps kS r ..)
    auto send = [&](int r) {
#pragma unroll
        for (int u = 0; u < kS; ++u) {            // a step past the end has zeros, and a scale in range
            const int ss = min(kS * r + u, nk - 1) * kMxStepScales;
            sb[u] = __builtin_amdgcn_raw_buffer_load_b16(rsb, 8 * lane + 2 * j, ss, 0);
            if constexpr (kXt < 0) {
                if constexpr (kMb == 4)
                    sa[u] = __builtin_amdgcn_raw_buffer_load_b32(rsa, 8 * lane + ((m0 >> 4) & 4), ss, 0);
                else
                    sa[u] = __builtin_amdgcn_raw_buffer_load_b8(rsa, 8 * lane + ((m0 >> 4) & 7), ss, 0);
            }
        }
#pragma unroll
        for (int d = 0; d < G::kBBytes / 1024; ++d) {
            constexpr int kC = 4 * kS;            // chunks of a row
            const int row = 64 / kC * d + lane / kC, at = G::kRow * r + 16 * G::b_chunk(row, lane % kC);
            to_lds(rb, lb + 1024 * d, at < p.kb ? row * p.kb + at : kPastEnd);
        }
        if constexpr (kXt < 0) {
#pragma unroll
            for (int d = 0; d < G::kABytes / 1024; ++d) {
                constexpr int kC = 4 * kS;
                const int row = 64 / kC * d + lane / kC, at = G::kRow * r + 16 * G::a_chunk(row, lane % kC);
                if (64 / kC * d < rows)           // rows past the matrix: whatever LDS holds, in columns not stored
                    to_lds(ra, la + 1024 * d, at < p.kb ? row * p.kb + at : kPastEnd);
            }
        } else if (whole) {
            constexpr int kChunks = G::kXRow / 16, kRows = 64 / kChunks;   // rows a load covers
#pragma unroll
            for (int u = 0; u < kS; ++u)
#pragma unroll
                for (int d = 0; d < 16 / kRows; ++d) {
                    const int row = kRows * d + lane / kChunks, c = G::x_chunk(row, lane % kChunks);
                    const int k = 128 * (kS * r + u) + 16 * c / G::kElem;
                    if (kRows * d < rows)
                        to_lds(ra, la + 1024 * (u * (16 / kRows) + d),
                               k < p.K ? (int)(row * p.ldx + k) * G::kElem : kPastEnd);
                }
        }
    };
    f32x4_t acc[kMb][2];
#pragma unroll
    for (int i = 0; i < kMb; ++i)
        acc[i][0] = acc[i][1] = f32x4_t{0.f, 0.f, 0.f, 0.f};
    const int runs = (nk + kS - 1) / kS;
    if (wave < runs)
        send(wave);
    for (int r = wave; r < runs; r += kFewWaves) {
        u32x4_t b[kS][2], a[kS][kMb];
        Vec8<(kXt < 0 ? 0 : kXt)> v[kS][4];
        uint32_t sb_now[kS], sa_now[kS];
        asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
        const int br = (x & 3) + 8 * (x >> 2);
#pragma unroll
        for (int u = 0; u < kS; ++u) {
            sb_now[u] = sb[u];
            sa_now[u] = sa[u];
#pragma unroll
            for (int h = 0; h < 2; ++h)
                b[u][h] = *reinterpret_cast<const u32x4_t *>(lb + G::kRow * (br + 4 * h) +
                                                               16 * G::b_chunk(br + 4 * h, 4 * u + q));
            if constexpr (kXt < 0) {
#pragma unroll
                for (int i = 0; i < kMb; ++i)
                    a[u][i] = *reinterpret_cast<const u32x4_t *>(la + G::kRow * (16 * i + x) +
                                                                   16 * G::a_chunk(x, 4 * u + q));
            } else if (whole) {
                constexpr int kVecs = kXt == 1 ? 2 : 1;   // 16-byte units of 8 elements
#pragma unroll
                for (int i = 0; i < 4 * kVecs; ++i) {
                    const u32x4_t t = *reinterpret_cast<const u32x4_t *>(
                        la + 16 * G::kXRow * u + G::kXRow * x + 16 * G::x_chunk(x, 4 * kVecs * q + i));
#pragma unroll
                    for (int w = 0; w < 4; ++w)
                        v[u][i / kVecs].w[4 * (i % kVecs) + w] = t[w];
                }
            } else {
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    v[u][i] = load8<(kXt < 0 ? 0 : kXt)>(p.x, p.ldx, m0 + x, p.M, 128 * (kS * r + u) + 32 * q + 8 * i, p.K, false);
            }
        }
        // the fragments are in registers: their LDS is free
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
        if (r + kFewWaves < runs)
            send(r + kFewWaves);
#pragma unroll
        for (int u = 0; u < kS; ++u) {
            if constexpr (kXt >= 0) {
                uint32_t big = 0;
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    big = max_u32(big, v[u][i].amax_bits());
                sa_now[u] = scale_code(big);
                const float s = scale_operand(sa_now[u]);
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    a[u][0][i] = sa_now[u] == kScaleNan ? 0u : v[u][i].codes(s);
            }
            acc[0][0] = mma_f4<0, 0>(b[u][0], a[u][0], acc[0][0], sb_now[u], sa_now[u]);
            acc[0][1] = mma_f4<1, 0>(b[u][1], a[u][0], acc[0][1], sb_now[u], sa_now[u]);
            if constexpr (kMb == 4) {
                acc[1][0] = mma_f4<0, 1>(b[u][0], a[u][1], acc[1][0], sb_now[u], sa_now[u]);
                acc[1][1] = mma_f4<1, 1>(b[u][1], a[u][1], acc[1][1], sb_now[u], sa_now[u]);
                acc[2][0] = mma_f4<0, 2>(b[u][0], a[u][2], acc[2][0], sb_now[u], sa_now[u]);
                acc[2][1] = mma_f4<1, 2>(b[u][1], a[u][2], acc[2][1], sb_now[u], sa_now[u]);
                acc[3][0] = mma_f4<0, 3>(b[u][0], a[u][3], acc[3][0], sb_now[u], sa_now[u]);
                acc[3][1] = mma_f4<1, 3>(b[u][1], a[u][3], acc[3][1], sb_now[u], sa_now[u]);
            }
        }
    }
    float(*part)[64][9] = reinterpret_cast<float(*)[64][9]>(smem);   // 9: neighbours' rows fall into other banks
#pragma unroll
    for (int i = 0; i < kMb; ++i) {
        // the sums are complete here for every lane: nothing below may move a
        // matrix instruction under a lane mask
        asm volatile("" : "+v"(acc[i][0]), "+v"(acc[i][1]));
        __syncthreads();
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            part[wave][lane][r] = acc[i][0][r];
            part[wave][lane][4 + r] = acc[i][1][r];
        }
        __syncthreads();
        // 16 x 32 results: lane 16 (c / 8) + r of the fragments holds row r, column c
#pragma unroll
        for (int o = threadIdx.x; o < 512; o += 64 * kFewWaves) {
            const int r = o >> 5, c = o & 31;
            float s = 0.f;
#pragma unroll
            for (int w = 0; w < kFewWaves; ++w)
                s += part[w][16 * (c >> 3) + r][c & 7];
            const int row = m0 + 16 * i + r, col = n0 + c;
            if (row < p.M && col < p.N) {
                const int64_t at = row * p.ldc + col;
                p.C[at] = (uint16_t)pack2_bf16(s, 0.f);
                if (p.C_f32)
                    p.C_f32[at] = s;
            }
        }
    }
}

// ---- the product without K ----------------------------------------------------
// Workgroups take 256 columns of a row, in turns in both directions.
__global__ __launch_bounds__(256) void mx4_zero_kernel(const Mx4GemmParams p)
{
    for (int64_t row = blockIdx.y; row < p.M; row += gridDim.y)
        for (int64_t col = (int64_t)blockIdx.x * 256 + threadIdx.x; col < p.N; col += (int64_t)gridDim.x * 256) {
            p.C[row * p.ldc + col] = 0;
            if (p.C_f32)
                p.C_f32[row * p.ldc + col] = 0.0f;
        }
}

template <int kXt, int kMb, int kS>
__global__ __launch_bounds__(64 * kFewWaves) void mx4_few_rows_kernel(const Mx4GemmParams p)
{
    __shared__ __attribute__((aligned(1024))) char smem[FewRows<kXt, kMb, kS>::kLds];
    mx4_few_rows<kXt, kMb, kS>(p, blockIdx.x, smem);
}

// Two products: the first `first` workgroups are product 0's.
struct FewRowsPair {
    Mx4GemmParams p[2];
    int first;
};
template <int kMb, int kS>
__global__ __launch_bounds__(64 * kFewWaves) void mx4_few_rows_pair_kernel(const FewRowsPair t)
{
    __shared__ __attribute__((aligned(1024))) char smem[FewRows<-1, kMb, kS>::kLds];
    const int which = (int)blockIdx.x >= t.first;
    mx4_few_rows<-1, kMb, kS>(t.p[which], blockIdx.x - (which ? t.first : 0), smem);
}

}  // namespace

hipError_t launch_mx4_quantize(ElemType t, const QuantParams &p, hipStream_t stream)
{
    const dim3 grid((unsigned)((p.rows + kQTile - 1) / kQTile) * ((p.K + kQTile - 1) / kQTile)), block(256);
    if (p.codes_t) {
        if (t == kElemBf16)
            hipLaunchKernelGGL((mx4_quantize_kernel<0, true>), grid, block, 0, stream, p);
        else
            hipLaunchKernelGGL((mx4_quantize_kernel<1, true>), grid, block, 0, stream, p);
    } else {
        if (t == kElemBf16)
            hipLaunchKernelGGL((mx4_quantize_kernel<0, false>), grid, block, 0, stream, p);
        else
            hipLaunchKernelGGL((mx4_quantize_kernel<1, false>), grid, block, 0, stream, p);
    }
    return hipGetLastError();
}

hipError_t launch_mx4_dequantize(ElemType t, const DequantParams &p, hipStream_t stream)
{
    // at most 2^23 workgroups, so that their threads stay below 2^32; the rest of a
    // very long matrix in turns
    const unsigned cols = (p.kp / 8 + 63) / 64, quads = (p.rows + 3) / 4, most = (1u << 23) / cols;
    const dim3 grid(cols * (quads < most ? quads : most)), block(256);
    if (t == kElemBf16)
        hipLaunchKernelGGL(mx4_dequantize_kernel<0>, grid, block, 0, stream, p);
    else
        hipLaunchKernelGGL(mx4_dequantize_kernel<1>, grid, block, 0, stream, p);
    return hipGetLastError();
}

template <int kXt, int kMb, int kS>
static hipError_t few_rows(const Mx4GemmParams &p, unsigned blocks, hipStream_t stream)
{
    hipLaunchKernelGGL((mx4_few_rows_kernel<kXt, kMb, kS>), dim3(blocks), dim3(64 * kFewWaves), 0, stream, p);
    return hipGetLastError();
}

// Two-step runs (96 KiB of LDS at 64 rows) where each of 256 compute units has at most
// one workgroup, or for a long K: 256 x 4096 x 14336 24.4 us against 27.1 in one-step
// runs, which let three workgroups share a unit (256 x 4096 x 4096: 9.3 against 10.5).
static bool two_steps(unsigned blocks, int K) { return blocks <= 256 || K >= 8192; }

static unsigned few_blocks(const Mx4GemmParams &p, int mb)
{
    return (unsigned)((p.N + 31) / 32) * (unsigned)((p.M + 16 * mb - 1) / (16 * mb));
}

hipError_t launch_mx4_zero(const Mx4GemmParams &p, hipStream_t stream)
{
    const int64_t cols = ((int64_t)p.N + 255) / 256;
    const dim3 grid((unsigned)(cols < 256 ? cols : 256), (unsigned)(p.M < 4096 ? p.M : 4096));
    hipLaunchKernelGGL(mx4_zero_kernel, grid, dim3(256), 0, stream, p);
    return hipGetLastError();
}

// A launch's threads have to stay below 2^32, or part of the grid is left out without an
// error: the columns of a very wide product in turns of 2^27 (2^22 workgroups for up to
// 16 rows; more rows come with at most 512 workgroups).
constexpr int kFewCols = 1 << 27;

hipError_t launch_mx4_few_rows(ElemType xt, const Mx4GemmParams &p, hipStream_t stream)
{
    if (p.N > kFewCols) {
        Mx4GemmParams head = p, rest = p;
        head.N = kFewCols;
        rest.N -= kFewCols;
        rest.B += (int64_t)kFewCols * p.kb;
        rest.SB += (int64_t)kFewCols / kMxStep * ((p.kb + 63) / 64) * kMxStepScales;
        rest.C += kFewCols;
        rest.C_f32 += p.C_f32 ? kFewCols : 0;
        const hipError_t e = launch_mx4_few_rows(xt, head, stream);
        return e != hipSuccess ? e : launch_mx4_few_rows(xt, rest, stream);
    }
    const int mb = p.A && p.M > 16 ? 4 : 1;
    const unsigned blocks = few_blocks(p, mb);
    const bool two = two_steps(blocks, p.K);
    if (p.A) {
        if (mb == 1)   // 48 KiB in two-step runs
            return few_rows<-1, 1, 2>(p, blocks, stream);
        return two ? few_rows<-1, 4, 2>(p, blocks, stream) : few_rows<-1, 4, 1>(p, blocks, stream);
    }
    if (xt == kElemF32)   // 80 KiB in one-step runs
        return few_rows<1, 1, 1>(p, blocks, stream);
    return two ? few_rows<0, 1, 2>(p, blocks, stream) : few_rows<0, 1, 1>(p, blocks, stream);
}

hipError_t launch_mx4_few_rows2(const Mx4GemmParams &p, const Mx4GemmParams &p2, hipStream_t stream)
{
    const unsigned first = few_blocks(p, 4), blocks = first + few_blocks(p2, 4);
    const FewRowsPair t = {{p, p2}, (int)first};
    if (two_steps(blocks, p.K > p2.K ? p.K : p2.K))
        hipLaunchKernelGGL((mx4_few_rows_pair_kernel<4, 2>), dim3(blocks), dim3(64 * kFewWaves), 0, stream, t);
    else
        hipLaunchKernelGGL((mx4_few_rows_pair_kernel<4, 1>), dim3(blocks), dim3(64 * kFewWaves), 0, stream, t);
    return hipGetLastError();
}

}  // namespace hkg
