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
// takes 32 of its rows and a lane 2 columns, one after the other.
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
// A lane turns one word of codes (8 elements) into 16 or 32 bytes.
template <int kElem>
__global__ __launch_bounds__(256) void mx4_dequantize_kernel(const DequantParams p)
{
    const int words = p.kp / 8, nk = (p.kp + kMxStep - 1) / kMxStep;
    const int cols = (words + 63) / 64;           // workgroups per 4 rows
    const int w = blockIdx.x % cols * 64 + (threadIdx.x & 63);
    const int row = blockIdx.x / cols * 4 + (threadIdx.x >> 6);
    if (w >= words || row >= p.rows)
        return;
    const uint32_t q = *reinterpret_cast<const uint32_t *>(p.codes + (int64_t)row * (p.kp / 2) + 4 * w);
    const int blk = w >> 2;
    const uint32_t code = p.packed[((int64_t)(row >> 7) * nk + (blk >> 2)) * kMxStepScales +
                                   scale_byte(p.operand, row & 127, blk & 3)];
    const float s = scale_operand(code);
    const bool nan = code == kScaleNan;
    const int64_t at = (int64_t)row * p.ldv + 8 * w;
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

// ---- the product, operands read straight from memory ------------------------
// One workgroup computes 16 rows (of A or x) x 32 columns (rows of B); its
// waves take every kWaves-th 128-k step and add their sums in LDS.  B is the
// matrix instruction's first operand: fragments 2 j and 2 j + 1 of a packed
// group then give a lane 8 consecutive columns of one row of C, one 16-byte
// store.  kXt: -1 A is codes, 0 / 1 x is bf16 / fp32 and each lane quantises
// the one block that its fragment holds (16 q + x holds row x, block q), so the
// quantised activations never leave the registers.
constexpr int kDirectWaves = 4;

template <int kXt>
__global__ __launch_bounds__(64 * kDirectWaves) void mx4_direct_kernel(const Mx4GemmParams p)
{
    __shared__ float part[kDirectWaves][64][9];   // 9: neighbours' rows fall into other banks
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int x = lane & 15, q = lane >> 4;
    const int n0 = 32 * blockIdx.x, m = 16 * blockIdx.y + x;
    const int nk = (p.kb + 63) / 64;              // 128-k steps
    const int g = n0 >> 7, j = (n0 >> 5) & 3;     // B's packed group, pair of fragments in it
    f32x4_t acc[2] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
    const int rb = n0 + (x & 3) + 8 * (x >> 2);
    const bool vec = ((reinterpret_cast<uintptr_t>(p.x) | (uintptr_t)(p.ldx * (kXt == 1 ? 4 : 2))) & 15) == 0;
    for (int t = wave; t < nk; t += kDirectWaves) {
        const int cb = 64 * t + 16 * q;           // byte of this lane's block in a row
        const bool in = cb < p.kb;
        u32x4_t b[2] = {{0, 0, 0, 0}, {0, 0, 0, 0}}, a = {0, 0, 0, 0};
        uint32_t sb = 0x7f7f, sa = kScaleOne;
#pragma unroll
        for (int h = 0; h < 2; ++h)
            if (in && rb + 4 * h < p.N)
                b[h] = *reinterpret_cast<const u32x4_t *>(p.B + (int64_t)(rb + 4 * h) * p.kb + cb);
        sb = *reinterpret_cast<const uint16_t *>(p.SB + ((int64_t)g * nk + t) * kMxStepScales + 8 * lane + 2 * j);
        if constexpr (kXt < 0) {
            if (in && m < p.M) {
                a = *reinterpret_cast<const u32x4_t *>(p.A + (int64_t)m * p.kb + cb);
                sa = p.SA[((int64_t)(m >> 7) * nk + t) * kMxStepScales + scale_byte(0, m & 127, q)];
            }
        } else {
            Vec8<kXt> v[4];
            uint32_t big = 0;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                v[i] = load8<kXt>(p.x, p.ldx, m, p.M, 2 * cb + 8 * i, p.K, vec);
                big = max_u32(big, v[i].amax_bits());
            }
            sa = scale_code(big);
            const float s = scale_operand(sa);
#pragma unroll
            for (int i = 0; i < 4; ++i)
                a[i] = sa == kScaleNan ? 0u : v[i].codes(s);
        }
        acc[0] = mma_f4<0, 0>(b[0], a, acc[0], sb, sa);
        acc[1] = mma_f4<1, 0>(b[1], a, acc[1], sb, sa);
    }
    // the sums are complete here for every lane: nothing below may move a
    // matrix instruction under a lane mask
    asm volatile("" : "+v"(acc[0]), "+v"(acc[1]));
#pragma unroll
    for (int r = 0; r < 4; ++r) {
        part[wave][lane][r] = acc[0][r];
        part[wave][lane][4 + r] = acc[1][r];
    }
    __syncthreads();
    // 512 sums for 256 threads: thread -> lane tid / 4 of the fragments, columns 2 (tid & 3), +1
    const int fl = threadIdx.x >> 2, c = 2 * (threadIdx.x & 3);
    float s0 = 0.f, s1 = 0.f;
#pragma unroll
    for (int w = 0; w < kDirectWaves; ++w) {
        s0 += part[w][fl][c];
        s1 += part[w][fl][c + 1];
    }
    const int row = 16 * blockIdx.y + (fl & 15), col = n0 + 8 * (fl >> 4) + c;
    if (row >= p.M || col >= p.N)
        return;
    const int64_t at = row * p.ldc + col;
    const uint32_t two = pack2_bf16(s0, s1);
    if (col + 1 < p.N && (p.ldc & 1) == 0) {
        *reinterpret_cast<uint32_t *>(p.C + at) = two;
    } else {
        p.C[at] = (uint16_t)two;
        if (col + 1 < p.N)
            p.C[at + 1] = (uint16_t)(two >> 16);
    }
    if (p.C_f32) {
        p.C_f32[at] = s0;
        if (col + 1 < p.N)
            p.C_f32[at + 1] = s1;
    }
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
    const dim3 grid((unsigned)((p.kp / 8 + 63) / 64) * ((p.rows + 3) / 4)), block(256);
    if (t == kElemBf16)
        hipLaunchKernelGGL(mx4_dequantize_kernel<0>, grid, block, 0, stream, p);
    else
        hipLaunchKernelGGL(mx4_dequantize_kernel<1>, grid, block, 0, stream, p);
    return hipGetLastError();
}

hipError_t launch_mx4_direct(ElemType xt, const Mx4GemmParams &p, hipStream_t stream)
{
    const dim3 grid((p.N + 31) / 32, (p.M + 15) / 16), block(64 * kDirectWaves);
    if (p.A)
        hipLaunchKernelGGL(mx4_direct_kernel<-1>, grid, block, 0, stream, p);
    else if (xt == kElemBf16)
        hipLaunchKernelGGL(mx4_direct_kernel<0>, grid, block, 0, stream, p);
    else
        hipLaunchKernelGGL(mx4_direct_kernel<1>, grid, block, 0, stream, p);
    return hipGetLastError();
}

}  // namespace hkg
