// mx4.h -- device helpers of the MXFP4 kernels (mxfp4_kernels.hip): the block
// format and the place of a scale in the packed order.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace hkg {

typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));
typedef float f32x4_t __attribute__((ext_vector_type(4)));
typedef int i32x4_t __attribute__((ext_vector_type(4)));
typedef int i32x8_t __attribute__((ext_vector_type(8)));
typedef unsigned int u32x2_t __attribute__((ext_vector_type(2)));
typedef unsigned int u32x4_t __attribute__((ext_vector_type(4)));

constexpr int kMxBlock = 32;          // elements per E8M0 scale
constexpr int kMxStep = 128;          // k per packed step, and rows per packed group
constexpr int kMxStepScales = 512;    // scale bytes of one step of one group
constexpr uint32_t kScaleOne = 127;   // E8M0 codes
constexpr uint32_t kScaleNan = 255;

// A buffer of `bytes` bytes: loads past it give zeros, stores past it are dropped.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t buffer_of(const void *base, uint32_t bytes)
{
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<void *>(base), 0, bytes, 0x00020000);
}
constexpr int kPastEnd = int(0x80000000u);       // a lane offset outside any buffer

// Byte of the scale of (row r of a 128-row group, block b of a 128-k step)
// inside the step's 512: 8 (16 b + x) + e, where fragment e gives lane x row r.
// Operand A: r = 16 e + x.  Operand B: r = 32 (e >> 1) + 4 (e & 1) + (x & 3) +
// 8 (x >> 2), so that two fragments give a lane 8 consecutive rows.
__device__ __forceinline__ int scale_byte(int operand, int r, int b)
{
    const int x = operand == 0 ? r & 15 : (r & 3) | ((r >> 1) & 12);
    const int e = operand == 0 ? r >> 4 : ((r >> 2) & 1) | ((r >> 4) & 6);
    return 8 * (16 * b + x) + e;
}

// E8M0 code of a block whose largest magnitude has fp32 bits `bits` (sign
// cleared): exponent floor(log2 amax) - 2, at least 2^-127 (code 0, which also
// takes subnormal amax); zero gives scale 1, NaN or infinity the NaN scale.
// Comparing magnitudes by their bits orders NaN above infinity above the rest.
__device__ __forceinline__ uint32_t scale_code(uint32_t bits)
{
    const uint32_t e = bits >> 23;
    const uint32_t c = e > 2 ? e - 2 : 0;
    return bits == 0 ? kScaleOne : e == 255 ? kScaleNan : c;
}

// The scale operand of the fp4 conversions: they use only the exponent field,
// with field 0 standing for 2^-127 (checked on gfx950 against every bf16 value
// and the neighbours of every rounding boundary in fp32).
__device__ __forceinline__ float scale_operand(uint32_t code)
{
    return __builtin_bit_cast(float, code << 23);
}

__device__ __forceinline__ uint32_t max_u32(uint32_t a, uint32_t b) { return a > b ? a : b; }

// A wave-wide exchange with lane ^ 1 / lane ^ 2 of a quad.
template <int kCtrl>
__device__ __forceinline__ uint32_t quad_xor(uint32_t v)
{
    return (uint32_t)__builtin_amdgcn_mov_dpp((int)v, kCtrl, 0xf, 0xf, true);
}
__device__ __forceinline__ uint32_t quad_max(uint32_t v)
{
    v = max_u32(v, quad_xor<0xB1>(v));   // quad_perm [1, 0, 3, 2]
    return max_u32(v, quad_xor<0x4E>(v)); // quad_perm [2, 3, 0, 1]
}

// Two bf16 magnitudes per word: the larger of each half.
__device__ __forceinline__ uint32_t pk_max_u16(uint32_t a, uint32_t b)
{
    typedef unsigned short u16x2 __attribute__((ext_vector_type(2)));
    const u16x2 r = __builtin_elementwise_max(__builtin_bit_cast(u16x2, a), __builtin_bit_cast(u16x2, b));
    return __builtin_bit_cast(uint32_t, r);
}

// Eight consecutive elements of a row.
template <int kElem>
struct Vec8;
template <>
struct Vec8<0> {                     // bf16, two a word
    uint32_t w[4];
    __device__ __forceinline__ uint32_t amax_bits() const
    {
        uint32_t m = pk_max_u16(pk_max_u16(w[0] & 0x7fff7fffu, w[1] & 0x7fff7fffu),
                                pk_max_u16(w[2] & 0x7fff7fffu, w[3] & 0x7fff7fffu));
        return max_u32(m << 16, m & 0xffff0000u);
    }
    __device__ __forceinline__ uint32_t codes(float scale) const
    {
        uint32_t r = 0;
        r = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(r, __builtin_bit_cast(bf16x2_t, w[0]), scale, 0);
        r = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(r, __builtin_bit_cast(bf16x2_t, w[1]), scale, 1);
        r = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(r, __builtin_bit_cast(bf16x2_t, w[2]), scale, 2);
        return __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(r, __builtin_bit_cast(bf16x2_t, w[3]), scale, 3);
    }
};
template <>
struct Vec8<1> {                     // fp32
    uint32_t w[8];
    __device__ __forceinline__ uint32_t amax_bits() const
    {
        uint32_t m = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i)
            m = max_u32(m, w[i] & 0x7fffffffu);
        return m;
    }
    __device__ __forceinline__ uint32_t codes(float scale) const
    {
        float f[8];
#pragma unroll
        for (int i = 0; i < 8; ++i)
            f[i] = __builtin_bit_cast(float, w[i]);
        uint32_t r = 0;
        r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, f[0], f[1], scale, 0);
        r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, f[2], f[3], scale, 1);
        r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, f[4], f[5], scale, 2);
        return __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, f[6], f[7], scale, 3);
    }
};

// Elements k .. k+7 of row `row` of x, zeros outside rows x K; kVec: rows are
// 16-byte aligned (base and pitch), so whole groups of 8 are 16-byte loads.
template <int kElem>
__device__ __forceinline__ Vec8<kElem> load8(const void *x, int64_t ldx, int row, int rows, int k,
                                             int K, bool vec)
{
    constexpr int kWords = kElem == 0 ? 4 : 8;
    Vec8<kElem> v;
#pragma unroll
    for (int i = 0; i < kWords; ++i)
        v.w[i] = 0;
    if (row >= rows || k >= K)
        return v;
    if constexpr (kElem == 0) {
        const uint16_t *p = static_cast<const uint16_t *>(x) + row * ldx + k;
        if (vec && k + 8 <= K) {
            const u32x4_t t = *reinterpret_cast<const u32x4_t *>(p);
#pragma unroll
            for (int i = 0; i < 4; ++i)
                v.w[i] = t[i];
        } else {
            const int n = K - k;
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (i < n)
                    v.w[i >> 1] |= (uint32_t)p[i] << (16 * (i & 1));
        }
    } else {
        const uint32_t *p = static_cast<const uint32_t *>(x) + row * ldx + k;
        if (vec && k + 8 <= K) {
            const u32x4_t t = *reinterpret_cast<const u32x4_t *>(p);
            const u32x4_t u = *reinterpret_cast<const u32x4_t *>(p + 4);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                v.w[i] = t[i];
                v.w[4 + i] = u[i];
            }
        } else {
            const int n = K - k;
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (i < n)
                    v.w[i] = p[i];
        }
    }
    return v;
}

__device__ __forceinline__ uint32_t pack2_bf16(float lo, float hi)
{
    const bf16x2_t v = {(__bf16)lo, (__bf16)hi};   // v_cvt_pk_bf16_f32: nearest even
    return __builtin_bit_cast(uint32_t, v);
}

// v_mfma_scale_f32_16x16x128_f8f6f4 on two e2m1 fragments: lane 16 q + x holds
// row x, elements 32 q .. 32 q + 31 of a 128-k step, and byte kOx / kOy of its
// scale word scales that block (checked on gfx950).
template <int kOx, int kOy>
__device__ __forceinline__ f32x4_t mma_f4(const u32x4_t &x, const u32x4_t &y, const f32x4_t &c,
                                          uint32_t sx, uint32_t sy)
{
    const i32x4_t a = __builtin_bit_cast(i32x4_t, x), b = __builtin_bit_cast(i32x4_t, y);
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
        __builtin_shufflevector(a, a, 0, 1, 2, 3, -1, -1, -1, -1),
        __builtin_shufflevector(b, b, 0, 1, 2, 3, -1, -1, -1, -1), c, 4, 4, kOx, (int)sx, kOy, (int)sy);
}

}  // namespace hkg
