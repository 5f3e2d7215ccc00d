// epilogue.h -- device code of what a product's results pass through on their way
// out: bias, activation, dropout, residual (linear_gemm.hip, linear_kernels.hip).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "linear_kernels.h"
#include "mx4.h"

namespace hkg {

// ---- the 16-bit types -----------------------------------------------------------
struct TypeBf16 {
    __device__ __forceinline__ static float low(uint32_t w) { return __builtin_bit_cast(float, w << 16); }
    __device__ __forceinline__ static float high(uint32_t w) { return __builtin_bit_cast(float, w & 0xffff0000u); }
    __device__ __forceinline__ static uint32_t pack2(float a, float b) { return pack2_bf16(a, b); }
};
struct TypeF16 {
    typedef _Float16 half2 __attribute__((ext_vector_type(2)));
    __device__ __forceinline__ static float low(uint32_t w) { return (float)__builtin_bit_cast(half2, w)[0]; }
    __device__ __forceinline__ static float high(uint32_t w) { return (float)__builtin_bit_cast(half2, w)[1]; }
    __device__ __forceinline__ static uint32_t pack2(float a, float b)   // nearest even; beyond 65504 infinity
    {
        const half2 v = {(_Float16)a, (_Float16)b};
        return __builtin_bit_cast(uint32_t, v);
    }
};

// Eight consecutive values of a row.  Rows start anywhere that suits their element:
// the hardware takes 16-byte accesses at any address.
typedef uint32_t u32x4_any_t __attribute__((ext_vector_type(4), aligned(2)));
// kStream: lines that nothing reads again soon, which then leave the L2 first.
template <bool kStream = false>
__device__ __forceinline__ u32x4_t load16(const void *p)
{
    if constexpr (kStream)
        return __builtin_nontemporal_load(static_cast<const u32x4_any_t *>(p));
    else
        return *static_cast<const u32x4_any_t *>(p);
}
template <bool kStream>
__device__ __forceinline__ void store16(void *p, const u32x4_t &v)
{
    if constexpr (kStream)
        __builtin_nontemporal_store((u32x4_any_t)v, static_cast<u32x4_any_t *>(p));
    else
        *static_cast<u32x4_any_t *>(p) = v;
}

// The first n < 8 of eight elements, as up to three accesses of 4, 2 and 1 of them, all
// sent before the first is needed.
typedef uint32_t u32x2_any_t __attribute__((ext_vector_type(2), aligned(2)));
typedef uint32_t u32_any_t __attribute__((aligned(2)));
// Eight elements of 16 bits in `a`, or of 32 in `a` and `b`.
struct Raw8 {
    u32x4_t a, b;
};
__device__ __forceinline__ u32x4_t load_tail16(const void *p, int n)
{
    const uint16_t *c = static_cast<const uint16_t *>(p);
    u32x2_t x = {0u, 0u};
    uint32_t y = 0u, z = 0u;
    n = n > 0 ? n : 0;
    if (n & 4)
        x = *reinterpret_cast<const u32x2_any_t *>(c);
    if (n & 2)
        y = *reinterpret_cast<const u32_any_t *>(c + (n & 4));
    if (n & 1)
        z = c[n & 6];
    return u32x4_t{(n & 4 ? x[0] : y) | (n == 1 ? z : 0u), x[1] | (n == 3 ? z : 0u), (n & 4 ? y : 0u) | (n == 5 ? z : 0u),
                   n == 7 ? z : 0u};
}
__device__ __forceinline__ void store_tail16(void *p, int n, const u32x4_t &w)
{
    uint16_t *c = static_cast<uint16_t *>(p);
    n = n > 0 ? n : 0;
    if (n & 4)
        *reinterpret_cast<u32x2_any_t *>(c) = u32x2_t{w[0], w[1]};
    if (n & 2)
        *reinterpret_cast<u32_any_t *>(c + (n & 4)) = n & 4 ? w[2] : w[0];
    if (n & 1)
        c[n & 6] = (uint16_t)(n == 1 ? w[0] : n == 3 ? w[1] : n == 5 ? w[2] : w[3]);
}
__device__ __forceinline__ Raw8 load_tail32(const void *p, int n)
{
    const uint32_t *c = static_cast<const uint32_t *>(p);
    u32x4_t x = {0u, 0u, 0u, 0u};
    u32x2_t y = {0u, 0u};
    uint32_t z = 0u;
    n = n > 0 ? n : 0;
    if (n & 4)
        x = *reinterpret_cast<const u32x4_any_t *>(c);
    if (n & 2)
        y = *reinterpret_cast<const u32x2_any_t *>(c + (n & 4));
    if (n & 1)
        z = c[n & 6];
    const bool f = n & 4;
    return Raw8{{f ? x[0] : n == 1 ? z : y[0], f ? x[1] : y[1], f ? x[2] : n == 3 ? z : 0u, x[3]},
                {f ? (n == 5 ? z : y[0]) : 0u, f ? y[1] : 0u, n == 7 ? z : 0u, 0u}};
}
__device__ __forceinline__ void store_tail32(void *p, int n, const Raw8 &w)
{
    uint32_t *c = static_cast<uint32_t *>(p);
    n = n > 0 ? n : 0;
    if (n & 4)
        *reinterpret_cast<u32x4_any_t *>(c) = w.a;
    if (n & 2)
        *reinterpret_cast<u32x2_any_t *>(c + (n & 4)) = n & 4 ? u32x2_t{w.b[0], w.b[1]} : u32x2_t{w.a[0], w.a[1]};
    if (n & 1)
        c[n & 6] = n == 1 ? w.a[0] : n == 3 ? w.a[2] : n == 5 ? w.b[0] : w.b[2];
}

// The first n of the eight elements from p (n < 1: none), the rest zeros.
template <bool kStream = false>
__device__ __forceinline__ Raw8 load_raw8(const void *p, int n, bool f32)
{
    Raw8 r = {{0u, 0u, 0u, 0u}, {0u, 0u, 0u, 0u}};
    if (n >= 8) {
        r.a = load16<kStream>(p);
        if (f32)
            r.b = load16<kStream>(static_cast<const char *>(p) + 16);
    } else if (f32) {
        r = load_tail32(p, n);
    } else {
        r.a = load_tail16(p, n);
    }
    return r;
}
template <class T>
__device__ __forceinline__ void unpack16(const u32x4_t &w, float (&v)[8])
{
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        v[2 * e] = T::low(w[e]);
        v[2 * e + 1] = T::high(w[e]);
    }
}
__device__ __forceinline__ void unpack32(const Raw8 &w, float (&v)[8])
{
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const uint32_t x = w.a[e], y = w.b[e];   // a bit cast of a vector's element reads element 0
        v[e] = __builtin_bit_cast(float, x);
        v[4 + e] = __builtin_bit_cast(float, y);
    }
}
template <class T, bool kStream = false>
__device__ __forceinline__ void load8_16(const void *p, int n, float (&v)[8])
{
    unpack16<T>(load_raw8<kStream>(p, n, false).a, v);
}
__device__ __forceinline__ void load8_32(const void *p, int n, float (&v)[8]) { unpack32(load_raw8(p, n, true), v); }
template <class T, bool kStream = false>
__device__ __forceinline__ void store8_16(void *p, int n, const float (&v)[8])
{
    const u32x4_t w = {T::pack2(v[0], v[1]), T::pack2(v[2], v[3]), T::pack2(v[4], v[5]), T::pack2(v[6], v[7])};
    if (n >= 8)
        store16<kStream>(p, w);
    else
        store_tail16(p, n, w);
}
template <bool kStream = false>
__device__ __forceinline__ void store8_32(void *p, int n, const float (&v)[8])
{
    Raw8 w;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        w.a[e] = __builtin_bit_cast(uint32_t, v[e]);
        w.b[e] = __builtin_bit_cast(uint32_t, v[4 + e]);
    }
    if (n >= 8) {
        store16<kStream>(p, w.a);
        store16<kStream>(static_cast<char *>(p) + 16, w.b);
    } else {
        store_tail32(p, n, w);
    }
}
__device__ __forceinline__ const char *element_at(const void *p, int64_t at, int bytes)
{
    return static_cast<const char *>(p) + at * bytes;
}
__device__ __forceinline__ char *element_at(void *p, int64_t at, int bytes)
{
    return static_cast<char *>(p) + at * bytes;
}

// ---- dropout ----------------------------------------------------------------------
// One call of Philox-4x32-10: a round multiplies two words by constants and mixes the
// products' halves with the other two words and the key; the key grows by constants.
// The 20 multiplications of 32 x 32 bits run at a quarter of the usual rate.
__device__ __forceinline__ u32x4_t philox(uint32_t c0, uint32_t c1, uint32_t c2, uint32_t c3, uint32_t k0, uint32_t k1)
{
#pragma unroll
    for (int r = 0; r < 10; ++r) {
        const uint64_t a = (uint64_t)c0 * 0xD2511F53u, b = (uint64_t)c2 * 0xCD9E8D57u;
        const uint32_t n0 = (uint32_t)(b >> 32) ^ c1 ^ k0, n2 = (uint32_t)(a >> 32) ^ c3 ^ k1;
        c1 = (uint32_t)b;
        c3 = (uint32_t)a;
        c0 = n0;
        c2 = n2;
        k0 += 0x9E3779B9u;
        k1 += 0xBB67AE85u;
    }
    return u32x4_t{c0, c1, c2, c3};
}

// Seed and offset of a launch, in scalar registers.
struct Key {
    uint32_t k0, k1, o0, o1;
    __device__ __forceinline__ explicit Key(const DropoutParams &d)
    {
        uint64_t seed = d.seed, offset = d.offset;
        if (d.rng) {
            seed = d.rng[0];
            offset = d.rng[1];
        }
        k0 = (uint32_t)seed;
        k1 = (uint32_t)(seed >> 32);
        o0 = (uint32_t)offset;
        o1 = (uint32_t)(offset >> 32);
    }
    // the eight numbers of columns 8 group .. 8 group + 7 of a row
    __device__ __forceinline__ u32x4_t numbers(int row, int group) const
    {
        return philox((uint32_t)group, (uint32_t)row, o0, o1, k0, k1);
    }
};
// Whether column e of a group is kept.
__device__ __forceinline__ bool kept(const u32x4_t &n, int e, uint32_t below)
{
    return (e & 1 ? n[e >> 1] >> 16 : n[e >> 1] & 0xffffu) >= below;
}
__device__ __forceinline__ void drop8(const DropoutParams &d, const u32x4_t &n, float (&v)[8])
{
#pragma unroll
    for (int e = 0; e < 8; ++e)
        v[e] = kept(n, e, d.below) ? v[e] * d.scale : 0.0f;
}

// ---- activations ------------------------------------------------------------------
// v_exp_f32 and v_rcp_f32, both within a unit of fp32's last place: a quarter of the
// usual rate each, where the library's functions take ten times as long.
//
// An exponential magnifies its argument's rounding: e^u of an fp32 u is off by up to |u|
// 2^-24, and u reaches 88 where results are still numbers of fp32.  Results of 16 bits are
// formed so (kWide = false: within 2^-15 of the value, where they are rounded by 2^-8 or
// 2^-11), results of 32 bits from arguments of two parts (kWide: within 2^-20; over every fp32 z of
// magnitude 2^-20 .. 2^7 gelu is off by 0.49 of that, silu by 0.23, gelu_tanh by 0.21).  16384 x 14336
// x 4096 with gelu, gelu_tanh and silu into fp32 1518, 1459 and 1410 us so, 1423, 1371 and 1365 as
// 16-bit results are formed; 1 x 14336 x 4096 21.1 either way.
__device__ __forceinline__ float exp2_of(float x) { return __builtin_amdgcn_exp2f(x); }
__device__ __forceinline__ float rcp_of(float x) { return __builtin_amdgcn_rcpf(x); }
constexpr float kLog2e = 1.44269504f;
constexpr float kTanhC = 2.0f * 0.79788456f * kLog2e;   // 2 sqrt(2 / pi), for powers of two
constexpr float kTanhA = 0.044715f;
constexpr float kLargest = 3.4e38f;

// z times a share s(z) of it that is 0 at -infinity: the product is 0 there too.  A NaN
// comes through s.
__device__ __forceinline__ float share(float z, float s) { return __builtin_fmaxf(z, -kLargest) * s; }

// 1 / (1 + 2^-u): 2^-u may be infinity, which gives 0.
__device__ __forceinline__ float sigmoid2(float u) { return rcp_of(1.0f + exp2_of(-u)); }

// h(a) = Phi(-a) exp(a^2 / 2), a >= 0, from k = 1 / (3.25 + a): k Q(k), Q a polynomial fitted for
// the smallest relative error over a < 14 (1.3e-7, 1.5e-7 with these fp32 coefficients), beyond
// which z Phi(z) is below 2^-126.  No cancellation on the left, where Phi is small.
__device__ __forceinline__ float phi_over_exp(float k)
{
    float q = 451.416382f;
    q = __builtin_fmaf(q, k, -562.613159f);
    q = __builtin_fmaf(q, k, 199.171753f);
    q = __builtin_fmaf(q, k, -9.12508869f);
    q = __builtin_fmaf(q, k, 12.8180742f);
    q = __builtin_fmaf(q, k, 3.63388824f);
    q = __builtin_fmaf(q, k, 1.30244911f);
    q = __builtin_fmaf(q, k, 0.398862779f);
    return q * k;
}
struct Normal {
    float g, phi;                  // exp(-z^2 / 2), Phi(z)
    __device__ __forceinline__ explicit Normal(float z)
    {
        g = exp2_of(z * z * (-0.5f * kLog2e));
        const float tail = g * phi_over_exp(rcp_of(__builtin_fabsf(z) + 3.25f));
        phi = z < 0.0f ? tail : 1.0f - tail;
    }
};

// The shares for results of 32 bits, |z| at most 100: 2^t with t a whole number and a rest r,
// and what z's powers and the constants lose in fp32 (x_lo, kXLo) carried along.
// (Written so that constants are inline or single literals: more scalar registers for them
// would spill out of the 256-tiles' epilogue.)
__device__ __forceinline__ float exp2_of(float n, float r) { return __builtin_amdgcn_ldexpf(exp2_of(r), (int)n); }
constexpr float kLog2eLo = 1.925963033e-8f;
constexpr float kTanhCube = 0.102943242f, kTanhCubeLo = -2.01619832e-09f;   // 2 sqrt(2 / pi) 0.044715 log2 e
constexpr float kTanhSum = 22.359375f, kTanhSumLo = 0.00448500225f;           // 1 / 0.044715; kTanhSum has 11 bits

__device__ __forceinline__ float silu_share(float z)
{
    const float n = __builtin_rintf(z * kLog2e), r = __builtin_fmaf(z, -kLog2eLo, __builtin_fmaf(z, -kLog2e, n));
    return rcp_of(1.0f + exp2_of(-n, r));
}
__device__ __forceinline__ float gelu_tanh_share(float z)
{
#pragma clang fp contract(off)   // s and p as rounded: what they lose is in s_lo and p_lo
    // t = -A z (z^2 + 1 / 0.044715), the sum u and the product p in two parts; u - kTanhSum is
    // exact, that constant's last bit being above u's
    const float s = z * z, s_lo = __builtin_fmaf(z, z, -s), u = s + kTanhSum, u_lo = (s - (u - kTanhSum)) + (s_lo + kTanhSumLo);
    const float p = z * u, p_lo = __builtin_fmaf(z, u_lo, __builtin_fmaf(z, u, -p)), n = __builtin_rintf(p * kTanhCube);
    const float r = __builtin_fmaf(p_lo, -kTanhCube, __builtin_fmaf(p, -kTanhCubeLo, __builtin_fmaf(p, -kTanhCube, n)));
    return rcp_of(1.0f + exp2_of(-n, r));
}
// k Q(k) turns an error of k into one three times as large, so what k misses goes in by the
// derivative: h' = a h - 1 / sqrt(2 pi), and k stands for a number that is `off` below a.
__device__ __forceinline__ float gelu_share(float z)
{
    const float s = z * z, s_lo = __builtin_fmaf(z, z, -s), n = __builtin_rintf(s * (0.5f * kLog2e));
    const float r = __builtin_fmaf(s_lo, -0.5f * kLog2e, __builtin_fmaf(s, -0.5f * kLog2eLo, __builtin_fmaf(s, -0.5f * kLog2e, n)));
    const float a = __builtin_fabsf(z), d = a + 3.25f, d_lo = a - (d - 3.25f), k = rcp_of(d), h = phi_over_exp(k);
    const float off = __builtin_fmaf(-d, __builtin_fmaf(-d, k, 1.0f), d_lo);
    const float tail = exp2_of(-n, r) * __builtin_fmaf(off * a, h, __builtin_fmaf(off, -0.39894228f, h));
    return z < 0.0f ? tail : 1.0f - tail;
}

template <int kAct, bool kWide>
__device__ __forceinline__ float act_of(float z)
{
    if constexpr (kAct == kActRelu)
        return z <= 0.0f ? 0.0f : z;
    if constexpr (kWide && kAct != kActNone) {
        // the share is constant beyond +-100, where z's powers are finite; a NaN's is lost here
        const float c = __builtin_amdgcn_fmed3f(z, -100.0f, 100.0f);
        const float v = share(z, kAct == kActGelu ? gelu_share(c) : kAct == kActGeluTanh ? gelu_tanh_share(c) : silu_share(c));
        return z != z ? z : v;
    }
    if constexpr (kAct == kActGelu)
        return share(z, Normal(z).phi);
    if constexpr (kAct == kActGeluTanh)
        return share(z, sigmoid2(z * __builtin_fmaf(kTanhC * kTanhA, z * z, kTanhC)));
    if constexpr (kAct == kActSilu)
        return share(z, sigmoid2(z * kLog2e));
    return z;
}
// Slopes, within 2^-19.  They are constant to fp32's last place beyond +-100; z^2 stays finite
// there.
template <int kAct>
__device__ __forceinline__ float slope_of(float z)
{
    if constexpr (kAct == kActRelu)
        return z <= 0.0f ? 0.0f : z > 0.0f ? 1.0f : z;
    const float c = z < -100.0f ? -100.0f : z > 100.0f ? 100.0f : z;
    if constexpr (kAct == kActGelu) {
        const Normal n(c);
        return __builtin_fmaf(c * 0.39894228f, n.g, n.phi);   // Phi(z) + z exp(-z^2 / 2) / sqrt(2 pi)
    }
    if constexpr (kAct == kActGeluTanh) {
        const float c2 = c * c, s = sigmoid2(c * __builtin_fmaf(kTanhC * kTanhA, c2, kTanhC));
        const float du = __builtin_fmaf(3.0f * kTanhA * 1.59576912f, c2, 1.59576912f);   // 2 u'
        return __builtin_fmaf(c * du, s * (1.0f - s), s);
    }
    if constexpr (kAct == kActSilu) {
        const float s = sigmoid2(c * kLog2e);
        return __builtin_fmaf(c, s * (1.0f - s), s);
    }
    return 1.0f;
}
// f on eight values with the activation a constant inside: one uniform branch.
template <class F>
__device__ __forceinline__ void with_activation(int act, F &&f)
{
    switch (act) {
    case kActRelu: f(std::integral_constant<int, kActRelu>{}); break;
    case kActGelu: f(std::integral_constant<int, kActGelu>{}); break;
    case kActGeluTanh: f(std::integral_constant<int, kActGeluTanh>{}); break;
    case kActSilu: f(std::integral_constant<int, kActSilu>{}); break;
    default: break;
    }
}
// And whether it is evaluated for a result of 32 bits.
template <class F>
__device__ __forceinline__ void with_evaluation(int act, int f32, F &&f)
{
    if (f32)
        with_activation(act, [&](auto a) __attribute__((always_inline)) { f(a, std::true_type{}); });
    else
        with_activation(act, [&](auto a) __attribute__((always_inline)) { f(a, std::false_type{}); });
}
__device__ __forceinline__ void act8(int act, int f32, float (&v)[8])
{
    with_evaluation(act, f32, [&](auto a, auto wide) __attribute__((always_inline)) {
#pragma unroll
        for (int e = 0; e < 8; ++e)
            v[e] = act_of<decltype(a)::value, decltype(wide)::value>(v[e]);
    });
}
__device__ __forceinline__ float act1(int act, int f32, float v)
{
    with_evaluation(act, f32, [&](auto a, auto wide)
                    __attribute__((always_inline)) { v = act_of<decltype(a)::value, decltype(wide)::value>(v); });
    return v;
}

}  // namespace hkg
