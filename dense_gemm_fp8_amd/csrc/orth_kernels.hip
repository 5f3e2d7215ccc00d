// orth_kernels.hip -- gfx950 kernels of the orthogonalised update: the norm, the
// conversion to scaled fp16 (with the transpose), and the three products of a
// step on tile16.h's loop.
//
// With m <= n the smaller and larger side, one step is
//   A = X X^T               m x m, symmetric: only tiles on and above the diagonal
//   B = b A + c A A         m x m, symmetric
//   X <- a X + B X          m x n
// The loop wants both operands with K contiguous: X [m][n] for the first, A for the
// second, B (symmetric) and X^T [n][m] for the third, so the third product's epilogue
// writes X and X^T, and the first two write each off-diagonal tile twice.
//
// What is rounded.  X is held in fp32; what goes into the matrix cores is fp16 (11
// significand bits at bf16's rate), summed in fp32:
// - an error in X that lies outside X's own singular directions grows by a a step, 485
//   times over five, so the state itself must not be rounded to 16 bits (done so, a
//   gradient of rank 1 came out 0.15 of its norm off, one of rank 64 0.02).  An error
//   that a product makes from the left, (B + E) X, stays inside X's row space and does
//   not grow.  Nor does B l, where l = X - h is what X's fp16 form h leaves out, so
//   the third product takes h alone.  X X^T does too, except in small blocks, where l
//   costs little: without it singular values move by up to fp16's step where X has few
//   columns that are not zero;
// - A and B are rounded off the diagonal only.  Their diagonals, where all entries are
//   alike for many gradients and would all be rounded the same way, are fp32 vectors;
//   the matrices hold zeros there;
// - B's diagonal also takes its part of l where it is large (t in OrthEpilogue).  Where
//   it is small beside a, the row still grows, and B_ii l has a part outside X's
//   singular directions that the whole B l has not.
// Against the 64-bit iteration results are 0.0017 .. 0.0019 of the norm off on
// full-rank, low-rank and mixed spectra; the rounding of the result to bf16 alone makes
// 0.0017, and so does the iteration in fp32.
// h is X times 2^12, so that entries, near 1 / sqrt(m n) at first, stay clear of fp16's
// subnormals; singular values may then reach 15.  A and B need no scale: what
// subnormals lose of their small entries (2^-25) is nothing beside a I.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "orth_kernels.h"
#include "tile16.h"

namespace hkg {
namespace {

// Element e of an 8-element group in fp32.
template <int kElem>
__device__ __forceinline__ float element(const Vec8<kElem> &v, int e)
{
    if constexpr (kElem == 0)
        return __builtin_bit_cast(float, e & 1 ? v.w[e >> 1] & 0xffff0000u : v.w[e >> 1] << 16);
    else
        return __builtin_bit_cast(float, v.w[e]);
}
template <int kElem>
__device__ __forceinline__ bool rows_aligned(const OrthInput &p)
{
    return ((reinterpret_cast<uintptr_t>(p.G) | (uintptr_t)(p.ldg * (kElem == 0 ? 2 : 4))) & 15) == 0;
}

// ---- |G|^2: partial sums in 64 bits, joined in a fixed order -----------------
// (64 bits because squares of fp32 values leave fp32's range; reading G bounds it:
// 117 MB of bf16 in 31 us, 3.8 TB/s)
template <int kElem>
__global__ __launch_bounds__(256) void orth_norm_kernel(const OrthInput p, double *partial)
{
    double s = 0.0;
    const bool vec = rows_aligned<kElem>(p);
    // rows without gaps or tails are one long row
    const bool flat = vec && p.ldg == p.cols && p.cols % 8 == 0;
    const int64_t vecs = flat ? (int64_t)p.rows * (p.cols / 8) : (p.cols + 7) / 8;
    const int64_t total = flat ? vecs : vecs * p.rows, stride = (int64_t)gridDim.x * 256;
    constexpr int kU = 4;
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < total; i += kU * stride) {
        Vec8<kElem> v[kU];
#pragma unroll
        for (int u = 0; u < kU; ++u) {
            const int64_t k = i + u * stride;
            if (flat) {
                const u32x4_t *q = static_cast<const u32x4_t *>(p.G) + (k < total ? k : i) * (kElem == 0 ? 1 : 2);
#pragma unroll
                for (int h = 0; h < (kElem == 0 ? 1 : 2); ++h)
#pragma unroll
                    for (int w = 0; w < 4; ++w)
                        v[u].w[4 * h + w] = q[h][w];
            } else {
                const int row = (int)(k / vecs), col = 8 * (int)(k % vecs);
                v[u] = load8<kElem>(p.G, p.ldg, row, p.rows, col, p.cols, vec);
            }
        }
#pragma unroll
        for (int u = 0; u < kU; ++u)
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const double f = (double)element<kElem>(v[u], e);
                s += i + u * stride < total ? f * f : 0.0;
            }
    }
    __shared__ double sums[256];
    sums[threadIdx.x] = s;
    __syncthreads();
    for (int d = 128; d > 0; d >>= 1) {
        if (threadIdx.x < d)
            sums[threadIdx.x] += sums[threadIdx.x + d];
        __syncthreads();
    }
    if (threadIdx.x == 0)
        partial[blockIdx.x] = sums[0];
}

// The fp32 value itself: h has to be the fp16 form of the x that is stored, and the
// compiler may otherwise round the sum behind x to fp16 in one step, to another h where
// x is a tie (an error of a fp16 ulp in B_ii h that the products do not share).
__device__ __forceinline__ float stored(float x)
{
    asm("" : "+v"(x));
    return x;
}

// What fp16 leaves out of eight values, in fp16.
__device__ __forceinline__ f16x8_t low_part(const float (&f)[8])
{
    f16x8_t l;
#pragma unroll
    for (int e = 0; e < 8; ++e)
        l[e] = (_Float16)(f[e] - (float)(_Float16)f[e]);
    return l;
}

// ---- X = G / (|G| + eps), its scaled fp16 form and that of its transpose -----
// A 64 x 64 tile a workgroup: rows x ps (straight) and cols x pt (transposed), and the
// fp32 state, zeros past the matrix.  out: with no steps at all, the bf16 result
// itself.  Bound by its bytes: 14336 x 4096 bf16 reads 117 and writes 470 MB in 105 to
// 118 us, 5.0 to 5.6 TB/s.
template <int kElem>
__global__ __launch_bounds__(256) void orth_convert_kernel(const OrthInput p, const double *partial, int parts,
                                                           float eps, const OrthState state, _Float16 *straight, int ps,
                                                           _Float16 *transposed, int pt, int low, uint16_t *out, int64_t ldo)
{
    __shared__ double sums[256];
    __shared__ __attribute__((aligned(16))) uint16_t tile[64 * 64];
    __shared__ float wide[64 * 65];      // the tile in fp32 where the state is its transpose
    const int tc = (p.cols + 63) / 64, r0 = blockIdx.x / tc * 64, c0 = blockIdx.x % tc * 64;
    const bool vec = rows_aligned<kElem>(p), tall = p.rows > p.cols;
    const int rl = threadIdx.x >> 3, u = threadIdx.x & 7;   // rows rl and rl + 32, unit of 8 columns
    Vec8<kElem> v[2];
#pragma unroll
    for (int h = 0; h < 2; ++h)
        v[h] = load8<kElem>(p.G, p.ldg, r0 + rl + 32 * h, p.rows, c0 + 8 * u, p.cols, vec);
    double s = 0.0;
    for (int i = threadIdx.x; i < parts; i += 256)
        s += partial[i];
    sums[threadIdx.x] = s;
    __syncthreads();
    for (int d = 128; d > 0; d >>= 1) {
        if (threadIdx.x < d)
            sums[threadIdx.x] += sums[threadIdx.x + d];
        __syncthreads();
    }
    // a norm that is no number makes every element NaN; a zero matrix stays zero
    const double norm = sqrt(sums[0]);
    const double mul = norm == 0.0 ? 0.0 : isfinite(norm) ? 1.0 / (norm + (double)eps) : (double)NAN;
    // mul as mantissa and exponent: G 2^exp is exact (the result is at most 1 in
    // size), so one rounding in fp32 is all there is, whatever the norm
    int exp = 0;
    const float mant = (float)frexp(mul, &exp);
    // row r, columns c .. c + 7 of the state
    auto keep = [&](int r, int c, const float (&f)[8]) {
        float *to = state.x + (r >> 4) * state.pitch + (c >> 5) * kOrthBlock + 4 * (16 * ((c >> 3) & 3) + (r & 15));
        *reinterpret_cast<f32x4_t *>(to) = f32x4_t{f[0], f[1], f[2], f[3]};
        *reinterpret_cast<f32x4_t *>(to + kOrthBlock / 2) = f32x4_t{f[4], f[5], f[6], f[7]};
    };
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int row = r0 + rl + 32 * h, col = c0 + 8 * u;
        float f[8];
        f16x8_t x;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            f[e] = stored(ldexpf(element<kElem>(v[h], e), exp + (out ? 0 : kOrthScaleLog2)) * mant);
            x[e] = (_Float16)f[e];
        }
        if (out) {
#pragma unroll
            for (int e = 0; e < 8; ++e)
                if (row < p.rows && col + e < p.cols)
                    out[row * ldo + col + e] = (uint16_t)pack2_bf16(f[e], 0.f);
            continue;
        }
        if (row < p.rows) {
            _Float16 *const to = straight + (int64_t)row * ps + col;
            *reinterpret_cast<f16x8_t *>(to) = x;
            if (low && !tall)
                *reinterpret_cast<f16x8_t *>(to + low) = low_part(f);
        }
        *reinterpret_cast<f16x8_t *>(tile + Stage<4>::place(rl + 32 * h, u)) = x;
        if (tall) {
#pragma unroll
            for (int e = 0; e < 8; ++e)
                wide[(rl + 32 * h) * 65 + 8 * u + e] = f[e];
        } else {
            keep(row, col, f);
        }
    }
    if (out)
        return;
    __syncthreads();
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int c = rl + 32 * h;   // column c, rows 8 u .. + 7
        _Float16 *const to = transposed + (int64_t)(c0 + c) * pt + r0 + 8 * u;
        if (tall) {
            float f[8];
#pragma unroll
            for (int e = 0; e < 8; ++e)
                f[e] = wide[(8 * u + e) * 65 + c];
            keep(c0 + c, r0 + 8 * u, f);
            if (low && c0 + c < p.cols)
                *reinterpret_cast<f16x8_t *>(to + low) = low_part(f);
        }
        if (c0 + c >= p.cols)
            continue;
        u32x4_t w = {0, 0, 0, 0};
#pragma unroll
        for (int e = 0; e < 8; ++e)
            w[e >> 1] |= (uint32_t)tile[Stage<4>::place(8 * u + e, c >> 3) + (c & 7)] << (16 * (e & 1));
        *reinterpret_cast<u32x4_t *>(to) = w;
    }
}

// ---- a product of a step -----------------------------------------------------
// Bound by the matrix cores at the clock the power cap leaves, and the update by its
// state besides: 4096 x 14336 takes 462 to 514 us by the card (378 to 423 in whole rounds of
// 256-tiles, the cores busy 54 % of the launch, the rest in a last round of 128-tiles), of
// which 235 MB of state read and written take 80 to 130, since the tiles of a round end
// together; the last update, which writes none, 412 to 484.  The triangle of a 4096^2
// product takes 66 us over K = 4096 and 202 to 212 over K = 14336 (253 192-tiles on 256
// compute units, the cores busy 64 %).
// Results leave as rows (straight) and / or as columns (transposed), both through a
// staged quarter of the tile (tile16.h): a symmetric product's D is loaded into it and
// each lane replaces D's units by its results; whole runs of rows or of columns leave.
enum ProductKind { kSymmetric, kUpdate, kLastUpdate };

template <bool kBf16>
__device__ __forceinline__ u32x4_t pack8(const float (&v)[8])
{
    u32x4_t w;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if constexpr (kBf16) {
            w[i] = pack2_bf16(v[2 * i], v[2 * i + 1]);
        } else {
            const f16x2_t h = {(_Float16)v[2 * i], (_Float16)v[2 * i + 1]};
            w[i] = __builtin_bit_cast(uint32_t, h);
        }
    }
    return w;
}

// a x + d (h + t (x - h)) as cx x + ch h.  t's 0.6 a: d is near -0.7 a in rows that have
// reached their size with the usual coefficients, and small beside a in those that grow.
struct RowFactors {
    float cx, ch;
    __device__ __forceinline__ RowFactors(float a, float d)
    {
        const float q = d / (0.6f * a);
        const float t = fminf(1.0f, q * q);    // a = 0: 1
        cx = fmaf(d, t, a);
        ch = d * (1.0f - t);
    }
    __device__ __forceinline__ float of(float acc, float x) const
    {
        return stored(fmaf(cx, x, fmaf(ch, (float)(_Float16)x, acc)));
    }
};

template <int kT, ProductKind kKind>
__global__ __launch_bounds__(256, kT == 128 ? 2 : 1) void orth_product_kernel(const TileOperands o, const OrthEpilogue p)
{
    using Loop = TileLoop<F16, kT>;
    constexpr int kB = Loop::kB;
    using St = Stage<kB>;
    static_assert(4 * St::kSide * St::kPitch * 2 <= Loop::kLds, "the four quarters fit the ring");
    __shared__ __attribute__((aligned(1024))) char smem[Loop::kLds];
    int tm, tn;
    if constexpr (kKind == kSymmetric)
        triangle_tile(blockIdx.x, o.Gm, tm, tn);
    else
        remap_tile(blockIdx.x, o.Gm, o.Gn, o.W, o.C, tm, tn);
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
    const int rows = o.rows_a - row0, cols = o.rows_b - col0;   // of the quarter that exist
    barrier();   // every wave has read its last fragments
    const St st(smem, loop.wave);
    const StageOut<kB> out(p.straight, row0 * p.lds + col0, p.lds, rows, p.cols_s - col0, p.cols_s);
    auto leave = [&](int i) __attribute__((always_inline)) {
        if (p.straight && i > 0)
            out.rows16(st, lane, 16 * (i - 1));   // while the next rows are formed
    };
    auto float_of = [](__amdgpu_buffer_rsrc_t rs, int at) {
        return __builtin_bit_cast(float, __builtin_amdgcn_raw_buffer_load_b32(rs, 4 * at, 0, 0));
    };
    auto four_of = [](__amdgpu_buffer_rsrc_t rs, int bytes) {
        return __builtin_bit_cast(f32x4_t, __builtin_amdgcn_raw_buffer_load_b128(rs, bytes, 0, 0));
    };
    if constexpr (kKind == kSymmetric) {
        constexpr int kSlots = St::kPitch / 8;   // units a staged row has room for
        float rj[kB / 2][8] = {}, ri[kB] = {};
        if (p.D) {
            // rows and columns past D read zeros, as do those past r
            const __amdgpu_buffer_rsrc_t rd = buffer_of(p.D + row0 * p.ldd + col0,
                                                        rows > 0 ? (uint32_t)min(rows, St::kSide) * (uint32_t)(2 * p.ldd) : 0u);
#pragma unroll
            for (int k = 0; k < St::kSide * kSlots / 64; ++k) {
                const int at = 64 * k + lane, row = at / kSlots;
                const int u = (St::place(row, at % kSlots) - row * St::kPitch) / 8;   // the permutation is its own inverse
                const bool in = u < St::kUnits && col0 + 8 * u < p.cols_d;
                __builtin_amdgcn_raw_ptr_buffer_load_lds(
                    rd, (__attribute__((address_space(3))) void *)(st.base + 512 * k), 16,
                    in ? (int)(2 * (row * p.ldd + 8 * u)) : kPastEnd, 0, 0, 0);
            }
            const __amdgpu_buffer_rsrc_t rr = buffer_of(p.r, (uint32_t)(4 * p.cols_d));
#pragma unroll
            for (int h = 0; h < kB / 2; ++h)
#pragma unroll
                for (int e = 0; e < 8; e += 4) {
                    const f32x4_t f = four_of(rr, 4 * (col0 + 8 * (4 * h + q) + e));
#pragma unroll
                    for (int w = 0; w < 4; ++w)
                        rj[h][e + w] = f[w];
                }
#pragma unroll
            for (int i = 0; i < kB; ++i)
                ri[i] = float_of(rr, row0 + 16 * i + x);
            wait_loads<0>();
        }
#pragma unroll
        for (int i = 0; i < kB; ++i) {
            settle_row(acc, i);
#pragma unroll
            for (int h = 0; h < kB / 2; ++h) {
                u32x4_t *w = st.unit(16 * i + x, 4 * h + q);
                float v[8];
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    v[e] = p.gamma * acc[i][2 * h + (e >> 2)][e & 3];
                if (p.D) {
                    const f16x8_t d = __builtin_bit_cast(f16x8_t, *w);
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        v[e] = fmaf(fmaf(p.gamma, ri[i] + rj[h][e], p.beta), (float)d[e], v[e]);
                }
                if (tm == tn) {
                    const int row = row0 + 16 * i + x, off = row - (col0 + 8 * (4 * h + q));   // the diagonal's column here
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        if (e == off) {
                            // D's diagonal is held as r, its place in D is zero
                            if (row < p.cols_s)
                                p.diag[row] = fmaf(fmaf(p.gamma, ri[i], p.beta), ri[i], v[e]);
                            v[e] = 0.0f;
                        }
                }
                *w = pack8<false>(v);
            }
            leave(i);
        }
    } else {
        const __amdgpu_buffer_rsrc_t rd = buffer_of(p.d, (uint32_t)(4 * p.rows_d));
        // the state's blocks of these rows; those past the matrix read zeros and are
        // not written
        const int pitch = (int)(4 * p.state.pitch);   // bytes, below 2^28
        const __amdgpu_buffer_rsrc_t rx =
            buffer_of(p.state.x + (row0 >> 4) * p.state.pitch,
                      rows > 0 ? (uint32_t)min((rows + 15) >> 4, kB) * (uint32_t)pitch : 0u);
        auto place = [&](int i, int h) {
            return (col0 >> 5) + h < p.state.blocks ? i * pitch + 4 * kOrthBlock * ((col0 >> 5) + h) + 16 * lane : kPastEnd;
        };
        auto take = [&](f32x4_t (&f)[kB / 2][2], int i) __attribute__((always_inline)) {
#pragma unroll
            for (int h = 0; h < kB / 2; ++h)
#pragma unroll
                for (int e = 0; e < 2; ++e)
                    f[h][e] = four_of(rx, place(i, h) + 2 * kOrthBlock * e);
        };
        f32x4_t now[kB / 2][2], next[kB / 2][2];
        float d = float_of(rd, row0 + x), d_next = 0.0f;
        take(now, 0);
#pragma unroll
        for (int i = 0; i < kB; ++i) {
            if (i + 1 < kB) {                         // in flight while this row is formed
                take(next, i + 1);
                d_next = float_of(rd, row0 + 16 * (i + 1) + x);
            }
            settle_row(acc, i);
            const RowFactors f(p.a, d);
#pragma unroll
            for (int h = 0; h < kB / 2; ++h) {
                float v[8];
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    v[e] = f.of(acc[i][2 * h + (e >> 2)][e & 3], now[h][e >> 2][e & 3]);
                if constexpr (kKind == kUpdate) {
#pragma unroll
                    for (int e = 0; e < 2; ++e)
                        __builtin_amdgcn_raw_buffer_store_b128(
                            __builtin_bit_cast(u32x4_t, f32x4_t{v[4 * e], v[4 * e + 1], v[4 * e + 2], v[4 * e + 3]}), rx,
                            place(i, h) + 2 * kOrthBlock * e, 0, 0);
                } else {
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        v[e] *= p.gamma;
                }
                *st.unit(16 * i + x, 4 * h + q) = pack8<kKind == kLastUpdate>(v);
            }
            leave(i);
#pragma unroll
            for (int h = 0; h < kB / 2; ++h)
#pragma unroll
                for (int e = 0; e < 2; ++e)
                    now[h][e] = next[h][e];
            d = d_next;
        }
    }
    if (p.straight) {
        out.rows16(st, lane, 16 * (kB - 1));
        out.odd_rows(st, lane);
    }
    if (!p.transposed || (kKind == kSymmetric && tm == tn))
        return;
    const bool units = ((reinterpret_cast<uintptr_t>(p.transposed) | (uintptr_t)(2 * p.ldt) | (uintptr_t)(2 * p.cols_t)) & 15) == 0 &&
                       p.ldt < (1 << 22);
    uint16_t *to = p.transposed + col0 * p.ldt + row0;
    const int tcols = p.cols_t - row0;
    const __amdgpu_buffer_rsrc_t rt =
        buffer_of(to, units && cols > 0 ? (uint32_t)min(cols, St::kSide) * (uint32_t)(2 * p.ldt) : 0u);
    lanes_in_step();
#pragma unroll 4
    for (int k = 0; k < St::kSide * St::kUnits / 64; ++k) {
        const int at = 64 * k + lane, u = at % St::kUnits, c = at / St::kUnits;   // rows 8 u .. of column c
        u32x4_t w = {0, 0, 0, 0};
#pragma unroll
        for (int e = 0; e < 8; ++e)
            w[e >> 1] |= (uint32_t)st.base[St::place(8 * u + e, c >> 3) + (c & 7)] << (16 * (e & 1));
        if (units) {
            __builtin_amdgcn_raw_buffer_store_b128(w, rt, 8 * u < tcols ? (int)(2 * (c * p.ldt + 8 * u)) : kPastEnd, 0, 0);
        } else if (c < cols) {
#pragma unroll
            for (int e = 0; e < 8; ++e)
                if (8 * u + e < tcols)
                    to[c * p.ldt + 8 * u + e] = (uint16_t)(w[e >> 1] >> (16 * (e & 1)));
        }
    }
}

// ---- a product of a step on a small matrix -----------------------------------
// What bounds it is the way to memory and back, once a launch and 15 launches an
// update: a workgroup takes 32 x 32 results and its 8 waves split K, each sending all
// loads of a 64-k run at once (whole lines, into LDS of its own) and multiplying when
// they are there; their sums are joined in LDS in a fixed order.  256 x 256: 4 us a
// product, launch included, against 6.5 on 128-tiles, whose loop keeps two K steps in
// flight.
constexpr int kSmallWaves = 8;
constexpr int kSmallPanel = 32 * kStepBytes;   // 32 rows of a run

// kLow: OrthProduct's low; a run's h, then its l, through the same LDS.
template <ProductKind kKind, bool kLow>
__global__ __launch_bounds__(64 * kSmallWaves) void orth_small_kernel(const TileOperands o, const OrthEpilogue p)
{
    __shared__ __attribute__((aligned(1024))) char smem[kSmallWaves * 2 * kSmallPanel];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    int tm = blockIdx.x / o.Gn, tn = blockIdx.x % o.Gn;
    if constexpr (kKind == kSymmetric)
        triangle_tile(blockIdx.x, o.Gm, tm, tn);
    const int row0 = 32 * tm, col0 = 32 * tn, rows = min(32, o.rows_a - row0), cols = min(32, o.rows_b - col0);
    const __amdgpu_buffer_rsrc_t ra = buffer_of(static_cast<const char *>(o.A) + (int64_t)row0 * o.pitch_a,
                                                panel_range(rows, o.pitch_a, o.kb));
    const __amdgpu_buffer_rsrc_t rb = buffer_of(static_cast<const char *>(o.B) + (int64_t)col0 * o.pitch_b,
                                                panel_range(cols, o.pitch_b, o.kb));
    char *const la = smem + wave * 2 * kSmallPanel, *const lb = la + kSmallPanel;
    auto send = [&](int at0) {
#pragma unroll
        for (int d = 0; d < kSmallPanel / kLoadBytes; ++d) {
            const int row = 8 * d + (lane >> 3), at = at0 + (((lane & 7) ^ swz_a(row)) << 4);
            __builtin_amdgcn_raw_ptr_buffer_load_lds(ra, (__attribute__((address_space(3))) void *)(la + d * kLoadBytes), 16,
                                                     row * o.pitch_a + at, 0, 0, 0);
            __builtin_amdgcn_raw_ptr_buffer_load_lds(rb, (__attribute__((address_space(3))) void *)(lb + d * kLoadBytes), 16,
                                                     row * o.pitch_b + at, 0, 0, 0);
        }
    };
    const int x = lane & 15, q = lane >> 4;
    f32x4_t acc[2][2] = {};
    typedef f16x8_t Run[2][2];   // [slice][block]
    auto take = [&](Run &a, Run &b) {
        wait_loads<0>();
#pragma unroll
        for (int s = 0; s < 2; ++s)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int at = (16 * i + x) * kStepBytes + (((4 * s + q) ^ swz_a(16 * i + x)) << 4);
                a[s][i] = *reinterpret_cast<const f16x8_t *>(la + at);
                b[s][i] = *reinterpret_cast<const f16x8_t *>(lb + at);
            }
        wait_lds();   // the fragments are in registers: their LDS is free
    };
    auto multiply = [&](const Run &a, const Run &b) {
#pragma unroll
        for (int s = 0; s < 2; ++s)
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int j = 0; j < 2; ++j)
                    acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_f16(b[s][j], a[s][i], acc[i][j], 0, 0, 0);
    };
    if (wave < o.nk)
        send(wave * kStepBytes);
    for (int t = wave; t < o.nk; t += kSmallWaves) {
        Run a, b;
        take(a, b);
        if constexpr (kLow) {
            send((o.nk + t) * kStepBytes);
            multiply(a, b);
            Run al, bl;
            take(al, bl);
            if (t + kSmallWaves < o.nk)
                send((t + kSmallWaves) * kStepBytes);
            multiply(a, bl);
            multiply(al, b);
        } else {
            if (t + kSmallWaves < o.nk)
                send((t + kSmallWaves) * kStepBytes);
            multiply(a, b);
        }
    }
    settle(acc);
    __syncthreads();
    // [wave][row][column], rows 33 apart: lane (x, q) of block (i, j) holds row 16 i + x,
    // columns 16 j + 4 q ..
    float(*part)[32][33] = reinterpret_cast<float(*)[32][33]>(smem);
    static_assert(kSmallWaves * 32 * 33 * 4 <= kSmallWaves * 2 * kSmallPanel, "the sums fit");
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e)
                part[wave][16 * i + x][16 * j + 4 * q + e] = acc[i][j][e];
    __syncthreads();
    // a thread takes two neighbouring columns of a row, then two neighbouring rows of a
    // column, whose results the others have left in the first wave's part.  Every row and
    // column lies within the padding to 64 of the state, the vectors and D.
    const int fast = 2 * (threadIdx.x & 15), slow = threadIdx.x >> 4;
    float v[2];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
        v[e] = 0.f;
#pragma unroll
        for (int k = 0; k < kSmallWaves; ++k)
            v[e] += part[k][slow][fast + e];
    }
    const int row = row0 + slow, col = col0 + fast;
    if constexpr (kKind == kSymmetric) {
        const float ri = p.D ? p.r[row] : 0.0f;
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            v[e] *= p.gamma;
            if (p.D && slow < rows)
                v[e] = fmaf(fmaf(p.gamma, ri + p.r[col + e], p.beta), (float)p.D[row * p.ldd + col + e], v[e]);
            if (row == col + e) {
                // D's diagonal is held as r, its place in D is zero
                p.diag[row] = fmaf(fmaf(p.gamma, ri, p.beta), ri, v[e]);
                v[e] = 0.0f;
            }
        }
    } else {
        typedef float f32x2_t __attribute__((ext_vector_type(2)));
        const RowFactors f(p.a, p.d[row]);
        f32x2_t *const at = reinterpret_cast<f32x2_t *>(
            p.state.x + (row >> 4) * p.state.pitch + (col >> 5) * kOrthBlock + (kOrthBlock / 2) * ((col >> 2) & 1) +
            4 * (16 * ((col >> 3) & 3) + (row & 15)) + (col & 3));
        const f32x2_t was = *at;
#pragma unroll
        for (int e = 0; e < 2; ++e)
            v[e] = f.of(v[e], was[e]);
        if constexpr (kKind == kUpdate)
            *at = f32x2_t{v[0], v[1]};
        else
            v[0] *= p.gamma, v[1] *= p.gamma;
    }
#pragma unroll
    for (int way = 0; way < 2; ++way) {
        uint16_t *const to = way == 0 ? p.straight : p.transposed;
        if (way == 1) {
            part[0][slow][fast] = v[0];   // read by this thread alone so far
            part[0][slow][fast + 1] = v[1];
            __syncthreads();
            v[0] = part[0][fast][slow];
            v[1] = part[0][fast + 1][slow];
        }
        if (!to)
            continue;
        uint16_t w[2], l[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            l[e] = __builtin_bit_cast(uint16_t, (_Float16)(v[e] - (float)(_Float16)v[e]));
            w[e] = kKind == kLastUpdate ? (uint16_t)pack2_bf16(v[e], 0.f) : __builtin_bit_cast(uint16_t, (_Float16)v[e]);
        }
        const int64_t ld = way == 0 ? p.lds : p.ldt;
        const int line = (way == 0 ? row0 : col0) + slow, at = (way == 0 ? col0 : row0) + fast;
        const int lines = way == 0 ? o.rows_a : o.rows_b, width = way == 0 ? p.cols_s : p.cols_t;
        if (line >= lines)
            continue;
        uint16_t *const d = to + line * ld + at;
        if (kKind == kUpdate && way == 0 && p.low)
            *reinterpret_cast<uint32_t *>(d + p.low) = l[0] | (uint32_t)l[1] << 16;
        if (at + 1 < width && (reinterpret_cast<uintptr_t>(d) & 3) == 0) {
            *reinterpret_cast<uint32_t *>(d) = w[0] | (uint32_t)w[1] << 16;
        } else {
            if (at < width)
                d[0] = w[0];
            if (at + 1 < width)
                d[1] = w[1];
        }
    }
}

}  // namespace

constexpr int kNormParts = 1024;
int orth_norm_parts() { return kNormParts; }

hipError_t launch_orth_norm(ElemType t, const OrthInput &p, double *partial, hipStream_t stream)
{
    if (t == kElemBf16)
        hipLaunchKernelGGL(orth_norm_kernel<0>, dim3(kNormParts), dim3(256), 0, stream, p, partial);
    else
        hipLaunchKernelGGL(orth_norm_kernel<1>, dim3(kNormParts), dim3(256), 0, stream, p, partial);
    return hipGetLastError();
}

hipError_t launch_orth_convert(ElemType t, const OrthInput &p, const double *partial, float eps, const OrthState &state,
                               void *straight, int ps, void *transposed, int pt, int low, uint16_t *out, int64_t ldo,
                               hipStream_t stream)
{
    const dim3 grid((unsigned)((p.rows + 63) / 64) * (unsigned)((p.cols + 63) / 64)), block(256);
    auto s = static_cast<_Float16 *>(straight), tr = static_cast<_Float16 *>(transposed);
    if (t == kElemBf16)
        hipLaunchKernelGGL(orth_convert_kernel<0>, grid, block, 0, stream, p, partial, kNormParts, eps, state, s, ps, tr,
                           pt, low, out, ldo);
    else
        hipLaunchKernelGGL(orth_convert_kernel<1>, grid, block, 0, stream, p, partial, kNormParts, eps, state, s, ps, tr,
                           pt, low, out, ldo);
    return hipGetLastError();
}

template <ProductKind kKind>
static hipError_t launch_product(int tile, bool low, const TileOperands &o, const OrthEpilogue &e, hipStream_t stream)
{
    const dim3 grid(o.triangle ? (unsigned)o.Gm * (unsigned)(o.Gm + 1) / 2 : (unsigned)o.Gm * (unsigned)o.Gn), block(256);
    if (tile == 256)
        hipLaunchKernelGGL((orth_product_kernel<256, kKind>), grid, block, 0, stream, o, e);
    else if (tile == 192)
        hipLaunchKernelGGL((orth_product_kernel<192, kKind>), grid, block, 0, stream, o, e);
    else if (tile == 32 && kKind == kSymmetric && low)
        hipLaunchKernelGGL((orth_small_kernel<kKind, kKind == kSymmetric>), grid, dim3(64 * kSmallWaves), 0, stream, o, e);
    else if (tile == 32)
        hipLaunchKernelGGL((orth_small_kernel<kKind, false>), grid, dim3(64 * kSmallWaves), 0, stream, o, e);
    else
        hipLaunchKernelGGL((orth_product_kernel<128, kKind>), grid, block, 0, stream, o, e);
    return hipGetLastError();
}

hipError_t launch_orth_product(int tile, const TileOrder &order, bool triangle, const OrthProduct &p,
                               const OrthEpilogue &e, hipStream_t stream)
{
    TileOperands o = {};
    o.A = p.A;
    o.B = p.B;
    o.pitch_a = o.pitch_b = o.kb = p.low ? 4 * p.K : 2 * p.K;
    o.rows_a = p.M;
    o.rows_b = p.N;
    o.Gm = order.Gm;
    o.Gn = order.Gn;
    o.W = order.W;
    o.C = order.C;
    o.nk = p.K / 64;
    o.triangle = triangle;
    if (triangle)
        return launch_product<kSymmetric>(tile, p.low, o, e, stream);
    return e.last ? launch_product<kLastUpdate>(tile, false, o, e, stream)
                  : launch_product<kUpdate>(tile, false, o, e, stream);
}

}  // namespace hkg
