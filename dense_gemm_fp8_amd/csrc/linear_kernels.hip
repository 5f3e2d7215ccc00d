// linear_kernels.hip -- gfx950 kernels of the 16-bit linear layer besides its tiles:
// dropout, the product of few rows, and what the gradients' products read.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "epilogue.h"
#include "linear_kernels.h"
#include "tile16.h"

namespace hkg {
namespace {

// ---- dropout ----------------------------------------------------------------------
// A lane takes 16 bytes of the result's rows, 8 columns or 4 of fp32, so that a wave's
// accesses are whole lines; a workgroup is 2^s lanes wide, 2^s near a row's but at most
// 256, and takes kDropRows rows a lane, whose loads are all sent before the first is used.
// Bound by its bytes, which it moves faster than a 2 GiB copy (4.8 TB/s read and written),
// since the last-level cache keeps a part of them: 16384 x 4096 bf16 with a residual 70 us,
// 5.8 TB/s; 8192 x 14336 fp32 150 us, 6.3; 16384 x 16384 bf16 172 us, 6.2; rows that are not
// aligned, 16384 x 4097, 92 us, 4.4.
constexpr int kDropRows = 4;

// Four values of 16 or 32 bits, the first n of them.
template <class T, int kBits>
__device__ __forceinline__ void load4(const void *p, int n, float (&v)[4])
{
    if constexpr (kBits == 16) {
        u32x2_t w;
        if (n >= 4) {
            w = __builtin_nontemporal_load(static_cast<const u32x2_any_t *>(p));
        } else {
            const u32x4_t t = load_tail16(p, n);
            w = u32x2_t{t[0], t[1]};
        }
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            v[2 * e] = T::low(w[e]);
            v[2 * e + 1] = T::high(w[e]);
        }
    } else {
        const u32x4_t w = n >= 4 ? load16<true>(p) : load_tail32(p, n).a;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const uint32_t x = w[e];
            v[e] = __builtin_bit_cast(float, x);
        }
    }
}
__device__ __forceinline__ void store4(float *p, int n, const float (&v)[4])
{
    Raw8 w = {{0u, 0u, 0u, 0u}, {0u, 0u, 0u, 0u}};
#pragma unroll
    for (int e = 0; e < 4; ++e)
        w.a[e] = __builtin_bit_cast(uint32_t, v[e]);
    if (n >= 4)
        store16<true>(p, w.a);
    else
        store_tail32(p, n, w);
}

// Results of 16 bits: a lane's 8 columns are one call of the generator.
template <class T>
__global__ __launch_bounds__(256) void dropout16_kernel(const DropoutCall p, int shift)
{
    const int wide = 1 << shift, tall = 256 >> shift;
    const int group = blockIdx.x * wide + (threadIdx.x & (wide - 1)), col = 8 * group, n = p.cols - col;
    if (n <= 0)
        return;
    const Key key(p.drop);
    for (int64_t top = (int64_t)blockIdx.y * (tall * kDropRows); top < p.rows; top += (int64_t)gridDim.y * (tall * kDropRows)) {
        const int64_t row0 = top + (threadIdx.x >> shift);
        float v[kDropRows][8], r[kDropRows][8];
#pragma unroll
        for (int i = 0; i < kDropRows; ++i) {
            const int64_t row = row0 + i * tall;
            const int m = row < p.rows ? n : 0;
            load8_16<T, true>(element_at(p.x, row * p.ldx + col, 2), m, v[i]);
            if (p.residual)
                load8_16<T, true>(element_at(p.residual, row * p.ldr + col, 2), m, r[i]);
        }
#pragma unroll
        for (int i = 0; i < kDropRows; ++i) {
            const int64_t row = row0 + i * tall;
            if (row >= p.rows)
                continue;
            if (p.drop.below > 0)
                drop8(p.drop, key.numbers((int)row, group), v[i]);
            if (p.residual)
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    v[i][e] += r[i][e];
            store8_16<T, true>(element_at(p.out, row * p.ldo + col, 2), n, v[i]);
        }
    }
}

// Results of 32 bits: a lane's 4 columns are half a call.  Two neighbours share a group of
// 8; the even one calls the generator for one row of each two, the odd one for the other,
// and they exchange the halves.  (With 8 columns a lane, in two accesses of half lines
// each: 8192 x 14336 170 us, and 185 with stores that leave the L2 first.)
template <class T, int kXBits>
__global__ __launch_bounds__(256) void dropout32_kernel(const DropoutCall p, int shift)
{
    const int wide = 1 << shift, tall = 256 >> shift;        // wide at least 2
    const int unit = blockIdx.x * wide + (threadIdx.x & (wide - 1)), col = 4 * unit, n = p.cols - col;
    const bool odd = unit & 1;
    const Key key(p.drop);
    for (int64_t top = (int64_t)blockIdx.y * (tall * kDropRows); top < p.rows; top += (int64_t)gridDim.y * (tall * kDropRows)) {
        const int64_t row0 = top + (threadIdx.x >> shift);
        float v[kDropRows][4], r[kDropRows][4];
#pragma unroll
        for (int i = 0; i < kDropRows; ++i) {
            const int64_t row = row0 + i * tall;
            const int m = row < p.rows ? n : 0;
            load4<T, kXBits>(element_at(p.x, row * p.ldx + col, kXBits / 8), m, v[i]);
            if (p.residual)
                load4<T, 32>(element_at(p.residual, row * p.ldr + col, 4), m, r[i]);
        }
        if (p.drop.below > 0)
#pragma unroll
            for (int i = 0; i < kDropRows; i += 2) {         // every lane, so that its neighbour gets its half
                const u32x4_t w = key.numbers((int)(row0 + (i + odd) * tall), unit >> 1);
                const uint32_t a = quad_xor<0xB1>(odd ? w[0] : w[2]), b = quad_xor<0xB1>(odd ? w[1] : w[3]);
                const uint32_t n0[2] = {odd ? a : w[0], odd ? b : w[1]}, n1[2] = {odd ? w[2] : a, odd ? w[3] : b};
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int s = 16 * (e & 1);
                    v[i][e] = (n0[e >> 1] >> s & 0xffffu) >= p.drop.below ? v[i][e] * p.drop.scale : 0.0f;
                    v[i + 1][e] = (n1[e >> 1] >> s & 0xffffu) >= p.drop.below ? v[i + 1][e] * p.drop.scale : 0.0f;
                }
            }
#pragma unroll
        for (int i = 0; i < kDropRows; ++i) {
            const int64_t row = row0 + i * tall;
            if (row >= p.rows)
                continue;
            if (p.residual)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    v[i][e] += r[i][e];
            store4(reinterpret_cast<float *>(element_at(p.out, row * p.ldo + col, 4)), n, v[i]);
        }
    }
}

// ---- the product of few rows --------------------------------------------------------
// What bounds it is reading B once, so each wave streams its own part of K and keeps a
// run of loads in flight.  One workgroup computes 16 kMb rows x 16 kNb columns; its 8 waves
// take runs of kS 32-k steps in turn: wait for the run in LDS, take its fragments into
// registers, send the next run's loads into the same LDS, multiply while they fly; the
// waves' sums are joined in LDS in a fixed order.  Loads go through LDS so that a wave's
// 16-byte chunks form whole lines of rows.  One token through 14336 x 4096 takes 20-22 us
// (5.3-5.8 TB/s), 16 through 8192 x 8192 28-29 us (4.6-4.8 TB/s; a copy reaches 4.8).
constexpr int kRowWaves = 8;

template <class T>
__device__ __forceinline__ f32x4_t mma16(const u32x4_t &a, const u32x4_t &b, const f32x4_t &c)
{
    if constexpr (std::is_same_v<T, TypeBf16>) {
        typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c,
                                                       0, 0, 0);
    } else {
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8_t, a), __builtin_bit_cast(f16x8_t, b), c,
                                                      0, 0, 0);
    }
}

// 16 kMb rows x 16 kNb columns, runs of kS steps.
template <int kMb, int kNb, int kS>
struct RowsPlan {
    static constexpr int kRow = 64 * kS;                    // bytes of a row in a run
    static constexpr int kChunks = 4 * kS;
    static constexpr int kB = 16 * kNb * kRow, kA = 16 * kMb * kRow;
    static constexpr int kWave = kA + kB;                   // LDS bytes of one wave
    static constexpr int kSums = kRowWaves * 64 * (4 * kNb + 1) * 4;
    static constexpr int kLds = kRowWaves * kWave > kSums ? kRowWaves * kWave : kSums;
    // B's row for lane x of block h: of two blocks interleaved, so that a lane's results
    // are 8 consecutive columns.
    __device__ __forceinline__ static int b_row(int x, int h) { return kNb == 1 ? x : (x & 3) + 8 * (x >> 2) + 4 * h; }
    // Places of a row's chunks in LDS, permuted so that the 16 rows of a fragment fall into
    // different 16-byte slots of the 256-byte bank line: by the four bits of the row that
    // vary among them, of which those that the row's own place does not tell apart.
    __device__ __forceinline__ static int chunk(int bits, int c) { return kS == 4 ? c ^ bits : c ^ (bits >> 1); }
    __device__ __forceinline__ static int a_chunk(int row, int c) { return chunk(row & 15, c); }
    __device__ __forceinline__ static int b_chunk(int row, int c)
    {
        return chunk(kNb == 1 ? row & 15 : (row & 3) | (row >> 3 & 3) << 2, c);
    }
};

template <class T, int kMb, int kNb, int kS>
__device__ __forceinline__ void few_rows_block(const LinearParams &p, int block, char *smem)
{
    using G = RowsPlan<kMb, kNb, kS>;
    constexpr int kCols = 16 * kNb;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int x = lane & 15, q = lane >> 4;
    const int gn = (p.N + kCols - 1) / kCols;
    const int n0 = kCols * (block % gn), m0 = 16 * kMb * (block / gn);
    const int kb = 2 * p.K, pitch_a = (int)(2 * p.lda), pitch_b = (int)(2 * p.ldb);
    const int rows = min(16 * kMb, p.M - m0);
    char *const lb = smem + wave * G::kWave, *const la = lb + G::kB;
    // buffers over the workgroup's rows: rows past the matrix read zeros
    const __amdgpu_buffer_rsrc_t ra = buffer_of(reinterpret_cast<const char *>(p.A) + (int64_t)m0 * pitch_a, panel_range(rows, pitch_a, kb));
    const __amdgpu_buffer_rsrc_t rb = buffer_of(reinterpret_cast<const char *>(p.B) + (int64_t)n0 * pitch_b, panel_range(min(kCols, p.N - n0), pitch_b, kb));
    auto to_lds = [&](__amdgpu_buffer_rsrc_t rs, char *to, int voff) __attribute__((always_inline)) {
        __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, (__attribute__((address_space(3))) void *)to, 16, voff, 0, 0, 0);
    };
    constexpr int kLoadRows = 64 / G::kChunks;              // rows of a wave-wide load
    auto send = [&](int r) __attribute__((always_inline)) {
#pragma unroll
        for (int d = 0; d < G::kB / 1024; ++d) {
            const int row = kLoadRows * d + lane / G::kChunks, at = G::kRow * r + 16 * G::b_chunk(row, lane % G::kChunks);
            to_lds(rb, lb + 1024 * d, at < kb ? row * pitch_b + at : kPastEnd);
        }
#pragma unroll
        for (int d = 0; d < G::kA / 1024; ++d) {
            const int row = kLoadRows * d + lane / G::kChunks, at = G::kRow * r + 16 * G::a_chunk(row, lane % G::kChunks);
            if (kLoadRows * d < rows)                       // past them: whatever LDS holds, in rows not stored
                to_lds(ra, la + 1024 * d, at < kb ? row * pitch_a + at : kPastEnd);
        }
    };
    f32x4_t acc[kMb][kNb];
#pragma unroll
    for (int i = 0; i < kMb; ++i)
#pragma unroll
        for (int h = 0; h < kNb; ++h)
            acc[i][h] = f32x4_t{0.f, 0.f, 0.f, 0.f};
    const int runs = (kb + G::kRow - 1) / G::kRow;
    if (wave < runs)
        send(wave);
    for (int r = wave; r < runs; r += kRowWaves) {
        u32x4_t b[kS][kNb], a[kS][kMb];
        wait_loads<0>();
#pragma unroll
        for (int u = 0; u < kS; ++u) {
#pragma unroll
            for (int h = 0; h < kNb; ++h)
                b[u][h] = *reinterpret_cast<const u32x4_t *>(lb + G::kRow * G::b_row(x, h) + 16 * G::b_chunk(G::b_row(x, h), 4 * u + q));
#pragma unroll
            for (int i = 0; i < kMb; ++i)
                a[u][i] = *reinterpret_cast<const u32x4_t *>(la + G::kRow * (16 * i + x) + 16 * G::a_chunk(x, 4 * u + q));
        }
        wait_lds();                                         // the fragments are in registers: their LDS is free
        if (r + kRowWaves < runs)
            send(r + kRowWaves);
#pragma unroll
        for (int u = 0; u < kS; ++u)
#pragma unroll
            for (int i = 0; i < kMb; ++i)
#pragma unroll
                for (int h = 0; h < kNb; ++h)
                    acc[i][h] = mma16<T>(b[u][h], a[u][i], acc[i][h]);
    }
    const Key key(p.drop);
    constexpr int kPer = 4 * kNb;                            // columns of a lane's results
    float(*part)[64][kPer + 1] = reinterpret_cast<float(*)[64][kPer + 1]>(smem);   // + 1: neighbours' rows fall into other banks
#pragma unroll
    for (int i = 0; i < kMb; ++i) {
        // the sums are complete here for every lane: nothing below may move a
        // matrix instruction under a lane mask
#pragma unroll
        for (int h = 0; h < kNb; ++h)
            asm volatile("" : "+v"(acc[i][h]));
        __syncthreads();
#pragma unroll
        for (int h = 0; h < kNb; ++h)
#pragma unroll
            for (int e = 0; e < 4; ++e)
                part[wave][lane][4 * h + e] = acc[i][h][e];
        __syncthreads();
        // 16 x 16 kNb results, one a thread: lane 16 (c / kPer) + r of the fragments holds row r, column c
        const int r = threadIdx.x / kCols, c = threadIdx.x % kCols, row = m0 + 16 * i + r, col = n0 + c;
        if (r >= 16)
            continue;                                        // 16 columns: half of the threads
        float v = 0.f;
#pragma unroll
        for (int w = 0; w < kRowWaves; ++w)
            v += part[w][16 * (c / kPer) + r][c % kPer];
        if (row >= p.M || col >= p.N)
            continue;
        if (p.bias)
            v += p.bias_f32 ? static_cast<const float *>(p.bias)[col] : T::low(static_cast<const uint16_t *>(p.bias)[col]);
        if (p.z)
            static_cast<uint16_t *>(p.z)[row * p.ldz + col] = (uint16_t)T::pack2(v, 0.f);
        v = act1(p.act, p.y_f32, v);
        if (p.drop.below > 0)
            v = kept(key.numbers(p.row0 + row, (p.col0 + col) >> 3), col & 7, p.drop.below) ? v * p.drop.scale : 0.0f;
        const int64_t at = row * p.ldy + col, from = row * p.ldr + col;
        if (p.y_f32) {
            if (p.residual)
                v += static_cast<const float *>(p.residual)[from];
            static_cast<float *>(p.y)[at] = v;
        } else {
            if (p.residual)
                v += T::low(static_cast<const uint16_t *>(p.residual)[from]);
            static_cast<uint16_t *>(p.y)[at] = (uint16_t)T::pack2(v, 0.f);
        }
    }
}

template <class T, int kMb, int kNb, int kS>
__global__ __launch_bounds__(64 * kRowWaves) void linear_few_rows_kernel(const LinearParams p)
{
    __shared__ __attribute__((aligned(1024))) char smem[RowsPlan<kMb, kNb, kS>::kLds];
    few_rows_block<T, kMb, kNb, kS>(p, blockIdx.x, smem);
}

// dbias: 16 columns a workgroup of the few-rows kernel's size, kTall rows of sums at a time,
// four of them in flight: 128 x 14336 4.2-5.0 us (with 32 columns, 8 rows and one in flight 9).
// One order of the sums, alone and in one launch with the products.
constexpr int kTall = 4 * kRowWaves;
struct BiasSum {
    const float *sums;
    int groups, N;
    float *dbias;
};
__device__ __forceinline__ void bias_sum_block(const BiasSum &b, int block, char *smem)
{
    float(*part)[16] = reinterpret_cast<float(*)[16]>(smem);
    const int c = threadIdx.x & 15, w = threadIdx.x >> 4, col = 16 * block + c;
    float s[4] = {0.f, 0.f, 0.f, 0.f};
    for (int g = w; g < b.groups; g += 4 * kTall)
#pragma unroll
        for (int k = 0; k < 4; ++k)
            s[k] += g + kTall * k < b.groups && col < b.N ? b.sums[(int64_t)(g + kTall * k) * b.N + col] : 0.f;
    part[w][c] = (s[0] + s[1]) + (s[2] + s[3]);
    __syncthreads();
    if (w == 0 && col < b.N) {
        float t = 0.f;
#pragma unroll
        for (int i = 0; i < kTall; ++i)
            t += part[i][c];
        b.dbias[col] = t;
    }
}
__global__ __launch_bounds__(16 * kTall) void linear_bias_sum_kernel(const BiasSum b)
{
    __shared__ char smem[kTall * 16 * 4];
    bias_sum_block(b, blockIdx.x, smem);
}

// Both gradients of a small layer and its bias's: the first `first` workgroups are the first
// product's, those up to `second` the other's, the rest sum.
struct FewRowsPair {
    LinearParams p[2];
    int first, second;
    BiasSum bias;
};
template <class T, int kMb, int kNb, int kS>
__global__ __launch_bounds__(64 * kRowWaves) void linear_few_rows_pair_kernel(const FewRowsPair t)
{
    __shared__ __attribute__((aligned(1024))) char smem[RowsPlan<kMb, kNb, kS>::kLds];
    const int block = blockIdx.x;
    if (block >= t.second)
        bias_sum_block(t.bias, block - t.second, smem);
    else if (block >= t.first)
        few_rows_block<T, kMb, kNb, kS>(t.p[1], block - t.first, smem);
    else
        few_rows_block<T, kMb, kNb, kS>(t.p[0], block, smem);
}

// ---- what the gradients' products read ------------------------------------------------
// 64 x 64 tiles through LDS: a tile of dz, of W or of x a workgroup.  A lane reads 8
// elements of a row, and for the transpose gathers 8 of a column from LDS, whose rows
// are 66 elements long so that the gather's neighbours meet different banks.  The products
// on tiles read the matrices as they are, so only dz is formed for them, once for both:
// 8192 x 14336 bf16 from dy and z (705 MB) 131-138 us, 5.1-5.4 TB/s, bound by its bytes;
// 8192 x 4096 from fp32 32 us, 6.3 TB/s, part of it out of the last-level cache.
// dz is rounded to 16 bits for both products, whose matrix instructions take nothing wider: the
// gradients are off by 0.0023 of their norm in bf16 and 0.0003 in fp16, 0.0017 and 0.0002 of
// which are their own rounding.  dbias sums what it was before.
constexpr int kPrep = 64;
constexpr int kPrepPitch = 66;

template <class T>
__global__ __launch_bounds__(256) void linear_prepare_kernel(const PrepareParams p, int dz_tiles, int w_tiles)
{
    __shared__ uint16_t tile[kPrep * kPrepPitch];
    __shared__ float part[32][kPrep];
    int b = blockIdx.x;
    const int what = b < dz_tiles ? 0 : b < dz_tiles + w_tiles ? 1 : 2;
    b -= what == 0 ? 0 : what == 1 ? dz_tiles : dz_tiles + w_tiles;
    const int rows = what == 1 ? p.N : p.M, cols = what == 0 ? p.N : p.K;
    const int gc = (cols + kPrep - 1) / kPrep, r0 = kPrep * (b / gc), c0 = kPrep * (b % gc);
    uint16_t *const to = what == 0 ? p.dz : nullptr, *const to_t = what == 0 ? p.dzt : what == 1 ? p.wt : p.xt;
    const int64_t ld = (cols + 7) & ~7, ld_t = (rows + 7) & ~7;
    const int g = threadIdx.x & 7, c = c0 + 8 * g;          // the lane's columns
    const Key key(p.drop);
    float sum[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int i = 0; i < kPrep / 32; ++i) {
        const int rl = (threadIdx.x >> 3) + 32 * i, row = r0 + rl, n = row < rows ? cols - c : 0;
        float v[8];
        if (what == 0) {
            if (p.dy_f32)
                load8_32(element_at(p.dy, row * p.lddy + c, 4), n, v);
            else
                load8_16<T>(element_at(p.dy, row * p.lddy + c, 2), n, v);
            if (p.act != kActNone) {
                float z[8];
                load8_16<T>(element_at(p.z, row * p.ldz + c, 2), n, z);
                with_activation(p.act, [&](auto a) __attribute__((always_inline)) {
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        v[e] = e < n ? v[e] * slope_of<decltype(a)::value>(z[e]) : 0.0f;
                });
            }
            if (p.drop.below > 0)
                drop8(p.drop, key.numbers(row, c >> 3), v);
#pragma unroll
            for (int e = 0; e < 8; ++e)
                sum[e] += v[e];
        } else {
            const int64_t at = (int64_t)row * (what == 1 ? p.ldw : p.ldx) + c;
            load8_16<T>(element_at(what == 1 ? p.W : p.x, at, 2), n, v);
        }
        const u32x4_t w = {T::pack2(v[0], v[1]), T::pack2(v[2], v[3]), T::pack2(v[4], v[5]), T::pack2(v[6], v[7])};
        if (to && row < rows && c < cols)
            store16<false>(to + row * ld + c, w);                  // rows of whole groups: zeros past the last column
#pragma unroll
        for (int e = 0; e < 4; ++e)
            *reinterpret_cast<uint32_t *>(&tile[rl * kPrepPitch + 8 * g + 2 * e]) = w[e];
    }
    if (what == 0 && p.sums) {
#pragma unroll
        for (int e = 0; e < 8; ++e)
            part[threadIdx.x >> 3][8 * g + e] = sum[e];
    }
    __syncthreads();
    if (to_t) {
#pragma unroll
        for (int i = 0; i < kPrep / 32; ++i) {
            const int cl = (threadIdx.x >> 3) + 32 * i, col = c0 + cl, row = r0 + 8 * g;
            u32x4_t w;
#pragma unroll
            for (int e = 0; e < 4; ++e)
                w[e] = tile[(8 * g + 2 * e) * kPrepPitch + cl] | (uint32_t)tile[(8 * g + 2 * e + 1) * kPrepPitch + cl] << 16;
            if (col < cols && row < rows)
                store16<false>(to_t + col * ld_t + row, w);        // rows past the matrix are zeros in the tile
        }
    }
    if (what == 0 && p.sums && threadIdx.x < kPrep && c0 + (int)threadIdx.x < cols) {
        float s = 0.f;
#pragma unroll
        for (int i = 0; i < 32; ++i)
            s += part[i][threadIdx.x];
        p.sums[(int64_t)(r0 / kPrep) * cols + c0 + threadIdx.x] = s;
    }
}

template <class T, int kMb, int kNb, int kS>
hipError_t few_rows(const LinearParams &p, hipStream_t stream)
{
    const unsigned blocks = (unsigned)((p.N + 16 * kNb - 1) / (16 * kNb)) * (unsigned)((p.M + 16 * kMb - 1) / (16 * kMb));
    hipLaunchKernelGGL((linear_few_rows_kernel<T, kMb, kNb, kS>), dim3(blocks), dim3(64 * kRowWaves), 0, stream, p);
    return hipGetLastError();
}

template <class T>
hipError_t few_rows_of(const LinearParams &p, hipStream_t stream)
{
    const RowsGrid g = rows_grid(p.M, p.N);
    if (g.mb == 1)
        return few_rows<T, 1, 1, 4>(p, stream);
    if (g.mb == 2)
        return g.nb == 1 ? few_rows<T, 2, 1, 2>(p, stream) : few_rows<T, 2, 2, 2>(p, stream);
    return g.nb == 1 ? few_rows<T, 4, 1, 2>(p, stream) : few_rows<T, 4, 2, 2>(p, stream);
}

template <class T, int kMb, int kNb, int kS>
hipError_t few_rows_pair(FewRowsPair &t, const RowsGrid &g, hipStream_t stream)
{
    t.first = (int)g.blocks(t.p[0].M, t.p[0].N);
    t.second = t.first + (int)g.blocks(t.p[1].M, t.p[1].N);
    const int blocks = t.second + (t.bias.dbias ? (t.bias.N + 15) / 16 : 0);
    hipLaunchKernelGGL((linear_few_rows_pair_kernel<T, kMb, kNb, kS>), dim3((unsigned)blocks), dim3(64 * kRowWaves), 0, stream, t);
    return hipGetLastError();
}
template <class T>
hipError_t few_rows_pair_of(const RowsGrid &g, FewRowsPair &t, hipStream_t stream)
{
    if (g.mb <= 2)
        return few_rows_pair<T, 2, 1, 2>(t, RowsGrid{2, 1, 0}, stream);
    return g.nb == 1 ? few_rows_pair<T, 4, 1, 2>(t, g, stream) : few_rows_pair<T, 4, 2, 2>(t, g, stream);
}

// f(grid, shift): shapes a launch whose lanes take `cols` columns of a row each.
template <class F>
hipError_t dropout_shape(const DropoutCall &p, int cols, F &&f)
{
    const int64_t units = ((int64_t)p.cols + cols - 1) / cols;
    int shift = cols == 4 ? 1 : 0;
    while (shift < 8 && (1 << shift) < units)
        ++shift;
    const int64_t tall = (256 >> shift) * kDropRows, high = (p.rows + tall - 1) / tall, wide = (units + (1 << shift) - 1) >> shift;
    // at most 2^23 workgroups, so that their threads stay below 2^32; more rows in turns
    int64_t turn = (int64_t(1) << 23) / wide;               // wide is at most 2^21
    turn = turn < 65535 ? turn : 65535;
    f(dim3((unsigned)wide, (unsigned)(high < turn ? high : turn)), shift);
    return hipGetLastError();
}
template <class T>
hipError_t dropout_of(int x_bits, int out_bits, const DropoutCall &p, hipStream_t stream)
{
    return dropout_shape(p, out_bits == 16 ? 8 : 4, [&](dim3 grid, int shift) {
        if (out_bits == 16)
            hipLaunchKernelGGL(dropout16_kernel<T>, grid, dim3(256), 0, stream, p, shift);
        else if (x_bits == 16)
            hipLaunchKernelGGL((dropout32_kernel<T, 16>), grid, dim3(256), 0, stream, p, shift);
        else
            hipLaunchKernelGGL((dropout32_kernel<TypeBf16, 32>), grid, dim3(256), 0, stream, p, shift);
    });
}

}  // namespace

hipError_t launch_dropout(bool f16, int x_bits, int out_bits, const DropoutCall &p, hipStream_t stream)
{
    return f16 ? dropout_of<TypeF16>(x_bits, out_bits, p, stream) : dropout_of<TypeBf16>(x_bits, out_bits, p, stream);
}

// A launch's threads have to stay below 2^32, or part of the grid is left out without an
// error: turns of at most 2^22 workgroups.
hipError_t launch_linear_few_rows(bool f16, const LinearParams &p, hipStream_t stream)
{
    constexpr int64_t kMost = int64_t(1) << 22;
    const int64_t high = ((int64_t)p.M + 31) / 32;          // a workgroup has 16 columns at least, and 32 rows if there are
    const int64_t turn_m = high < kMost ? p.M : 32 * kMost, turn_n = 16 * (high < kMost ? kMost / high : 1);
    hipError_t e = hipSuccess;
    for (int64_t m = 0; m < p.M && e == hipSuccess; m += turn_m)
        for (int64_t n = 0; n < p.N && e == hipSuccess; n += turn_n) {
            const LinearParams q = linear_part(p, m, p.M - m < turn_m ? p.M - m : turn_m, n, p.N - n < turn_n ? p.N - n : turn_n);
            e = f16 ? few_rows_of<TypeF16>(q, stream) : few_rows_of<TypeBf16>(q, stream);
        }
    return e;
}

hipError_t launch_linear_few_rows2(bool f16, const RowsGrid &g, const LinearParams &p, const LinearParams &p2, const float *sums, int groups, int N,
                                   float *dbias, hipStream_t stream)
{
    FewRowsPair t = {{p, p2}, 0, 0, {sums, groups, N, dbias}};
    return f16 ? few_rows_pair_of<TypeF16>(g, t, stream) : few_rows_pair_of<TypeBf16>(g, t, stream);
}

hipError_t launch_linear_prepare(bool f16, const PrepareParams &p, hipStream_t stream)
{
    const auto tiles = [](int64_t r, int64_t c) { return (r + kPrep - 1) / kPrep * ((c + kPrep - 1) / kPrep); };
    const int64_t dz = p.dz || p.dzt || p.sums ? tiles(p.M, p.N) : 0, w = p.wt ? tiles(p.N, p.K) : 0,
                  x = p.xt ? tiles(p.M, p.K) : 0;
    if (dz + w + x == 0)
        return hipSuccess;
    if (f16)
        hipLaunchKernelGGL(linear_prepare_kernel<TypeF16>, dim3((unsigned)(dz + w + x)), dim3(256), 0, stream, p, (int)dz, (int)w);
    else
        hipLaunchKernelGGL(linear_prepare_kernel<TypeBf16>, dim3((unsigned)(dz + w + x)), dim3(256), 0, stream, p, (int)dz, (int)w);
    return hipGetLastError();
}

hipError_t launch_linear_bias_sum(const float *sums, int groups, int N, float *dbias, hipStream_t stream)
{
    hipLaunchKernelGGL(linear_bias_sum_kernel, dim3((unsigned)((N + 15) / 16)), dim3(16 * kTall), 0, stream, BiasSum{sums, groups, N, dbias});
    return hipGetLastError();
}

}  // namespace hkg
