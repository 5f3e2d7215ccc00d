// ops_api.cpp -- entry points of the MXFP4 linear layer (hkg_ops.h): argument
// checks, workspace layout and launches.  As in hkg_api.cpp every check runs
// before the first HIP call.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "ops_internal.h"
#include "ops_kernels.h"

namespace hkg::api {
namespace {

bool operand_ok(int32_t o) { return o == HKG_MX_OPERAND_A || o == HKG_MX_OPERAND_B; }

int quantize(int32_t operand, int32_t operand_t, int64_t rows, int64_t K, const void *x,
             int32_t x_type, int64_t ldx, void *codes, void *packed, void *codes_t, void *packed_t,
             bool both, void *stream)
{
    const int64_t e = elem_size(x_type);
    if (!operand_ok(operand) || !operand_ok(operand_t) || !e)
        return HKG_ERR_OPTS;
    if (rows < 0 || K < 0)
        return HKG_ERR_SHAPE;
    if (rows == 0 || K == 0)
        return HKG_OK;
    if (!x || !codes || !packed || (both && (!codes_t || !packed_t)))
        return HKG_ERR_NULL;
    int rc = check_matrix(x, rows, K, e, &ldx);
    if (rc != HKG_OK)
        return rc;
    if (!aligned16(codes) || !aligned16(packed) || !aligned16(codes_t) || !aligned16(packed_t))
        return HKG_ERR_ALIGN;
    if (!mx4_fits(rows, K) || (both && !mx4_fits(K, rows)))
        return HKG_ERR_SIZE;
    const Range r[] = {{codes, mx4_codes(rows, K)},
                       {packed, mx4_scales(rows, K)},
                       {both ? codes_t : nullptr, mx4_codes(K, rows)},
                       {both ? packed_t : nullptr, mx4_scales(K, rows)},
                       {x, extent(rows, K, ldx, e)}};
    if (any_overlap(r, 4))
        return HKG_ERR_OVERLAP;
    rc = prepare_launch(stream);
    if (rc != HKG_OK)
        return rc;
    const hkg::QuantParams p = {x, ldx, static_cast<int>(rows), static_cast<int>(K), operand, operand_t,
                                static_cast<uint8_t *>(codes), static_cast<uint8_t *>(packed),
                                both ? static_cast<uint8_t *>(codes_t) : nullptr,
                                both ? static_cast<uint8_t *>(packed_t) : nullptr};
    return launched(hkg::launch_mx4_quantize(x_type == HKG_T_F32 ? hkg::kElemF32 : hkg::kElemBf16, p,
                                             static_cast<hipStream_t>(stream)));
}

// Shape and operand checks of one product; a pointer may be null where its
// matrix is empty.
int check_product(int64_t M, int64_t N, int64_t K, const void *B, const void *SB, const void *C,
                  int64_t *ldc)
{
    if (M < 0 || N < 0 || K < 0)
        return HKG_ERR_SHAPE;
    if (M == 0 || N == 0)
        return HKG_OK;
    if (!C || (K > 0 && (!B || !SB)))
        return HKG_ERR_NULL;
    int rc = check_matrix(C, M, N, 2, ldc);
    if (rc != HKG_OK)
        return rc;
    if (!aligned16(B) || !aligned16(SB) || !aligned16(C))
        return HKG_ERR_ALIGN;
    if (!mx4_fits(M, K) || !mx4_fits(N, K) ||
        ceil_div(M, kTile) * ceil_div(N, kTile) >= (int64_t(1) << 30))
        return HKG_ERR_SIZE;
    return HKG_OK;
}

hkg::Mx4GemmParams product(int64_t M, int64_t N, int64_t K, const void *A, const void *SA,
                           const void *B, const void *SB, void *C, float *C_f32, int64_t ldc)
{
    hkg::Mx4GemmParams p = {};
    p.A = static_cast<const uint8_t *>(A);
    p.SA = static_cast<const uint8_t *>(SA);
    p.B = static_cast<const uint8_t *>(B);
    p.SB = static_cast<const uint8_t *>(SB);
    p.C = static_cast<uint16_t *>(C);
    p.C_f32 = C_f32;
    p.ldc = ldc;
    p.M = static_cast<int>(M);
    p.N = static_cast<int>(N);
    p.K = static_cast<int>(K);
    p.kb = static_cast<int>(pad32(K) / 2);
    return p;
}

// The product of two MXFP4 matrices: up to 512 blocks of 64 x 32 results (two for each
// compute unit) the kernel for few rows, which splits K over a workgroup's waves; above,
// tiles, which read each operand fewer times.  Measured at 512 blocks: 256 x 4096 x 4096
// 9.3 us against 10.7 on 128-tiles, 512 x 2048 x 2048 6.3 against 7.2, 256 x 4096 x 14336
// 24.4 against 35.8; at 896 and 1024: 128 x 14336 x 4096 17.6 against 13.4, 256 x 8192 x
// 8192 34.5 against 23.2.  Up to 128 tiles of 256 (one round of 512 at two a compute unit)
// 128-tiles: 2048 x 4096 22.9 us against 27.3 at K = 4096 and 65 against 72 at 14336, 2816 x
// 2816 (121) 22.3 against 26.8; above, 256-tiles: 2048 x 4352 (136) 27.0 against 31.4 and 72
// against 93.  At K = 512 128-tiles are a tenth faster there, 10.1 against 11.3.
int product_tile(const hkg::Mx4GemmParams &p)   // 0: the kernel for few rows
{
    if (ceil_div(p.M, 64) * ceil_div(p.N, 32) <= 512)
        return 0;
    return ceil_div(p.M, 256) * ceil_div(p.N, 256) <= 128 ? 128 : 256;
}

hipError_t run_product(const hkg::Mx4GemmParams &p, void *stream)
{
    const hipStream_t st = static_cast<hipStream_t>(stream);
    if (p.K == 0)
        return hkg::launch_mx4_zero(p, st);
    const int tile = product_tile(p);
    if (tile == 0)
        return hkg::launch_mx4_few_rows(hkg::kElemBf16, p, st);
    if (tile == 128)
        return hkg::launch_mx4_tiles(128, order_of(p.M, p.N, p.kb, 128), p, st);
    const TileSplit split = split_last_round(p.M, p.N);
    hkg::Mx4GemmParams head = p, rest = p;
    if (split.keep > 0) {
        // a multiple of 256 rows or columns: whole groups of packed scales
        const int64_t packed = mx_packed_bytes(split.keep, 2 * (int64_t)p.kb), codes = split.keep * p.kb;
        const int64_t at = split.by_rows ? split.keep * p.ldc : split.keep;
        (split.by_rows ? head.M : head.N) = static_cast<int>(split.keep);
        (split.by_rows ? rest.M : rest.N) -= static_cast<int>(split.keep);
        (split.by_rows ? rest.A : rest.B) += codes;
        (split.by_rows ? rest.SA : rest.SB) += packed;
        rest.C += at;
        rest.C_f32 += rest.C_f32 ? at : 0;
    }
    const hipError_t e = hkg::launch_mx4_tiles(256, order_of(head.M, head.N, p.kb, 256), head, st);
    if (e != hipSuccess || split.keep == 0)
        return e;
    return hkg::launch_mx4_tiles(128, order_of(rest.M, rest.N, p.kb, 128), rest, st);
}

// Two independent products (K > 0 in both), in one launch where both take the same kernel: a launch less
// for small ones (the gradients of 500 x 1000 x 768: 17.2 us against 20.8), one partial
// last round instead of two for large ones, the longer tiles first (8192 x 14336 x 4096:
// 484 us against 490).
hipError_t run_products(const hkg::Mx4GemmParams &p, const hkg::Mx4GemmParams &p2, void *stream)
{
    const hipStream_t st = static_cast<hipStream_t>(stream);
    const int tile = product_tile(p);
    if (tile != product_tile(p2)) {
        const hipError_t e = run_product(p, stream);
        return e != hipSuccess ? e : run_product(p2, stream);
    }
    if (tile == 0)
        return hkg::launch_mx4_few_rows2(p, p2, st);
    const hkg::Mx4GemmParams &a = p.kb >= p2.kb ? p : p2, &b = p.kb >= p2.kb ? p2 : p;
    return hkg::launch_mx4_tiles2(tile, order_of(a.M, a.N, a.kb, tile), a, order_of(b.M, b.N, b.kb, tile), b, st);
}

// Whether the linear layer quantises x inside the product: up to 16 rows, whose part of
// the work each workgroup then repeats, while that costs less than a launch of its own.
// In replayed graphs, one launch against two: 1 and 16 x 4096 x 4096 5.0 and 5.7 us against
// 6.8 and 7.2, x 14336 x 4096 7.7 and 9.7 against 10.0 and 10.6; even at K = 8192 (x 4096 7.7
// and 8.9 against 8.1 and 8.7); at K = 14336 two are better for one row as for
// sixteen (x 4096 11.8 and 14.4 against 10.6 and 11.5).
bool fused_linear(int64_t M, int64_t K) { return M <= 16 && K <= 10240; }

}  // namespace
}  // namespace hkg::api

using namespace hkg::api;

extern "C" {

int64_t hkg_mxfp4_code_bytes(int64_t rows, int64_t K)
{
    if (rows < 0 || K < 0)
        return HKG_ERR_SHAPE;
    if (!mx4_fits(rows, K))
        return HKG_ERR_SIZE;
    return mx4_codes(rows, K);
}

int hkg_mxfp4_quantize(int32_t operand, int64_t rows, int64_t K, const void *x, int32_t x_type,
                       int64_t ldx, void *codes, void *packed, void *stream)
{
    return quantize(operand, operand, rows, K, x, x_type, ldx, codes, packed, nullptr, nullptr, false,
                    stream);
}

int hkg_mxfp4_quantize_both(int32_t operand, int32_t operand_t, int64_t rows, int64_t K,
                            const void *x, int32_t x_type, int64_t ldx, void *codes, void *packed,
                            void *codes_t, void *packed_t, void *stream)
{
    return quantize(operand, operand_t, rows, K, x, x_type, ldx, codes, packed, codes_t, packed_t,
                    true, stream);
}

int hkg_mxfp4_dequantize(int32_t operand, int64_t rows, int64_t K, const void *codes,
                         const void *packed, void *values, int32_t v_type, int64_t ldv,
                         void *stream)
{
    const int64_t e = elem_size(v_type);
    if (!operand_ok(operand) || !e)
        return HKG_ERR_OPTS;
    if (rows < 0 || K < 0)
        return HKG_ERR_SHAPE;
    if (rows == 0 || K == 0)
        return HKG_OK;
    if (!codes || !packed || !values)
        return HKG_ERR_NULL;
    if (!mx4_fits(rows, K))
        return HKG_ERR_SIZE;
    const int64_t kp = pad32(K);
    int rc = check_matrix(values, rows, kp, e, &ldv);
    if (rc != HKG_OK)
        return rc;
    if (!aligned16(codes) || !aligned16(packed))
        return HKG_ERR_ALIGN;
    const Range r[] = {{values, extent(rows, kp, ldv, e)},
                       {codes, mx4_codes(rows, K)},
                       {packed, mx4_scales(rows, K)}};
    if (any_overlap(r, 1))
        return HKG_ERR_OVERLAP;
    rc = prepare_launch(stream);
    if (rc != HKG_OK)
        return rc;
    const hkg::DequantParams p = {static_cast<const uint8_t *>(codes), static_cast<const uint8_t *>(packed),
                                  values, ldv, static_cast<int>(rows), static_cast<int>(kp), operand};
    return launched(hkg::launch_mx4_dequantize(v_type == HKG_T_F32 ? hkg::kElemF32 : hkg::kElemBf16, p,
                                               static_cast<hipStream_t>(stream)));
}

int hkg_gemm_mxfp4(int64_t M, int64_t N, int64_t K, const void *A, const void *B, const void *SA,
                   const void *SB, void *C, float *C_f32, int64_t ldc, void *stream)
{
    int rc = check_product(M, N, K, B, SB, C, &ldc);
    if (rc != HKG_OK || M == 0 || N == 0)
        return rc;
    if (K > 0 && (!A || !SA))
        return HKG_ERR_NULL;
    if (!aligned16(A) || !aligned16(SA) || !aligned16(C_f32))
        return HKG_ERR_ALIGN;
    const Range r[] = {{C, extent(M, N, ldc, 2)}, {C_f32, extent(M, N, ldc, 4)},
                       {A, mx4_codes(M, K)},      {SA, mx4_scales(M, K)},
                       {B, mx4_codes(N, K)},      {SB, mx4_scales(N, K)}};
    if (any_overlap(r, 2))
        return HKG_ERR_OVERLAP;
    rc = prepare_launch(stream);
    if (rc != HKG_OK)
        return rc;
    return launched(run_product(product(M, N, K, A, SA, B, SB, C, C_f32, ldc), stream));
}

int64_t hkg_linear_mxfp4_workspace_bytes(int64_t M, int64_t N, int64_t K)
{
    if (M < 0 || N < 0 || K < 0)
        return HKG_ERR_SHAPE;
    if (!mx4_fits(M, K) || !mx4_fits(N, K))
        return HKG_ERR_SIZE;
    return fused_linear(M, K) || N == 0 ? 0 : round16(mx4_codes(M, K)) + mx4_scales(M, K);
}

int hkg_linear_mxfp4(int64_t M, int64_t N, int64_t K, const void *x, int32_t x_type, int64_t ldx,
                     const void *W, const void *SW, void *y, int64_t ldy, void *workspace,
                     int64_t workspace_bytes, void *stream)
{
    const int64_t e = elem_size(x_type);
    if (!e)
        return HKG_ERR_OPTS;
    int rc = check_product(M, N, K, W, SW, y, &ldy);
    if (rc != HKG_OK || M == 0 || N == 0)
        return rc;
    if (K > 0) {
        if (!x)
            return HKG_ERR_NULL;
        rc = check_matrix(x, M, K, e, &ldx);
        if (rc != HKG_OK)
            return rc;
    }
    const int64_t need = hkg_linear_mxfp4_workspace_bytes(M, N, K);
    if (need > 0) {
        if (!workspace)
            return HKG_ERR_NULL;
        if (!aligned16(workspace))
            return HKG_ERR_ALIGN;
        if (workspace_bytes < need)
            return HKG_ERR_WORKSPACE;
    }
    const Range r[] = {{y, extent(M, N, ldy, 2)},
                       {need > 0 ? workspace : nullptr, need},
                       {x, extent(M, K, ldx, e)},
                       {W, mx4_codes(N, K)},
                       {SW, mx4_scales(N, K)}};
    if (any_overlap(r, 2))
        return HKG_ERR_OVERLAP;
    rc = prepare_launch(stream);
    if (rc != HKG_OK)
        return rc;
    const hkg::ElemType t = x_type == HKG_T_F32 ? hkg::kElemF32 : hkg::kElemBf16;
    const hipStream_t st = static_cast<hipStream_t>(stream);
    if (need == 0 && K > 0) {
        hkg::Mx4GemmParams p = product(M, N, K, nullptr, nullptr, W, SW, y, nullptr, ldy);
        p.x = x;
        p.ldx = ldx;
        return launched(hkg::launch_mx4_few_rows(t, p, st));
    }
    uint8_t *codes = static_cast<uint8_t *>(workspace), *packed = codes + round16(mx4_codes(M, K));
    const hkg::QuantParams q = {x, ldx, static_cast<int>(M), static_cast<int>(K), HKG_MX_OPERAND_A,
                                HKG_MX_OPERAND_A, codes, packed, nullptr, nullptr};
    rc = K > 0 ? launched(hkg::launch_mx4_quantize(t, q, st)) : HKG_OK;
    if (rc != HKG_OK)
        return rc;
    return launched(run_product(product(M, N, K, codes, packed, W, SW, y, nullptr, ldy), stream));
}

int64_t hkg_linear_mxfp4_backward_workspace_bytes(int64_t M, int64_t N, int64_t K)
{
    if (M < 0 || N < 0 || K < 0)
        return HKG_ERR_SHAPE;
    if (!mx4_fits(M, N) || !mx4_fits(N, M) || !mx4_fits(K, N) || !mx4_fits(K, M))
        return HKG_ERR_SIZE;
    return round16(mx4_codes(M, N)) + mx4_scales(M, N) + round16(mx4_codes(N, M)) + mx4_scales(N, M);
}

int hkg_linear_mxfp4_backward(int64_t M, int64_t N, int64_t K, const void *dy, int32_t dy_type,
                              int64_t lddy, const void *Wt, const void *SWt, const void *Xt,
                              const void *SXt, void *dx, int64_t lddx, void *dw, int64_t lddw,
                              void *workspace, int64_t workspace_bytes, void *stream)
{
    const int64_t e = elem_size(dy_type);
    if (!e)
        return HKG_ERR_OPTS;
    if (M < 0 || N < 0 || K < 0)
        return HKG_ERR_SHAPE;
    const bool want_x = dx && M > 0 && K > 0, want_w = dw && N > 0 && K > 0;
    if (!want_x && !want_w)
        return HKG_OK;
    // the pitch of a gradient that is not asked for means nothing
    lddx = want_x ? lddx : K;
    lddw = want_w ? lddw : K;
    int rc = want_x ? check_product(M, K, N, Wt, SWt, dx, &lddx) : HKG_OK;
    if (rc == HKG_OK && want_w)
        rc = check_product(N, K, M, Xt, SXt, dw, &lddw);
    if (rc != HKG_OK)
        return rc;
    const bool have = M > 0 && N > 0;
    const int64_t need = hkg_linear_mxfp4_backward_workspace_bytes(M, N, K);
    if (need < 0)
        return static_cast<int>(need);
    if (have) {
        if (!dy || !workspace)
            return HKG_ERR_NULL;
        rc = check_matrix(dy, M, N, e, &lddy);
        if (rc != HKG_OK)
            return rc;
        if (!aligned16(workspace))
            return HKG_ERR_ALIGN;
        if (workspace_bytes < need)
            return HKG_ERR_WORKSPACE;
    }
    const Range r[] = {{want_x ? dx : nullptr, extent(M, K, lddx, 2)},
                       {want_w ? dw : nullptr, extent(N, K, lddw, 2)},
                       {have ? workspace : nullptr, need},
                       {dy, extent(M, N, lddy, e)},
                       {want_x ? Wt : nullptr, mx4_codes(K, N)},
                       {want_x ? SWt : nullptr, mx4_scales(K, N)},
                       {want_w ? Xt : nullptr, mx4_codes(K, M)},
                       {want_w ? SXt : nullptr, mx4_scales(K, M)}};
    if (any_overlap(r, 3))
        return HKG_ERR_OVERLAP;
    rc = prepare_launch(stream);
    if (rc != HKG_OK)
        return rc;
    const hipStream_t st = static_cast<hipStream_t>(stream);
    uint8_t *q = static_cast<uint8_t *>(workspace), *s = q + round16(mx4_codes(M, N)),
            *qt = s + mx4_scales(M, N), *stt = qt + round16(mx4_codes(N, M));
    if (have) {
        const hkg::QuantParams p = {dy, lddy, static_cast<int>(M), static_cast<int>(N), HKG_MX_OPERAND_A,
                                    HKG_MX_OPERAND_A, q, s, want_w ? qt : nullptr, want_w ? stt : nullptr};
        rc = launched(hkg::launch_mx4_quantize(dy_type == HKG_T_F32 ? hkg::kElemF32 : hkg::kElemBf16, p, st));
    }
    if (rc != HKG_OK)
        return rc;
    const hkg::Mx4GemmParams px = product(M, K, N, q, s, Wt, SWt, dx, nullptr, lddx);
    const hkg::Mx4GemmParams pw = product(N, K, M, qt, stt, Xt, SXt, dw, nullptr, lddw);
    return launched(want_x && want_w ? run_products(px, pw, stream) : run_product(want_x ? px : pw, stream));
}

}  // extern "C"
