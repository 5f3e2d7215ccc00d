// linear_api.cpp -- entry points of hkg_linear.h: argument checks, workspace layout
// and launches.  As in hkg_api.cpp every check runs before the first HIP call.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/hkg_linear.h"
#include "linear_kernels.h"
#include "ops_internal.h"

namespace hkg::api {
namespace {

bool operand_type(int32_t t) { return t == HKG_T_BF16 || t == HKG_T_F16; }

// Element size of a type of this interface that goes with operands of `type`; 0 if it
// is none: `type` itself or fp32.
int64_t size_beside(int32_t t, int32_t type) { return t == HKG_T_F32 ? 4 : t == type ? 2 : 0; }

// Dropout's options as the kernels take them: HKG_ERR_OPTS, HKG_ERR_ALIGN or HKG_OK.
int dropout_params(const hkg_dropout_opts *o, hkg::DropoutParams *d)
{
    *d = {0, 1.0f, 0, 0, nullptr};
    if (!o || o->p == 0.0f)
        return HKG_OK;
    if (!(o->p > 0.0f && o->p <= 1.0f))
        return HKG_ERR_OPTS;
    const double below = static_cast<double>(static_cast<int64_t>(static_cast<double>(o->p) * 65536.0 + 0.5));
    d->below = static_cast<uint32_t>(below);
    d->scale = below < 65536.0 ? static_cast<float>(65536.0 / (65536.0 - below)) : 0.0f;
    if (d->below == 0)
        return HKG_OK;
    if (reinterpret_cast<uintptr_t>(o->rng) & 7u)
        return HKG_ERR_ALIGN;
    d->seed = o->seed;
    d->offset = o->offset;
    d->rng = o->rng;
    return HKG_OK;
}
// The bytes of {seed, offset} that a call reads.
Range rng_range(const hkg::DropoutParams &d) { return {d.rng, d.rng ? 16 : 0}; }

// An operand of the matrix cores [rows][cols], pitch *ld (0 becomes cols).
int check_operand(const void *p, int64_t rows, int64_t cols, int64_t *ld)
{
    const int rc = check_matrix(p, rows, cols, 2, ld);
    if (rc != HKG_OK)
        return rc;
    if (!aligned16(p) || *ld % 8)
        return HKG_ERR_ALIGN;
    return *ld < (int64_t(1) << 31) / (kTile * 2) ? HKG_OK : HKG_ERR_SIZE;
}

// Whether out may share its bytes with the input at `in`: the same matrix, element for element.
bool same_matrix(const void *out, int64_t ldo, const void *in, int64_t ldi) { return out == in && ldo == ldi; }

// How a product runs: the kernel for few rows, 128-tiles with K over `splits` workgroups
// of `steps` K steps each, or tiles.
struct How {
    enum Kind { kFewRows, kSplit, kTiles } kind;
    int splits, steps;
    int64_t few_over;            // how much longer the kernel for few rows takes, ns
};
// The cheapest by what each takes in ns, fitted to replayed graphs over weights in turn (M
// 17 .. 1024; N, K 1024 .. 14336), which they meet within a third:
//   few rows  2000 + rows_grid's a step, for each 256 workgroups; 4000 more where its
//             operands have to be transposed first
//   split     8500 + 750 a step of a part; a part for each compute unit, of 8 steps at least
//   tiles     3000 + 600 a step, for each 256 tiles of 128
// in us: 32 x 4096 x 4096 10.3, 15.1 (8 parts), 34.3; 256 x 4096 x 4096 29.0, 21.3 (4), 37.2;
// 100 x 4096 x 14336 42.9, 32.4 (8), 135; 512 x 1024 x 1024 5.6, 10.5 (2), 9.8; 1024 x 1024 x
// 8192 37.4, 29.9 (4), 56.5; 32 x 8192 x 8192 34.6, 39.2 (4), 71.3; 256 x 14336 x 4096 115, -,
// 45.5.
How how_to(int64_t M, int64_t N, int64_t K, bool transposed)
{
    if (M == 0 || N == 0 || K == 0 || (!transposed && M <= 16))
        return {How::kFewRows, 0, 0, 0};
    const int64_t tiles = ceil_div(M, 128) * ceil_div(N, 128), steps = ceil_div(K, 64);
    if (tiles >= int64_t(1) << 20)      // nothing else comes near, and the products below stay in range
        return {How::kTiles, 0, 0, INT64_MAX / 4};
    const hkg::RowsGrid rows = hkg::rows_grid(M, N);
    const int64_t few = (transposed ? 6000 : 2000) + rows.step_ns * steps * ceil_div(rows.blocks(M, N), 256);
    const int64_t whole = 3000 + 600 * steps * ceil_div(tiles, 256);
    const int64_t most = steps / 8 < 256 / tiles ? steps / 8 : 256 / tiles;
    if (most >= 2) {
        const int64_t each = ceil_div(steps, most), split = 8500 + 750 * each;
        if (split < few && split < whole)
            return {How::kSplit, static_cast<int>(ceil_div(steps, each)), static_cast<int>(each), few - split};
    }
    return {few < whole ? How::kFewRows : How::kTiles, 0, 0, few < whole ? 0 : few - whole};
}
int64_t parts_bytes(const How &h, int64_t M, int64_t N)
{
    return h.kind == How::kSplit ? hkg::linear_parts_bytes(M, N, h.splits) : 0;
}

// The product and its epilogue, on arguments that are checked.
hipError_t run_product(bool f16, const How &h, const hkg::LinearParams &p, void *parts, hipStream_t stream)
{
    if (h.kind == How::kFewRows)
        return hkg::launch_linear_few_rows(f16, p, stream);
    if (h.kind == How::kSplit) {
        const hkg::TileOrder o = order_of(p.M, p.N, 2 * static_cast<int64_t>(p.K), 128);
        return hkg::launch_linear_split(f16, {128, o.Gm, o.Gn, o.W, o.C}, h.splits, h.steps, static_cast<float *>(parts), p, stream);
    }
    // The tile that the GEMM takes for this shape (operands with K along their rows have no
    // 192-tiles, as MXFP8 has none).  Where 256-tiles end in a partial round of the 256
    // compute units, and at least a tenth of the whole would idle, the whole rounds' rows or
    // columns on 256-tiles and the rest on 128-tiles: by columns too, unlike the GEMM (a
    // gradient of 4096 x 14336, K = 8192, 896 tiles: 786 us in four rounds, 735 so).
    const bool transposed = p.tr_a || p.tr_b;
    const int64_t edge = tile_edge(default_schedule(transposed ? hkg::kMx : hkg::kBf16, p.M, p.N)), bytes = 2 * static_cast<int64_t>(p.K);
    const int64_t tiles = ceil_div(p.M, 256) * ceil_div(p.N, 256);
    TileSplit cut = {0, false};
    if (edge == 256 && (256 - tiles % 256) * 10 >= 256 * (tiles / 256 + 1))
        cut = split_last_round(p.M, p.N);
    const auto launch = [&](const hkg::LinearParams &q, int tile) {
        const hkg::TileOrder o = order_of(q.M, q.N, bytes, tile);
        return hkg::launch_linear_tiles(f16, {tile, o.Gm, o.Gn, o.W, o.C}, q, stream);
    };
    if (cut.keep == 0)
        return launch(p, static_cast<int>(edge));
    const int64_t m = cut.by_rows ? cut.keep : p.M, n = cut.by_rows ? p.N : cut.keep;
    const hipError_t e = launch(hkg::linear_part(p, 0, m, 0, n), 256);
    if (e != hipSuccess)
        return e;
    return launch(cut.by_rows ? hkg::linear_part(p, m, p.M - m, 0, p.N) : hkg::linear_part(p, 0, p.M, n, p.N - n), 128);
}

int64_t round8(int64_t n) { return (n + 7) / 8 * 8; }
constexpr int64_t kSumRows = 64;   // rows of dz whose sum is one row of partial sums

// How the gradients' products run, and their workspace: what they read that is formed
// first, whose parts are in this order, and room for the parts of split products.
struct BackwardLayout {
    How x, w;                                    // dx, dw
    int64_t dz, dzt, wt, xt, sums, parts, total;
    BackwardLayout(int64_t M, int64_t N, int64_t K)
    {
        x = how_to(M, K, N, true);
        w = how_to(N, K, M, true);
        // both by the kernel for few rows are one launch, with the bias's sums: worth 5 us of
        // the host's and the GPU's time (500 x 1000 x 768 in fp16 27.6 us a call in four launches,
        // 21.8 in two).  In replayed graphs, where the host's part is gone, in us apart and
        // together: 150 x 140 x 72 16.0 and 7.2, 300 x 300 x 304 19.2 and 8.8, 256 x 512 x 512 13.8 and
        // 10.0, 768 x 768 x 768 24.3 and 22.5; 500 x 1000 x 768 20.7 and 21.4, 400 x 1200 x 800 24.1 and
        // 25.4, 64 x 2048 x 512 15.0 and 16.8, 128 x 1024 x 1024 14.5 and 17.1
        if (x.few_over + w.few_over < 5000 && x.few_over < 4000 && w.few_over < 4000)
            x = w = {How::kFewRows, 0, 0, 0};
        // the kernel for few rows takes transposed copies, tiles the matrices themselves
        dz = 0;
        dzt = dz + 2 * M * round8(N);
        wt = dzt + (w.kind == How::kFewRows ? 2 * N * round8(M) : 0);
        xt = wt + (x.kind == How::kFewRows ? 2 * K * round8(N) : 0);
        sums = xt + (w.kind == How::kFewRows ? 2 * K * round8(M) : 0);
        parts = sums + round16(4 * ceil_div(M, kSumRows) * N);
        const int64_t px = parts_bytes(x, M, K), pw = parts_bytes(w, N, K);
        total = parts + (px > pw ? px : pw);
    }
};
// Operands of the gradients' products are M, N and K long, and their preparation is one
// launch of 64 x 64 tiles.
bool backward_fits(int64_t M, int64_t N, int64_t K)
{
    const int64_t most = (int64_t(1) << 31) / (kTile * 2) - 8;
    return M < most && N < most && K < most &&
           ceil_div(M, 64) * ceil_div(N, 64) + ceil_div(N, 64) * ceil_div(K, 64) + ceil_div(M, 64) * ceil_div(K, 64) <
               (int64_t(1) << 23);
}

}  // namespace
}  // namespace hkg::api

using namespace hkg::api;

extern "C" {

int hkg_dropout(int64_t rows, int64_t cols, const void *x, int32_t x_type, int64_t ldx,
                const hkg_dropout_opts *dropout, const void *residual, int64_t ldr, void *out,
                int32_t out_type, int64_t ldo, void *stream)
{
    if (!operand_type(x_type) && x_type != HKG_T_F32)
        return HKG_ERR_OPTS;
    const int64_t xe = x_type == HKG_T_F32 ? 4 : 2, oe = size_beside(out_type, x_type);
    if (!oe)
        return HKG_ERR_OPTS;
    hkg::DropoutCall p = {};
    int rc = dropout_params(dropout, &p.drop);
    if (rc == HKG_ERR_OPTS)
        return rc;
    if (rows < 0 || cols < 0)
        return HKG_ERR_SHAPE;
    if (rows == 0 || cols == 0)
        return HKG_OK;
    if (!x || !out)
        return HKG_ERR_NULL;
    if (rc != HKG_OK)
        return rc;
    if (cols >= (int64_t(1) << 31))
        return HKG_ERR_SIZE;
    if ((rc = check_matrix(x, rows, cols, xe, &ldx)) != HKG_OK || (rc = check_matrix(out, rows, cols, oe, &ldo)) != HKG_OK ||
        (residual && (rc = check_matrix(residual, rows, cols, oe, &ldr)) != HKG_OK))
        return rc;
    const bool on_x = xe == oe && same_matrix(out, ldo, x, ldx), on_r = same_matrix(out, ldo, residual, ldr);
    const Range r[] = {{out, extent(rows, cols, ldo, oe)},
                       {on_x ? nullptr : x, extent(rows, cols, ldx, xe)},
                       {on_r ? nullptr : residual, extent(rows, cols, ldr, oe)},
                       rng_range(p.drop)};
    if (any_overlap(r, 1))
        return HKG_ERR_OVERLAP;
    rc = prepare_launch(stream);
    if (rc != HKG_OK)
        return rc;
    p.x = x;
    p.residual = residual;
    p.out = out;
    p.ldx = ldx;
    p.ldr = ldr;
    p.ldo = ldo;
    p.rows = static_cast<int>(rows);
    p.cols = static_cast<int>(cols);
    return launched(hkg::launch_dropout(x_type == HKG_T_F16, static_cast<int>(8 * xe), static_cast<int>(8 * oe), p,
                                        static_cast<hipStream_t>(stream)));
}

int64_t hkg_linear_workspace_bytes(int64_t M, int64_t N, int64_t K)
{
    if (M < 0 || N < 0 || K < 0 || K % 8)
        return HKG_ERR_SHAPE;
    if (M >= (int64_t(1) << 31) || N >= (int64_t(1) << 31) || K >= (int64_t(1) << 31) / (kTile * 2) ||
        (M > 16 && ceil_div(M, 128) * ceil_div(N, 128) >= (int64_t(1) << 24)))
        return HKG_ERR_SIZE;
    return M == 0 || N == 0 ? 0 : parts_bytes(how_to(M, N, K, false), M, N);
}

int hkg_linear(int64_t M, int64_t N, int64_t K, int32_t type, const void *x, int64_t ldx,
               const void *W, int64_t ldw, const hkg_epilogue *epilogue, void *y, int32_t y_type,
               int64_t ldy, void *workspace, int64_t workspace_bytes, void *stream)
{
    const hkg_epilogue none = {};
    const hkg_epilogue &e = epilogue ? *epilogue : none;
    const int64_t ye = operand_type(type) ? size_beside(y_type, type) : 0;
    if (!ye || e.activation < HKG_ACT_NONE || e.activation > HKG_ACT_SILU ||
        (e.bias && !size_beside(e.bias_type, type)))
        return HKG_ERR_OPTS;
    hkg::LinearParams p = {};
    const int rng = dropout_params(&e.dropout, &p.drop);
    if (rng == HKG_ERR_OPTS)
        return rng;
    const int64_t need = hkg_linear_workspace_bytes(M, N, K);
    if (need == HKG_ERR_SHAPE)
        return HKG_ERR_SHAPE;
    if (M == 0 || N == 0)
        return HKG_OK;
    if (!y || (K > 0 && (!x || !W)))
        return HKG_ERR_NULL;
    if (rng != HKG_OK)
        return rng;
    int64_t ldr = e.ldr, ldz = e.ldz;
    int rc = K > 0 ? check_operand(x, M, K, &ldx) : HKG_OK;
    if (rc == HKG_OK && K > 0)
        rc = check_operand(W, N, K, &ldw);
    if (rc == HKG_OK)
        rc = check_matrix(y, M, N, ye, &ldy);
    if (rc == HKG_OK && e.residual)
        rc = check_matrix(e.residual, M, N, ye, &ldr);
    if (rc == HKG_OK && e.z)
        rc = check_matrix(e.z, M, N, 2, &ldz);
    if (rc != HKG_OK)
        return rc;
    const int64_t be = e.bias ? size_beside(e.bias_type, type) : 1;
    if (reinterpret_cast<uintptr_t>(e.bias) % static_cast<uintptr_t>(be))
        return HKG_ERR_ALIGN;
    if (need < 0 || N >= (int64_t(1) << 31))
        return HKG_ERR_SIZE;
    if (need > 0) {
        if (!workspace)
            return HKG_ERR_NULL;
        if (!aligned16(workspace))
            return HKG_ERR_ALIGN;
        if (workspace_bytes < need)
            return HKG_ERR_WORKSPACE;
    }
    const bool on_r = same_matrix(y, ldy, e.residual, ldr);
    const Range r[] = {{y, extent(M, N, ldy, ye)},
                       {e.z, e.z ? extent(M, N, ldz, 2) : 0},
                       {need > 0 ? workspace : nullptr, need},
                       {x, extent(M, K, ldx, 2)},
                       {W, extent(N, K, ldw, 2)},
                       {e.bias, N * be},
                       {on_r ? nullptr : e.residual, e.residual ? extent(M, N, ldr, ye) : 0},
                       rng_range(p.drop)};
    if (any_overlap(r, 3))
        return HKG_ERR_OVERLAP;
    rc = prepare_launch(stream);
    if (rc != HKG_OK)
        return rc;
    p.A = static_cast<const uint16_t *>(x);
    p.B = static_cast<const uint16_t *>(W);
    p.lda = K > 0 ? ldx : 0;
    p.ldb = K > 0 ? ldw : 0;
    p.M = static_cast<int>(M);
    p.N = static_cast<int>(N);
    p.K = static_cast<int>(K);
    p.bias = e.bias;
    p.residual = e.residual;
    p.y = y;
    p.z = e.z;
    p.ldr = ldr;
    p.ldy = ldy;
    p.ldz = ldz;
    p.bias_f32 = e.bias_type == HKG_T_F32;
    p.y_f32 = y_type == HKG_T_F32;
    p.act = e.activation;
    return launched(run_product(type == HKG_T_F16, how_to(M, N, K, false), p, workspace, static_cast<hipStream_t>(stream)));
}

int64_t hkg_linear_backward_workspace_bytes(int64_t M, int64_t N, int64_t K)
{
    if (M < 0 || N < 0 || K < 0 || K % 8)
        return HKG_ERR_SHAPE;
    if (!backward_fits(M, N, K))
        return HKG_ERR_SIZE;
    return BackwardLayout(M, N, K).total;
}

int hkg_linear_backward(int64_t M, int64_t N, int64_t K, int32_t type, const void *dy,
                        int32_t dy_type, int64_t lddy, const void *x, int64_t ldx, const void *W,
                        int64_t ldw, const void *z, int64_t ldz, int32_t activation,
                        const hkg_dropout_opts *dropout, void *dx, int64_t lddx, void *dw,
                        int64_t lddw, float *dbias, void *workspace, int64_t workspace_bytes,
                        void *stream)
{
    const int64_t de = operand_type(type) ? size_beside(dy_type, type) : 0;
    if (!de || activation < HKG_ACT_NONE || activation > HKG_ACT_SILU)
        return HKG_ERR_OPTS;
    hkg::PrepareParams p = {};
    const int rng = dropout_params(dropout, &p.drop);
    if (rng == HKG_ERR_OPTS)
        return rng;
    if (M < 0 || N < 0 || K < 0 || K % 8)
        return HKG_ERR_SHAPE;
    const bool want_x = dx && M > 0 && K > 0, want_w = dw && N > 0 && K > 0, want_b = dbias && N > 0;
    if (!want_x && !want_w && !want_b)
        return HKG_OK;
    const bool have = M > 0 && N > 0, act = activation != HKG_ACT_NONE;
    if (have && (!dy || (act && !z) || (want_x && !W) || (want_w && !x)))
        return HKG_ERR_NULL;
    if (rng != HKG_OK)
        return rng;
    int rc = HKG_OK;
    if (have) {
        rc = check_matrix(dy, M, N, de, &lddy);
        if (rc == HKG_OK && act)
            rc = check_matrix(z, M, N, 2, &ldz);
        if (rc == HKG_OK && want_x)
            rc = check_operand(W, N, K, &ldw);
        if (rc == HKG_OK && want_w)
            rc = check_operand(x, M, K, &ldx);
    }
    if (rc == HKG_OK && want_x)
        rc = check_matrix(dx, M, K, 2, &lddx);
    if (rc == HKG_OK && want_w)
        rc = check_matrix(dw, N, K, 2, &lddw);
    if (rc != HKG_OK)
        return rc;
    if (reinterpret_cast<uintptr_t>(want_b ? dbias : nullptr) & 3u)
        return HKG_ERR_ALIGN;
    const int64_t need = hkg_linear_backward_workspace_bytes(M, N, K);
    if (need < 0)
        return static_cast<int>(need);
    if (have) {
        if (!workspace)
            return HKG_ERR_NULL;
        if (!aligned16(workspace))
            return HKG_ERR_ALIGN;
        if (workspace_bytes < need)
            return HKG_ERR_WORKSPACE;
    }
    const Range r[] = {{want_x ? dx : nullptr, want_x ? extent(M, K, lddx, 2) : 0},
                       {want_w ? dw : nullptr, want_w ? extent(N, K, lddw, 2) : 0},
                       {want_b ? dbias : nullptr, 4 * N},
                       {have ? workspace : nullptr, need},
                       {have ? dy : nullptr, have ? extent(M, N, lddy, de) : 0},
                       {have && act ? z : nullptr, have && act ? extent(M, N, ldz, 2) : 0},
                       {have && want_w ? x : nullptr, have && want_w ? extent(M, K, ldx, 2) : 0},
                       {have && want_x ? W : nullptr, have && want_x ? extent(N, K, ldw, 2) : 0},
                       rng_range(p.drop)};
    if (any_overlap(r, 4))
        return HKG_ERR_OVERLAP;
    rc = prepare_launch(stream);
    if (rc != HKG_OK)
        return rc;
    const BackwardLayout at(M, N, K);
    char *const ws = static_cast<char *>(workspace);
    const bool f16 = type == HKG_T_F16;
    const hipStream_t st = static_cast<hipStream_t>(stream);
    if (have) {
        p.dy = dy;
        p.z = z;
        p.x = x;
        p.W = W;
        p.lddy = lddy;
        p.ldz = ldz;
        p.ldx = ldx;
        p.ldw = ldw;
        const bool few_x = want_x && at.x.kind == How::kFewRows, few_w = want_w && at.w.kind == How::kFewRows;
        p.dz = want_x || (want_w && !few_w) ? reinterpret_cast<uint16_t *>(ws + at.dz) : nullptr;
        p.dzt = few_w ? reinterpret_cast<uint16_t *>(ws + at.dzt) : nullptr;
        p.wt = few_x ? reinterpret_cast<uint16_t *>(ws + at.wt) : nullptr;
        p.xt = few_w ? reinterpret_cast<uint16_t *>(ws + at.xt) : nullptr;
        p.sums = want_b ? reinterpret_cast<float *>(ws + at.sums) : nullptr;
        p.M = static_cast<int>(M);
        p.N = static_cast<int>(N);
        p.K = static_cast<int>(K);
        p.dy_f32 = dy_type == HKG_T_F32;
        p.act = activation;
        rc = launched(hkg::launch_linear_prepare(f16, p, st));
    }
    const int groups = static_cast<int>(ceil_div(M, kSumRows));
    // one launch for both, also where one of them is not wanted (it has no rows then): the
    // same blocks, and the same bits
    const bool pair = have && (want_x || want_w) && at.x.kind == How::kFewRows && at.w.kind == How::kFewRows;
    const hkg::RowsGrid rows_of_both = hkg::rows_grid(M > N ? M : N, K);   // the larger product's
    hkg::LinearParams q = {}, qx = {}, qw = {};
    q.drop = {0, 1.0f, 0, 0, nullptr};
    q.N = static_cast<int>(K);
    if (rc == HKG_OK && want_x) {
        q.A = p.dz;
        q.lda = round8(N);
        q.tr_b = at.x.kind != How::kFewRows;
        q.B = q.tr_b ? static_cast<const uint16_t *>(W) : p.wt;
        q.ldb = q.tr_b ? ldw : round8(N);
        q.M = static_cast<int>(M);
        q.K = static_cast<int>(q.tr_b ? N : round8(N));
        q.y = dx;
        q.ldy = lddx;
        if (pair)
            qx = q;
        else
            rc = launched(run_product(f16, at.x, q, ws + at.parts, st));
    }
    if (rc == HKG_OK && want_w) {
        q.tr_a = q.tr_b = at.w.kind != How::kFewRows;
        q.A = q.tr_a ? p.dz : p.dzt;
        q.lda = q.tr_a ? round8(N) : round8(M);
        q.B = q.tr_b ? static_cast<const uint16_t *>(x) : p.xt;
        q.ldb = q.tr_b ? ldx : round8(M);
        q.M = static_cast<int>(N);
        q.K = static_cast<int>(q.tr_a ? M : round8(M));
        q.y = dw;
        q.ldy = lddw;
        if (pair)
            qw = q;
        else
            rc = launched(run_product(f16, at.w, q, ws + at.parts, st));
    }
    if (rc == HKG_OK && pair)
        rc = launched(hkg::launch_linear_few_rows2(f16, rows_of_both, qx, qw, p.sums, groups, static_cast<int>(N),
                                                   want_b ? dbias : nullptr, st));
    if (rc == HKG_OK && want_b && !pair)
        rc = launched(hkg::launch_linear_bias_sum(p.sums, groups, static_cast<int>(N), dbias, st));
    return rc;
}

}  // extern "C"
