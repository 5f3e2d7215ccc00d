// orth_api.cpp -- hkg_orthogonalize (hkg_ops.h): argument checks, workspace
// layout and the launches of its steps, single ones or two at a time.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "ops_internal.h"
#include "orth_kernels.h"

namespace hkg::api {
namespace {

int64_t pad64(int64_t n) { return (n + 63) / 64 * 64; }

// Byte offsets in the workspace: X [m][np], two X^T [n][mp] (the third product
// reads one while it writes the other), three symmetric matrices [m][mp], the norm's
// partial sums.
struct OrthLayout {
    int64_t m, n, mp, np;
    int64_t x, xt[2], a, p, b, sums, bytes;
};
OrthLayout layout(int64_t rows, int64_t cols)
{
    OrthLayout l;
    l.m = rows < cols ? rows : cols;
    l.n = rows < cols ? cols : rows;
    l.mp = pad64(l.m);
    l.np = pad64(l.n);
    int64_t at = 0;
    auto take = [&](int64_t elems) {
        const int64_t here = at;
        at += 2 * elems;         // rows of 128 bytes: every part stays aligned
        return here;
    };
    l.x = take(l.m * l.np);
    l.xt[0] = take(l.n * l.mp);
    l.xt[1] = take(l.n * l.mp);
    l.a = take(l.m * l.mp);
    l.p = take(l.m * l.mp);
    l.b = take(l.m * l.mp);
    l.sums = at;
    l.bytes = at + round16(8 * hkg::orth_norm_parts());
    return l;
}

// A 256-row panel is read through a 32-bit buffer range.
bool sizes_fit(int64_t rows, int64_t cols)
{
    constexpr int64_t kMax = (int64_t(1) << 31) / (256 * 2) - 64;
    return rows <= kMax && cols <= kMax;
}

// Up to so many 32 x 32 blocks a product runs on the kernel for small matrices (five
// steps on it against five on tiles: 256 x 256 68 us against 108, 1024 x 2048 -- 2048
// blocks in its third product -- 213 against 236, 2048 x 2048 665 against 336).
constexpr int64_t kSmallBlocks = 2048;

// The tile of a product (M x N, or the triangle of an M x M): the one whose rounds
// of the 256 compute units take least, a unit's time for a tile growing with its
// area and, for smaller tiles, with the LDS bytes per matrix instruction (two
// 128-tiles share a compute unit).  256-tiles are priced with their last round
// split off (split_last_round), where that is done.
int pick_tile(int64_t M, int64_t N, bool triangle)
{
    const int64_t bm = pad64(M) / 32, bn = pad64(N) / 32;
    if ((triangle ? bm * (bm + 1) / 2 : bm * bn) <= kSmallBlocks)
        return 32;
    int best = 256;
    double least = 0.0;
    for (const int t : {256, 192, 128}) {
        const int64_t gm = ceil_div(M, t), gn = ceil_div(N, t), tiles = triangle ? gm * (gm + 1) / 2 : gm * gn;
        double cost = (double)ceil_div(tiles, 256) * t * t * (t == 256 ? 1.0 : t == 192 ? 1.05 : 1.2);
        if (t == 256 && !triangle && split_last_round(M, N).keep > 0)
            cost = (double)(tiles / 256 + 0.78) * t * t;
        if (least == 0.0 || cost < least) {
            least = cost;
            best = t;
        }
    }
    return best;
}

// Tiles cover the padding of a result's rows and columns too (multiples of 64): it
// holds zeros where the next product takes it for K.
hkg::TileOrder tiles_of(int64_t M, int64_t N, int64_t K, int tile)
{
    return order_of(pad64(M), pad64(N), 2 * K, tile);
}

// X <- P X (m x n), whole or in the two parts of split_last_round.
hipError_t launch_update(int tile, const hkg::OrthProduct &p, const hkg::OrthEpilogue &e, hipStream_t stream)
{
    const TileSplit split = tile == 256 ? split_last_round(p.M, p.N) : TileSplit{0, false};
    if (split.keep == 0)
        return hkg::launch_orth_product(tile, tiles_of(p.M, p.N, p.K, tile), false, p, e, stream);
    hkg::OrthProduct head = p, rest = p;
    hkg::OrthEpilogue re = e;
    const int keep = static_cast<int>(split.keep);
    const int64_t skip = 2 * (int64_t)keep * p.K;   // bytes of its operand rows
    if (split.by_rows) {
        head.M = keep;
        rest.M -= keep;
        rest.A = static_cast<const char *>(p.A) + skip;
        re.straight += e.straight ? keep * e.lds : 0;
        re.transposed += e.transposed ? keep : 0;
        re.cols_t -= keep;
    } else {
        head.N = keep;
        rest.N -= keep;
        rest.B = static_cast<const char *>(p.B) + skip;
        re.straight += e.straight ? keep : 0;
        re.cols_s -= keep;
        re.transposed += e.transposed ? keep * e.ldt : 0;
    }
    const hipError_t err = hkg::launch_orth_product(256, tiles_of(head.M, head.N, p.K, 256), false, head, e, stream);
    if (err != hipSuccess)
        return err;
    return hkg::launch_orth_product(128, tiles_of(rest.M, rest.N, p.K, 128), false, rest, re, stream);
}

// Whether two steps share one pass over X: the second step's A' = X' X'^T is P A P,
// since P is a polynomial of A, so X'' = (P' P) X needs three symmetric m x m products
// more and one product over X's n columns and one update less.  Worth it from n = 1.5 m
// where the update runs on tiles (4096 x 14336: 2574 us against 3368; 4096 x 6144: 1580
// against 1757; 1024 x 2304: even; 2048 x 2560: 408 against 396; small matrices are bound
// by their launches, one more here: 256 x 1024 92 us against 86).  P' P, near a^2 where
// singular values are small, is rounded to fp16 as a whole, which shows next to its
// smaller values, those of the largest singular values: with these between 1 and 1e-4 a
// result's singular values end within 0.02 of the exact ones (0.01 by single steps); a
// larger a takes single steps.
bool steps_in_pairs(int64_t m, int64_t n, int update_tile, float a)
{
    return update_tile != 32 && 2 * n >= 3 * m && a <= 4.0f && a >= -4.0f;
}

}  // namespace
}  // namespace hkg::api

using namespace hkg::api;

extern "C" {

int64_t hkg_orthogonalize_workspace_bytes(int64_t rows, int64_t cols)
{
    if (rows < 0 || cols < 0)
        return HKG_ERR_SHAPE;
    if (!sizes_fit(rows, cols))
        return HKG_ERR_SIZE;
    return rows == 0 || cols == 0 ? 0 : layout(rows, cols).bytes;
}

int hkg_orthogonalize(int64_t rows, int64_t cols, const void *G, int32_t g_type, int64_t ldg,
                      int32_t steps, float a, float b, float c, float eps, void *out, int64_t ldo,
                      void *workspace, int64_t workspace_bytes, void *stream)
{
    const int64_t e = elem_size(g_type);
    if (!e || steps < 0 || steps > 64 || !(eps >= 0.0f))
        return HKG_ERR_OPTS;
    if (rows < 0 || cols < 0)
        return HKG_ERR_SHAPE;
    if (rows == 0 || cols == 0)
        return HKG_OK;
    if (!G || !out || !workspace)
        return HKG_ERR_NULL;
    int rc = check_matrix(G, rows, cols, e, &ldg);
    if (rc == HKG_OK)
        rc = check_matrix(out, rows, cols, 2, &ldo);
    if (rc != HKG_OK)
        return rc;
    if (!aligned16(workspace))
        return HKG_ERR_ALIGN;
    if (!sizes_fit(rows, cols))
        return HKG_ERR_SIZE;
    const OrthLayout l = layout(rows, cols);
    if (workspace_bytes < l.bytes)
        return HKG_ERR_WORKSPACE;
    // G is read to the end before out is written, except with no steps at all,
    // where each element is read and written by one lane: G itself is a valid out
    const bool same = out == G && g_type == HKG_T_BF16 && ldo == ldg;
    const int64_t ob = extent(rows, cols, ldo, 2), gb = extent(rows, cols, ldg, e);
    if ((!same && overlaps(out, ob, G, gb)) || overlaps(workspace, l.bytes, G, gb) ||
        overlaps(workspace, l.bytes, out, ob))
        return HKG_ERR_OVERLAP;
    rc = prepare_launch(stream);
    if (rc != HKG_OK)
        return rc;

    const hipStream_t st = static_cast<hipStream_t>(stream);
    char *ws = static_cast<char *>(workspace);
    uint16_t *x = reinterpret_cast<uint16_t *>(ws + l.x), *am = reinterpret_cast<uint16_t *>(ws + l.a),
             *pm = reinterpret_cast<uint16_t *>(ws + l.p), *bm = reinterpret_cast<uint16_t *>(ws + l.b);
    uint16_t *xt[2] = {reinterpret_cast<uint16_t *>(ws + l.xt[0]), reinterpret_cast<uint16_t *>(ws + l.xt[1])};
    double *sums = reinterpret_cast<double *>(ws + l.sums);
    const hkg::ElemType t = g_type == HKG_T_F32 ? hkg::kElemF32 : hkg::kElemBf16;
    const hkg::OrthInput in = {G, ldg, static_cast<int>(rows), static_cast<int>(cols)};
    const bool tall = rows > cols;
    const int m = static_cast<int>(l.m), n = static_cast<int>(l.n), mp = static_cast<int>(l.mp),
              np = static_cast<int>(l.np);

    rc = launched(hkg::launch_orth_norm(t, in, sums, st));
    if (rc != HKG_OK)
        return rc;
    if (steps == 0)
        return launched(hkg::launch_orth_convert(t, in, sums, eps, nullptr, 0, nullptr, 0,
                                                 static_cast<uint16_t *>(out), ldo, st));
    rc = launched(tall ? hkg::launch_orth_convert(t, in, sums, eps, xt[0], mp, x, np, nullptr, 0, st)
                       : hkg::launch_orth_convert(t, in, sums, eps, x, np, xt[0], mp, nullptr, 0, st));

    const float s = 1.0f / hkg::kOrthScale;
    const int sym = pick_tile(m, m, true), upd = pick_tile(m, n, false);
    // out = alpha A B^T + beta D + diag I, symmetric m x m; A and B have rows of K elements
    auto symmetric = [&](const uint16_t *A, const uint16_t *B, int K, float alpha, float beta, float diag,
                         const uint16_t *D, uint16_t *to) {
        if (rc == HKG_OK)
            rc = launched(hkg::launch_orth_product(
                sym, tiles_of(m, m, K, sym), true, {A, B, m, m, K},
                {alpha, beta, diag, reinterpret_cast<const _Float16 *>(D), mp, mp, to, mp, mp, to, mp, mp, 0}, st));
    };
    const bool pairs = steps_in_pairs(m, n, upd, a);
    for (int i = 0, xi = 0; i < steps && rc == HKG_OK; ++i, xi ^= 1) {
        symmetric(x, x, np, s * s, 0.0f, 0.0f, nullptr, am);   // A = X X^T
        symmetric(am, am, mp, c, b, a, am, pm);                // P = a I + b A + c A A
        const uint16_t *by = pm;
        if (pairs && i + 1 < steps) {
            symmetric(pm, am, mp, 1.0f, 0.0f, 0.0f, nullptr, bm);
            symmetric(pm, bm, mp, 1.0f, 0.0f, 0.0f, nullptr, am);   // A' = P A P
            symmetric(am, am, mp, c, b, a, am, bm);                 // P' = a I + b A' + c A' A'
            symmetric(bm, pm, mp, 1.0f, 0.0f, 0.0f, nullptr, am);   // P' P
            by = am;
            ++i;
        }
        // X <- P X (or P' P X), as X and X^T, or the result in its own orientation
        hkg::OrthEpilogue ep = {1.0f, 0.0f, 0.0f, nullptr, 0, 0, x, np, np, xt[xi ^ 1], mp, mp, 0};
        if (i + 1 == steps) {
            ep = {s, 0.0f, 0.0f, nullptr, 0, 0, nullptr, 0, 0, nullptr, 0, 0, 1};
            if (tall) {
                ep.transposed = static_cast<uint16_t *>(out);
                ep.ldt = ldo;
                ep.cols_t = m;
            } else {
                ep.straight = static_cast<uint16_t *>(out);
                ep.lds = ldo;
                ep.cols_s = n;
            }
        }
        if (rc == HKG_OK)
            rc = launched(launch_update(upd, {by, xt[xi], m, n, mp}, ep, st));
    }
    return rc;
}

}  // extern "C"
