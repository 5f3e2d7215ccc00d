// orth_api.cpp -- hkg_orthogonalize (hkg_ops.h): argument checks, workspace
// layout and the launches of its steps.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "ops_internal.h"
#include "orth_kernels.h"

namespace hkg::api {
namespace {

int64_t pad64(int64_t n) { return (n + 63) / 64 * 64; }

// Byte offsets in the workspace: X [m][np], two X^T [n][mp] (the third product
// reads one while it writes the other), A and P [m][mp], the norm's partial sums.
struct OrthLayout {
    int64_t m, n, mp, np;
    int64_t x, xt[2], a, p, sums, bytes;
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
             *pm = reinterpret_cast<uint16_t *>(ws + l.p);
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
    for (int i = 0; i < steps && rc == HKG_OK; ++i) {
        const bool last = i + 1 == steps;
        // A = X X^T
        rc = launched(hkg::launch_orth_product(sym, tiles_of(m, m, np, sym), true, {x, x, m, m, np},
                                               {s * s, 0.0f, 0.0f, nullptr, 0, 0, am, mp, mp, am, mp, mp, 0}, st));
        // P = a I + b A + c A A
        if (rc == HKG_OK)
            rc = launched(hkg::launch_orth_product(
                sym, tiles_of(m, m, mp, sym), true, {am, am, m, m, mp},
                {c, b, a, reinterpret_cast<const _Float16 *>(am), mp, mp, pm, mp, mp, pm, mp, mp, 0}, st));
        // X <- P X, as X and X^T, or the result in its own orientation
        hkg::OrthEpilogue ep = {1.0f, 0.0f, 0.0f, nullptr, 0, 0, x, np, np, xt[(i + 1) & 1], mp, mp, 0};
        if (last) {
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
            rc = launched(launch_update(upd, {pm, xt[i & 1], m, n, mp}, ep, st));
    }
    return rc;
}

}  // extern "C"
