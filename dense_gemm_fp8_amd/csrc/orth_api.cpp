// orth_api.cpp -- hkg_orthogonalize (hkg_ops.h): argument checks, workspace
// layout and the launches of its steps.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "ops_internal.h"
#include "orth_kernels.h"

namespace hkg::api {
namespace {

int64_t pad64(int64_t n) { return (n + 63) / 64 * 64; }

// Up to so many 32 x 32 blocks a product runs on the kernel for small matrices (five
// steps on it against five on tiles: 256 x 256 67 us against 116, 1024 x 2048 -- 2048
// blocks in its third product -- 211 against 250 without with_low's addition, 2048 x
// 2048 866 against 354).
constexpr int64_t kSmallBlocks = 2048;

// Whether X X^T takes what fp16 leaves out of X too: where every product runs on the
// kernel for small matrices, bound by latency, and K is short.  768 x 768 130 us, 118 without;
// 1024 x 2048 259 and 211; 64 x 14336, which is beyond the rule, would take 262 and
// takes 163.  On tiles it would cost X X^T twice over.
bool with_low(int64_t mp, int64_t np) { return (mp / 32) * (np / 32) <= kSmallBlocks && np <= 2048; }

// Byte offsets in the workspace: X in fp32 (OrthState), its fp16 forms X [m][xp] and two
// X^T [n][mp] (the third product reads one while it writes the other), two symmetric
// matrices [m][mp] with their diagonals in fp32, the norm's partial sums.
struct OrthLayout {
    int64_t m, n, mp, np, xp;
    int64_t state, x, xt[2], a, b, da, db, sums, bytes;
};
OrthLayout layout(int64_t rows, int64_t cols)
{
    OrthLayout l;
    l.m = rows < cols ? rows : cols;
    l.n = rows < cols ? cols : rows;
    l.mp = pad64(l.m);
    l.np = pad64(l.n);
    l.xp = with_low(l.mp, l.np) ? 2 * l.np : l.np;
    int64_t at = 0;
    auto take = [&](int64_t elems, int64_t size) {
        const int64_t here = at;
        at += size * elems;      // multiples of 64 elements: every part stays aligned
        return here;
    };
    l.state = take(l.mp * l.np, 4);
    l.x = take(l.m * l.xp, 2);
    l.xt[0] = take(l.n * l.mp, 2);
    l.xt[1] = take(l.n * l.mp, 2);
    l.a = take(l.m * l.mp, 2);
    l.b = take(l.m * l.mp, 2);
    l.da = take(l.mp, 4);
    l.db = take(l.mp, 4);
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

// The update of X (m x n), whole or in the two parts of split_last_round.
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
        re.state.x += keep / 16 * e.state.pitch;
        re.d += keep;
        re.rows_d -= keep;
    } else {
        head.N = keep;
        rest.N -= keep;
        rest.B = static_cast<const char *>(p.B) + skip;
        re.straight += e.straight ? keep : 0;
        re.cols_s -= keep;
        re.transposed += e.transposed ? keep * e.ldt : 0;
        re.state.x += keep / 32 * hkg::kOrthBlock;
        re.state.blocks -= keep / 32;
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
    auto half = [&](int64_t at) { return reinterpret_cast<uint16_t *>(ws + at); };
    auto full = [&](int64_t at) { return reinterpret_cast<float *>(ws + at); };
    uint16_t *const x = half(l.x), *const xt[2] = {half(l.xt[0]), half(l.xt[1])}, *const am = half(l.a), *const bm = half(l.b);
    float *const da = full(l.da), *const db = full(l.db);
    double *sums = reinterpret_cast<double *>(ws + l.sums);
    const hkg::ElemType t = g_type == HKG_T_F32 ? hkg::kElemF32 : hkg::kElemBf16;
    const hkg::OrthInput in = {G, ldg, static_cast<int>(rows), static_cast<int>(cols)};
    const bool tall = rows > cols;
    const int m = static_cast<int>(l.m), n = static_cast<int>(l.n), mp = static_cast<int>(l.mp),
              np = static_cast<int>(l.np), xp = static_cast<int>(l.xp), low = xp - np;

    rc = launched(hkg::launch_orth_norm(t, in, sums, st));
    if (rc != HKG_OK)
        return rc;
    if (steps == 0)
        return launched(hkg::launch_orth_convert(t, in, sums, eps, {}, nullptr, 0, nullptr, 0, 0,
                                                 static_cast<uint16_t *>(out), ldo, st));
    const hkg::OrthState state = {full(l.state), 16 * l.np, np / 32};
    rc = launched(tall ? hkg::launch_orth_convert(t, in, sums, eps, state, xt[0], mp, x, xp, low, nullptr, 0, st)
                       : hkg::launch_orth_convert(t, in, sums, eps, state, x, xp, xt[0], mp, low, nullptr, 0, st));

    const float s = 1.0f / hkg::kOrthScale;
    const int sym = pick_tile(m, m, true), upd = pick_tile(m, n, false);
    // from rows of K elements: to = gamma (from from^T) alone (D null), or with D = from
    // and its diagonal r beta S + gamma S S for their matrix S; the diagonal to diag
    auto symmetric = [&](const uint16_t *from, int K, float gamma, float beta, const uint16_t *D, const float *r,
                         uint16_t *to, float *diag) {
        hkg::OrthEpilogue ep = {};
        ep.gamma = gamma;
        ep.beta = beta;
        ep.D = reinterpret_cast<const _Float16 *>(D);
        ep.r = r;
        ep.diag = diag;
        ep.straight = ep.transposed = to;
        ep.ldd = ep.lds = ep.ldt = ep.cols_d = ep.cols_s = ep.cols_t = mp;
        if (rc == HKG_OK)
            rc = launched(hkg::launch_orth_product(sym, tiles_of(m, m, K, sym), true, {from, from, m, m, K, !D && low > 0}, ep, st));
    };
    for (int i = 0; i < steps && rc == HKG_OK; ++i) {
        symmetric(x, np, s * s, 0.0f, nullptr, nullptr, am, da);   // A = X X^T
        symmetric(am, mp, c, b, am, da, bm, db);                   // B = b A + c A A
        // X <- a X + B X, as X and X^T, or the result in its own orientation
        hkg::OrthEpilogue ep = {};
        ep.gamma = s;
        ep.state = state;
        ep.a = a;
        ep.d = db;
        ep.rows_d = mp;
        ep.last = i + 1 == steps;
        if (!ep.last) {
            ep.straight = x;
            ep.lds = xp;
            ep.cols_s = np;
            ep.low = low;
            ep.transposed = xt[(i & 1) ^ 1];
            ep.ldt = ep.cols_t = mp;
        } else if (tall) {
            ep.transposed = static_cast<uint16_t *>(out);
            ep.ldt = ldo;
            ep.cols_t = m;
        } else {
            ep.straight = static_cast<uint16_t *>(out);
            ep.lds = ldo;
            ep.cols_s = n;
        }
        if (rc == HKG_OK)
            rc = launched(launch_update(upd, {bm, xt[i & 1], m, n, mp, false}, ep, st));
    }
    return rc;
}

}  // extern "C"
