// ops_internal.h -- host checks shared by the entry points of hkg_ops.h
// (ops_api.cpp, orth_api.cpp) and those of hkg.h (hkg_api.cpp, which defines
// the ones declared here without a body).  Not part of the installed interface.
#pragma once

#include <stdint.h>

#include "../../include/hkg_ops.h"
#include "api_internal.h"
#include "ops_kernels.h"

namespace hkg::api {

bool mx_sizes_fit(int64_t rows, int64_t K);
bool aligned16(const void *p);
int64_t extent(int64_t rows, int64_t cols, int64_t ld, int64_t elem);
bool overlaps(const void *p, int64_t pb, const void *q, int64_t qb);

inline int64_t pad32(int64_t K) { return (K + 31) / 32 * 32; }

// An MXFP4 matrix [rows][K] within the limits; K is compared before it is
// rounded up, so no value can wrap.
inline bool mx4_fits(int64_t rows, int64_t K)
{
    return K < (int64_t(1) << 23) - 32 && mx_sizes_fit(rows, pad32(K));
}
inline int64_t mx4_codes(int64_t rows, int64_t K) { return rows * (pad32(K) / 2); }
inline int64_t mx4_scales(int64_t rows, int64_t K) { return mx_packed_bytes(rows, pad32(K)); }

// Element size of an HKG_T_* value, 0 if it is none.
inline int64_t elem_size(int32_t t) { return t == HKG_T_BF16 ? 2 : t == HKG_T_F32 ? 4 : 0; }

// A matrix [rows][cols] of elements with pitch *ld (0 becomes cols): pitch at
// least the row (HKG_ERR_OPTS), base aligned to its element (HKG_ERR_ALIGN),
// extents that cannot wrap (HKG_ERR_SIZE).
inline int check_matrix(const void *p, int64_t rows, int64_t cols, int64_t elem, int64_t *ld)
{
    if (*ld == 0)
        *ld = cols;
    if (*ld < cols)
        return HKG_ERR_OPTS;
    if (reinterpret_cast<uintptr_t>(p) % static_cast<uintptr_t>(elem))
        return HKG_ERR_ALIGN;
    if (rows >= (int64_t(1) << 31) || *ld >= (int64_t(1) << 31) || rows * *ld >= (int64_t(1) << 60))
        return HKG_ERR_SIZE;
    return HKG_OK;
}

struct Range {
    const void *p;
    int64_t n;
};

// Whether the first `outs` ranges share a byte with each other or with a later one.
template <int kN>
bool any_overlap(const Range (&r)[kN], int outs)
{
    for (int i = 0; i < outs; ++i)
        for (int j = i + 1; j < kN; ++j)
            if (overlaps(r[i].p, r[i].n, r[j].p, r[j].n))
                return true;
    return false;
}

inline int64_t round16(int64_t n) { return (n + 15) / 16 * 16; }

// Grid order of a tile grid whose operand rows hold row_bytes: the rule of the
// GEMM of hkg.h (launch.cpp), measured there; other orders of e2m1 tiles are within 2 %.
inline hkg::TileOrder order_of(int64_t M, int64_t N, int64_t row_bytes, int tile)
{
    const bool big = row_bytes > 18944;
    int64_t Gm = ceil_div(M, tile), Gn = ceil_div(N, tile), w = big ? 16 : 8, c = big ? 4 : 32;
    clamp_remap(Gm, Gn, &w, &c);
    return {static_cast<int>(Gm), static_cast<int>(Gn), static_cast<int>(w), static_cast<int>(c)};
}

// A grid of 256-tiles whose last round of the 256 compute units is at most half full,
// as two launches: whole rounds of 256-tiles over the first `keep` rows (by_rows) or
// columns of the result, 128-tiles over the rest (512 of them at most: one round at two
// a compute unit, which takes 0.74 of a round of 256-tiles: 20.3 against 27.3 us at
// K = 4096 e2m1).  keep 0: one launch.
struct TileSplit {
    int64_t keep;
    bool by_rows;
};
inline TileSplit split_last_round(int64_t M, int64_t N)
{
    const int64_t gm = ceil_div(M, 256), gn = ceil_div(N, 256), whole = gm * gn / 256 * 256;
    if (whole == 0 || gm * gn == whole)
        return {0, false};
    for (const bool by_rows : {true, false}) {
        const int64_t lines = by_rows ? gm : gn, other = by_rows ? gn : gm, keep = whole / other;
        const int64_t rest = ceil_div((by_rows ? M : N) - 256 * keep, 128) * ceil_div(by_rows ? N : M, 128);
        // the kept part may leave a few tiles of its last round out
        if (keep > 0 && keep < lines && rest <= 512 && ceil_div(keep * other, 256) == whole / 256)
            return {256 * keep, by_rows};
    }
    return {0, false};
}

// Record a launch's HIP error, if it has one, as the entry points of hkg.h do.
inline int launched(hipError_t e)
{
    if (e == hipSuccess)
        return HKG_OK;
    set_last_hip_error(static_cast<int>(e));
    return HKG_ERR_LAUNCH;
}

}  // namespace hkg::api
