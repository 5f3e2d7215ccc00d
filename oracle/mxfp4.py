"""MXFP4 (e2m1 codes, one E8M0 scale per 32 elements) from the format's
definition, in numpy and 64 bits -- TEST INFRASTRUCTURE, like the rest of this
package; shares no code with the GPU path.

A code's low three bits count up through the magnitudes 0, 0.5, 1, 1.5, 2, 3, 4,
6; bit 3 is the sign.  OCP Microscaling Formats v1.0 sets a block's scale to the
largest power of two not above its largest magnitude, divided by the largest
power of two that the element type holds (4)."""
from __future__ import annotations

import numpy as np

MAGNITUDES = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
BLOCK = 32


def pad32(k: int) -> int:
    return -(-k // BLOCK) * BLOCK


def nearest_code(y):
    """e2m1 codes (0..7) of non-negative values: by distance to every magnitude,
    the even code where two are equally near."""
    d = np.abs(np.asarray(y, dtype=np.float64)[..., None] - MAGNITUDES)
    d = np.where(np.isnan(d), np.inf, d)
    first = d.argmin(-1)
    tie = np.take_along_axis(d, np.minimum(first + 1, 7)[..., None], -1)[..., 0] == d.min(-1)
    return np.where(tie & (first % 2 == 1) & (first < 7), first + 1, first).astype(np.uint8)


def quantize(x):
    """x [R, K] -> (codes [R, Kp] one a byte, scales [R, Kp / 32])."""
    x = np.asarray(x, dtype=np.float64)
    R, K = x.shape
    z = np.zeros((R, pad32(K)))
    z[:, :K] = x
    b = z.reshape(R, -1, BLOCK)
    with np.errstate(invalid="ignore"):
        amax = np.abs(b).max(-1)
    bad = ~np.isfinite(b).all(-1)
    _, e = np.frexp(np.where(bad, 1.0, amax))         # amax = f 2^e, f in [0.5, 1)
    s = np.where(amax > 0, np.maximum(e - 1 - 2, -127), 0)
    codes = nearest_code(np.ldexp(np.where(bad[..., None], 0.0, np.abs(b)), -s[..., None]))
    codes |= (np.signbit(b) & ~bad[..., None]).astype(np.uint8) << np.uint8(3)
    scales = np.where(bad, 255, s + 127).astype(np.uint8)
    return codes.reshape(R, -1), scales


def values(codes, scales):
    """float64 values of (codes one a byte, scales)."""
    v = np.where(codes & 8, -1.0, 1.0) * MAGNITUDES[codes & 7]
    s = np.where(scales == 255, np.nan, np.ldexp(1.0, scales.astype(np.int64) - 127))
    return v * np.repeat(s, BLOCK, axis=1)


def pack_codes(codes):
    """One code a byte -> two a byte, the lower k in the low four bits."""
    return (codes[:, 0::2] | (codes[:, 1::2] << 4)).astype(np.uint8)


def unpack_codes(b):
    out = np.empty((b.shape[0], 2 * b.shape[1]), dtype=np.uint8)
    out[:, 0::2], out[:, 1::2] = b & 15, b >> 4
    return out


def pack_scales(scales, operand):
    """The packed order that include/hkg.h defines for block scales, byte by byte."""
    rows, nblk = scales.shape
    groups, nk = -(-rows // 128), -(-nblk // 4)
    out = np.full((groups, nk, 64, 8), 127, dtype=np.uint8)
    for l in range(64):
        x, q = l & 15, l >> 4
        for e in range(8):
            rho = 16 * e + x if operand == 0 else 32 * (e >> 1) + 4 * (e & 1) + (x & 3) + 8 * (x >> 2)
            for g in range(groups):
                r = 128 * g + rho
                blks = np.arange(q, nblk, 4)
                if r < rows and blks.size:
                    out[g, :blks.size, l, e] = scales[r, blks]
    return out.reshape(-1)


def product(A, SA, B, SB):
    """(exact fp64 A·Bᵀ, tolerance per entry) of two MXFP4 matrices with codes one
    a byte.  The matrix instruction sums the 128 products of a step with about 13
    bits below the largest of them before it adds the fp32 accumulator, so an
    entry is within sum_steps 128 2^-13 max|a_k b_k| + steps 2^-24 sum|a_k b_k|."""
    a, b = values(A, SA), values(B, SB)
    K = a.shape[1]
    ref = a @ b.T
    tol = np.zeros_like(ref)
    total = np.abs(a) @ np.abs(b).T
    for k in range(0, K, 128):
        aa, bb = np.abs(a[:, k:k + 128]), np.abs(b[:, k:k + 128])
        # max_k of products, bounded block by block to stay cheap
        m = np.zeros_like(ref)
        for j in range(0, aa.shape[1], 32):
            m = np.maximum(m, np.outer(aa[:, j:j + 32].max(1), bb[:, j:j + 32].max(1)))
        tol += 2.0 ** -6 * m
    return ref, tol + (K // 128 + 1) * 2.0 ** -24 * total
