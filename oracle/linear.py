"""The 16-bit linear layer with its epilogue, its gradients and dropout, from the
definitions in include/hkg_linear.h, in numpy and 64 bits -- TEST INFRASTRUCTURE,
like the rest of this package; shares no code with the GPU path.

Every function that returns a result returns how far a correct computation may be
from it too: sums of n products in fp32 in any order are within n 2^-23 of the sum
of magnitudes, other fp32 operations round by 2^-24 of their result, an activation
is evaluated within `act_error`, and a result that is stored in 16 bits is rounded
by at most half a step (`HALF`; for fp16 at least 2^-25, half its smallest step)."""
from __future__ import annotations

import math

import numpy as np

HALF = {"bf16": 2.0 ** -8, "fp16": 2.0 ** -11, "fp32": 2.0 ** -24}
TINY = {"bf16": 2.0 ** -133, "fp16": 2.0 ** -25, "fp32": 2.0 ** -126}


def stored(v, kind):
    """v, but what fp16 cannot hold, from 65520 on (half a step above its largest number,
    65504), as infinity."""
    return np.where(np.abs(v) >= 65520.0, np.copysign(np.inf, v), v) if kind == "fp16" else v


def erfc(x):
    return np.vectorize(math.erfc, otypes=[np.float64])(x)


# ---- the generator ---------------------------------------------------------------

def philox4x32(counter, key, rounds=10):
    """Four 32-bit words (Python integers) of Philox-4x32 for a counter of four and a
    key of two, as the paper defines it."""
    c, k = list(counter), list(key)
    for _ in range(rounds):
        a, b = c[0] * 0xD2511F53, c[2] * 0xCD9E8D57
        c = [(b >> 32) ^ c[1] ^ k[0], b & 0xFFFFFFFF, (a >> 32) ^ c[3] ^ k[1], a & 0xFFFFFFFF]
        k = [(k[0] + 0x9E3779B9) & 0xFFFFFFFF, (k[1] + 0xBB67AE85) & 0xFFFFFFFF]
    return c


def numbers(rows, cols, seed, offset, row0=0):
    """The 16-bit numbers of rows row0 .. of a matrix, uint32 [rows, cols]; the rounds of
    philox4x32 on arrays."""
    low = np.uint64(0xFFFFFFFF)
    groups = -(-cols // 8)
    c0, c1 = np.meshgrid(np.arange(groups, dtype=np.uint64), np.arange(row0, row0 + rows, dtype=np.uint64))
    c = [c0, c1, np.full_like(c0, offset & 0xFFFFFFFF), np.full_like(c0, offset >> 32)]
    k = [seed & 0xFFFFFFFF, seed >> 32]
    s = np.uint64(32)
    for _ in range(10):
        a, b = c[0] * np.uint64(0xD2511F53), c[2] * np.uint64(0xCD9E8D57)
        c = [(b >> s) ^ c[1] ^ np.uint64(k[0]), b & low, (a >> s) ^ c[3] ^ np.uint64(k[1]), a & low]
        k = [(k[0] + 0x9E3779B9) & 0xFFFFFFFF, (k[1] + 0xBB67AE85) & 0xFFFFFFFF]
    out = np.empty((rows, 8 * groups), dtype=np.uint32)
    for w in range(4):
        out[:, 2 * w::8] = c[w] & np.uint64(0xFFFF)
        out[:, 2 * w + 1::8] = c[w] >> np.uint64(16)
    return out[:, :cols]


def below(p):
    """65536 q for the probability p as an fp32 number."""
    return int(math.floor(float(np.float32(p)) * 65536.0 + 0.5))


def keep(rows, cols, p, rng, row0=0):
    return numbers(rows, cols, rng[0], rng[1], row0) >= below(p)


def scale(p):
    return 65536.0 / (65536 - below(p)) if below(p) < 65536 else 0.0


# ---- activations -------------------------------------------------------------------

def act(z, name):
    z = np.asarray(z, dtype=np.float64)
    with np.errstate(over="ignore", invalid="ignore"):
        if name is None:
            return z.copy()
        if name == "relu":
            return np.where(z <= 0, 0.0, z)
        if name == "gelu":
            v = z * (0.5 * erfc(-z / math.sqrt(2.0)))
        elif name == "gelu_tanh":
            v = z / (1.0 + np.exp(-2.0 * math.sqrt(2.0 / math.pi) * (z + 0.044715 * z ** 3)))
        else:
            v = z / (1.0 + np.exp(-z))
    return np.where(np.isneginf(z), 0.0, v)


def slope(z, name):
    z = np.asarray(z, dtype=np.float64)
    if name is None:
        return np.ones_like(z)
    if name == "relu":
        return np.where(z > 0, 1.0, np.where(z <= 0, 0.0, z))
    c = np.clip(z, -800.0, 800.0)     # a NaN stays one; constant in 64 bits beyond
    with np.errstate(over="ignore"):
        if name == "gelu":
            return 0.5 * erfc(-c / math.sqrt(2.0)) + c * np.exp(-0.5 * c * c) / math.sqrt(2.0 * math.pi)
        if name == "gelu_tanh":
            k = 2.0 * math.sqrt(2.0 / math.pi)
            e = np.exp(-k * (c + 0.044715 * c ** 3))
            s = 1.0 / (1.0 + e)
            rest = 1.0 / (1.0 + np.exp(k * (c + 0.044715 * c ** 3)))
            return s + c * s * rest * k * (1.0 + 3 * 0.044715 * c * c)
        return (1.0 + c / (1.0 + np.exp(c))) / (1.0 + np.exp(-c))


def act_error(z, name, y_type="fp32"):
    """What include/hkg_linear.h states (none and relu are exact).  fp32: an exponential and a
    reciprocal, each within a unit of the last place (2^-23), and at most ten roundings of
    2^-24 (gelu's polynomial and products), the exponential's argument being below 1.  16 bits: the
    exponential's argument goes through at most five roundings of 2^-24 in fp32, and is at
    most 88 where the result is not 0."""
    z = np.asarray(z, dtype=np.float64)
    if name in (None, "relu"):
        return np.zeros_like(z)
    return np.abs(act(z, name)) * (2.0 ** -20 if y_type == "fp32" else 2.0 ** -15) + 2.0 ** -116


SLOPE_ERROR = 2.0 ** -19              # absolute, as stated: a few roundings of terms up to 1.2
STEEPEST = 1.13                       # no slope exceeds it


# ---- the operators -----------------------------------------------------------------

def dropout(x, p, rng, residual=None, out_type="bf16"):
    """-> (out, tolerance)."""
    x = np.asarray(x, dtype=np.float64)
    v = np.where(keep(*x.shape, p, rng), x * scale(p), 0.0) if below(p) else x.copy()
    tol = 2.0 ** -23 * np.abs(v)
    if residual is not None:
        v = v + residual
        tol = tol + 2.0 ** -24 * np.abs(v)
    return stored(v, out_type), tol + HALF[out_type] * np.abs(v) * (1 + 2.0 ** -7) + TINY[out_type]


def linear(x, W, bias=None, activation=None, residual=None, p=0.0, rng=None, y_type="bf16", z_type="bf16", row0=0):
    """-> (y, tolerance of y, z, tolerance of z)."""
    x, W = np.asarray(x, dtype=np.float64), np.asarray(W, dtype=np.float64)
    z = x @ W.T
    err = (x.shape[1] + 1) * 2.0 ** -23 * (np.abs(x) @ np.abs(W).T)
    if bias is not None:
        z = z + bias
        err = err + 2.0 ** -24 * np.abs(z)
    v = act(z, activation)
    e = STEEPEST * err + act_error(z, activation, y_type)
    if below(p):
        k = keep(*v.shape, p, rng, row0)
        v = np.where(k, v * scale(p), 0.0)
        e = np.where(k, e * scale(p), 0.0) + 2.0 ** -23 * np.abs(v)
    if residual is not None:
        v = v + residual
        e = e + 2.0 ** -24 * np.abs(v)
    zt = err + HALF[z_type] * (np.abs(z) + err) + TINY[z_type]
    return v, e + HALF[y_type] * (np.abs(v) + e) + TINY[y_type], z, zt


def backward(dy, x, W, z=None, activation=None, p=0.0, rng=None, kind="bf16"):
    """-> ((dx, tolerance), (dw, tolerance), (dbias, tolerance))."""
    dy = np.asarray(dy, dtype=np.float64)
    M, N = dy.shape
    dz = dy.copy()
    e = np.zeros_like(dy)
    if activation is not None:
        s = slope(z, activation)
        e = np.abs(dz) * (0.0 if activation == "relu" else SLOPE_ERROR)
        dz = dz * s
    if below(p):
        k = keep(M, N, p, rng)
        dz, e = np.where(k, dz * scale(p), 0.0), np.where(k, e * scale(p), 0.0)
    e = e + 2.0 ** -22 * np.abs(dz)
    b = dz.sum(0)
    out_b = b, e.sum(0) + (M + 1) * 2.0 ** -24 * np.abs(dz).sum(0) + TINY["fp32"]
    e16 = e + HALF[kind] * (np.abs(dz) + e) + TINY[kind]
    a16 = np.abs(dz) + e16
    x, W = np.asarray(x, dtype=np.float64), np.asarray(W, dtype=np.float64)
    dx, dw = dz @ W, dz.T @ x
    tx = e16 @ np.abs(W) + (N + 1) * 2.0 ** -23 * (a16 @ np.abs(W))
    tw = e16.T @ np.abs(x) + (M + 1) * 2.0 ** -23 * (a16.T @ np.abs(x))
    return ((dx, tx + HALF[kind] * (np.abs(dx) + tx) + TINY[kind]), (dw, tw + HALF[kind] * (np.abs(dw) + tw) + TINY[kind]), out_b)
