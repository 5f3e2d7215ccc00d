"""Pins of oracle/mxfp4.py (CPU): the e2m1 rounding by brute force, the scale rule
on hand-made blocks, the packed order against the MXFP8 oracle's definition, and
the plain-C form of include/hkg_ops.h."""
import os
import shutil
import subprocess

import numpy as np
import pytest

from oracle import mxfp4 as ref

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_codes_stand_for_sign_exponent_mantissa():
    # OCP e2m1: exponent bias 1, one mantissa bit, exponent 0 subnormal
    for c in range(8):
        e, m = c >> 1, c & 1
        assert ref.MAGNITUDES[c] == (m * 0.5 if e == 0 else (1 + m / 2) * 2.0 ** (e - 1))


def test_nearest_code_between_every_pair():
    for lo in range(7):
        a, b = ref.MAGNITUDES[lo], ref.MAGNITUDES[lo + 1]
        mid = (a + b) / 2
        even = lo if lo % 2 == 0 else lo + 1
        got = ref.nearest_code([a, np.nextafter(mid, 0), mid, np.nextafter(mid, 9), b])
        assert got.tolist() == [lo, lo, even, lo + 1, lo + 1]
    assert ref.nearest_code([6.0, 6.5, 100.0, np.inf]).tolist()[:3] == [7, 7, 7]


@pytest.mark.parametrize("amax,scale", [(4.0, 127), (7.99, 127), (8.0, 128), (1.0, 125), (3.999, 126), (0.0, 127),
                                        (2.0 ** -126, 0), (2.0 ** -125, 0), (2.0 ** -124, 1), (2.0 ** -149, 0),
                                        (3.4e38, 252), (np.inf, 255), (np.nan, 255)])
def test_scale_rule(amax, scale):
    x = np.zeros((1, 32))
    x[0, 17] = -amax
    codes, scales = ref.quantize(x)
    assert scales[0, 0] == scale
    if 0 < amax < np.inf and scale > 0:
        v = ref.values(codes, scales)[0, 17]
        assert abs(v + amax) <= amax / 4          # 7.99 rounds to 6, the format's largest


def test_round_trip_of_every_code_and_padding():
    x = np.concatenate([ref.MAGNITUDES, -ref.MAGNITUDES, [4.0] * 17])[None, :]
    codes, scales = ref.quantize(x)
    assert codes.shape == (1, 64) and scales.tolist() == [[127, 127]]
    np.testing.assert_array_equal(ref.values(codes, scales)[0, :33], x[0])
    assert (codes[0, 33:] == 0).all()
    np.testing.assert_array_equal(ref.unpack_codes(ref.pack_codes(codes)), codes)
    assert ref.pack_codes(codes)[0, 0] == codes[0, 0] | codes[0, 1] << 4


@pytest.mark.parametrize("operand", [0, 1])
def test_packed_order_is_a_permutation_of_a_group(operand):
    s = np.arange(128 * 4, dtype=np.int64).reshape(128, 4)
    lo, hi = (s & 255).astype(np.uint8), (s >> 8).astype(np.uint8)
    back = ref.pack_scales(lo, operand).astype(np.int64) + 256 * ref.pack_scales(hi, operand).astype(np.int64)
    assert sorted(back.tolist()) == list(range(512))
    # the row and block that include/hkg.h gives byte 8 l + e
    l, e = 37, 5
    row = 16 * e + l % 16 if operand == 0 else 32 * (e >> 1) + 4 * (e & 1) + (l & 3) + 8 * (l % 16 >> 2)
    assert back[8 * l + e] == 4 * row + l // 16


@pytest.mark.skipif(not shutil.which("gcc"), reason="gcc not available")
def test_header_is_plain_c(tmp_path):
    src = tmp_path / "t.c"
    src.write_text('#include "hkg_ops.h"\nint main(void) { return HKG_T_BF16; }\n')
    subprocess.run(["gcc", "-std=c99", "-Wall", "-Wextra", "-Werror", "-pedantic", "-fsyntax-only", "-I",
                    os.path.join(ROOT, "include"), str(src)], check=True)
