"""Pins of oracle/linear.py (CPU): the generator against the published answers of
Philox-4x32-10, its array form against the single one, activations and slopes
against known values and differences."""
import math

import numpy as np
import pytest

from oracle import linear as ref

# known answers of Philox-4x32 with 10 rounds, from the generator's authors
KNOWN = [
    ((0, 0, 0, 0), (0, 0), (0x6627e8d5, 0xe169c58d, 0xbc57ac4c, 0x9b00dbd8)),
    ((0xffffffff,) * 4, (0xffffffff,) * 2, (0x408f276d, 0x41c83b0e, 0xa20bc7c6, 0x6d5451fd)),
    ((0x243f6a88, 0x85a308d3, 0x13198a2e, 0x03707344), (0xa4093822, 0x299f31d0),
     (0xd16cfe09, 0x94fdcceb, 0x5001e420, 0x24126ea1)),
]


@pytest.mark.parametrize("counter,key,want", KNOWN)
def test_generator(counter, key, want):
    assert tuple(ref.philox4x32(counter, key)) == want


def test_numbers_are_the_generators_halves():
    seed, offset = 0x299f31d0a4093822, 0x0370734413198a2e
    got = ref.numbers(3, 21, seed, offset, row0=7)
    for r in range(3):
        for c in range(21):
            w = ref.philox4x32((c // 8, 7 + r, offset & 0xffffffff, offset >> 32), (seed & 0xffffffff, seed >> 32))
            assert got[r, c] == (w[c % 8 // 2] >> (16 * (c % 2))) & 0xffff


def test_share_of_dropped_elements():
    n = 1 << 20
    for p in (0.05, 0.1, 0.5, 0.9):
        dropped = n - int(ref.keep(1024, 1024, p, (11, 5)).sum())
        # five standard deviations of a binomial count
        assert abs(dropped - n * ref.below(p) / 65536) < 5 * math.sqrt(n * p * (1 - p))
    assert ref.below(0.1) == 6554 and ref.below(1.0) == 65536 and ref.below(1e-6) == 0


@pytest.mark.parametrize("name", ["relu", "gelu", "gelu_tanh", "silu"])
def test_slopes_are_the_activations_differences(name):
    z = np.linspace(-8.0, 8.0, 161) + 0.013
    h = 1e-5
    d = (ref.act(z + h, name) - ref.act(z - h, name)) / (2 * h)
    # h^2 / 6 times third derivatives below 2, and 2^-53 x 8 / h
    np.testing.assert_allclose(ref.slope(z, name), d, rtol=0, atol=2e-10)
    np.testing.assert_allclose(ref.slope(0.0, name), 0.0 if name == "relu" else 0.5)


def test_values_at_the_ends():
    for name in ("relu", "gelu", "gelu_tanh", "silu"):
        z = np.array([-np.inf, np.inf, np.nan, -3e38, 3e38])
        np.testing.assert_array_equal(ref.act(z, name)[:2], [0.0, np.inf])
        np.testing.assert_array_equal(ref.slope(z, name)[[0, 1, 3, 4]], [0.0, 1.0, 0.0, 1.0])
        assert np.isnan(ref.act(z, name)[2]) and np.isnan(ref.slope(z, name)[2])
    assert abs(ref.act(1.0, "gelu") - 0.8413447460685429) < 1e-15
    assert abs(ref.act(1.0, "silu") - 0.7310585786300049) < 1e-15
    assert abs(ref.act(1.0, "gelu_tanh") - 0.5 * (1 + math.tanh(math.sqrt(2 / math.pi) * 1.044715))) < 1e-15
