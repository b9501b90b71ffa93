"""Fractions of a turn in whole numbers: those of exact rational arithmetic."""
from fractions import Fraction

import numpy as np

import bit_block_quantized_nibble_amd as qbn

PI = Fraction("3.14159265358979323846264338327950288419716939937510582097494459")


def test_turns_are_those_of_rational_arithmetic():
    rng = np.random.default_rng(0)
    f = [0.0, -0.0, 1.0, -1.0, 5e-324, -5e-324, 1.7976931348623157e308, -1.7976931348623157e308, 2.0 ** -64, 3.4e-19, -3.4e-19]
    f += (rng.standard_normal(500) * 10.0 ** rng.uniform(-22, 22, 500)).tolist() + rng.uniform(-7, 7, 497).tolist()
    want = [round(Fraction(x) / (2 * PI) * (1 << 64)) % (1 << 64) for x in f]
    assert [t % (1 << 64) for t in qbn.Rope(f, device="cpu").turns.tolist()] == want


def test_frequencies_of_any_numbers():
    """Numbers of other types are taken in binary64."""
    f = [1, 2, np.float32(0.1), np.float64(0.3), True, 7, Fraction(1, 3), 0.5]
    got = qbn.Rope(f, device="cpu")
    assert got.frequencies == [float(x) for x in f]
    assert qbn.Rope([float(x) for x in f], device="cpu").turns.tolist() == got.turns.tolist()
