"""Contracts of the attention step that are kept on the host: the rotary table's range."""
import math
from fractions import Fraction

import pytest

import nvfp4_speculative_draft_gb300 as nd


def test_rotary_table_of_any_finite_frequency():
    """Finite frequencies beyond what 2^64 turns leave of binary64's range: their fraction of a turn."""
    f = [1e300, -1e300, 1.7976931348623157e308, 5e-324, 1e17, -3.5, 2.0 ** -40, 0.0]
    t = nd.rotary_table(16, inv_freq=f, device="cpu")
    for x, got in zip(f, t.turns.tolist()):
        assert got % 2 ** 64 == int(Fraction(x / (2 * math.pi)) * 2 ** 64) % 2 ** 64
    t = nd.rotary_table(64, theta=1e-308, device="cpu")  # up to 1e298 radians
    assert t.turns[0].item() % 2 ** 64 == int(Fraction(1 / (2 * math.pi)) * 2 ** 64)


def test_rotary_table_refuses_frequencies_out_of_range():
    with pytest.raises(ValueError):
        nd.rotary_table(256, theta=5e-324, device="cpu")  # theta^(-254 / 256) is no binary64
