"""Contracts of the attention step that are kept on the host: the rotary table's range, the launch of the kernel that
joins partial results."""
import ctypes
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


@pytest.mark.parametrize("tokens,batch,kv_heads,group,blocks", [
    (1, 1, 8, 4, 8), (5, 1, 8, 4, 20), (6, 1, 8, 4, 24), (7, 1, 8, 4, 8),   # one sequence: its rows, up to 24
    (2, 2, 8, 4, 8), (4, 4, 8, 4, 8), (6, 6, 8, 4, 8), (6, 3, 8, 4, 8),     # an item's 4 or 8 rows, whatever the batch's
    (10, 2, 8, 4, 20), (15, 3, 8, 4, 8), (20, 4, 4, 4, 20), (40, 8, 8, 4, 8),  # parts of an item: more than 8, or not
    (3, 1, 4, 8, 24), (1, 1, 1, 16, 16), (9, 2, 2, 4, 20), (2 ** 31 - 600, 2 ** 20 - 1, 1, 1, 8)])
def test_blocks_that_join(tokens, batch, kv_heads, group, blocks):
    from nvfp4_speculative_draft_gb300 import build
    build.build()
    f = ctypes.CDLL(build.WITHHOLD_LIB).nvfp4_test_join_blocks
    f.argtypes = [ctypes.c_int, ctypes.c_int64, ctypes.c_int64] + [ctypes.c_int] * 4
    assert f(1, tokens, batch, kv_heads, group, 128 // group, 152) == blocks
    assert f(2, tokens, batch, kv_heads, group, 256 // group, 152) == 16
