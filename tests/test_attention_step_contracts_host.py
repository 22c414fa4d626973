"""Contracts of the attention step that are kept on the host: the rotary table's range, the launch of the kernel that
joins partial results; and what the GPU tests' bound on an error's norm tells apart."""
import ctypes
import math
from fractions import Fraction

import pytest
import torch

import attention_step_ref as ref
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


def test_the_norm_sees_a_tile_that_is_lost_or_doubled():
    """The tests' bound on the error's norm, with the kernels' roundings, and with a tile's weights 0 or twice."""
    g = torch.Generator().manual_seed(3)
    n, heads, m, d = 1, 4, 60000, 64
    q = (torch.randn((n, heads, d), generator=g) * 0.5).to(torch.bfloat16)
    k, v = (torch.randn((m, 1, d), generator=g).to(torch.bfloat16) for _ in range(2))
    want, most = ref.norm_bound(q, k, v, m - n)
    assert torch.allclose(want, ref.attend(q, k, v, m - n)[0], rtol=1e-12, atol=1e-15)

    def kernel(weight):  # weights in BF16 relative to the maximum, their sum before rounding
        s = q.float()[0] @ k.float()[:, 0].t() * d ** -0.5
        p = (s - s.amax(1, keepdim=True)).exp() * weight
        return ((p.to(torch.bfloat16).double() @ v[:, 0].double()) / p.double().sum(1, keepdim=True)).to(torch.bfloat16)

    ones = torch.ones(m)
    assert (kernel(ones).double() - want[0]).norm().item() <= most
    for tile in torch.randint(0, m // 128, (20,), generator=g).tolist():
        for factor in (0.0, 2.0):
            weight = ones.clone()
            weight[128 * tile:128 * tile + 128] = factor
            assert (kernel(weight).double() - want[0]).norm().item() > most
