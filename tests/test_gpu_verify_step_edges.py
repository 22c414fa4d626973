"""Edges of the verify step's operators on the GPU: signs of zeros, code bytes.

Codes are compared byte by byte, so that -0 (0x80) and +0 (0x00) differ: the
contract gives every code the sign of its value, also where it rounds to zero.
"""
import pytest
import torch

import verify_step_ref as ref
from test_gpu_verify_step import nd, randn, u8

pytestmark = pytest.mark.gpu


def code_bytes(y, s):
    """E4M3 bytes of the correctly rounded binary32 quotients; +0 where the scale is 0."""
    q = torch.where(s > 0, y / torch.where(s > 0, s, torch.ones_like(s)), torch.zeros_like(y))
    return q.clamp(-448.0, 448.0).to(ref.F8).view(torch.uint8)


def signed_zeros(dev, seed, n, k):
    """Values with zeros of both signs and values far below the block's largest among them."""
    x = randn(dev, seed, n, k)
    kind = torch.randint(0, 8, (n, k), generator=torch.Generator(device=dev).manual_seed(seed + 1), device=dev)
    x = torch.where(kind == 0, torch.zeros_like(x), x)
    x = torch.where(kind == 1, torch.full_like(x, -0.0), x)
    return torch.where(kind == 2, x * 2.0 ** -24, x).to(torch.bfloat16)


# the largest magnitude decides how the quotients are formed: ordinary, tiny and huge
@pytest.mark.parametrize("scale", [1.0, 2.0 ** -90, 2.0 ** 124])
@pytest.mark.parametrize("n,k", [(1, 16), (130, 272), (256, 1040)])
def test_quantize_sign_of_zero(dev, n, k, scale):
    w = (signed_zeros(dev, n + k, n, k).float() * scale).to(torch.bfloat16)
    q = nd().fp8b_quantize(w)
    s = q.scales.repeat_interleave(ref.BLOCK, 0)[:n].repeat_interleave(ref.BLOCK, 1)[:, :k]
    assert torch.equal(u8(q.codes), code_bytes(w.float(), s))
    assert (u8(q.codes) == 0x80).any()


@pytest.mark.parametrize("m,k", [(1, 16), (5, 272), (37, 5120), (400, 5120)])
@pytest.mark.parametrize("with_res", [False, True])
def test_norm_sign_of_zero_without_gamma(dev, m, k, with_res):
    """y is h itself, a BF16 value: its codes are those of the rounded quotients."""
    x = signed_zeros(dev, m + k, m, k)
    r = signed_zeros(dev, m + k + 9, m, k) if with_res else None
    acts, h = nd().fp8b_rmsnorm(x, None, residual=r)
    y = (x if r is None else h).float()
    s = acts.scales.t().repeat_interleave(ref.BLOCK, 1)[:, :k]
    assert torch.equal(u8(acts.codes), code_bytes(y, s))
    assert (u8(acts.codes) == 0x80).any()


@pytest.mark.parametrize("m,k", [(1, 16), (5, 272), (37, 5120), (400, 5120)])
@pytest.mark.parametrize("with_res", [False, True])
def test_norm_sign_of_zero_with_gamma(dev, m, k, with_res):
    """The sign of h times the sign of gamma, zeros included."""
    x = signed_zeros(dev, m + k, m, k)
    r = signed_zeros(dev, m + k + 9, m, k) if with_res else None
    g = randn(dev, k, k).to(torch.bfloat16)
    acts, h = nd().fp8b_rmsnorm(x, g, 1e-6, residual=r)
    y = torch.signbit(x if r is None else h) ^ torch.signbit(g)[None]
    s = acts.scales.t().repeat_interleave(ref.BLOCK, 1)[:, :k]
    assert torch.equal((u8(acts.codes) >= 0x80)[s > 0], y[s > 0])
