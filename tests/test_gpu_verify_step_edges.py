"""Edges of the verify step's operators on the GPU: signs of zeros, tiny values, the range of scales, memory
of other streams.

Codes are compared byte by byte, so that -0 (0x80) and +0 (0x00) differ: the
contract gives every code the sign of its value, also where it rounds to zero.
"""
import pytest
import torch

import verify_step_ref as ref
from test_gpu_verify_step import check_gemm, check_norm, gemm_tol, make_gemm, nd, randn, u8

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


# ------------------------------------------ rows whose squares leave binary32's range

# magnitudes of a row; around 2^-50 the squares' mean passes from the plain sum to the scaled one
TINY = [2.0 ** -e for e in (40, 48, 49, 50, 51, 52, 60, 63, 64, 70, 76, 100, 120, 126, 130)]


@pytest.mark.parametrize("eps", [0.0, 2.0 ** -148, 1e-38, 2.0 ** -101, 2.0 ** -100, 1e-24])
@pytest.mark.parametrize("k", [16, 128, 272, 2064, 5120, 17408])
@pytest.mark.parametrize("with_res", [False, True])
def test_norm_of_tiny_rows(dev, k, eps, with_res):
    """Finite rows are normalised whatever their magnitude: the squares of values below 2^-63 are not
    normal binary32 numbers, those below 2^-75 are zero.  (Tolerance: that of every other row; scaling a
    row by a power of two rounds nothing.)"""
    eps = torch.tensor(eps).item()  # as binary32
    x = randn(dev, k, 3 * len(TINY) + 2, k)
    x[0] = 0.0
    x[1, k // 2:] = 0.0
    for i, t in enumerate(TINY):
        x[3 * i + 2] *= t          # between rows of other magnitudes, which share a CTA with it
        x[3 * i + 3, : k // 2] *= t
    x = x.to(torch.bfloat16)
    x[4, 0] = 2.0 ** -133          # the smallest of all values, alone in its row
    x[4, 1:] = 0.0
    r = x.flip(0) * 2.0 ** -20 if with_res else None
    g = (1 + 0.05 * randn(dev, k + 1, k)).to(torch.bfloat16)
    status = torch.zeros(1, dtype=torch.int32, device=dev)
    acts, h = nd().fp8b_rmsnorm(x, g, eps, residual=r, dev_status=status)
    assert status.item() == 0
    check_norm(acts, h, x, r, g, eps)


def test_norm_of_tiny_rows_leaves_the_residual_stream(dev):
    """h is written as it is, also in place, where the row is scaled to be summed."""
    m = nd()
    x = (randn(dev, 1, 8, 512) * 2.0 ** -80).to(torch.bfloat16)
    r = (randn(dev, 2, 8, 512) * 2.0 ** -81).to(torch.bfloat16)
    g = torch.ones(512, dtype=torch.bfloat16, device=dev)
    want, h = m.fp8b_rmsnorm(x, g, 0.0, residual=r)
    check_norm(want, h, x, r, g, 0.0)
    target = r.clone()
    got, _ = m.fp8b_rmsnorm(x, g, 0.0, residual=target, residual_out=target)
    assert torch.equal(target, h)
    assert torch.equal(u8(got.codes), u8(want.codes)) and torch.equal(got.scales, want.scales)


# --------------------------------------------------- outputs on the call's stream

def segment_stream(t):
    """The stream whose memory pool holds t."""
    for s in torch.cuda.memory_snapshot():
        if s["address"] <= t.data_ptr() < s["address"] + s["total_size"]:
            return s["stream"]
    raise AssertionError("not in the allocator's memory")


@pytest.mark.parametrize("handle", [False, True])
def test_outputs_are_allocated_on_the_calls_stream(dev, handle):
    """With ``stream`` given: memory that the current stream's queued work may still use is not taken."""
    m = nd()
    s = torch.cuda.Stream()
    stream = s.cuda_stream if handle else s
    w = torch.ones((128, 256), dtype=torch.bfloat16, device=dev)
    x = torch.ones((4, 256), dtype=torch.bfloat16, device=dev)
    g = torch.ones(256, dtype=torch.bfloat16, device=dev)
    p = torch.full((2, 3, 64), 1 / 64, device=dev)
    tok, u, r = torch.zeros((2, 2), dtype=torch.int32, device=dev), torch.zeros((2, 2), device=dev), torch.zeros(2, device=dev)

    def outputs(st):
        q = m.fp8b_quantize(w, stream=st)
        a, h = m.fp8b_rmsnorm(x, g, residual=x, stream=st)
        c = m.fp8b_gemm(a, q, stream=st)
        tokens, accepted = m.spec_verify(p, tok, u, r, stream=st)
        return q.codes, q.scales, a.codes, a.scales, h, c, tokens, accepted

    torch.cuda.synchronize()
    current = torch.cuda.current_stream().cuda_stream
    got = outputs(stream)
    assert all(segment_stream(t) == s.cuda_stream for t in got)
    assert torch.cuda.current_stream().cuda_stream == current  # restored
    s.synchronize()
    for st in (None, torch.cuda.current_stream(), current):
        want = outputs(st)
        assert all(segment_stream(t) == current for t in want)
        torch.cuda.synchronize()
        assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(got, want))
    with torch.cuda.stream(s):  # the current stream's outputs while another one is current
        want = outputs(current)
    assert all(segment_stream(t) == current for t in want)
    torch.cuda.synchronize()
    for st in (1, 0):  # the default stream by its legacy handle, and by none
        assert all(segment_stream(t) == 0 for t in outputs(st))
    torch.cuda.synchronize()
    bad = torch.zeros((3, 3), dtype=torch.int32, device=dev)
    with pytest.raises(ValueError):  # a refusal restores it too
        m.spec_verify(p, bad, u, r, stream=stream)
    with pytest.raises(ValueError):
        m.spec_verify(p, tok, u, r, out_accepted=bad, stream=stream)
    assert torch.cuda.current_stream().cuda_stream == current


# ------------------------------------------------------ products of scales

# every tile: few tokens (split over K and not), many, with a ragged last block of rows and columns
RANGE_SIZES = [(1, 300, 2064), (20, 260, 272), (50, 200, 400), (100, 500, 1040), (300, 20000, 272)]


@pytest.mark.parametrize("m,n,k", RANGE_SIZES)
def test_gemm_reports_scales_out_of_range(dev, m, n, k):
    """A product of scales past binary32's range makes its results not finite, even where the
    block's sum is zero: the status says so; other results are as they were."""
    mod = nd()
    a, w = make_gemm(dev, m, n, k)
    last = ref.BLOCK * (ref.blocks(n) - 1)
    w.codes[last:, :ref.BLOCK] = 0
    status = torch.zeros(1, dtype=torch.int32, device=dev)
    want = mod.fp8b_gemm(a, w, out_dtype=torch.float32, dev_status=status)
    assert status.item() == 0
    check_gemm(want, a, w)
    for sa, sw in ((1e30, 1e30), (float("inf"), 1.0), (1.0, float("nan"))):
        a2 = mod.Fp8BlockActs(a.codes, a.scales.clone(), m, k)
        w2 = mod.Fp8BlockWeight(w.codes, w.scales.clone(), n, k)
        a2.scales[0, m - 1] = sa
        w2.scales[-1, 0] = sw
        status.zero_()
        got = mod.fp8b_gemm(a2, w2, out_dtype=torch.float32, dev_status=status)
        assert status.item() == 7
        assert not torch.isfinite(got[m - 1, last:]).any()
        assert torch.equal(got[:m - 1, :last], want[:m - 1, :last])


@pytest.mark.parametrize("m,n,k", RANGE_SIZES)
def test_gemm_of_tiny_scales(dev, m, n, k):
    """Products of scales below 2^-126 round to multiples of 2^-149: by at most 2^-150 times a block's
    sum, which is below 128 x 448^2 < 2^24.7; so 2^-125 for each block beside the usual tolerance, and
    sums below 2^-126 another 2^-150 each."""
    a, w = make_gemm(dev, m, n, k)
    a.scales.mul_(2.0 ** -80)   # 2^-10 .. 2^-2 of make_gemm, times this
    w.scales.mul_(2.0 ** -52)
    status = torch.zeros(1, dtype=torch.int32, device=dev)
    got = nd().fp8b_gemm(a, w, out_dtype=torch.float32, dev_status=status)
    c, s = ref.gemm(a.codes, a.scales, w.codes, w.scales)
    assert status.item() == 0
    assert ((got.double() - c).abs() <= gemm_tol(c, s, k, False) + ref.blocks(k) * 2.0 ** -124).all()
