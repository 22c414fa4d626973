"""The verify step's kernels at sizes that reach each of their variants and loops on 152 SMs.

Tolerances: those of test_gpu_verify_step.py, derived there.
"""
import pytest
import torch

import verify_step_ref as ref
from test_gpu_verify_step import check_gemm, check_norm, make_gemm, nd, randn, u8

pytestmark = pytest.mark.gpu


# rows for every SM (more than 2 x 152): two vectors a thread, in blocks of 160 to 512 threads;
# and beside them the same widths with few rows, and 16384 columns
@pytest.mark.parametrize("m,k", [(310, 2064), (400, 5120), (320, 8192), (305, 16384), (304, 2064), (304, 8192), (9, 16384)])
@pytest.mark.parametrize("with_res", [False, True])
@pytest.mark.parametrize("eps", [1e-6, 0.0])
def test_norm_of_many_rows(dev, m, k, with_res, eps):
    x = randn(dev, m + k, m, k)
    x[3] = 0.0
    x[4] *= 2.0 ** -70 if eps == 0.0 else 1.0
    x = x.to(torch.bfloat16)
    r = (randn(dev, m + k + 1, m, k) * 3).to(torch.bfloat16) if with_res else None
    if with_res:
        r[3:5] = x[3:5]
    g = (1 + 0.05 * randn(dev, k, k)).to(torch.bfloat16)
    status = torch.zeros(1, dtype=torch.int32, device=dev)
    acts, h = nd().fp8b_rmsnorm(x, g, eps, residual=r, dev_status=status)
    assert status.item() == 0
    check_norm(acts, h, x, r, g, eps)
    first = u8(acts.codes).clone(), acts.scales.clone()
    again, _ = nd().fp8b_rmsnorm(x, g, eps, residual=r)
    assert torch.equal(u8(again.codes), first[0]) and torch.equal(again.scales, first[1])


@pytest.mark.parametrize("m,k", [(310, 2064), (400, 5120)])
def test_norm_of_many_rows_in_place(dev, m, k):
    x, r = randn(dev, 2, m, k).to(torch.bfloat16), randn(dev, 3, m, k).to(torch.bfloat16)
    g = torch.ones(k, dtype=torch.bfloat16, device=dev)
    want, h = nd().fp8b_rmsnorm(x, g, residual=r)
    for target in (x.clone(), r.clone()):
        a, b = (target, r) if torch.equal(target, x) else (x, target)
        got, _ = nd().fp8b_rmsnorm(a, g, residual=b, residual_out=target)
        assert torch.equal(target, h)
        assert torch.equal(u8(got.codes), u8(want.codes)) and torch.equal(got.scales, want.scales)


# More output tiles than CTAs at once, so that a CTA takes several one after another: tiles of 16 columns
# (304 CTAs), 32 (304), 64 (152, two issuing warps), 128 (152, two issuing warps), 256 (152).  Odd numbers of K
# blocks move rings, phases and issuers on from tile to tile.
@pytest.mark.parametrize("m,n,k", [(5, 60000, 272), (16, 120001, 16), (20, 60000, 272), (32, 151936, 144), (17, 40000, 1104),
                                   (33, 151936, 144), (40, 40000, 336), (64, 50001, 16), (50, 20000, 1104),
                                   (20000, 100, 272), (40001, 128, 336), (19500, 77, 1104), (39000, 100, 16),
                                   (129, 60000, 272), (300, 40001, 16)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_gemm_of_several_tiles_a_cta(dev, m, n, k, dtype):
    a, w = make_gemm(dev, m, n, k)
    status = torch.zeros(1, dtype=torch.int32, device=dev)
    got = nd().fp8b_gemm(a, w, out_dtype=dtype, dev_status=status)
    assert status.item() == 0
    check_gemm(got, a, w)
    assert torch.equal(nd().fp8b_gemm(a, w, out_dtype=dtype), got)


# 129 to 1024 rows against narrow outputs: a server's batch x (drafts + 1) rows
@pytest.mark.parametrize("m,n,k", [(129, 5120, 5120), (256, 5120, 1040), (511, 5120, 2064), (512, 5120, 5120), (1024, 5120, 528)])
def test_gemm_of_middle_sizes(dev, m, n, k):
    a, w = make_gemm(dev, m, n, k)
    check_gemm(nd().fp8b_gemm(a, w, out_dtype=torch.float32), a, w)
