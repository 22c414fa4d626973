"""The block-scaled GEMM's bounded waits run out, on the GPU, without faulting or hanging it.

The test build of the library (libnvfp4draft_withhold.so; see NVFP4_TEST_WITHHOLD in csrc/common.cuh)
never issues the first stage's loads of CTA 0 and shortens the wait limit to 20 ms.  Nothing of the
withheld copies is ever in flight.  Each call must return and report NVFP4_ERR_TIMEOUT; the context stays
usable: the library's own call on the same inputs afterwards is right, TMEM and clusters included."""
import ctypes
import os

import pytest
import torch

import verify_step_ref as ref

pytestmark = pytest.mark.gpu

NVFP4_ERR_TIMEOUT = 6


@pytest.fixture(scope="module")
def wl():
    import nvfp4_speculative_draft_gb300 as m
    from nvfp4_speculative_draft_gb300 import build
    if not os.path.exists(build.WITHHOLD_LIB):
        build.build(withhold=True)
    L = ctypes.CDLL(build.WITHHOLD_LIB)
    P = ctypes.POINTER
    L.fp8b_gemm.argtypes = [P(m._Fp8BlockActs), P(m._Fp8BlockWeight), ctypes.c_void_p, ctypes.c_int, ctypes.c_int64,
                            P(m._Exec)]
    L.fp8b_gemm.restype = ctypes.c_int
    return L


# one token over split K and not, each tile of few tokens, both tiles of many, several waves of tiles
@pytest.mark.parametrize("m,n,k", [(1, 1024, 5120), (1, 40000, 1024), (20, 512, 2048), (50, 900, 1024), (100, 640, 2560),
                                   (300, 3000, 1024), (600, 20000, 512)])
def test_gemm_wait_runs_out_and_the_call_returns(dev, wl, m, n, k):
    import nvfp4_speculative_draft_gb300 as nd
    g = torch.Generator(device=dev)
    g.manual_seed(m + n + k)
    x = torch.randn((m, k), generator=g, device=dev).to(torch.bfloat16)
    w = nd.fp8b_quantize((torch.randn((n, k), generator=g, device=dev) * 0.02).to(torch.bfloat16))
    a, _ = nd.fp8b_rmsnorm(x, None)
    out = torch.empty((m, n), device=dev)
    status = torch.zeros(1, dtype=torch.int32, device=dev)
    ca = nd._Fp8BlockActs(a.codes.data_ptr(), k, a.scales.data_ptr(), m, m, k)
    cw = nd._Fp8BlockWeight(w.codes.data_ptr(), w.scales.data_ptr(), n, k)
    ex = nd._Exec(torch.cuda.current_stream().cuda_stream, None, 0, status.data_ptr())
    torch.cuda.synchronize()
    assert wl.fp8b_gemm(ctypes.byref(ca), ctypes.byref(cw), out.data_ptr(), nd.DTYPE_F32, n, ctypes.byref(ex)) == 0
    torch.cuda.synchronize()
    assert status.item() == NVFP4_ERR_TIMEOUT
    status.zero_()
    got = nd.fp8b_gemm(a, w, out_dtype=torch.float32, dev_status=status)
    c, s = ref.gemm(a.codes, a.scales, w.codes, w.scales)
    assert status.item() == 0
    assert ((got.double() - c).abs() <= (128 + 2 * ref.blocks(k)) * 2.0 ** -24 * s).all()
