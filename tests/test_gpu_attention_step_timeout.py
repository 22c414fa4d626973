"""Attention's bounded waits run out, on the GPU, without faulting or hanging it.

The test build of the library (libnvfp4draft_withhold.so; see NVFP4_TEST_WITHHOLD in csrc/common.cuh) never issues the
first load of K of CTA 0 and shortens the wait limit to 20 ms.  Nothing of the withheld copy is ever in flight.  Each
call must return and report NVFP4_ERR_TIMEOUT; the context stays usable: the library's own call on the same inputs
afterwards is right, TMEM included."""
import ctypes
import os

import pytest
import torch

import attention_step_ref as ref

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
    L.prompt_attention.argtypes = [P(m._PromptInput), P(m._Rows), P(m._Exec)]
    L.prompt_attention.restype = ctypes.c_int
    return L


# both forms of the kernel at each head size; one item, several, items that many CTAs share
@pytest.mark.parametrize("d,lens,hq,hk", [(64, [5], 2, 2), (64, [900, 40], 8, 2), (128, [5], 2, 2), (128, [900, 40], 8, 2),
                                          (128, [1], 4, 1), (256, [3], 2, 2), (256, [900, 40], 8, 2), (128, [3000], 2, 2)])
def test_attention_wait_runs_out_and_the_call_returns(dev, wl, d, lens, hq, hk):
    import nvfp4_speculative_draft_gb300 as nd
    g = torch.Generator(device=dev)
    g.manual_seed(sum(lens) + d)
    t = sum(lens)
    q, k, v = (torch.randn((t, h, d), generator=g, device=dev).to(torch.bfloat16) for h in (hq, hk, hk))
    cu = torch.tensor([sum(lens[:i]) for i in range(len(lens) + 1)], dtype=torch.int32, device=dev)
    out = torch.empty_like(q)
    ws = torch.zeros(nd.ATTENTION_WS_BYTES, dtype=torch.uint8, device=dev)
    status = torch.zeros(1, dtype=torch.int32, device=dev)

    def rows(x):
        return nd._Rows(x.data_ptr(), x.stride(0), x.stride(1))

    a = nd._PromptInput(rows(q), rows(k), rows(v), cu.data_ptr(), t, len(lens), hq, hk, d, d ** -0.5)
    ex = nd._Exec(torch.cuda.current_stream().cuda_stream, ws.data_ptr(), ws.numel(), status.data_ptr())
    torch.cuda.synchronize()
    assert wl.prompt_attention(ctypes.byref(a), ctypes.byref(rows(out)), ctypes.byref(ex)) == 0
    torch.cuda.synchronize()
    assert status.item() == NVFP4_ERR_TIMEOUT
    status.zero_()
    got = nd.prompt_attention(q, k, v, cu, dev_status=status)
    assert status.item() == 0
    for s in range(len(lens)):
        part = slice(int(cu[s]), int(cu[s + 1]))
        want, tol = ref.attend(q[part], k[part], v[part], 0)
        assert ((got[part].double() - want).abs() <= tol).all()
