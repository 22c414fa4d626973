"""Host-side checks of the verify step's calls: the C ABI's status codes and the
binding's refusals, before anything is launched (no GPU), and the tests' own plain
implementations against closed forms."""
import ctypes

import numpy as np
import pytest
import torch

import nvfp4_speculative_draft_gb300 as nd
import verify_step_ref as ref

P = 0x10000  # a well-aligned address that nothing reads: every call below is refused


@pytest.fixture(scope="module")
def L():
    from nvfp4_speculative_draft_gb300 import build
    build.build()
    return nd.load()


def ex():
    return ctypes.byref(nd._Exec(None, None, 0, None))


@pytest.mark.parametrize("args,code", [
    ((None, 4, 64, 64, P, P), 1), ((P, 4, 64, 64, None, P), 1), ((P, 4, 64, 64, P, None), 1),
    ((P, 0, 64, 64, P, P), 2), ((P, 4, 0, 64, P, P), 2), ((P, 4, 24, 24, P, P), 2), ((P, 4, 64, 56, P, P), 2),
    ((P, 2 ** 31, 64, 64, P, P), 2),
    ((P + 2, 4, 64, 64, P, P), 3), ((P, 4, 64, 68, P, P), 3), ((P, 4, 64, 64, P + 8, P), 3),
    ((P, 4, 64, 64, P, P + 2), 3),
])
def test_quantize_status(L, args, code):
    assert L.fp8b_quantize(*args, ex()) == code


def norm_input(x=P, ld_x=64, r=None, ld_r=0, ro=None, ld_ro=0, gamma=P, eps=1e-6):
    return nd._NormInput(x, ld_x, r, ld_r, ro, ld_ro, gamma, eps)


def acts(codes=P, ld=64, scales=P, lds=4, m=4, k=64):
    return nd._Fp8BlockActs(codes, ld, scales, lds, m, k)


@pytest.mark.parametrize("inp,out,code", [
    (norm_input(x=None), acts(), 1), (norm_input(), acts(codes=None), 1), (norm_input(), acts(scales=None), 1),
    (norm_input(), acts(m=0), 2), (norm_input(), acts(k=40, ld=48), 2), (norm_input(), acts(ld=48), 2),
    (norm_input(), acts(lds=3), 2), (norm_input(ld_x=56), acts(), 2), (norm_input(eps=-1.0), acts(), 2),
    (norm_input(eps=float("nan")), acts(), 2), (norm_input(r=P, ld_r=32), acts(), 2),
    (norm_input(ro=P, ld_ro=32), acts(), 2),
    (norm_input(ld_x=32784), acts(k=32784, ld=32784), 2),
    (norm_input(x=P + 8), acts(), 3), (norm_input(gamma=P + 2), acts(), 3), (norm_input(r=P + 4, ld_r=64), acts(), 3),
    (norm_input(r=P, ld_r=68), acts(), 3), (norm_input(ro=P, ld_ro=68), acts(), 3),
    (norm_input(ld_x=68), acts(), 3), (norm_input(), acts(ld=72), 3), (norm_input(), acts(codes=P + 8), 3),
    (norm_input(), acts(scales=P + 2), 3),
])
def test_rmsnorm_status(L, inp, out, code):
    assert L.fp8b_rmsnorm(ctypes.byref(inp), ctypes.byref(out), ex()) == code


def weight(codes=P, scales=P, n=8, k=64):
    return nd._Fp8BlockWeight(codes, scales, n, k)


@pytest.mark.parametrize("a,w,c,dt,ldc,code", [
    (acts(), weight(), None, 0, 8, 1), (acts(), weight(codes=None), P, 0, 8, 1),
    (acts(), weight(scales=None), P, 0, 8, 1), (acts(codes=None), weight(), P, 0, 8, 1),
    (acts(), weight(n=0), P, 0, 8, 2), (acts(), weight(k=80), P, 0, 8, 2), (acts(), weight(), P, 0, 7, 2),
    (acts(m=0), weight(), P, 0, 8, 2),
    (acts(), weight(codes=P + 4), P, 0, 8, 3), (acts(), weight(), P + 2, 0, 8, 3), (acts(), weight(), P + 1, 1, 8, 3),
    (acts(), weight(scales=P + 1), P, 1, 8, 3), (acts(), weight(), P, 7, 8, 8),
])
def test_gemm_status(L, a, w, c, dt, ldc, code):
    assert L.fp8b_gemm(ctypes.byref(a), ctypes.byref(w), c, dt, ldc, ex()) == code


def verify_input(**kw):
    d = dict(target=P, ld_target_seq=30, ld_target_pos=10, draft=P, ld_draft_seq=20, ld_draft_pos=10,
             draft_vocab=10, dtype=0, tokens=P, ld_tokens=2, num_draft=None, accept_u=P, ld_accept_u=2,
             sample_u=P, batch=3, g=2, vocab=10)
    d.update(kw)
    return nd._VerifyInput(**d)


@pytest.mark.parametrize("kw,out,ld,acc,code", [
    (dict(target=None), P, 3, P, 1), (dict(tokens=None), P, 3, P, 1), (dict(accept_u=None), P, 3, P, 1),
    (dict(sample_u=None), P, 3, P, 1), ({}, None, 3, P, 1), ({}, P, 3, None, 1),
    (dict(batch=0), P, 3, P, 2), (dict(g=-1), P, 3, P, 2), (dict(g=1025), P, 1026, P, 2), (dict(vocab=0), P, 3, P, 2),
    (dict(vocab=2 ** 30 + 1), P, 3, P, 2), (dict(draft_vocab=11), P, 3, P, 2), (dict(draft_vocab=0), P, 3, P, 2),
    (dict(ld_tokens=1), P, 3, P, 2), (dict(ld_accept_u=1), P, 3, P, 2), ({}, P, 2, P, 2),
    (dict(target=P + 2), P, 3, P, 3), (dict(target=P + 1, dtype=1), P, 3, P, 3), (dict(draft=P + 2), P, 3, P, 3),
    (dict(tokens=P + 1), P, 3, P, 3), (dict(num_draft=P + 1), P, 3, P, 3), ({}, P + 2, 3, P, 3), ({}, P, 3, P + 2, 3),
    (dict(dtype=5), P, 3, P, 8),
])
def test_verify_status(L, kw, out, ld, acc, code):
    assert L.spec_verify(ctypes.byref(verify_input(**kw)), out, ld, acc, ex()) == code


def bf16(*shape):
    return torch.zeros(shape, dtype=torch.bfloat16)


def test_binding_refuses_host_tensors(L):
    w = nd.Fp8BlockWeight(torch.zeros((8, 64), dtype=torch.uint8), torch.zeros((1, 1)), 8, 64)
    a = nd.Fp8BlockActs(torch.zeros((2, 64), dtype=torch.uint8), torch.zeros((1, 2)), 2, 64)
    f = torch.zeros((1, 2, 8))
    i = torch.zeros((1, 1), dtype=torch.int32)
    for call in (lambda: nd.fp8b_quantize(bf16(8, 64)), lambda: nd.fp8b_rmsnorm(bf16(2, 64), bf16(64)),
                 lambda: nd.fp8b_gemm(a, w), lambda: nd.spec_verify(f, i, torch.zeros((1, 1)), torch.zeros(1))):
        with pytest.raises(ValueError, match="CUDA"):
            call()


def test_binding_refuses_other_objects(L):
    a = nd.Fp8BlockActs(torch.zeros((2, 64), dtype=torch.uint8), torch.zeros((1, 2)), 2, 64)
    for call in (lambda: nd.fp8b_quantize(None), lambda: nd.fp8b_rmsnorm("x", None), lambda: nd.fp8b_rmsnorm([1.0], None),
                 lambda: nd.spec_verify(3, None, None, None)):
        with pytest.raises(ValueError, match="CUDA"):
            call()
    with pytest.raises(AttributeError):
        nd.fp8b_gemm(torch.zeros(2, 64), a)


def test_binding_needs_the_library_first():
    """The native module refuses calls before bind(), and bad arguments of bind()."""
    native = nd._load_binding()
    with pytest.raises(TypeError):
        native.bind(1, 2)
    with pytest.raises((TypeError, ValueError)):
        native.bind(0, 0, 0, 0, nd.Nvfp4Error)
    with pytest.raises(TypeError):
        native.quantize(None)


# ---------------------------------------- the plain implementations themselves

def test_ref_e4m3_matches_torch():
    codes = torch.arange(256, dtype=torch.uint8)
    v = codes.view(ref.F8).double()
    v = v[torch.isfinite(v)]
    assert torch.equal(ref.e4m3(v), v)
    x = torch.linspace(-470, 470, 20001, dtype=torch.float64)
    x = torch.cat([x, x * 2.0 ** -8, x * 2.0 ** -14]).float().clamp(-448, 448)
    assert torch.equal(ref.e4m3(x.double()), x.to(ref.F8).double())


def test_ref_verify_closed_forms():
    t = np.array([[[0.25, 0.5, 0.25, 0.0], [0.1, 0.2, 0.3, 0.4]]], np.float32)
    tok = np.array([[1]], np.int32)
    # u < p(d): accepted, then the bonus row: 0.6 of its mass is reached at token 2
    out, acc = ref.verify(t, None, tok, np.array([[0.49]]), np.array([0.55]))
    assert acc[0] == 1 and out[0].tolist() == [1, 2]
    # u = p(d): refused; what is left is 0.25, 0, 0.25
    out, acc = ref.verify(t, None, tok, np.array([[0.5]]), np.array([0.49]))
    assert acc[0] == 0 and out[0].tolist() == [0, -1]
    out, acc = ref.verify(t, None, tok, np.array([[0.5]]), np.array([0.5]))
    assert out[0].tolist() == [2, -1]
