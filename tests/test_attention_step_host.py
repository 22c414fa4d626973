"""Host-side checks of the attention step's calls: the C ABI's status codes and the binding's refusals before
anything is launched (no GPU), the rotary table, and the tests' own plain implementations against closed forms."""
import ctypes
import math

import pytest
import torch

import attention_step_ref as ref
import nvfp4_speculative_draft_gb300 as nd

P = 0x10000  # a well-aligned address that nothing reads: every call below is refused


@pytest.fixture(scope="module")
def L():
    from nvfp4_speculative_draft_gb300 import build
    build.build()
    return nd.load()


def ex(ws=None, size=0):
    return ctypes.byref(nd._Exec(None, ws, size, None))


PLAN_IN = dict(lens=P, num_new=P, held=None, block_table=P, ld_table=8, max_pages=8, free_pages=P, free_capacity=9,
               free_count=P, batch=3, page_size=16, tokens=5)
PLAN_OUT = dict(cu_new=P, kv_lens=P, positions=P, slots=P, held=None, free_count=None)


@pytest.mark.parametrize("kin,kout,code", [
    (dict(lens=None), {}, 1), (dict(num_new=None), {}, 1), (dict(block_table=None), {}, 1), (dict(free_pages=None), {}, 1),
    (dict(free_count=None), {}, 1), ({}, dict(cu_new=None), 1), ({}, dict(kv_lens=None), 1), ({}, dict(positions=None), 1),
    ({}, dict(slots=None), 1),
    (dict(batch=-1), {}, 2), (dict(batch=8193), {}, 2), (dict(page_size=0), {}, 2), (dict(page_size=65537), {}, 2),
    (dict(tokens=-1), {}, 2), (dict(tokens=2 ** 31), {}, 2), (dict(max_pages=0), {}, 2), (dict(max_pages=9), {}, 2),
    (dict(free_capacity=-1), {}, 2), (dict(free_capacity=2 ** 31), {}, 2),
    (dict(lens=P + 2), {}, 3), (dict(held=P + 1), {}, 3), (dict(free_count=P + 2), {}, 3), ({}, dict(slots=P + 2), 3),
    ({}, dict(held=P + 3), 3),
])
def test_plan_status(L, kin, kout, code):
    i, o = nd._PlanInput(**{**PLAN_IN, **kin}), nd._PlanOutput(**{**PLAN_OUT, **kout})
    assert L.kv_plan(ctypes.byref(i), ctypes.byref(o), ex()) == code
    assert L.kv_plan(None, ctypes.byref(o), ex()) == 1 and L.kv_plan(ctypes.byref(i), None, ex()) == 1


def rows(data=P, ld_token=512, ld_head=128):
    return nd._Rows(data, ld_token, ld_head)


def pages(data=P, ld_page=8192, ld_token=512, ld_head=128):
    return nd._Pages(data, ld_page, ld_token, ld_head)


ROPE_IN = dict(q=rows(), k=rows(), v=rows(), tokens=4, heads=4, kv_heads=2, dim=128, rot_dim=64, positions=P, ld_positions=4,
               axes=1, turns=P, axis=None, k_cache=pages(), v_cache=pages(), pages=10, page_size=16, slots=P)


@pytest.mark.parametrize("kin,kout,code", [
    (dict(q=rows(None)), {}, 1), (dict(k=rows(None)), {}, 1), (dict(v=rows(None)), {}, 1), (dict(positions=None), {}, 1),
    (dict(turns=None), {}, 1), (dict(slots=None), {}, 1), (dict(v_cache=pages(None)), {}, 1), ({}, dict(q=rows(None)), 1),
    (dict(tokens=-1), {}, 2), (dict(heads=0), {}, 2), (dict(kv_heads=0), {}, 2), (dict(dim=24), {}, 2), (dict(dim=528), {}, 2),
    (dict(rot_dim=144), {}, 2), (dict(rot_dim=8), {}, 2), (dict(rot_dim=0), {}, 2), (dict(axes=0), {}, 2), (dict(ld_positions=3), {}, 2),
    (dict(pages=0), {}, 2), (dict(page_size=0), {}, 2), (dict(pages=2 ** 28, page_size=16), {}, 2),
    (dict(q=rows(P + 2)), {}, 3), (dict(k=rows(ld_head=132)), {}, 3), (dict(v=rows(ld_token=516)), {}, 3),
    (dict(k_cache=pages(ld_page=4)), {}, 3), (dict(v_cache=pages(P + 8)), {}, 3), (dict(turns=P + 4), {}, 3),
    (dict(positions=P + 2), {}, 3), (dict(slots=P + 1), {}, 3), ({}, dict(q=rows(ld_token=4)), 3), ({}, dict(k=rows(P + 4)), 3),
])
def test_rope_status(L, kin, kout, code):
    i, o = nd._RopeInput(**{**ROPE_IN, **kin}), nd._RopeOutput(**{**dict(q=rows(), k=rows(None)), **kout})
    assert L.rope_kv_write(ctypes.byref(i), ctypes.byref(o), ex()) == code


ATTEND = dict(tokens=4, batch=2, heads=8, kv_heads=2, dim=128, scale=0.1, cu=P, q=rows())
PROMPT_IN = dict(ATTEND, k=rows(), v=rows())
PAGED_IN = dict(ATTEND, k=pages(), v=pages(), pages=10, page_size=16, block_table=P, ld_table=8, max_pages=8, kv_lens=P)
BOTH = [
    (dict(q=rows(None)), 1), (dict(cu=None), 1), (dict(tokens=-1), 2), (dict(tokens=2 ** 31 - 1), 2), (dict(batch=-1), 2),
    (dict(batch=2 ** 20), 2), (dict(kv_heads=0), 2), (dict(heads=0), 2), (dict(heads=9), 2), (dict(heads=258), 2), (dict(dim=96), 2),
    (dict(dim=512), 2), (dict(scale=float("nan")), 2), (dict(scale=float("inf")), 2), (dict(q=rows(ld_token=-8)), 2),
    (dict(q=rows(ld_token=2 ** 39)), 2), (dict(q=rows(P + 8)), 3), (dict(q=rows(ld_head=100)), 3), (dict(cu=P + 2), 3)]


@pytest.mark.parametrize("kw,code", BOTH + [(dict(k=rows(None)), 1), (dict(v=rows(P + 2)), 3), (dict(v=rows(ld_token=-512)), 2)])
def test_prompt_status(L, kw, code):
    i = nd._PromptInput(**{**PROMPT_IN, **kw})
    assert L.prompt_attention(ctypes.byref(i), ctypes.byref(rows()), ex(P, nd.ATTENTION_WS_BYTES)) == code


@pytest.mark.parametrize("kw,code", BOTH + [
    (dict(k=pages(None)), 1), (dict(block_table=None), 1), (dict(kv_lens=None), 1), (dict(pages=0), 2), (dict(page_size=8), 2),
    (dict(page_size=24), 2), (dict(page_size=65552), 2), (dict(max_pages=0), 2), (dict(max_pages=9), 2), (dict(v=pages(P + 2)), 3),
    (dict(k=pages(ld_page=4)), 3), (dict(kv_lens=P + 1), 3), (dict(block_table=P + 2), 3)])
def test_paged_status(L, kw, code):
    i = nd._PagedInput(**{**PAGED_IN, **kw})
    assert L.paged_attention(ctypes.byref(i), ctypes.byref(rows()), ex(P, nd.ATTENTION_WS_BYTES)) == code


def test_attention_outputs_and_workspace(L):
    for f, i in ((L.prompt_attention, nd._PromptInput(**PROMPT_IN)), (L.paged_attention, nd._PagedInput(**PAGED_IN))):
        full = ex(P, nd.ATTENTION_WS_BYTES)
        assert f(None, ctypes.byref(rows()), full) == 1 and f(ctypes.byref(i), None, full) == 1
        assert f(ctypes.byref(i), ctypes.byref(rows(None)), full) == 1
        assert f(ctypes.byref(i), ctypes.byref(rows(P + 4)), full) == 3
        for e in (ex(), ex(P, nd.ATTENTION_WS_BYTES - 1), ex(P + 16, nd.ATTENTION_WS_BYTES), None):
            assert f(ctypes.byref(i), ctypes.byref(rows()), e) == 4
        i.tokens = 0  # nothing to do
        assert f(ctypes.byref(i), ctypes.byref(rows()), ex()) == 0


def test_binding_refuses_host_tensors(L):
    i = torch.zeros(2, dtype=torch.int32)
    x = torch.zeros((2, 2, 64), dtype=torch.bfloat16)
    table = nd.rotary_table(64, device="cpu")
    for call in (lambda: nd.kv_plan(i, i, i.view(1, 2), i, i, 16, 4), lambda: nd.rope_kv_write(x, x, x, i, table),
                 lambda: nd.prompt_attention(x, x, x, i), lambda: nd.paged_attention(x, x[None], x[None], i.view(1, 2), i, i),
                 lambda: nd.kv_plan(None, i, i, i, i, 16, 4), lambda: nd.prompt_attention("x", x, x, i)):
        with pytest.raises(ValueError, match="CUDA"):
            call()


def test_rotary_table():
    t = nd.rotary_table(32, theta=500.0, device="cpu")
    assert t.turns.dtype == torch.int64 and t.axis.dtype == torch.uint8 and t.axes == 1 and t.axis.sum() == 0
    for i, v in enumerate(t.turns.tolist()):
        want = 500.0 ** (-2.0 * i / 32) / (2 * math.pi)
        assert abs((v % 2 ** 64) / 2.0 ** 64 - want) <= want * 2.0 ** -51
    t = nd.rotary_table(16, inv_freq=[0.0, -1.0, 7.0, 1e-20, 2 * math.pi, 0.5, 1.0, 3.0], device="cpu")
    turns = [(v % 2 ** 64) / 2.0 ** 64 for v in t.turns.tolist()]
    assert turns[0] == 0 and abs(turns[1] - (1 - 1 / (2 * math.pi))) < 1e-15 and turns[4] == 0
    assert abs(turns[2] - (7 / (2 * math.pi) - 1)) < 1e-15
    t = nd.rotary_table(32, sections=[4, 6, 6], device="cpu")
    assert t.axis.tolist() == [0] * 4 + [1] * 6 + [2] * 6 and t.axes == 3
    t = nd.rotary_table(32, sections=[8, 4, 4], interleaved=True, device="cpu")
    assert t.axis.tolist() == [0, 1, 2, 0, 1, 2, 0, 1, 2, 0, 1, 2, 0, 0, 0, 0]


@pytest.mark.parametrize("kw", [dict(rot_dim=8), dict(rot_dim=40), dict(rot_dim=32, sections=[8, 9]), dict(rot_dim=32, sections=[]),
                                dict(rot_dim=32, sections=[17, -1]), dict(rot_dim=32, theta=0.0), dict(rot_dim=32, inv_freq=[1.0]),
                                dict(rot_dim=16, inv_freq=[float("inf")] * 8), dict(rot_dim=32, sections=[2, 7, 7], interleaved=True)])
def test_rotary_table_refuses(kw):
    with pytest.raises(ValueError):
        nd.rotary_table(device="cpu", **kw)


# ---------------------------------------- the plain implementations themselves

def test_ref_attend_closed_forms():
    v = 1 + torch.arange(12, dtype=torch.float64).view(6, 1, 2)
    q, k = torch.zeros((6, 3, 2)), torch.randn(6, 1, 2)
    out, tol = ref.attend(q, k, v, 0)  # equal scores: running means
    for i in range(6):
        assert torch.allclose(out[i, 2], v[: i + 1, 0].mean(0)) and (tol[i] > 0).all()
    out, _ = ref.attend(q[:2], k, v, -1)  # the first query sees nothing
    assert (out[0] == 0).all() and torch.equal(out[1, 0], v[0, 0])
    k[:] = 0.0
    k[4] = 1e4
    out, _ = ref.attend(torch.ones((1, 3, 2)), k, v, 5)
    assert torch.equal(out[0, 1], v[4, 0])


def test_ref_rotate_keeps_lengths_and_adds_angles():
    x = torch.randn(5, 2, 8, dtype=torch.float64)
    f, axis = [1.0, 0.1, 0.01], [0, 0, 0]
    a, b = torch.arange(5)[None], torch.full((1, 5), 7)
    y = ref.rotate(x, a, f, axis)
    assert torch.allclose(y[..., :6].norm(dim=-1), x[..., :6].norm(dim=-1)) and torch.equal(y[..., 6:], x[..., 6:])
    assert torch.allclose(ref.rotate(y, b, f, axis), ref.rotate(x, a + b, f, axis))


def test_ref_plan_by_hand():
    # two pages held; 3 + 2 tokens fit the first sequence's page, 16 + 1 need a second one
    table, cu, kv, pos, slots, held, left = ref.plan([3, 16, 5], [2, 1, 0], None, [[7, 0], [4, 0], [9, 0]], [1, 2, 8], 3, 16, 4)
    assert table == [[7, 0], [4, 8], [9, 0]] and cu == [0, 2, 3, 3] and kv == [5, 17, 5] and held == [1, 2, 1] and left == 2
    assert pos == [3, 4, 16, 0] and slots == [7 * 16 + 3, 7 * 16 + 4, 8 * 16, -1]
