"""The attention step's operators where they can go wrong: offsets past 32 bits, very many sequences, very long ones,
padded batches, streams, values that are not finite, calls that are refused."""
import random

import pytest
import torch

import attention_step_ref as ref
from test_gpu_attention_step import BF16, check, check_paged, check_rope, gen, ints, nd, paged_inputs, prefix, randn

pytestmark = pytest.mark.gpu


def test_cache_past_32_bits(dev):
    """Pages whose elements lie past 2^31 and 2^32: written by rope_kv_write, read by paged_attention."""
    m, g = nd(), gen(dev, 1)
    page, hk, d, hq = 32, 4, 256, 8
    count = 2 ** 32 // (page * hk * d) + 40
    kc, vc = (torch.empty((count, page, hk, d), dtype=BF16, device=dev) for _ in range(2))
    assert kc.numel() > 2 ** 32
    table = ints(dev, [[count - 1, 3, count - 20, 2 ** 31 // (page * hk * d) + 1], [0, count - 2, 7, 8]])
    lens = [100, 64]
    t = sum(lens)
    q, k, v = (randn(g, t, h, d).to(BF16) for h in (hq, hk, hk))
    pos = torch.cat([torch.arange(n, device=dev) for n in lens]).int()
    slots = torch.cat([table[s].long()[torch.arange(n, device=dev) // page] * page + torch.arange(n, device=dev) % page
                       for s, n in enumerate(lens)]).int()
    rotary = m.rotary_table(d, device=dev)
    qr, kr = m.rope_kv_write(q, k, v, pos, rotary, kc, vc, slots, k_out=torch.empty_like(k))
    assert torch.equal(kc.view(-1, hk, d)[slots.long()], kr) and torch.equal(vc.view(-1, hk, d)[slots.long()], v)
    out = m.paged_attention(qr, kc, vc, table, ints(dev, lens), ints(dev, prefix(lens)))
    at = 0
    for s, n in enumerate(lens):
        p = slice(at, at + n)
        check(out[p], *ref.attend(qr[p], kr[p], v[p], 0))
        at += n


@pytest.mark.parametrize("d", [64, 128, 256])
def test_thousands_of_sequences(dev, d):
    m, g, r = nd(), gen(dev, d), random.Random(d)
    batch, page, hq, hk = 5000, 16, 4, 1
    kv = [r.choice([1, 2, 15, 16, 17, 40]) for _ in range(batch)]
    pages = sum(-(-n // page) for n in kv)
    kc, vc = (randn(g, pages, page, hk, d).to(BF16) for _ in range(2))
    table, at = torch.zeros((batch, 3), dtype=torch.int32), 0
    for s, n in enumerate(kv):
        for j in range(-(-n // page)):
            table[s, j] = at
            at += 1
    table = table.to(dev)
    q = randn(g, batch, hq, d).to(BF16)
    out = m.paged_attention(q, kc, vc, table, ints(dev, kv), ints(dev, list(range(batch + 1))))
    for s in r.sample(range(batch), 150) + [0, batch - 1]:
        check(out[s:s + 1], *ref.attend(q[s:s + 1], ref.gather(kc, table[s], kv[s]), ref.gather(vc, table[s], kv[s]), kv[s] - 1))


@pytest.mark.parametrize("d,page", [(64, 16), (128, 256), (256, 4096)])
def test_very_long_sequence(dev, d, page):
    check_paged(dev, [2, 1], [260003, 7], 2, 1, d, page)


def test_as_many_positions_as_an_int32_counts(dev):
    """2^31 - 1 cached tokens, by a table that names one page over and over: equal scores, so the
    values' mean, and nothing of the slot behind the last token."""
    m, page, pages = nd(), 65536, 32768
    kc = torch.zeros((2, page, 1, 64), dtype=BF16, device=dev)
    value = torch.tensor([1.0, 0.5, 0.0, -1.0], dtype=BF16, device=dev).repeat(16)
    vc = value.expand(2, page, 1, 64).contiguous()
    kc[1, -1], vc[1, -1] = float("nan"), float("nan")
    table = torch.zeros((1, pages), dtype=torch.int32, device=dev)
    table[0, -1] = 1
    q = randn(gen(dev, 1), 1, 4, 64).to(BF16)
    status = ints(dev, [0])
    out = m.paged_attention(q, kc, vc, table, ints(dev, [2 ** 31 - 1]), ints(dev, [0, 1]), dev_status=status)
    assert torch.equal(out, value.expand(1, 4, 64)) and status.item() == 0


def test_padded_batch_and_rows(dev):
    """Sequences without tokens at the end, rows of q behind the last one: as they were."""
    m = nd()
    for d in (64, 128, 256):
        new, kv = [3, 0, 1, 0, 0], [40, 0, 300, 9, 0]
        q, kc, vc, table, lens, cu = paged_inputs(dev, d, new, kv, 8, 2, d, 16)
        wide = torch.cat([q, torch.full((60, 8, d), float("nan"), dtype=BF16, device=dev)])
        out = torch.full_like(wide, 5.0)
        m.paged_attention(wide, kc, vc, table, lens, cu, out=out)
        assert torch.equal(out[:4], m.paged_attention(q, kc, vc, table, lens, cu)) and (out[4:] == 5).all()


def test_outputs_do_not_reach_further(dev):
    """Guard rows and columns around outputs, for each form of the kernel, and outputs that are only 16-byte aligned."""
    m = nd()
    for d, new, kv, hq, hk in ((64, [5, 1], [300, 20], 6, 2), (128, [5, 1], [300, 20], 6, 2), (256, [5, 70], [300, 90], 6, 2),
                               (128, [300], [900], 6, 2), (64, [300], [900], 6, 2), (128, [1], [20000], 6, 1)):
        q, kc, vc, table, lens, cu = paged_inputs(dev, d, new, kv, hq, hk, d, 16)
        want = m.paged_attention(q, kc, vc, table, lens, cu)
        t = sum(new)
        buf = torch.full((t + 4, hq + 2, d + 24), 3.0, dtype=BF16, device=dev)
        out = buf[2:2 + t, 1:1 + hq, 8:8 + d]  # (heads d + 24 apart: rows on 16 bytes, not 32)
        m.paged_attention(q, kc, vc, table, lens, cu, out=out)
        assert torch.equal(out, want)
        out.fill_(3.0)
        assert (buf == 3).all()


def test_values_that_are_not_finite(dev):
    """A key of a query's own that is not a number makes that query's result so, and no other sequence's."""
    m = nd()
    for d in (64, 128, 256):
        q, kc, vc, table, lens, cu = paged_inputs(dev, 3, [1, 1, 1], [200, 300, 2000], 4, 2, d, 16)
        clean = m.paged_attention(q, kc, vc, table, lens, cu)
        kc[table[1, 2], 5, 0] = float("nan")
        vc[table[2, 9], 3, 1, 7] = float("inf")
        out = m.paged_attention(q, kc, vc, table, lens, cu)
        assert torch.equal(out[0], clean[0])
        assert torch.isnan(out[1, :2]).all() and torch.equal(out[1, 2:], clean[1, 2:])
        assert torch.isinf(out[2, 2:, 7]).all() or torch.isnan(out[2, 2:, 7]).all()
        keep = torch.ones(d, dtype=torch.bool, device=dev)
        keep[7] = False
        assert torch.equal(out[2, 2:, keep], clean[2, 2:, keep]) and torch.equal(out[2, :2], clean[2, :2])
    # all scores of a row not numbers
    q = torch.full((3, 2, 64), float("nan"), dtype=BF16, device=dev)
    k = torch.ones((3, 2, 64), dtype=BF16, device=dev)
    assert torch.isnan(m.prompt_attention(q, k, k, ints(dev, [0, 3]))).all()


def test_values_behind_the_tokens_of_an_item(dev):
    """Later tokens of the same prompt that are not finite: queries of earlier items are untouched."""
    m = nd()
    for d, hq, hk in ((64, 8, 1), (128, 8, 1), (256, 8, 1)):
        g = gen(dev, d)
        t = 500
        q, k, v = (randn(g, t, h, d).to(BF16) for h in (hq, hk, hk))
        clean = m.prompt_attention(q, k, v, ints(dev, [0, t]))
        k[300:], v[300:] = float("nan"), float("nan")
        out = m.prompt_attention(q, k, v, ints(dev, [0, t]))
        # an item is 32 tokens at most (256 rows of 8 heads): it ends before token 300 up to token 288
        assert torch.equal(out[:288], clean[:288]) and torch.isnan(out[300:]).all()


def test_rope_on_another_stream_and_captured(dev):
    m, g = nd(), gen(dev, 4)
    x = randn(g, 700, 12, 128).to(BF16)
    q, k, v = x.split([8, 2, 2], 1)
    table = m.rotary_table(128, device=dev)
    pos = torch.arange(700, device=dev).int()
    kc, vc = (torch.zeros((50, 16, 2, 128), dtype=BF16, device=dev) for _ in range(2))
    slots = torch.randperm(800, generator=g, device=dev)[:700].int()
    want, _ = m.rope_kv_write(q, k, v, pos, table, kc, vc, slots)
    wk, wv = kc.clone(), vc.clone()
    side = torch.cuda.Stream()
    kc.zero_()
    vc.zero_()
    side.wait_stream(torch.cuda.current_stream())
    got, _ = m.rope_kv_write(q, k, v, pos, table, kc, vc, slots, stream=side)
    side.synchronize()
    assert torch.equal(got, want) and torch.equal(kc, wk) and torch.equal(vc, wv)
    graph = torch.cuda.CUDAGraph()
    lens, new = ints(dev, [100, 0, 37]), ints(dev, [5, 2, 1])
    block, free, count = torch.full((3, 20), -1, dtype=torch.int32, device=dev), torch.arange(60, device=dev).int(), ints(dev, [60])
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        plan = m.kv_plan(lens, new, block, free, count, 16, 10)
        out, _ = m.rope_kv_write(q, k, v, pos, table, kc, vc, slots)
    kc.zero_()
    lens.copy_(ints(dev, [0, 16, 31]))
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want) and torch.equal(kc, wk)
    ref_plan = ref.plan([0, 16, 31], [5, 2, 1], None, [[-1] * 20] * 3, list(range(60)), 60, 16, 10)
    assert plan.kv_lens.tolist() == ref_plan[2] and plan.cu_new.tolist() == ref_plan[1] and plan.positions.tolist() == ref_plan[3]


def test_rope_very_wide_and_many_tokens(dev):
    m, g = nd(), gen(dev, 5)
    for t, hq, hk, d, rot in ((3, 300, 40, 256, 256), (5001, 3, 1, 64, 32), (2432, 5, 5, 48, 48)):
        q, k = randn(g, t, hq, d).to(BF16), randn(g, t, hk, d).to(BF16)
        pos = torch.randint(0, 10 ** 6, (1, t), generator=g, device=dev, dtype=torch.int32)
        qo, ko = m.rope_kv_write(q, k, None, pos[0], m.rotary_table(rot, device=dev))
        inv = [1e4 ** (-2.0 * i / rot) for i in range(rot // 2)]
        check_rope(qo, q, pos, inv, [0] * (rot // 2))
        check_rope(ko, k, pos, inv, [0] * (rot // 2))


# --------------------------------------------------------------- refusals

def refused(call, what=ValueError):
    with pytest.raises(what):
        call()


def test_attention_refuses(dev):
    m = nd()
    q, kc, vc, table, lens, cu = paged_inputs(dev, 1, [2, 1], [20, 30], 4, 2, 64, 16)
    good = (q, kc, vc, table, lens, cu)

    def paged(i, x, **kw):
        return lambda: m.paged_attention(*good[:i], x, *good[i + 1:], **kw)

    for i, bad in ((0, q.float()), (0, q[0]), (0, q.transpose(1, 2)), (0, q.cpu()), (1, kc.float()), (1, kc[0]), (1, kc[..., :32]),
                   (2, vc[1:]), (2, vc.cpu()), (3, table.long()), (3, table[:1]), (3, table.t().contiguous().t()), (4, lens[:1]), (4, lens.float()),
                   (5, cu[:2]), (5, cu.long()), (4, torch.stack([lens, lens], 1)[:, 0])):
        refused(paged(i, bad))
    refused(paged(0, q[:, :3]), m.Nvfp4Error)                     # heads that do not divide
    refused(lambda: m.paged_attention(q[..., :32].contiguous(), kc[..., :32].contiguous(), vc[..., :32].contiguous(), *good[3:]), m.Nvfp4Error)
    odd = torch.zeros(q.numel() + 8, dtype=BF16, device=dev)[1:1 + q.numel()].view_as(q)
    refused(paged(0, odd), m.Nvfp4Error)                           # 2-byte aligned
    small = torch.zeros((9, 8, 2, 64), dtype=BF16, device=dev)
    refused(lambda: m.paged_attention(q, small, small, *good[3:]), m.Nvfp4Error)  # pages of 8
    for out in (q[:2], q.float(), q[:, :, :32], q[:1].expand(3, 4, 64)):
        refused(paged(0, q, out=out))
    refused(paged(0, q, workspace=torch.zeros(100, dtype=torch.uint8, device=dev)), m.Nvfp4Error)
    refused(paged(0, q, workspace=torch.zeros(100, dtype=torch.uint8)))
    refused(paged(0, q, dev_status=torch.zeros(1, device=dev)))
    refused(paged(0, q, scale=float("nan")), m.Nvfp4Error)
    refused(paged(0, q, scale="x"), TypeError)
    k = torch.zeros((3, 2, 64), dtype=BF16, device=dev)
    for args in ((q, k[:2], k, cu), (q, k, k[:, :1], cu), (q, k, k, cu.long()), (q, k, k, cu[:0]), (q, k.float(), k, cu), (q, None, k, cu)):
        refused(lambda: m.prompt_attention(*args))


def test_rope_refuses(dev):
    m = nd()
    q = torch.zeros((5, 4, 64), dtype=BF16, device=dev)
    k = torch.zeros((5, 2, 64), dtype=BF16, device=dev)
    kc = torch.zeros((4, 16, 2, 64), dtype=BF16, device=dev)
    pos, slots, table = ints(dev, [0] * 5), ints(dev, [1, 2, 3, 4, 5]), m.rotary_table(64, device=dev)
    three = m.rotary_table(64, sections=[8, 12, 12], device=dev)
    for args, kw in (((q, k, k, pos[:4], table), {}), ((q, k, k, pos.long(), table), {}), ((q, k[:4], k, pos, table), {}),
                     ((q, k.float(), k, pos, table), {}), ((q, k, k, pos, m.rotary_table(128, device=dev)), {}),
                     ((q, k, k, pos, m.rotary_table(64, device="cpu")), {}), ((q, k, k, pos.view(1, 5), three), {}),
                     ((q, k, k, pos, table), dict(k_cache=kc)), ((q, k, k, pos, table), dict(k_cache=kc, v_cache=kc)),
                     ((q, k, None, pos, table), dict(k_cache=kc, v_cache=kc, slots=slots)),
                     ((q, k, k, pos, table), dict(k_cache=kc, v_cache=kc[:3], slots=slots)),
                     ((q, k, k, pos, table), dict(k_cache=kc[:, :, :1], v_cache=kc[:, :, :1], slots=slots)),
                     ((q, k, k, pos, table), dict(k_cache=kc, v_cache=kc, slots=slots[:3])),
                     ((q, k, k, pos, table), dict(k_cache=kc[:1].expand(4, 16, 2, 64), v_cache=kc, slots=slots)),
                     ((q, k, k, pos, table), dict(q_out=q[:, :3])), ((q, k, k, pos, table), dict(k_out=k.float())),
                     ((q, k, k, pos, table), dict(q_out=q[:1].expand(5, 4, 64)))):
        refused(lambda: m.rope_kv_write(*args, **kw))
    refused(lambda: m.rope_kv_write(q[..., :40].contiguous(), k[..., :40].contiguous(), None, pos, m.rotary_table(32, device=dev)), m.Nvfp4Error)


def test_plan_refuses(dev):
    m = nd()
    i = ints(dev, [1, 2, 3])
    good = (i, i, torch.zeros((3, 4), dtype=torch.int32, device=dev), i, i[:1])
    for j, bad in ((0, i.long()), (0, i.view(3, 1)), (1, i[:2]), (2, good[2][:2]), (2, i), (2, good[2].long()), (3, i.view(1, 3)), (4, i), (4, None)):
        refused(lambda: m.kv_plan(*good[:j], bad, *good[j + 1:], 16, 8))
    refused(lambda: m.kv_plan(*good, 16, -1))
    refused(lambda: m.kv_plan(*good, 16, 8, held=i[:2]))
    refused(lambda: m.kv_plan(*good, 0, 8), m.Nvfp4Error)
    refused(lambda: m.kv_plan(*good, 1 << 20, 8), m.Nvfp4Error)
    refused(lambda: m.kv_plan(*good, 16, 8, out=m.KvPlan(i, i, i, i, i, i)))
