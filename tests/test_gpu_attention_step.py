"""The attention step's operators on the GPU against plain 64-bit implementations.

Tolerances: the plan exactly; rotary results to the rounding of the result (BF16, 2^-8 relative) and
the sines' and FP32 products' error, (|x| + |y|) 6e-7 (sines 4e-7, two products and a sum 3 x 2^-24);
attention to the bound that ``attention_step_ref.attend`` derives."""
import random

import pytest
import torch

import attention_step_ref as ref

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


def nd():
    import nvfp4_speculative_draft_gb300 as m
    return m


def gen(dev, seed):
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    return g


def randn(g, *shape):
    return torch.randn(shape, generator=g, device=g.device)


def ints(dev, x):
    return torch.tensor(x, dtype=torch.int32, device=dev)


def prefix(n):
    out = [0]
    for x in n:
        out.append(out[-1] + x)
    return out


# ------------------------------------------------------------------- plan

def run_plan(dev, lens, new, held, table, free, count, page, tokens, **kw):
    m = nd()
    t = ints(dev, table).view(len(lens), -1)
    status = torch.zeros(1, dtype=torch.int32, device=dev)
    p = m.kv_plan(ints(dev, lens), ints(dev, new), t, ints(dev, free), ints(dev, [count]), page, tokens,
                  held=None if held is None else ints(dev, held), dev_status=status, **kw)
    got = (t.tolist(), p.cu_new.tolist(), p.kv_lens.tolist(), p.positions.tolist(), p.slots.tolist(),
           p.held.tolist(), p.free_count.item())
    return got, status.item()


def plan_case(seed, batch, page, most_len, most_new, spare=50, with_held=True):
    r = random.Random(seed)
    lens = [r.randint(0, most_len) for _ in range(batch)]
    new = [r.choice([-1, 0, 1, 1, 2, r.randint(1, most_new)]) for _ in range(batch)]
    held = [-(-n // page) + r.choice([0, 0, 1, 3]) for n in lens]
    width = max(held + [1]) + -(-most_new // page) + 1
    ids = list(range(sum(held) + sum(max(n, 0) // page + 1 for n in new) + spare))
    r.shuffle(ids)
    table = [[-1] * width for _ in lens]
    for row, n in zip(table, held):
        for j in range(n):
            row[j] = ids.pop()
    if not with_held:
        held = None
    return lens, new, held, table, ids, page, sum(max(n, 0) for n in new)


@pytest.mark.parametrize("batch,page,most_len,most_new", [
    (1, 16, 0, 1), (1, 16, 100, 1), (3, 1, 9, 4), (24, 16, 3000, 5), (33, 7, 500, 90), (511, 32, 200, 3), (513, 16, 60, 40),
    (1000, 64, 4000, 300), (2, 16, 50, 20000), (8192, 16, 40, 2)])
def test_plan(dev, batch, page, most_len, most_new):
    lens, new, held, table, ids, page, total = plan_case(batch + page, batch, page, most_len, most_new)
    for tokens in (total, total + 13):  # exact and padded
        want = ref.plan(lens, new, held, table, ids, len(ids), page, tokens)
        got, status = run_plan(dev, lens, new, held, table, ids, len(ids), page, tokens)
        for g, w in zip(got, want):
            assert g == w
        assert status == 0


def test_plan_without_held(dev):
    lens, new, _, table, ids, page, total = plan_case(5, 40, 16, 300, 30)
    want = ref.plan(lens, new, None, table, ids, len(ids), page, total)
    got, status = run_plan(dev, lens, new, None, table, ids, len(ids), page, total)
    assert tuple(got) == tuple(want) and status == 0


@pytest.mark.parametrize("count", [0, 1, 7, 20, 10 ** 6, -4])
def test_plan_short_of_pages(dev, count):
    lens, new, held, table, ids, page, total = plan_case(9, 60, 16, 300, 60)
    want = ref.plan(lens, new, held, table, ids, count, page, total)
    got, status = run_plan(dev, lens, new, held, table, ids, count, page, total)
    assert tuple(got) == tuple(want)
    refused = any(n > 0 and k == a for a, n, k in zip(lens, new, want[2]))
    clamped = count < 0 or count > len(ids)
    assert status in ([10] if refused else []) + ([9] if clamped else []) + ([0] if not refused and not clamped else [])


def test_plan_refuses_single_sequences(dev):
    # a row too short for its sequence, tokens that end early, lengths next to 2^31
    lens, new = [10, 30, 5, 2 ** 31 - 3, 7, 0], [3, 10, 4, 5, 60, 2]
    table = [[0, 90], [1, 2], [3, 91], [4, 92], [5, 93], [94, 95]]
    ids = list(range(10, 30))
    for tokens in (84, 30, 12, 3, 0):
        want = ref.plan(lens, new, None, table, ids, len(ids), 16, tokens)
        got, status = run_plan(dev, lens, new, None, table, ids, len(ids), 16, tokens)
        assert tuple(got) == tuple(want) and status == 10


def test_plan_empty_batch(dev):
    m = nd()
    e = torch.zeros(0, dtype=torch.int32, device=dev)
    p = m.kv_plan(e, e, e.view(0, 3), ints(dev, [1, 2]), ints(dev, [2]), 16, 5)
    assert p.cu_new.tolist() == [0] and p.slots.tolist() == [-1] * 5 and p.positions.tolist() == [0] * 5
    assert p.free_count.item() == 2


def test_plan_in_place_and_repeated(dev):
    """lens, held and the free count updated in place, step by step; the same call twice elsewhere."""
    m = nd()
    r = random.Random(3)
    batch, page, width = 700, 8, 40
    lens, held, ids = [0] * batch, [0] * batch, list(range(batch * 12))
    table = [[-1] * width for _ in lens]
    t, tl, th = ints(dev, table), ints(dev, lens), ints(dev, held)
    free, count = ints(dev, ids), ints(dev, [len(ids)])
    left = len(ids)
    for step in range(6):
        new = [r.choice([0, 1, 3, 20]) for _ in lens]
        total = sum(new)
        want = ref.plan(lens, new, held, table, ids, left, page, total)
        once = m.kv_plan(tl, ints(dev, new), t, free, count, page, total, held=th)
        twice = m.kv_plan(tl, ints(dev, new), t, free, count, page, total, held=th)
        for f in ("cu_new", "kv_lens", "positions", "slots", "held", "free_count"):
            assert torch.equal(getattr(once, f), getattr(twice, f))
        out = m.KvPlan(once.cu_new, tl, once.positions, once.slots, th, count)
        p = m.kv_plan(tl, ints(dev, new), t, free, count, page, total, held=th, out=out)
        table, cu, lens, positions, slots, held, left = want
        assert p is out and t.tolist() == table and tl.tolist() == lens and th.tolist() == held
        assert p.slots.tolist() == slots and p.cu_new.tolist() == cu and count.item() == left
        # refused drafts: the length goes back, the pages stay
        lens = [max(0, n - r.choice([0, 0, 2])) for n in lens]
        tl.copy_(ints(dev, lens))


def test_plan_padded_table_and_slot_range(dev):
    m = nd()
    wide = torch.full((3, 9), 77, dtype=torch.int32, device=dev)
    t = wide[:, 2:6]
    t[:, 0] = ints(dev, [2 ** 27, 2 ** 31 - 1, -5])
    status = torch.zeros(1, dtype=torch.int32, device=dev)
    p = m.kv_plan(ints(dev, [3, 3, 3]), ints(dev, [1, 1, 14]), t, ints(dev, [8, 9]), ints(dev, [2]), 16, 16,
                  dev_status=status)
    assert p.slots.tolist() == [-1, -1] + [-1] * 13 + [9 * 16] and status.item() == 9
    assert (wide[:, :2] == 77).all() and (wide[:, 6:] == 77).all() and t[2, 1].item() == 9 and t[0, 1].item() == 77


# ----------------------------------------------------------------- rotary

def check_rope(got, x, positions, inv_freq, axis):
    want = ref.rotate(x, positions, inv_freq, axis)
    half = len(inv_freq)
    size = x[..., :half].double().abs() + x[..., half:2 * half].double().abs()
    tol = want.abs() * 2.0 ** -8 + 1e-40
    tol[..., :2 * half] += torch.cat([size, size], -1) * 6e-7
    assert bool(((got.double() - want).abs() <= tol).all())
    assert torch.equal(got[..., 2 * half:], x[..., 2 * half:])


@pytest.mark.parametrize("tokens,hq,hk,dim,rot,sections,interleaved", [
    (1, 1, 1, 16, 16, None, False), (1, 32, 4, 256, 64, None, False), (5, 7, 1, 64, 48, None, False),
    (77, 28, 4, 128, 128, None, False), (300, 6, 2, 128, 128, (16, 24, 24), False), (130, 5, 5, 96, 96, (24, 12, 12), True),
    (33, 3, 3, 512, 512, (200, 28, 28), True), (1001, 2, 2, 80, 32, (0, 16), False), (9, 12, 12, 64, 64, (8, 8, 8, 8), False)])
def test_rope(dev, tokens, hq, hk, dim, rot, sections, interleaved):
    m, g = nd(), gen(dev, tokens + dim)
    axes = 1 if sections is None else len(sections)
    table = m.rotary_table(rot, theta=1e6, sections=sections, interleaved=interleaved, device=dev)
    inv = [1e6 ** (-2.0 * i / rot) for i in range(rot // 2)]
    axis = table.axis.tolist()
    assert sorted(axis) == sorted(a for a, n in enumerate(sections or [rot // 2]) for _ in range(n))
    qkv = randn(g, tokens, hq + 2 * hk, dim).to(BF16)
    q, k, v = qkv.split([hq, hk, hk], 1)
    pos = torch.randint(0, 1 << 20, (axes, tokens), generator=g, device=dev, dtype=torch.int32)
    pos[:, 0] = 2 ** 31 - 1 if tokens > 1 else 5
    page, pages = 16, tokens // 16 + 3
    kc = randn(g, pages, page, hk, dim).to(BF16)
    vc = randn(g, pages, page, hk, dim).to(BF16)
    slots = torch.randperm(pages * page, generator=g, device=dev)[:tokens].to(torch.int32)
    if tokens > 4:
        slots[3] = -1
    k0, v0 = kc.clone(), vc.clone()
    status = torch.zeros(1, dtype=torch.int32, device=dev)
    qo, ko = m.rope_kv_write(q, k, v, pos if axes > 1 else pos[0], table, kc, vc, slots, dev_status=status)
    assert ko is None and status.item() == 0
    check_rope(qo, q, pos, inv, axis)
    ok = slots >= 0
    at = slots[ok].long()
    check_rope(kc.view(-1, hk, dim)[at], k[ok], pos[:, ok], inv, axis)
    assert torch.equal(vc.view(-1, hk, dim)[at], v[ok])
    kept = torch.ones(pages * page, dtype=torch.bool, device=dev)
    kept[at] = False
    assert torch.equal(kc.view(-1, hk, dim)[kept], k0.view(-1, hk, dim)[kept])
    assert torch.equal(vc.view(-1, hk, dim)[kept], v0.view(-1, hk, dim)[kept])
    # without a cache, in new tensors and in place
    q2, k2 = m.rope_kv_write(q, k, None, pos if axes > 1 else pos[0], table)
    assert torch.equal(q2, qo)
    check_rope(k2, k, pos, inv, axis)
    q3, k3, rest = q.clone(), k.clone(), qkv.clone()
    out = m.rope_kv_write(rest[:, :hq], rest[:, hq:hq + hk], None, pos if axes > 1 else pos[0], table,
                          q_out=rest[:, :hq], k_out=rest[:, hq:hq + hk])
    assert torch.equal(out[0], qo) and torch.equal(out[1], k2) and torch.equal(rest[:, hq + hk:], qkv[:, hq + hk:])
    assert torch.equal(q, q3) and torch.equal(k, k3)


def test_rope_layouts(dev):
    """Heads before tokens, caches with heads before tokens and with keys and values in one tensor."""
    m, g = nd(), gen(dev, 1)
    t, hq, hk, d = 50, 6, 2, 128
    table = m.rotary_table(d, device=dev)
    inv = [1e4 ** (-2.0 * i / d) for i in range(d // 2)]
    q = randn(g, hq, t, d + 8).to(BF16)[..., :d].transpose(0, 1)
    k, v = (randn(g, hk, t, d).to(BF16).transpose(0, 1) for _ in range(2))
    pos = torch.arange(-20, t - 20, device=dev, dtype=torch.int32)  # negative ones too
    both = torch.full((9, 2, hk, 16, d), 3.0, dtype=BF16, device=dev)
    kc, vc = both[:, 0].transpose(1, 2), both[:, 1].transpose(1, 2)
    slots = torch.randperm(9 * 16, generator=g, device=dev)[:t].to(torch.int32)
    qo = torch.full((t, hq + 1, d), 5.0, dtype=BF16, device=dev)
    ko = torch.empty((t, hk, d), dtype=BF16, device=dev)
    m.rope_kv_write(q, k, v, pos, table, kc, vc, slots, q_out=qo[:, :hq], k_out=ko)
    check_rope(qo[:, :hq], q, pos[None], inv, [0] * (d // 2))
    check_rope(ko, k, pos[None], inv, [0] * (d // 2))
    assert (qo[:, hq] == 5).all()
    flat_k, flat_v = kc.reshape(-1, hk, d), vc.reshape(-1, hk, d)
    assert torch.equal(flat_k[slots.long()], ko) and torch.equal(flat_v[slots.long()], v)
    untouched = torch.ones(9 * 16, dtype=torch.bool, device=dev)
    untouched[slots.long()] = False
    assert (flat_k[untouched] == 3).all() and (flat_v[untouched] == 3).all()


def test_rope_far_positions(dev):
    """A unit pair at far positions: the angle itself, where FP32 products would be off by tenths."""
    m = nd()
    pos = torch.tensor([0, 1, 12345, 999999, 123456789, 2 ** 31 - 1, -2 ** 31, -77], dtype=torch.int32, device=dev)
    table = m.rotary_table(16, inv_freq=[1.0, 0.5, 3.0, -0.25, 1e-3, 1e-9, 0.0, 6.283185307179586], device=dev)
    x = torch.zeros((8, 1, 16), dtype=BF16, device=dev)
    x[..., :8] = 1.0
    q, k = m.rope_kv_write(x, x, None, pos, table)
    import math
    for i, f in enumerate([1.0, 0.5, 3.0, -0.25, 1e-3, 1e-9, 0.0, 6.283185307179586]):
        for t, p in enumerate(pos.tolist()):
            c, s = math.cos(p * f), math.sin(p * f)
            # p f itself is rounded here: 2^-53 of up to 1.4e10 is 1.5e-6
            assert abs(q[t, 0, i].item() - c) <= abs(c) * 2 ** -8 + 3e-6
            assert abs(q[t, 0, 8 + i].item() - s) <= abs(s) * 2 ** -8 + 3e-6
    assert torch.equal(q, k)


def test_rope_slot_past_the_cache(dev):
    m, g = nd(), gen(dev, 2)
    x = randn(g, 3, 1, 16).to(BF16)
    buf = torch.full((4, 16, 1, 16), 2.0, dtype=BF16, device=dev)
    vb = buf.clone()
    status = torch.zeros(1, dtype=torch.int32, device=dev)
    m.rope_kv_write(x, x, x, ints(dev, [0, 1, 2]), m.rotary_table(16, device=dev), buf[:2], vb[:2],
                    ints(dev, [32, 2 ** 31 - 1, 31]), dev_status=status)
    assert status.item() == 9 and (buf[2:] == 2).all() and (vb[2:] == 2).all()
    assert torch.equal(vb[1, 15], x[2]) and (vb[0] == 2).all()


def test_rope_no_tokens(dev):
    m = nd()
    e = torch.zeros((0, 2, 32), dtype=BF16, device=dev)
    q, k = m.rope_kv_write(e, e, None, torch.zeros(0, dtype=torch.int32, device=dev), m.rotary_table(32, device=dev))
    assert q.shape == (0, 2, 32) and k.shape == (0, 2, 32)


# -------------------------------------------------------------- attention

def check(got, want, tol):
    err = (got.double() - want).abs()
    assert bool((err <= tol + 1e-30).all()), f"off by {(err / (tol + 1e-30)).max().item():.2f} of the bound"


def prompt_inputs(dev, seed, lens, hq, hk, d, tail=0):
    g, t = gen(dev, seed), sum(lens) + tail
    q = randn(g, t, hq, d) * (0.5 + 2.5 * torch.rand((hq, 1), generator=g, device=dev))
    return q.to(BF16), randn(g, t, hk, d).to(BF16), randn(g, t, hk, d).to(BF16), ints(dev, prefix(lens))


def check_prompt(dev, lens, hq, hk, d, tail=0, scale=None, seed=None):
    q, k, v, cu = prompt_inputs(dev, seed or sum(lens) + hq + d, lens, hq, hk, d, tail)
    status = torch.zeros(1, dtype=torch.int32, device=dev)
    out = torch.full_like(q, 9.0)
    r = nd().prompt_attention(q, k, v, cu, scale=scale, out=out, dev_status=status)
    assert r is out and status.item() == 0
    at = 0
    for n in lens:
        part = slice(at, at + n)
        check(out[part], *ref.attend(q[part], k[part], v[part], 0, scale))
        at += n
    assert (out[at:] == 9).all()


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("hq,hk,lens", [
    (1, 1, [1]), (4, 1, [2, 1, 3]), (8, 8, [5, 0, 33]), (32, 8, [77]), (7, 1, [127, 128, 129]), (10, 2, [64, 300]),
    (28, 4, [257, 1, 0, 0, 513]), (12, 1, [1000]), (96, 1, [40, 9]), (128, 1, [3, 200]), (16, 16, [700])])
def test_prompt(dev, d, hq, hk, lens):
    check_prompt(dev, lens, hq, hk, d, tail=3)


@pytest.mark.parametrize("d", [64, 128, 256])
def test_prompt_long(dev, d):
    check_prompt(dev, [3001, 17, 1500], 4, 2, d)


def test_prompt_many_short(dev):
    r = random.Random(1)
    check_prompt(dev, [r.randint(0, 40) for _ in range(900)], 4, 2, 64)


@pytest.mark.parametrize("scale", [0.0, 1.0, -0.3, 1e-30])
def test_prompt_scale(dev, scale):
    check_prompt(dev, [150, 60], 4, 2, 128, scale=scale)


def test_prompt_strided(dev):
    g = gen(dev, 8)
    hq, hk, d, lens = 6, 2, 128, [90, 200]
    t = sum(lens)
    qkv = randn(g, t, (hq + 2 * hk) * d + 40).to(BF16)[:, 8:8 + (hq + 2 * hk) * d].unflatten(1, (-1, d))
    q, k, v = qkv.split([hq, hk, hk], 1)
    vt = v.permute(1, 0, 2).contiguous().permute(1, 0, 2)  # heads before tokens
    wide = torch.full((t, hq, d + 16), 4.0, dtype=BF16, device=dev)
    out = nd().prompt_attention(q, k, vt, ints(dev, prefix(lens)), out=wide[..., 8:8 + d])
    at = 0
    for n in lens:
        check(out[at:at + n], *ref.attend(q[at:at + n], k[at:at + n], v[at:at + n], 0))
        at += n
    assert (wide[..., :8] == 4).all() and (wide[..., 8 + d:] == 4).all()


def paged_inputs(dev, seed, new, kv, hq, hk, d, page, junk=float("nan")):
    """A shuffled cache; whatever no query may use is NaN: unused pages, slots behind a sequence's end."""
    g = gen(dev, seed)
    need = [-(-n // page) for n in kv]
    pages = sum(need) + 4
    width = max(need + [1]) + 2
    order = torch.randperm(pages, generator=g, device=dev)
    table = torch.randint(-5, 2 * pages, (len(kv), width), generator=g, device=dev, dtype=torch.int32)
    kc, vc = randn(g, pages, page, hk, d).to(BF16), randn(g, pages, page, hk, d).to(BF16)
    used = torch.zeros(pages * page, dtype=torch.bool, device=dev)
    at = 0
    for s, n in enumerate(need):
        mine = order[at:at + n]
        table[s, :n] = mine.int()
        used.view(pages, page)[mine] = (torch.arange(n * page, device=dev) < kv[s]).view(n, page)
        at += n
    kc.view(-1, hk, d)[~used] = junk
    vc.view(-1, hk, d)[~used] = junk
    q = randn(g, sum(new), hq, d) * (0.5 + 2.5 * torch.rand((hq, 1), generator=g, device=dev))
    return q.to(BF16), kc, vc, table, ints(dev, kv), ints(dev, prefix(new))


def check_paged(dev, new, kv, hq, hk, d, page, seed=None, transform=None):
    q, kc, vc, table, lens, cu = paged_inputs(dev, seed or sum(kv) + hq + d, new, kv, hq, hk, d, page)
    a, b = (kc, vc) if transform is None else transform(kc, vc)
    status = torch.zeros(1, dtype=torch.int32, device=dev)
    out = nd().paged_attention(q, a, b, table, lens, cu, dev_status=status)
    assert status.item() == 0
    at = 0
    for s, (n, m) in enumerate(zip(new, kv)):
        want, tol = ref.attend(q[at:at + n], ref.gather(kc, table[s], m), ref.gather(vc, table[s], m), m - n)
        check(out[at:at + n], want, tol)
        at += n


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("hq,hk,page,new,kv", [
    (8, 1, 16, [1], [1]), (32, 4, 16, [1], [4000]), (4, 4, 16, [1, 1, 1], [17, 16, 1000]), (32, 8, 16, [5, 3, 1, 5], [900, 5, 129, 128]),
    (28, 4, 32, [6] * 5, [700, 6, 31, 33, 2000]), (12, 1, 48, [9, 2], [500, 1500]), (10, 2, 64, [40, 1, 0, 300], [1000, 64, 77, 300]),
    (14, 2, 128, [130, 257], [130, 2000]), (16, 16, 256, [3, 70], [513, 700]), (8, 2, 16, [0, 2, 0], [50, 300, 0]),
    (128, 1, 80, [2, 1], [400, 81])])
def test_paged(dev, d, hq, hk, page, new, kv):
    check_paged(dev, new, kv, hq, hk, d, page)


@pytest.mark.parametrize("d,hq,hk", [(64, 8, 8), (128, 16, 2), (256, 8, 1)])
def test_paged_batches(dev, d, hq, hk):
    r = random.Random(d)
    new = [r.choice([0, 1, 1, 5]) for _ in range(300)]
    check_paged(dev, new, [n + r.choice([0, r.randint(0, 60), r.randint(0, 1500)]) for n in new], hq, hk, d, 16)


@pytest.mark.parametrize("d,hq,hk,new,kv", [(128, 8, 1, [1], [60000]), (256, 8, 1, [3], [20001]), (64, 4, 1, [2, 1], [30000, 5]),
                                            (128, 4, 2, [700], [9000])])
def test_paged_split_over_many(dev, d, hq, hk, new, kv):
    """Few items over a long axis: the sums of many CTAs joined."""
    check_paged(dev, new, kv, hq, hk, d, 16)


def test_paged_layouts(dev):
    def heads_first(kc, vc):
        return tuple(x.permute(0, 2, 1, 3).contiguous().permute(0, 2, 1, 3) for x in (kc, vc))

    def together(kc, vc):
        both = torch.stack([kc, vc], 1)
        return both[:, 0], both[:, 1]

    def padded(kc, vc):
        wide = torch.full((*kc.shape[:3], kc.shape[3] + 24), float("nan"), dtype=BF16, device=dev)
        wide[..., 8:8 + kc.shape[3]] = kc
        return wide[..., 8:8 + kc.shape[3]], vc

    for f in (heads_first, together, padded):
        check_paged(dev, [5, 1, 30], [300, 900, 45], 8, 2, 128, 16, transform=f)


def test_queries_before_the_first_position_see_nothing(dev):
    m = nd()
    for d in (64, 128, 256):
        new, kv = [5, 3, 200], [3, 3, 120]
        q, kc, vc, table, lens, cu = paged_inputs(dev, d, [5, 3, 200], [3, 3, 120], 8, 2, d, 16)
        lens = ints(dev, [3, -4, 120])
        out = m.paged_attention(q, kc, vc, table, lens, cu)
        assert (out[:2] == 0).all() and (out[5:8] == 0).all() and (out[8:88] == 0).all()
        for s, at, skip in ((0, 0, 2), (2, 8, 80)):
            n, mm = new[s], kv[s]
            want, tol = ref.attend(q[at + skip:at + n], ref.gather(kc, table[s], mm), ref.gather(vc, table[s], mm), 0)
            check(out[at + skip:at + n], want, tol)


def test_scores_of_any_size(dev):
    """Large scores of either sign, keys whose scores rise along the axis, equal ones."""
    m, g = nd(), gen(dev, 11)
    for d in (64, 128, 256):
        n, hq, hk = 700, 4, 2
        k, v = randn(g, n, hk, d).to(BF16), randn(g, n, hk, d).to(BF16)
        for rise in (3.0, -3.0, 0.0):
            q = randn(g, n, hq, d).to(BF16)
            q[..., 0] = 8.0
            k[..., 0] = (torch.arange(n, device=dev) * rise).to(BF16)[:, None]
            check(m.prompt_attention(q, k, v, ints(dev, [0, n])), *ref.attend(q, k, v, 0))
        z = torch.zeros_like(q)
        check(m.prompt_attention(z, k, v, ints(dev, [0, n])), *ref.attend(z, k, v, 0))
        q, k = torch.full_like(q, 30.0), torch.full_like(k, -30.0)
        check(m.prompt_attention(q, k, v, ints(dev, [0, n])), *ref.attend(q, k, v, 0))


def test_other_sequences_and_rows_do_not_matter(dev):
    """NaN and infinities in another prompt, and in rows that no prompt covers."""
    m = nd()
    for d in (64, 128, 256):
        lens = [70, 90, 100]
        q, k, v, cu = prompt_inputs(dev, 3, lens, 6, 2, d, tail=60)
        clean = m.prompt_attention(q, k, v, cu)
        for x in (q, k, v):
            x[70:160] = float("nan")
            x[75] = float("inf")
            x[260:] = float("-inf")
        out = m.prompt_attention(q, k, v, cu)
        assert torch.equal(out[:70], clean[:70]) and torch.equal(out[160:260], clean[160:260])


def test_bad_device_values_are_clamped(dev):
    """Offsets and lengths that contradict the tensors: reported, within bounds."""
    m = nd()
    q, kc, vc, table, lens, cu = paged_inputs(dev, 5, [4, 4, 4], [40, 50, 60], 4, 2, 64, 16, junk=0.0)

    def call(table=table, lens=lens, cu=cu):
        status = torch.zeros(1, dtype=torch.int32, device=dev)
        out = torch.full_like(q, 7.0)
        m.paged_attention(q, kc, vc, table, lens, cu, out=out, dev_status=status)
        return out, status.item()

    good, code = call()
    assert code == 0
    out, code = call(cu=ints(dev, [0, 4, 8, 500]))
    assert code == 9 and torch.equal(out[:8], good[:8])
    out, code = call(cu=ints(dev, [0, 4, 2, 12]))  # (two sequences claim rows 2 and 3)
    assert code == 9 and torch.equal(out[:2], good[:2])
    out, code = call(cu=ints(dev, [-3, 4, 8, 12]))
    assert code == 9 and torch.equal(out[4:], good[4:])
    out, code = call(lens=ints(dev, [40, 50, 10 ** 9]))
    assert code == 9 and torch.equal(out[:8], good[:8])
    bad = table.clone()
    bad[1, 0] = 10 ** 6
    bad[1, 1] = -1
    out, code = call(table=bad)
    assert code == 9 and torch.equal(out[:4], good[:4]) and torch.equal(out[8:], good[8:])
    kz, vz = ref.gather(kc, table[1], 50).clone(), ref.gather(vc, table[1], 50).clone()
    kz[:32] = 0
    vz[:32] = 0
    check(out[4:8], *ref.attend(q[4:8], kz, vz, 46))


def test_no_tokens_or_sequences(dev):
    m = nd()
    e = torch.zeros((0, 4, 64), dtype=BF16, device=dev)
    assert m.prompt_attention(e, e, e, ints(dev, [0])).shape == (0, 4, 64)
    q = torch.ones((5, 4, 64), dtype=BF16, device=dev)
    out = torch.full_like(q, 3.0)
    m.prompt_attention(q, q, q, ints(dev, [0]), out=out)
    assert (out == 3).all()
    m.prompt_attention(q, q, q, ints(dev, [2, 2, 2]), out=out)
    assert (out == 3).all()


def test_same_bits_twice_and_any_batch_position(dev):
    m = nd()
    q, kc, vc, table, lens, cu = paged_inputs(dev, 6, [5] * 40, [3000 + 13 * i for i in range(40)], 16, 2, 128, 16)
    a = m.paged_attention(q, kc, vc, table, lens, cu)
    for _ in range(5):
        assert torch.equal(a, m.paged_attention(q, kc, vc, table, lens, cu))


def test_streams_graphs_and_workspaces(dev):
    """A captured step replayed on new inputs beside eager calls on another stream."""
    m = nd()
    args = paged_inputs(dev, 7, [1] * 6, [4000] * 6, 8, 1, 128, 16)
    other = paged_inputs(dev, 8, [2] * 3, [5000] * 3, 8, 2, 128, 16)
    want, want_other = m.paged_attention(*args), m.paged_attention(*other)
    q = args[0].clone()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        m.paged_attention(q, *args[1:])
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = m.paged_attention(q, *args[1:])
    second = torch.cuda.CUDAGraph()
    with torch.cuda.graph(second):
        out2 = m.paged_attention(other[0], *other[1:])
    q.zero_()
    for _ in range(3):
        q.copy_(args[0])
        graph.replay()
        with torch.cuda.stream(side):
            second.replay()
            b = m.paged_attention(*other)
        c = m.paged_attention(*other, stream=side)
        torch.cuda.synchronize()
        assert torch.equal(out, want) and torch.equal(out2, want_other)
        assert torch.equal(b, want_other) and torch.equal(c, want_other)
        out.zero_()
    ws = torch.full((m.ATTENTION_WS_BYTES,), 0xFF, dtype=torch.uint8, device=dev)  # nothing need be in it
    assert torch.equal(m.paged_attention(*args, workspace=ws), want)


# ------------------------------------------------------------ the whole step

def test_step_by_step_equals_whole_prompt(dev):
    """Prompts prefilled in one pass; the same tokens in chunks, drafts and single tokens over the paged
    cache: both within the bound of one definition, and of what the verify step accepts."""
    m, g = nd(), gen(dev, 20)
    r = random.Random(20)
    hq, hk, d, page = 8, 2, 128, 16
    lens = [150, 333, 41]
    total, batch = sum(lens), len(lens)
    cu = prefix(lens)
    rotary = m.rotary_table(d, theta=1e6, device=dev)
    qkv = randn(g, total, (hq + 2 * hk) * d).to(BF16).view(total, -1, d)
    q, k, v = qkv.split([hq, hk, hk], 1)
    pos = torch.cat([torch.arange(n, device=dev) for n in lens]).int()
    qr, kr = m.rope_kv_write(q, k, None, pos, rotary)
    whole = m.prompt_attention(qr, kr, v, ints(dev, cu))

    table = torch.full((batch, 30), -1, dtype=torch.int32, device=dev)
    pages = 70
    free = torch.randperm(pages, generator=g, device=dev).int()
    count, held, have = ints(dev, [pages]), ints(dev, [0] * batch), [0] * batch
    kc = torch.full((pages, page, hk, d), float("nan"), dtype=BF16, device=dev)
    vc = torch.full_like(kc, float("nan"))
    got = torch.zeros_like(whole)
    status = torch.zeros(1, dtype=torch.int32, device=dev)
    while any(a < n for a, n in zip(have, lens)):
        new = [min(n - a, r.choice([0, 1, 5, 64, 100])) for a, n in zip(have, lens)]
        rows = torch.cat([torch.arange(cu[s] + have[s], cu[s] + have[s] + new[s], device=dev) for s in range(batch)])
        pad = 3
        x = torch.cat([qkv[rows], torch.full((pad, *qkv.shape[1:]), float("nan"), dtype=BF16, device=dev)])
        xq, xk, xv = x.split([hq, hk, hk], 1)
        plan = m.kv_plan(ints(dev, have), ints(dev, new), table, free, count, page, x.shape[0], held=held, dev_status=status)
        xr, _ = m.rope_kv_write(xq, xk, xv, plan.positions, rotary, kc, vc, plan.slots, dev_status=status)
        o = m.paged_attention(xr, kc, vc, table, plan.kv_lens, plan.cu_new, dev_status=status)
        got[rows] = o[: len(rows)]
        keep = [max(0, n - (r.choice([0, 2]) if n == 5 else 0)) for n in new]  # refused drafts are drafted again
        have = [a + n for a, n in zip(have, keep)]
        held, count = plan.held, plan.free_count
    assert status.item() == 0
    for s in range(batch):
        part = slice(cu[s], cu[s + 1])
        want, tol = ref.attend(qr[part], kr[part], v[part], 0)
        check(whole[part], want, tol)
        check(got[part], want, tol)


def test_step_feeds_the_verify_step(dev):
    """plan -> rotary and cache -> attention -> norm -> head -> verification; then the next plan from what
    was accepted, with the pages of the refused drafts."""
    m, g = nd(), gen(dev, 21)
    batch, drafts, hq, hk, d, page, vocab = 5, 3, 4, 1, 64, 16, 512
    n = drafts + 1
    lens = ints(dev, [30, 1, 100, 15, 64])
    table = torch.full((batch, 12), -1, dtype=torch.int32, device=dev)
    have = (lens + page - 1) // page
    ids = torch.arange(40, device=dev, dtype=torch.int32)
    at = 0
    for s in range(batch):
        c = int(have[s])
        table[s, :c] = ids[at:at + c]
        at += c
    kc, vc = randn(g, 40, page, hk, d).to(BF16), randn(g, 40, page, hk, d).to(BF16)
    free, count = ids[at:].clone(), ints(dev, [40 - at])
    status = torch.zeros(1, dtype=torch.int32, device=dev)
    plan = m.kv_plan(lens, ints(dev, [n] * batch), table, free, count, page, batch * n, dev_status=status)
    qkv = randn(g, batch * n, hq + 2 * hk, d).to(BF16)
    q, k, v = qkv.split([hq, hk, hk], 1)
    q, _ = m.rope_kv_write(q, k, v, plan.positions, m.rotary_table(d, device=dev), kc, vc, plan.slots, dev_status=status)
    o = m.paged_attention(q, kc, vc, table, plan.kv_lens, plan.cu_new, dev_status=status)
    for s in range(batch):
        part, total = slice(s * n, s * n + n), int(lens[s]) + n
        check(o[part], *ref.attend(q[part], ref.gather(kc, table[s], total), ref.gather(vc, table[s], total), total - n))
    gamma = torch.ones(hq * d, dtype=BF16, device=dev)
    acts, _ = m.fp8b_rmsnorm(o.view(batch * n, hq * d), gamma)
    head = m.fp8b_quantize((randn(g, vocab, hq * d) * 0.05).to(BF16))
    probs = torch.softmax(m.fp8b_gemm(acts, head, out_dtype=torch.float32).view(batch, n, vocab), -1)
    drafted = probs[:, :drafts].argmax(-1).int()
    u = torch.rand((batch, drafts), generator=g, device=dev)
    tokens, accepted = m.spec_verify(probs, drafted, u, torch.rand(batch, generator=g, device=dev))
    after = lens + accepted + 1
    again = m.kv_plan(after, ints(dev, [n] * batch), table, free, plan.free_count, page, batch * n, held=plan.held,
                      dev_status=status)
    want = ref.plan(after.tolist(), [n] * batch, plan.held.tolist(), table.tolist(), free.tolist(),
                    plan.free_count.item(), page, batch * n)
    assert again.slots.tolist() == want[4] and again.free_count.item() == want[6] and status.item() == 0
