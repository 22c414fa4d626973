"""Attention shared out over the CTAs: every tile of keys is counted once, whatever the shares' borders; many sequences
in each form of the kernel; long and short sequences together; sequences at any place of the batch.

A tile of 128 keys among thousands moves a result of random values by less than the bound of its roundings, so a tile
lost or doubled is looked for in two other ways: values that are 1 in one tile and channel only, under equal scores, and
the error's norm (``attention_step_ref.norm_bound``)."""
import random

import pytest
import torch

import attention_step_ref as ref
from test_gpu_attention_step import BF16, check_paged, check_prompt, gen, ints, nd, paged_inputs, prefix, randn

pytestmark = pytest.mark.gpu

TILE = 128


def one_hot(keys, base, heads, d, dev):
    """[keys, heads, d]: 1 where channel c of head h stands for the key's tile, base + h d + c."""
    tile = torch.arange(keys, device=dev) // TILE - base
    v = torch.zeros((keys, heads * d), dtype=BF16, device=dev)
    ours = (tile >= 0) & (tile < heads * d)
    v[torch.arange(keys, device=dev)[ours], tile[ours]] = 1.0
    return v.view(keys, heads, d)


def check_counts(got, first, keys, base, hk):
    """Under equal scores: the keys of each tile that the query sees among all that it sees.

    All weights are 1 and all sums are whole numbers below 2^24, exact in FP32, as are the parts' weights exp2(0); the
    quotient is rounded twice in FP32 (2^-23 in all) and once to BF16 (2^-8)."""
    n, heads, d = got.shape
    seen = first + 1 + torch.arange(n, device=got.device, dtype=torch.float64)
    tile = base + torch.arange(hk * d, device=got.device).view(hk, d).double()
    count = (seen[:, None, None] - tile * TILE).clamp(0, TILE)
    want = (count / seen[:, None, None]).repeat_interleave(heads // hk, 1)
    bad = (got.double() - want).abs() > want * (2.0 ** -8 + 2.0 ** -22)
    assert not bool(bad.any()), f"row, head, channel {bad.nonzero()[0].tolist()}: {got[bad][0].item()}, not {want[bad][0].item()}"


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("hq,hk,page,new,kv", [
    (8, 1, 16, [1], [60000]),                          # one token, many parts: a block a row
    (4, 2, 64, [5], [20001]),                          # some parts
    (32, 8, 16, [5] * 3, [4000, 129, 9001]),           # few parts an item: a warp a row
    (32, 8, 32, [1] * 40, [300 + 171 * i for i in range(40)]),
    (8, 2, 16, [40, 3], [30000, 7000]),                # more rows than blocks
    (8, 2, 16, [200, 1, 0, 300], [1500, 40000, 5, 9000]),  # full tiles of rows, cut
    (8, 2, 16, [300] * 9, [300 + 97 * i for i in range(9)]),  # whole and cut items
    (4, 2, 16, [700], [9000])])
def test_every_tile_counts_once(dev, d, hq, hk, page, new, kv):
    m = nd()
    _, kc, vc, table, lens, cu = paged_inputs(dev, d, new, kv, hq, hk, d, page)
    q = torch.zeros((sum(new), hq, d), dtype=BF16, device=dev)
    slots = [table[s].long()[torch.arange(n, device=dev) // page] * page + torch.arange(n, device=dev) % page
             for s, n in enumerate(kv)]
    flat, status = vc.view(-1, hk, d), ints(dev, [0])
    for base in range(0, -(-max(kv) // TILE), hk * d):
        for s, n in enumerate(kv):
            flat[slots[s]] = one_hot(n, base, hk, d, dev)
        out = m.paged_attention(q, kc, vc, table, lens, cu, dev_status=status)
        at = 0
        for n, keys in zip(new, kv):
            check_counts(out[at:at + n], keys - n, keys, base, hk)
            at += n
    assert status.item() == 0


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("hq,hk,lens", [(4, 2, [9000]), (8, 8, [3001, 17, 1500]), (7, 1, [1024, 1025, 1152, 0, 1]), (16, 2, [5, 6200, 40]),
                                        (8, 2, [400 + 90 * i for i in range(40)])])
def test_every_tile_of_a_prompt_counts_once(dev, d, hq, hk, lens):
    m, t = nd(), sum(lens)
    q, k = torch.zeros((t, hq, d), dtype=BF16, device=dev), randn(gen(dev, t), t, hk, d).to(BF16)
    for base in range(0, -(-max(lens) // TILE), hk * d):
        v = torch.cat([one_hot(n, base, hk, d, dev) for n in lens])
        out = m.prompt_attention(q, k, v, ints(dev, prefix(lens)))
        at = 0
        for n in lens:
            check_counts(out[at:at + n], 0, n, base, hk)
            at += n


@pytest.mark.parametrize("d,hq,hk,page,new,kv", [
    (64, 4, 1, 16, [1], [60000]), (128, 8, 1, 16, [1], [60000]), (256, 8, 1, 16, [3], [20001]), (64, 4, 1, 16, [2, 1], [30000, 5]),
    (128, 2, 1, 256, [2, 1], [260003, 7]), (256, 2, 1, 4096, [2], [260003]), (128, 32, 8, 16, [5] * 4, [9000, 800, 3000, 129]),
    (64, 4, 2, 16, [700], [9000]), (128, 4, 2, 16, [700], [9000]), (256, 4, 2, 16, [700], [9000])])
def test_errors_in_norm(dev, d, hq, hk, page, new, kv):
    """Flat scores over random values: a result is no larger than its parts' errors would be."""
    m, g = nd(), gen(dev, d + sum(kv))
    _, kc, vc, table, lens, cu = paged_inputs(dev, sum(kv), new, kv, hq, hk, d, page)
    q = (randn(g, sum(new), hq, d) * 0.5).to(BF16)
    out = m.paged_attention(q, kc, vc, table, lens, cu)
    at = 0
    for s, (n, keys) in enumerate(zip(new, kv)):
        want, most = ref.norm_bound(q[at:at + n], ref.gather(kc, table[s], keys), ref.gather(vc, table[s], keys), keys - n)
        assert (out[at:at + n].double() - want).norm().item() <= most
        at += n


# ------------------------------------------------- many sequences, uneven ones

@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("batch,most", [(33, 300), (70, 200), (1100, 80)])
def test_prompts_of_many_sequences_in_full_tiles(dev, d, batch, most):
    """More sequences than a warp has lanes (and than 32 lanes of 32), with more rows than a tile on average."""
    r = random.Random(batch)
    lens = [r.choice([0, 1, r.randint(1, most), most, most]) for _ in range(batch)]
    assert sum(lens) * 4 > 128 * batch
    check_prompt(dev, lens, 4, 1, d, tail=5)


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("batch", [40, 130])
def test_chunks_of_many_sequences(dev, d, batch):
    r = random.Random(batch + d)
    new = [r.choice([0, 1, 40, 64, 129]) for _ in range(batch)]
    assert sum(new) * 4 > 128 * batch
    check_paged(dev, new, [n + r.choice([0, r.randint(0, 300), r.randint(0, 1500)]) for n in new], 4, 1, d, 16)


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("chunk", [700, 1100])
def test_a_chunk_beside_decoding_sequences(dev, d, chunk):
    """One tile of rows an item (700 tokens among 31 sequences, group 4), and two: all sequences in the same form."""
    r = random.Random(chunk)
    new = [1] * 30
    kv = [r.randint(1, 3000) for _ in new]
    new.insert(17, chunk)
    kv.insert(17, chunk + 900)
    assert (sum(new) * 4 > 128 * len(new)) == (chunk == 1100)
    check_paged(dev, new, kv, 8, 2, d, 16)


@pytest.mark.parametrize("new", [1, 5, 150])
def test_a_sequence_at_any_place_of_the_batch(dev, new):
    """Shares' borders depend on the other sequences, so its bits may differ: its result is within the bound anywhere."""
    r = random.Random(new)
    kv = [new + r.randint(0, 4000) for _ in range(12)]
    for _ in range(3):
        r.shuffle(kv)
        check_paged(dev, [new] * len(kv), kv, 8, 2, 128, 16)


def test_same_bits_beside_other_work(dev):
    """Results do not depend on when the CTAs run: the same bits while another stream keeps the GPU busy."""
    m = nd()
    side, x = torch.cuda.Stream(), torch.randn((2048, 2048), device=dev)
    for new, kv in (([5] * 20, [2000 + 131 * i for i in range(20)]), ([1], [30000]), ([400, 30], [5000, 700])):
        args = paged_inputs(dev, 6, new, kv, 16, 2, 128, 16)
        want = m.paged_attention(*args)
        torch.cuda.synchronize()
        for _ in range(5):
            with torch.cuda.stream(side):
                for _ in range(4):
                    y = x @ x
            got = m.paged_attention(*args)
            torch.cuda.synchronize()
            assert torch.equal(got, want) and y.shape == x.shape
