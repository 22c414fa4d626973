"""The attention step's contracts that its other tests leave open: calls in place one right behind the other,
counts past a table's row."""
import random

import pytest
import torch

import attention_step_ref as ref
from test_gpu_attention_step import ints, nd

pytestmark = pytest.mark.gpu


# (one CTA; a cluster; a cluster whose threads have several sequences each)
@pytest.mark.parametrize("captured", [False, True])
@pytest.mark.parametrize("batch,most", [(24, 5), (700, 20), (3000, 4)])
def test_plan_in_place_back_to_back(dev, batch, most, captured):
    """Calls that update lens, held and the free count in place, with nothing between them: each sees
    what the one before it wrote."""
    m, r, page, width, calls = nd(), random.Random(batch + most), 8, 40, 8
    new = [[r.choice([-1, 0, 1, most]) for _ in range(batch)] for _ in range(calls)]
    tokens = max(sum(max(n, 0) for n in x) for x in new)
    ids = list(range(batch * 25))
    r.shuffle(ids)
    lens, held, count, free = ints(dev, [0] * batch), ints(dev, [0] * batch), ints(dev, [len(ids)]), ints(dev, ids)
    table = torch.full((batch, width), -1, dtype=torch.int32, device=dev)
    news = [ints(dev, x) for x in new]
    outs = [m.KvPlan(ints(dev, [0] * (batch + 1)), lens, ints(dev, [0] * tokens), ints(dev, [0] * tokens), held, count)
            for _ in new]

    def steps():
        for n, out in zip(news, outs):
            m.kv_plan(lens, n, table, free, count, page, tokens, held=held, out=out)

    torch.cuda.synchronize()
    if captured:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            steps()
        graph.replay()
    else:
        steps()
    torch.cuda.synchronize()
    state = [[-1] * width for _ in range(batch)], [0] * batch, [0] * batch, len(ids)
    for n, out in zip(new, outs):
        t, cu, kv, positions, slots, h, left = ref.plan(state[1], n, state[2], state[0], ids, state[3], page, tokens)
        state = t, kv, h, left
        assert out.cu_new.tolist() == cu and out.positions.tolist() == positions and out.slots.tolist() == slots
    assert table.tolist() == state[0] and lens.tolist() == state[1] and held.tolist() == state[2]
    assert count.item() == state[3]


def test_plan_keeps_counts_past_the_row(dev):
    """held comes back as max(held, need), also where it is more than a table's row has; such a sequence takes
    no page, and one whose tokens do not fit its row is refused with its count unchanged."""
    m, page, width = nd(), 16, 2
    lens, new, held = [20, 0, 40, 3, 31], [1, 0, 8, 20, 2], [5, 3, 9, 2 ** 31 - 1, 2]
    table = ints(dev, [[7, 4], [1, 2], [3, 5], [6, 8], [9, 10]])
    before, status = table.clone(), ints(dev, [0])
    p = m.kv_plan(ints(dev, lens), ints(dev, new), table, ints(dev, [11, 12, 13]), ints(dev, [3]), page, 31,
                  held=ints(dev, held), dev_status=status)
    assert p.held.tolist() == held and p.free_count.item() == 3 and torch.equal(table, before)
    # 40 + 8 tokens are three pages of two, 31 + 2 as well
    assert p.kv_lens.tolist() == [21, 0, 40, 23, 31] and status.item() == 10
    slots = [4 * 16 + 4] + [-1] * 8 + [6 * 16 + i for i in range(3, 16)] + [8 * 16 + i for i in range(7)] + [-1] * 2
    assert p.slots.tolist() == slots
