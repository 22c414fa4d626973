"""The attention step's contracts that its other tests leave open: calls in place one right behind the other,
outputs given in part, counts past a table's row, host queries that every batch size would repeat."""
import ctypes
import os
import random

import pytest
import torch

import attention_step_ref as ref
from test_gpu_attention_step import ints, nd

pytestmark = pytest.mark.gpu


def test_plan_outputs_given_in_part(dev):
    """A plan whose `out` holds only the state that is updated in place: the others are made and come with it."""
    m = nd()
    lens, new, held, table = [3, 16, 5], [2, 1, 0], [1, 1, 1], [[7, 0], [4, 0], [9, 0]]
    tl, th, tc, t = ints(dev, lens), ints(dev, held), ints(dev, [3]), ints(dev, table)
    out = m.KvPlan(None, tl, None, None, th, tc)
    p = m.kv_plan(tl, ints(dev, new), t, ints(dev, [1, 2, 8]), tc, 16, 4, held=th, out=out)
    want = ref.plan(lens, new, held, table, [1, 2, 8], 3, 16, 4)
    assert p is out and p.kv_lens is tl and p.held is th and p.free_count is tc
    assert (t.tolist(), p.cu_new.tolist(), tl.tolist(), p.positions.tolist(), p.slots.tolist(), th.tolist(), tc.item()) == tuple(want)


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


def test_batch_sizes_of_the_plan_do_not_fill_the_table_of_queries(dev):
    """Several hundred batch sizes: the runtime is asked about kv_plan's kernel once, and a kernel that is first
    used behind them once too.  (The test build counts its queries; none of these calls withholds anything.)"""
    from nvfp4_speculative_draft_gb300 import build
    m = nd()
    if not os.path.exists(build.WITHHOLD_LIB):
        build.build(withhold=True)
    L = ctypes.CDLL(build.WITHHOLD_LIB)
    L.nvfp4_test_occupancy_asked.restype = ctypes.c_long
    L.fp8w_quantize.argtypes = [ctypes.c_void_p, ctypes.c_int64, ctypes.c_int64, ctypes.c_void_p, ctypes.c_void_p,
                                ctypes.POINTER(m._Exec)]
    most = 700
    zeros = lambda n: ints(dev, [0] * n)  # noqa: E731
    lens, new, table, free, count = zeros(most), ints(dev, [1] * most), zeros(most * 2), ints(dev, list(range(most))), ints(dev, [most])
    cu, kv, positions, slots = zeros(most + 1), zeros(most), zeros(most), zeros(most)
    ex = m._Exec(torch.cuda.current_stream().cuda_stream, None, 0, None)

    def plan(batch):
        i = m._PlanInput(lens.data_ptr(), new.data_ptr(), None, table.data_ptr(), 2, 2, free.data_ptr(), most, count.data_ptr(),
                         batch, 16, most)
        o = m._PlanOutput(cu.data_ptr(), kv.data_ptr(), positions.data_ptr(), slots.data_ptr(), None, None)
        assert L.kv_plan(ctypes.byref(i), ctypes.byref(o), ctypes.byref(ex)) == 0

    w = torch.ones((64, 64), dtype=torch.bfloat16, device=dev)
    codes, scale = torch.zeros((64, 64), dtype=torch.uint8, device=dev), torch.zeros(64, device=dev)

    def other():
        assert L.fp8w_quantize(w.data_ptr(), 64, 64, codes.data_ptr(), scale.data_ptr(), ctypes.byref(ex)) == 0

    plan(1)
    asked = L.nvfp4_test_occupancy_asked()
    for batch in range(1, most + 1):
        plan(batch)
    assert L.nvfp4_test_occupancy_asked() == asked
    other()
    asked = L.nvfp4_test_occupancy_asked()
    for _ in range(5):
        other()
        plan(most)
    assert L.nvfp4_test_occupancy_asked() == asked
    torch.cuda.synchronize()
    assert cu.tolist() == list(range(most + 1)) and slots.tolist() == [16 * (most - 1 - s) for s in range(most)]
