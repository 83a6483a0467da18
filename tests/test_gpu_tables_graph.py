"""Block tables and slots captured once and replayed for steps that differ: every step
fits the captured list, and comes more than once."""

import numpy as np
import pytest
import torch

import speculative_decoding_verification_13_gb300 as sv
from oracle import tables as ot
from test_gpu_tables import i32, reserve_case

pytestmark = pytest.mark.gpu
DEV = "cuda"
B, COLS, S, SPARE, CAPACITY, ROWS = 30, 12, 16, 200, 800, 6000


def expected(case):
    got = ot.reserve(*case, S)
    return got, ot.slots(got[0], [0] * B, case[2], ROWS, S)


def error_of(want):
    status, all_ = want
    if all_:
        return all_, -1, -1
    return (int(status[status != 0][0]), int(np.flatnonzero(status)[0]), -1) if status.any() else \
        (0, -1, -1)


@pytest.mark.parametrize("apart", [True, False])
def test_every_replay_is_its_own_step(apart):
    cases = [reserve_case(seed, B, COLS, S, SPARE if seed != 5 else 3, CAPACITY)
             for seed in (1, 2, 3, 4, 5)]
    assert all(sum(c[1]) + c[4] <= CAPACITY for c in cases)
    cases[3][0][4, :] = -1   # a request of the fourth has nothing to give back
    want = [expected(c) for c in cases]
    assert len({tuple(w[0][0].reshape(-1)) for w in want}) == 5
    assert want[4][0][4].any()   # one of them runs out of pages

    def tensors(c):
        return [torch.as_tensor(c[0]).to(DEV), i32(c[1]), i32(c[2]), torch.as_tensor(c[3]).to(DEV),
                i32([c[4]])]

    a = tensors(cases[0])
    kw = {}
    if apart:
        kw = dict(out_table=torch.empty_like(a[0]), out_held=torch.empty_like(a[1]),
                  out_free=torch.empty_like(a[3]), out_count=torch.empty_like(a[4]))
    zero = i32([0] * B)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = sv.kv_reserve(*a, S, **kw)
        slots = sv.kv_slots(got.block_table, zero, a[2], ROWS, S)
    replays = 0
    for i in (0, 1, 2, 3, 4, 0, 4, 3, 1, 1):
        for x, y in zip(a, tensors(cases[i])):
            x.copy_(y)
        graph.replay()
        # the stream's own workspaces in between
        sv.kv_slots(a[0], zero, a[2], 100, S)
        table, where = want[i]
        for x, y in zip(got, table):
            assert np.array_equal(x.cpu().numpy(), np.atleast_1d(y)), i
        for x, y in zip(slots, where):
            assert np.array_equal(x.cpu().numpy(), y), i
        assert sv.kv_reserve_error() == error_of(table[4:])
        replays += 1
    assert replays == 10
