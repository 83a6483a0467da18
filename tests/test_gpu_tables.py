"""Block tables, slot maps and writes to the slots on the GPU against the oracles
(oracle/tables.py), bit for bit."""

import random

import numpy as np
import pytest
import torch

import speculative_decoding_verification_13_gb300 as sv
from oracle import tables as ot

pytestmark = pytest.mark.gpu
DEV = "cuda"


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def reserve_case(seed, B, cols, S, spare, capacity=None):
    rng = random.Random(seed)
    held = [rng.choice([0, rng.randint(0, cols), rng.randint(0, min(cols, 3))]) for _ in range(B)]
    lengths = [rng.choice([0, h * S, min(cols * S, h * S + rng.randint(0, 3 * S)),
                           rng.randint(0, cols * S)]) for h in held]
    pages = sum(held) + spare
    order = list(range(pages))
    rng.shuffle(order)
    table = np.full((B, cols), -1, np.int32)
    for b, h in enumerate(held):
        for c in range(h):
            table[b, c] = order.pop()
    free = np.full(capacity or pages, -1, np.int32)
    free[:spare] = order
    free[spare:] = rng.randint(-1, 5)
    return table, held, lengths, free, spare


def run_reserve(case, S, apart):
    table, held, lengths, free, n = case
    a = [torch.as_tensor(table).to(DEV), i32(held), i32(lengths), torch.as_tensor(free).to(DEV),
         i32([n])]
    before = [x.clone() for x in a]
    kw = {}
    if apart:
        kw = dict(out_table=torch.full_like(a[0], 77), out_held=torch.full_like(a[1], 77),
                  out_free=torch.full_like(a[3], 77), out_count=torch.full_like(a[4], 77))
    got = sv.kv_reserve(*a, S, **kw)
    error = sv.kv_reserve_error()
    want = ot.reserve(table, held, lengths, free, n, S)
    for x, y in zip(got, want):
        assert np.array_equal(x.cpu().numpy(), np.atleast_1d(y))
    for x, y in zip(a, before):
        if apart:
            assert torch.equal(x, y)
    status, all_ = want[4], want[5]
    if all_:
        assert error == (all_, -1, -1)
    elif status.any():
        b = int(np.flatnonzero(status)[0])
        assert error == (int(status[b]), b, -1)
    else:
        assert error == (0, -1, -1)
    return want


@pytest.mark.parametrize("apart", [False, True])
@pytest.mark.parametrize("B,cols,S,spare", [(1, 1, 16, 0), (1, 40, 1, 100), (8, 128, 16, 64),
                                            (33, 7, 7, 30), (300, 20, 16, 9000), (257, 64, 64, 90),
                                            (700, 12, 32, 0), (5000, 4, 16, 20000)])
def test_reserve_matches_oracle(B, cols, S, spare, apart):
    for seed in range(3):
        run_reserve(reserve_case(seed * 100 + B, B, cols, S, spare), S, apart)


@pytest.mark.parametrize("apart", [False, True])
def test_reserve_takes_what_is_there(apart):
    # the stack's end first; a request that cannot be served stops those behind it
    table = np.full((5, 4), -1, np.int32)
    table[0, :3] = [10, 11, 12]
    case = (table, [3, 0, 0, 0, 0], [16, 20, 60, 16, 0], np.array([1, 2, 3, -1, -1, -1], np.int32), 3)
    want = run_reserve(case, 16, apart)
    assert want[0].tolist() == [[10, -1, -1, -1], [12, 11, -1, -1], [-1] * 4, [-1] * 4, [-1] * 4]
    assert want[2].tolist() == [1, 2, 3, -1, -1, -1] and want[3] == 3
    assert want[4].tolist() == [0, 0, 30, 30, 0]


@pytest.mark.parametrize("apart", [False, True])
def test_reserve_errors(apart):
    table = np.arange(12, dtype=np.int32).reshape(3, 4)
    free = np.array([20, 21, 22, -1], np.int32)
    for held, lengths in (([4, 5, 2], [64, 16, 1]), ([4, -1, 2], [64, 16, 40]),
                          ([4, 1, 2], [65, 20, 1]), ([4, 1, 2], [64, -1, 0]),
                          ([4, 1, 2], [64, 2 ** 31 - 1, 33])):
        run_reserve((table, held, lengths, free, 3), 16, apart)
    for n in (-1, 5, 4):   # 4: full, and a page comes back
        run_reserve((table, [4, 1, 2], [64, 0, 20], free, n), 16, apart)


def test_reserve_beside_memory_that_is_not_aligned():
    case = reserve_case(4, 20, 8, 16, 40)
    want = ot.reserve(case[0], case[1], case[2], case[3], case[4], 16)
    flat = torch.zeros(20 * 8 + 1, dtype=torch.int32, device=DEV)
    flat[1:] = torch.as_tensor(case[0]).to(DEV).reshape(-1)
    got = sv.kv_reserve(flat[1:].view(20, 8), i32(case[1]), i32(case[2]),
                        torch.as_tensor(case[3]).to(DEV), i32([case[4]]), 16,
                        out_table=torch.empty(20, 8, dtype=torch.int32, device=DEV))
    for x, y in zip(got, want):
        assert np.array_equal(x.cpu().numpy(), np.atleast_1d(y))


def test_no_request():
    none = i32([])
    free, n = i32([1, 2]), i32([2])
    sv.kv_reserve(i32([]).view(0, 3), none, none, free, n, 16)
    assert free.tolist() == [1, 2] and sv.kv_reserve_error() == (0, -1, -1)
    s = sv.kv_slots(i32([]).view(0, 3), none, none, 5, 16)
    assert s.offsets.tolist() == [0] and (s.slots == -1).all()


def run_slots(table, start, count, rows, S):
    got = sv.kv_slots(torch.as_tensor(table).to(DEV), i32(start), i32(count), rows, S)
    error = sv.kv_slots_error()
    want = ot.slots(table, start, count, rows, S)
    for x, y in zip(got, want):
        assert np.array_equal(x.cpu().numpy(), y)
    status, all_ = want[4], want[5]
    if all_:
        assert error == (all_, -1, -1)
    elif status.any():
        b = int(np.flatnonzero(status)[0])
        assert error == (int(status[b]), b, -1)
    else:
        assert error == (0, -1, -1)


@pytest.mark.parametrize("B,most,S,more", [(1, 1, 16, 0), (1, 3000, 16, 0), (8, 16, 16, 5),
                                           (70, 500, 7, 0), (300, 4, 1, 2000), (3000, 3, 64, 1)])
def test_slots_match_oracle(B, most, S, more):
    rng = random.Random(B)
    start = [rng.randint(0, 300) for _ in range(B)]
    count = [rng.choice([0, 1, rng.randint(0, most)]) for _ in range(B)]
    count[-1] = most
    cols = (300 + most) // S + 1
    table = np.random.default_rng(B).integers(0, 2 ** 31 - 1, (B, cols), dtype=np.int64)
    run_slots(table.astype(np.int32), start, count, sum(count) + more, S)


def test_slots_errors():
    table = np.arange(20, dtype=np.int32).reshape(4, 5)
    table[2, 1] = -1
    ok = ([0, 3, 10, 60], [5, 0, 20, 3])
    run_slots(table, *ok, 28, 16)                            # a page is missing in the middle
    table[2, 1] = 11
    run_slots(table, *ok, 28, 16)
    run_slots(table, *ok, 27, 16)                            # one row too few
    run_slots(table, [0, -3, 10, 60], ok[1], 30, 16)
    run_slots(table, [0, -3, 10, 60], [5, 4, 20, 3], 40, 16)
    run_slots(table, ok[0], [5, -1, 20, 3], 30, 16)
    run_slots(table, ok[0], [5, 0, 20, 21], 60, 16)          # past the table
    run_slots(table, [0, 2 ** 31 - 1, 10, 60], [5, 4, 20, 3], 40, 16)


@pytest.mark.parametrize("rows,Hk,D,S,dtype,layers", [
    (1, 1, 128, 16, torch.bfloat16, 1), (201, 8, 128, 16, torch.bfloat16, 4),
    (70, 2, 80, 7, torch.float16, 2), (33, 3, 5, 1, torch.bfloat16, 2),
    (64, 2, 64, 64, torch.float32, 2), (40, 1, 7, 16, torch.float32, 1),
    (5000, 4, 256, 16, torch.bfloat16, 1)])
@pytest.mark.parametrize("how", ["slices", "apart", "unaligned"])
def test_write_matches_oracle(rows, Hk, D, S, dtype, layers, how):
    g = torch.Generator().manual_seed(rows)
    pool = -(-rows // S) + 2
    slots = torch.randperm(pool * S, generator=g)[:rows]
    slots[torch.rand(rows, generator=g) < 0.1] = -1
    ref = torch.randn(pool, layers, 2, S, Hk * D, generator=g).to(dtype)
    k, v = (torch.randn(rows, Hk, D, generator=g).to(dtype) for _ in range(2))
    cache = ref.to(DEV)
    assert ot.write(ref, layers - 1, k, v, slots) == -1
    if how == "slices":
        kd, vd = torch.cat([k, v, k], 1).to(DEV).split([Hk, Hk, Hk], 1)[:2]
    elif how == "apart":
        kd = k.to(DEV).transpose(0, 1).contiguous().transpose(0, 1)
        vd = torch.cat([v, v], 2).to(DEV)[:, :, :D]
    else:
        kd, vd = (torch.cat([x.reshape(-1)[:1], x.reshape(-1)]).to(DEV)[1:].view(x.shape)
                  for x in (k, v))
    assert sv.kv_write(cache, layers - 1, kd, vd, slots.to(DEV)) is cache
    assert sv.kv_write_error() == (0, -1, -1)
    assert torch.equal(cache.cpu(), ref)


def test_write_leaves_out_slots_outside_the_pool():
    cache = torch.zeros(2, 1, 2, 4, 8, device=DEV)
    k = torch.ones(5, 1, 8, device=DEV)
    sv.kv_write(cache, 0, k, k, torch.tensor([-1, 3, 8, -2, 2 ** 40], device=DEV))
    assert sv.kv_write_error() == (27, -1, 2)
    assert float(cache.sum()) == 16 and float(cache[0, 0, :, 3].sum()) == 16
    sv.kv_write(cache, 0, k[:0], k[:0], torch.tensor([], dtype=torch.int64, device=DEV))
    assert sv.kv_write_error() == (0, -1, -1)


def test_a_step_of_tables_in_a_graph():
    table, held, lengths, free, n = reserve_case(1, 30, 12, 16, 200)
    a = [torch.as_tensor(table).to(DEV), i32(held), i32(lengths), torch.as_tensor(free).to(DEV),
         i32([n])]
    out = [torch.empty_like(a[0]), torch.empty_like(a[1]), torch.empty_like(a[3]),
           torch.empty_like(a[4])]
    zero = i32([0] * 30)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        sv.kv_reserve(*a, 16, out_table=out[0], out_held=out[1], out_free=out[2], out_count=out[3])
        s = sv.kv_slots(out[0], zero, a[2], 6000, 16)
    for seed in (2, 3):
        case = reserve_case(seed, 30, 12, 16, 200, len(free) + 2000)
        m = len(free)
        want = ot.reserve(case[0], case[1], case[2], case[3][:m], case[4], 16) \
            if sum(case[1]) + 200 <= m else None
        if want is None:
            continue
        a[0].copy_(torch.as_tensor(case[0]))
        a[1].copy_(i32(case[1]))
        a[2].copy_(i32(case[2]))
        a[3].copy_(torch.as_tensor(case[3][:m]))
        g.replay()
        for x, y in zip(out, want):
            assert np.array_equal(x.cpu().numpy(), np.atleast_1d(y))
        w = ot.slots(want[0], [0] * 30, case[2], 6000, 16)
        for x, y in zip(s, w):
            assert np.array_equal(x.cpu().numpy(), y)
