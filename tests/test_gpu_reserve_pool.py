"""The free list of kv_reserve in calls at the edges: no request at all, pages that
cannot be given back."""

import random

import numpy as np
import pytest
import torch

import speculative_decoding_verification_13_gb300 as sv
from test_gpu_tables import reserve_case, run_reserve

pytestmark = pytest.mark.gpu
DEV = "cuda"


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


@pytest.mark.parametrize("n", [0, 2, 5])
@pytest.mark.parametrize("outs", ["list", "count", "both", "all"])
def test_no_request_copies_the_list_and_its_count(n, outs):
    none, table = i32([]), i32([]).view(0, 3)
    free, count = i32([4, 1, 9, -1, -1]), i32([n])
    kw = {}
    if outs in ("list", "both", "all"):
        kw["out_free"] = torch.full_like(free, 77)
    if outs in ("count", "both", "all"):
        kw["out_count"] = torch.full_like(count, 77)
    if outs == "all":
        kw.update(out_table=table.clone(), out_held=none.clone())
    got = sv.kv_reserve(table, none, none, free, count, 16, **kw)
    assert sv.kv_reserve_error() == (0, -1, -1)
    assert got.free_pages.tolist() == [4, 1, 9, -1, -1] and got.free_count.tolist() == [n]
    assert free.tolist() == [4, 1, 9, -1, -1] and count.tolist() == [n]


def test_no_request_in_place_by_another_name():
    free, count = i32([4, -1]), i32([-5])    # not looked at
    sv.kv_reserve(i32([]).view(0, 3), i32([]), i32([]), free, count, 16, out_free=free[:],
                  out_count=count[:])
    assert sv.kv_reserve_error() == (0, -1, -1) and free.tolist() == [4, -1]


@pytest.mark.parametrize("n", [-1, 6])
def test_no_request_and_a_count_that_is_none(n):
    none, table = i32([]), i32([]).view(0, 3)
    free, count = i32([4, 1, 9, -1, -1]), i32([n])
    got = sv.kv_reserve(table, none, none, free, count, 16, out_free=torch.full_like(free, 77),
                        out_count=torch.full_like(count, 77))
    assert sv.kv_reserve_error() == (30, -1, -1)
    assert got.free_pages.tolist() == [4, 1, 9, -1, -1] and got.free_count.tolist() == [n]


def test_a_large_list_without_requests():
    g = torch.Generator().manual_seed(1)
    free = torch.randperm(100003, generator=g).int().to(DEV)
    for at in (0, 1):   # whole vectors, and memory that is not aligned
        x = free[at:]
        got = sv.kv_reserve(i32([]).view(0, 3), i32([]), i32([]), x, i32([5000]), 16,
                            out_free=torch.full_like(x, 77))
        assert np.array_equal(got.free_pages.cpu().numpy(), x.cpu().numpy())
        assert got.free_count.tolist() == [5000]


# ------------------------------------------------- pages that cannot be given back
@pytest.mark.parametrize("apart", [False, True])
@pytest.mark.parametrize("holes", [1, 3, 40])
@pytest.mark.parametrize("B,cols,S,spare", [(1, 8, 16, 3), (3, 4, 16, 2), (30, 12, 16, 10),
                                            (300, 20, 16, 900), (257, 7, 1, 0), (700, 64, 4, 90)])
def test_missing_pages_are_not_given_back(B, cols, S, spare, holes, apart):
    for seed in range(3):
        case = reserve_case(seed * 100 + B, B, cols, S, spare)
        rng = random.Random(seed)
        for _ in range(holes):
            b = rng.randrange(B)
            if case[1][b]:
                case[0][b, rng.randrange(case[1][b])] = rng.choice([-1, -2 ** 31])
        run_reserve(case, S, apart)


@pytest.mark.parametrize("apart", [False, True])
def test_all_requests_but_one_keep_their_holes(apart):
    B = 600
    table = np.arange(B * 4, dtype=np.int32).reshape(B, 4)
    table[:, 2] = -1
    table[333, 2] = 5000
    lengths = [0] * B
    lengths[599] = 64
    free = np.full(B * 4, -1, np.int32)
    want = run_reserve((table, [4] * B, lengths, free, 0), 16, apart)
    assert want[3] == 4 and want[2][:4].tolist() == [333 * 4, 333 * 4 + 1, 5000, 333 * 4 + 3]
    assert (want[4] != 0).sum() == B - 2


def test_pages_come_from_behind_a_hole():
    # the pages handed out are released in the same call by requests around one that fails
    table = np.full((5, 6), -1, np.int32)
    table[0, :3], table[1, :3], table[2, :3] = [1, 2, 3], [4, -1, 6], [7, 8, 9]
    case = (table, [3, 3, 3, 0, 0], [16, 16, 0, 64, 16], np.full(20, -1, np.int32), 0)
    want = run_reserve(case, 16, False)
    assert want[0].tolist()[3] == [9, 8, 7, 3, -1, -1] and want[0].tolist()[4][0] == 2
    assert want[0].tolist()[1] == [4, -1, 6, -1, -1, -1] and want[1].tolist() == [1, 3, 0, 4, 1]
