"""The free list of kv_reserve in calls at the edges: no request at all, pages that
cannot be given back."""

import numpy as np
import pytest
import torch

import speculative_decoding_verification_13_gb300 as sv

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
