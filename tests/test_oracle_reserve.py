"""The oracle of the block tables where a request would give back pages it does not
have, worked by hand."""

import numpy as np

from oracle import tables as ot


def test_a_request_with_a_hole_keeps_its_row():
    table = np.array([[5, -1, 6, -1], [7, 8, 9, -1], [-1, -1, -1, -1]], np.int32)
    free = np.array([1, 2, -1, -1, -1, -1, -1], np.int32)
    got = ot.reserve(table, [3, 3, 0], [16, 10, 60], free, 2, 16)
    # request 0 would give back -1 and 6; 1 gives back 8 and 9; 2 wants four and gets them
    assert got[0].tolist() == [[5, -1, 6, -1], [7, -1, -1, -1], [9, 8, 2, 1]]
    assert got[1].tolist() == [3, 1, 4] and got[3] == 0
    assert got[2].tolist() == [-1] * 7
    assert got[4].tolist() == [27, 0, 0] and got[5] == 0


def test_a_hole_among_the_pages_that_stay_is_nothing_to_the_list():
    table = np.array([[-1, 3, 4]], np.int32)
    got = ot.reserve(table, [3], [32], np.array([1, -1, -1], np.int32), 1, 16)
    assert got[0].tolist() == [[-1, 3, -1]] and got[2].tolist() == [1, 4, -1]
    assert got[4].tolist() == [0] and got[3] == 2


def test_the_capacity_is_asked_for_all_that_would_come_back():
    table = np.array([[3, -1], [4, 5]], np.int32)
    got = ot.reserve(table, [2, 2], [0, 0], np.array([1, 2, -1], np.int32), 2, 16)
    assert got[5] == 30 and got[0].tolist() == table.tolist() and got[3] == 2
