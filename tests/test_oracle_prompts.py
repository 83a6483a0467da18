"""Pins of the oracles of prompts, trees and tables: hand-worked examples and
properties computed another way, and planted mistakes that a comparison catches."""

import math

import numpy as np
import pytest
import torch

from oracle import attention as oa
from oracle import prompt as op
from oracle import tables as ot
from oracle import tree as otr


@pytest.mark.parametrize("window", [0, 1, 3])
def test_prompt_attention_equals_dense_softmax(window):
    rng = np.random.default_rng(1)
    at, D, Hk, G = [0, 5, 5, 12], 6, 2, 3
    q, k, v = (rng.normal(size=(12, h, D)) for h in (Hk * G, Hk, Hk))
    out, lse = op.prompt_attention(q, k, v, at, window=window)
    seq = torch.tensor([0] * 5 + [2] * 7)
    i = torch.arange(12)
    see = (seq[:, None] == seq) & (i[None] <= i[:, None])
    if window:
        see &= i[None] > i[:, None] - window
    kk, vv = (torch.as_tensor(x).repeat_interleave(G, 1) for x in (k, v))
    s = torch.einsum("ihd,jhd->hij", torch.as_tensor(q), kk) / math.sqrt(D)
    s = s.masked_fill(~see, -math.inf)
    assert np.allclose(lse, torch.logsumexp(s, -1).T, atol=1e-12)
    assert np.allclose(out, torch.einsum("hij,jhd->ihd", torch.softmax(s, -1), vv), atol=1e-12)


def test_prompt_attention_by_hand():
    # equal scores: the mean of the values so far; rows of no sequence are none
    v = np.array([9., 1, 3, 5, 9])[:, None, None]
    out, lse = op.prompt_attention(np.ones((5, 1, 1)), np.zeros((5, 1, 1)), v, [1, 4])
    assert out[1:4, 0, 0].tolist() == [1, 2, 3]
    assert np.allclose(lse[1:4, 0], np.log([1, 2, 3]))
    assert np.isnan(out[[0, 4]]).all() and np.isnan(lse[[0, 4]]).all()


def tree(seed, n=7, k=6, S=4, D=4, Hk=2, G=2):
    rng = np.random.default_rng(seed)
    pages = -(-n // S) + 1
    cache = rng.normal(size=(pages, 1, 2, S, Hk * D))
    spec = rng.normal(size=(1, k + 1, 1, 2, Hk * D))
    return rng.normal(size=(k + 1, Hk * G, D)), cache, [n], rng.permutation(pages)[None], [k], spec


@pytest.mark.parametrize("window", [0, 2, 5])
def test_a_node_sees_what_a_chain_of_its_ancestors_sees(window):
    q, cache, n, table, k, spec = tree(3)
    parent = [-1, 0, 0, 1, 3, 2, 3]
    out, lse = otr.attention(q, cache, 0, n, table, k, parent, spec, window=window)
    for j in range(7):
        way = otr.way(parent, j)
        assert way[0] == 0 and way[-1] == j
        o, l = oa.attention(q[way], cache, 0, n, table, [len(way) - 1], spec[:, way],
                            window=window)
        assert np.allclose(out[j], o[-1]) and np.allclose(lse[j], l[-1])
    # seeing a sibling instead is another result
    wrong, _ = otr.attention(q, cache, 0, n, table, k, [-1, 0, 1, 1, 3, 2, 3], spec, window=window)
    assert not np.allclose(out[2], wrong[2])


def test_tree_verification_by_hand():
    # 0 -> 1, 2; 2 -> 3, 4; the target wants 8, then 5, then 1
    parent, drafts = [-1, 0, 0, 2, 2], [7, 8, 5, 5]
    accept, tokens, path = otr.verify_greedy([8, 0, 5, 1, 2], drafts, parent, [4])
    assert accept.tolist() == [2]
    assert tokens.tolist() == [8, 5, 1, -1, -1] and path.tolist() == [0, 2, 3, -1, -1]
    accept, tokens, path = otr.verify_greedy([9, 0, 5, 1, 2], drafts, parent, [4])
    assert accept.tolist() == [0] and tokens.tolist() == [9] + [-1] * 4
    assert path.tolist() == [0] + [-1] * 4


def test_a_chain_accepts_the_longest_prefix():
    rng = np.random.default_rng(5)
    k = rng.integers(0, 6, 40)
    argmax, drafts = rng.integers(0, 3, k.sum() + 40), rng.integers(0, 3, k.sum())
    parent = np.concatenate([np.arange(-1, x) for x in k])
    accept, tokens, _ = otr.verify_greedy(argmax, drafts, parent, k)
    t = d = 0
    for b, x in enumerate(k):
        same = np.concatenate([argmax[t:t + x] == drafts[d:d + x], [False]])
        assert accept[b] == np.argmin(same)
        assert (tokens[t:t + accept[b] + 1] == argmax[t:t + accept[b] + 1]).all()
        t, d = t + x + 1, d + x


def test_reserve_by_hand_and_no_page_is_lost():
    table = np.array([[5, 6, -1], [7, -1, -1], [-1, -1, -1]])
    got = ot.reserve(table, [2, 1, 0], [3, 9, 1], [1, 2, -1, -1, -1], 2, 4)
    assert got[0].tolist() == [[5, -1, -1], [7, 6, 2], [1, -1, -1]]
    assert got[1].tolist() == [1, 3, 1] and got[2].tolist() == [-1, -1, -1, -1, -1] and got[3] == 0
    assert not got[4].any() and got[5] == 0
    rng = np.random.default_rng(0)
    table, held = np.full((9, 6), -1), np.zeros(9, int)
    free, n = rng.permutation(30), 30
    for _ in range(20):
        table, held, free, n, _, bad = ot.reserve(table, held, rng.integers(0, 49, 9), free, n, 8)
        own = [p for b in range(9) for p in table[b, :held[b]]]
        assert bad == 0 and sorted(own + list(free[:n])) == list(range(30))
        assert all((table[b, held[b]:] == -1).all() for b in range(9)) and (free[n:] == -1).all()


def test_slots_by_hand_and_write():
    table = np.array([[3, 1], [0, -1], [2, -1]])
    out, req, pos, at, st, _ = ot.slots(table, [3, 0, 4], [2, 0, 1], 5, 4)
    assert out.tolist() == [15, 4, -1, -1, -1]               # the last request has no such page
    assert req.tolist() == [0, 0, 2, -1, -1] and pos.tolist() == [3, 4, 4, -1, -1]
    assert at.tolist() == [0, 2, 2, 3] and st.tolist() == [0, 0, 27]
    cache = np.zeros((4, 1, 2, 4, 2))
    k = np.arange(6.).reshape(3, 1, 2) + 1
    assert ot.write(cache, 0, k, -k, out[:3]) == -1
    assert cache[3, 0, 0, 3].tolist() == [1, 2] and cache[1, 0, 1, 0].tolist() == [-3, -4]
    assert np.count_nonzero(cache) == 8 and ot.write(cache, 0, k, k, [-1, 16, -2]) == 1
