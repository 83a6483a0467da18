"""Pins of the oracles of attention, accumulated weights, eviction and log
probabilities: hand-worked examples and properties computed another way."""

import math

import numpy as np
import pytest
import torch

from oracle import attention as oa
from oracle import evict as oe
from oracle import logprobs as ol


def paged(n, S, layers, E, seed):
    rng = np.random.default_rng(seed)
    pages = -(-max(n, 1) // S) + 2
    cache = rng.normal(size=(pages, layers, 2, S, E))
    table = rng.permutation(pages)[None].astype(np.int32)
    return cache, table


@pytest.mark.parametrize("window,with_spec", [(0, True), (0, False), (3, True), (5, False)])
def test_attention_equals_dense_softmax(window, with_spec):
    n, k, S, D, Hk, G = 11, 3, 4, 6, 2, 3
    cache, table = paged(n, S, 2, Hk * D, 1)
    rng = np.random.default_rng(2)
    spec = rng.normal(size=(1, k + 1, 2, 2, Hk * D)) if with_spec else None
    q = rng.normal(size=(k + 1, Hk * G, D))
    out, lse = oa.attention(q, cache, 1, [n], table, [k], spec, window=window)
    # the dense sequence, and a full score matrix with a mask, by torch
    seq = torch.as_tensor(cache)[torch.as_tensor(table[0]).long(), 1].transpose(0, 1)
    seq = seq.reshape(2, -1, Hk * D)[:, :n]
    if with_spec:
        seq = torch.cat([seq, torch.as_tensor(spec[0, :, 1]).transpose(0, 1)], 1)
    total = seq.shape[1]
    kv = seq.reshape(2, total, Hk, D).repeat_interleave(G, 2)
    s = torch.einsum("jhd,nhd->hjn", torch.as_tensor(q), kv[0]) / math.sqrt(D)
    at = torch.arange(total - k - 1, total)[:, None]
    p = torch.arange(total)[None]
    see = (p <= at) & ((p > at - window) if window else True)
    s = s.masked_fill(~see, -math.inf)
    assert np.allclose(lse, torch.logsumexp(s, -1).T, atol=1e-12)
    assert np.allclose(out, torch.einsum("hjn,nhd->jhd", torch.softmax(s, -1), kv[1]), atol=1e-12)


def test_attention_hand_example_and_empty_row():
    # one head of size 1: equal scores average the values; no key gives 0 and -inf
    cache = np.zeros((2, 1, 2, 2, 1))
    cache[1, 0, 1, 0, 0], cache[1, 0, 1, 1, 0], cache[0, 0, 1, 0, 0] = 3.0, 6.0, 9.0
    out, lse = oa.attention(np.ones((1, 1, 1)), cache, 0, [3], np.array([[1, 0]]), [0])
    assert out[0, 0, 0] == pytest.approx(6.0) and lse[0, 0] == pytest.approx(math.log(3))
    out, lse = oa.attention(np.ones((1, 1, 1)), cache, 0, [0], np.array([[1, 0]]), [0])
    assert out[0, 0, 0] == 0 and lse[0, 0] == -math.inf


@pytest.mark.parametrize("accept", [None, 0, 2, -1])
def test_weights_of_a_token_sum_to_one_per_head(accept):
    n, k, S, D, Hk, G = 9, 2, 4, 4, 2, 2
    cache, table = paged(n, S, 1, Hk * D, 3)
    rng = np.random.default_rng(4)
    spec = rng.normal(size=(1, k + 1, 1, 2, Hk * D))
    q = rng.normal(size=(k + 1, Hk * G, D))
    _, lse = oa.attention(q, cache, 0, [n], table, [k], spec)
    acc = None if accept is None else [accept]
    score = oa.weights(q, cache, 0, [n], table, [k], lse, np.zeros((1, 20)), spec, acc)
    tokens = k + 1 if accept is None else accept + 1
    assert score.sum() == pytest.approx(tokens * Hk * G)
    assert (score[0, n + tokens:] == 0).all()


def test_evict_hand_example():
    score = np.array([[5., 1., 9., 9., 2., 9., 0., 3., np.nan, 7.]])
    assert oe.choose(score[0], 10, 5, 1, 2) == [0, 2, 3, 8, 9]     # ties: the lowest positions
    assert oe.choose(score[0], 10, 9, 0, 0) == [0, 1, 2, 3, 4, 5, 6, 7, 9]  # NaN goes first
    assert oe.choose(score[0], 4, 5, 1, 2) == [0, 1, 2, 3]
    S = 2
    cache = np.arange(6 * 1 * 2 * S * 1, dtype=np.float32).reshape(6, 1, 2, S, 1)
    table = np.array([[4, 0, 5, 1, 3]], np.int32)
    before = cache.copy()
    lengths, kept, st = oe.kv_evict(cache, score, [10], table, 5, 1, 2)
    assert st[0] == 0 and lengths[0] == 5 and kept[0].tolist() == [0, 2, 3, 8, 9]
    for i, p in enumerate([0, 2, 3, 8, 9]):
        assert (cache[table[0, i // S], :, :, i % S] == before[table[0, p // S], :, :, p % S]).all()
    assert score[0, :5].tolist()[:4] == [5, 9, 9, pytest.approx(np.nan, nan_ok=True)]
    assert (score[0, 5:] == 0).all()


def test_evict_errors_touch_nothing():
    cache = np.zeros((2, 1, 2, 2, 1), np.float32)
    score = np.ones((3, 8))
    table = np.array([[0, -1], [0, 1], [5, 1]], np.int32)
    lengths, kept, st = oe.kv_evict(cache, score, [3, 5, 2], table, 2, 0, 0)
    assert st.tolist() == [27, 28, 27] and lengths.tolist() == [3, 5, 2]
    assert (kept == -1).all() and (score == 1).all()


def test_logprobs_equal_log_softmax_and_hand_entropy():
    rng = np.random.default_rng(0)
    x = rng.normal(size=50) * 3
    lp, H, m, ls, tok, top, _, _ = ol.row(x, 7, 0.7, 4)
    want = torch.log_softmax(torch.as_tensor(x) / 0.7, 0)
    assert lp == pytest.approx(float(want[7]), abs=1e-12)
    assert ls + m / 0.7 == pytest.approx(float(torch.logsumexp(torch.as_tensor(x) / 0.7, 0)))
    v, i = torch.topk(want, 4)
    assert tok.tolist() == i.tolist() and np.allclose(top, v)
    # a uniform row of 8, one of them masked: entropy ln 7; ties in index order
    x = np.zeros(8)
    x[2] = -np.inf
    lp, H, _, _, tok, top, _, _ = ol.row(x, 2, 0, 8)
    assert lp == -np.inf and H == pytest.approx(math.log(7))
    assert tok.tolist() == [0, 1, 3, 4, 5, 6, 7, -1] and top[7] == -np.inf


@pytest.mark.parametrize("T", [0, 0.6, 2.0])
def test_logprobs_gradient_equals_differences(T):
    rng = np.random.default_rng(1)
    x, g, h, t = rng.normal(size=9), 1.3, -0.7, 4

    def loss(x):
        lp, H = ol.row(x, t, T, 0)[:2]
        return g * lp + h * H

    d = ol.grad_row(x, t, T, g, h)
    for i in range(9):
        e = np.zeros(9)
        e[i] = 1e-6
        # central differences: an error of about 1e-12 (curvature) + 1e-10 (rounding)
        assert d[i] == pytest.approx((loss(x + e) - loss(x - e)) / 2e-6, abs=1e-8)
    assert d.sum() == pytest.approx(0, abs=1e-12)
