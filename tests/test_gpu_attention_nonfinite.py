"""Infinite keys and values in attention over the paged cache and in its
accumulated weights: what the formulas give in 64 bits, at every place of the
kernels' tiles.

Finite results keep the tolerances of test_gpu_attention.py; infinite ones and
NaN have to be the formula's."""

import math

import numpy as np
import pytest
import torch

import speculative_decoding_verification_13_gb300 as sv
from oracle import attention as oa
from test_gpu_attention import B16, DEV, F16, F32, Case, check, score_error

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [B16, F16, F32])
@pytest.mark.parametrize("k,G", [(0, 4), (16, 1), (15, 4)])
@pytest.mark.parametrize("sign", [1, -1])
def test_a_key_of_weight_zero_leaves_the_score(dtype, k, G, sign):
    # an infinite component whose products are -inf for every query of the head: the
    # position weighs nothing there, whatever the number of rows
    c = Case(21, [300], [k], 2, G, 64, 16, dtype)
    bad = (3, 70, 299)
    for p in bad:
        c.cache[c.table[0, p // 16], c.layer, 0, p % 16, 5] = sign * math.inf
    c.q[:, :G, 5] = -sign * (c.q[:, :G, 5].abs() + 1)
    with np.errstate(invalid="ignore"):
        out, lse = oa.attention(c.q, c.cache, c.layer, c.n, c.table, c.k, c.spec)
    assert np.isfinite(lse).all()
    truth = torch.as_tensor(lse, dtype=torch.float32)
    score = torch.rand(1, 340, generator=torch.Generator().manual_seed(2))
    ref = oa.weights(c.q, c.cache, c.layer, c.n, c.table, c.k, truth, score, c.spec)
    assert np.isfinite(ref).all()
    args, sp = c.gpu()
    got = sv.attention_weights(*args, truth.to(DEV), score.to(DEV), sp).double().cpu().numpy()
    assert sv.attention_weights_error()[0] == 0
    # sizes of the scores without the infinite component
    K = c.cache.clone()
    K[..., 5] = 0
    size = oa.attention(c.q, K, c.layer, c.n, c.table, c.k, c.spec, magnitude=True)[3]
    rel = 2 * score_error(c, float(size.max()) + 64) + 2.0 ** -22 * np.abs(lse).max()
    tol = (rel + ((k + 1) * 2 * G + 4) * 2.0 ** -24) * ref + 1e-30
    assert np.isfinite(got).all()
    assert (np.abs(got - ref) <= tol).all()


def expect(c, out, lse, window=0):
    """Checks against the oracle; what is not finite there has to be the same here."""
    with np.errstate(invalid="ignore"):
        o, l, mag, size = c.oracle(window=window)
    got = out.double().cpu().numpy()
    assert np.isfinite(l).all()
    fine = np.isfinite(o)
    assert not fine.all()
    assert np.array_equal(got[~fine], o[~fine], equal_nan=True)
    assert np.isfinite(got[fine]).all()
    clean = torch.where(torch.as_tensor(fine), out.cpu(), torch.zeros((), dtype=out.dtype))
    check(c, clean, lse, [np.where(fine, o, 0), l, np.where(fine, mag, 0), size])


def put(c, b, p, d, v):
    c.cache[c.table[b, p // c.cache.shape[3]], c.layer, 1, p % c.cache.shape[3], d] = v


# rows a head: 4 lie four times in the product, 52 twice, 128 and 132 once or in two tiles
@pytest.mark.parametrize("k,G", [(0, 4), (12, 4), (31, 4), (32, 4)])
@pytest.mark.parametrize("dtype,D,S", [(B16, 128, 16), (F16, 64, 5), (B16, 256, 64), (F16, 80, 16),
                                       (F32, 64, 16)])
def test_infinite_values_in_inner_tiles(dtype, D, S, k, G):
    c = Case(22, [700, 40], [k, 0], 2, G, D, S, dtype)
    put(c, 0, 130, 3, math.inf)
    put(c, 0, 200, 5, -math.inf)
    put(c, 0, 310, 7, math.nan)
    put(c, 0, 150, 9, math.inf)        # both signs, and one sign in several places
    put(c, 0, 420, 9, -math.inf)
    for p in (7, 260, 300, 500):
        put(c, 0, p, D - 1, -math.inf)
        put(c, 0, p, D + 4, math.inf)  # the other head
    args, sp = c.gpu()
    expect(c, *sv.attention(*args, sp))


@pytest.mark.parametrize("dtype,D", [(B16, 128), (F16, 64)])
@pytest.mark.parametrize("k", [0, 15])
def test_infinite_values_of_a_long_request(dtype, D, k):
    # the request lies in parts over many blocks
    c = Case(23, [9001], [k], 1, 2, D, 16, dtype, layers=1, junk=False)
    put(c, 0, 4000, 1, math.inf)
    put(c, 0, 8999, 2, -math.inf)
    put(c, 0, 77, 3, math.inf)
    put(c, 0, 6000, 3, math.inf)
    put(c, 0, 20, 4, math.nan)
    args, sp = c.gpu()
    expect(c, *sv.attention(*args, sp))


def test_an_infinite_value_of_little_weight_in_half_precision():
    # a weight of e^-25, below the smallest number of fp16
    c = Case(24, [600], [0], 1, 4, 64, 16, F16, layers=1)
    c.cache[..., 0, :, 0] = 0
    c.q[..., 0] = 8
    c.q[..., 1:] *= 0.1
    put(c, 0, 200, 6, math.inf)
    c.cache[c.table[0, 200 // 16], 0, 0, 200 % 16, 0] = -25
    args, sp = c.gpu()
    expect(c, *sv.attention(*args, sp))


@pytest.mark.parametrize("dtype,D", [(B16, 128), (F16, 64), (B16, 256), (F32, 64)])
@pytest.mark.parametrize("k,G", [(0, 4), (9, 4)])
def test_infinite_values_that_only_the_last_columns_of_a_tile_see(dtype, D, k, G):
    # a window that leaves the first columns of the only tile to nobody
    c = Case(25, [100, 127], [k, 0], 2, G, D, 16, dtype)
    put(c, 0, 97, 3, math.inf)
    put(c, 0, 96, 4, -math.inf)
    put(c, 1, 120, 5, math.nan)
    put(c, 1, 40, 6, math.inf)         # in front of the window: seen by none
    args, sp = c.gpu()
    expect(c, *sv.attention(*args, sp, window=15), window=15)


@pytest.mark.parametrize("dtype,D,G,k,window", [(B16, 256, 4, 32, 900), (B16, 128, 4, 0, 0),
                                                (F16, 64, 16, 32, 700)])
@pytest.mark.parametrize("value", [math.inf, -math.inf, math.nan])
def test_nothing_but_infinite_or_nan_values(dtype, D, G, k, window, value):
    # every row and column takes the second look, which has to end in a wait's time
    n, Hk, S = 40000, 2, 16
    g = torch.Generator(device=DEV).manual_seed(1)
    cache = torch.randn(n // S, 1, 2, S, Hk * D, device=DEV, generator=g).to(dtype)
    spec = torch.randn(1, k + 1, 1, 2, Hk * D, device=DEV, generator=g).to(dtype)
    cache[:, :, 1], spec[:, :, :, 1] = value, value
    q = torch.randn(k + 1, Hk * G, D, device=DEV, generator=g).to(dtype)
    i32 = dict(dtype=torch.int32, device=DEV)
    out, lse = sv.attention(q, cache, 0, torch.tensor([n], **i32),
                            torch.arange(n // S, **i32)[None], torch.tensor([k], **i32), spec,
                            window=window)
    assert sv.attention_error()[0] == 0
    assert torch.isfinite(lse).all()
    assert (torch.isnan(out) if math.isnan(value) else out == value).all()
