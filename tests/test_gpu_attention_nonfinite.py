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
