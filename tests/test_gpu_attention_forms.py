"""Attention and its weights with a caller's own scale, and the weights with a
window and an output of their own, against the oracle; tolerances as in
test_gpu_attention.py."""

import numpy as np
import pytest
import torch

import speculative_decoding_verification_13_gb300 as sv
from oracle import attention as oa
from test_gpu_attention import B16, DEV, F16, F32, Case, check, score_error

pytestmark = pytest.mark.gpu


def check_weights(c, got, ref, want, terms):
    rel = 2 * score_error(c, float(want[3].max())) + \
        2.0 ** -22 * np.abs(want[1][np.isfinite(want[1])]).max()
    tol = (rel + (terms + 4) * 2.0 ** -24) * np.abs(ref) + 1e-30
    assert (np.abs(got.double().cpu().numpy() - ref) <= tol).all()


@pytest.mark.parametrize("scale", [0.31, 1.0, 1e-3, 0.0, -0.2])
@pytest.mark.parametrize("dtype,D", [(B16, 128), (F16, 64), (B16, 80), (F32, 64)])
def test_a_caller_s_scale(dtype, D, scale):
    # one of 0 or below takes attention to the ordinary cores
    n, k, Hk, G = [300, 64, 0, 700], [5, 0, 15, 1], 2, 3
    c = Case(31, n, k, Hk, G, D, 16, dtype)
    args, sp = c.gpu()
    out, lse = sv.attention(*args, sp, scale=scale, window=200)
    assert sv.attention_error()[0] == 0
    want = c.oracle(scale=scale, window=200)
    check(c, out, lse, want)
    truth = torch.as_tensor(want[1], dtype=torch.float32)
    score = torch.rand(4, 720, generator=torch.Generator().manual_seed(1))
    ref = oa.weights(c.q, c.cache, c.layer, n, c.table, k, truth, score, c.spec, scale=scale,
                     window=200)
    got = sv.attention_weights(*args, truth.to(DEV), score.to(DEV), sp, scale=scale, window=200)
    assert sv.attention_weights_error()[0] == 0
    check_weights(c, got, ref, want, 16 * Hk * G)


@pytest.mark.parametrize("window", [1, 70, 128, 400])
@pytest.mark.parametrize("spec", [True, False])
@pytest.mark.parametrize("dtype,D", [(B16, 128), (F16, 64), (B16, 256), (F32, 64)])
def test_scores_in_front_of_the_window_reach_another_output(dtype, D, spec, window):
    n, k, Hk, G = [600, 129, 3, 1000], [5, 0, 2, 15], 2, 2
    c = Case(32, n, k, Hk, G, D, 16, dtype, spec=spec)
    args, sp = c.gpu()
    want = c.oracle(window=window)
    truth = torch.as_tensor(want[1], dtype=torch.float32)
    score = torch.rand(4, 1020, generator=torch.Generator().manual_seed(1))
    accept = np.array([2, 0, -1, 15], np.int32)
    ref = oa.weights(c.q, c.cache, c.layer, n, c.table, k, truth, score, c.spec, accept,
                     window=window)
    out = torch.full((4, 1020), 7.0, device=DEV)
    kept = score.to(DEV)
    got = sv.attention_weights(*args, truth.to(DEV), kept, sp, torch.as_tensor(accept).to(DEV),
                               window=window, out_score=out)
    assert got is out and sv.attention_weights_error()[0] == 0
    assert torch.equal(kept.cpu(), score)
    for b, x in enumerate(n):
        end = 0 if accept[b] < 0 else x + accept[b] + 1 if spec else x
        assert (out[b, end:] == 7).all()
        check_weights(c, out[b, :end], ref[b, :end], want, 16 * Hk * G)
        front = max(0, (x if spec else x - 1 - k[b]) - window + 1)   # seen by no counted token
        front = min(front, end)
        assert torch.equal(out[b, :front].cpu(), score[b, :front])
