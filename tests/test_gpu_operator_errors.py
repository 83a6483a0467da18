"""What the operators' *_error calls report after calls with nothing to do."""

import pytest
import torch

import speculative_decoding_verification_13_gb300 as sv

pytestmark = pytest.mark.gpu
DEV = "cuda"


def i32(*x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def test_an_empty_call_has_no_error():
    cache = torch.zeros(4, 1, 2, 16, 128, dtype=torch.bfloat16, device=DEV)
    q = torch.zeros(1, 2, 64, dtype=torch.bfloat16, device=DEV)
    bad, none = i32(99).view(1, 1), torch.zeros(0, 1, dtype=torch.int32, device=DEV)
    lse, score = torch.zeros(1, 2, device=DEV), torch.zeros(1, 64, device=DEV)
    zero = none[:, 0].contiguous()
    x = torch.zeros(1, 100, device=DEV)
    calls = [
        (lambda: sv.attention(q, cache, 0, i32(8), bad, i32(0)),
         lambda: sv.attention(q[:0], cache, 0, zero, none, zero), sv.attention_error, (27, 0, -1)),
        (lambda: sv.attention_weights(q, cache, 0, i32(8), bad, i32(0), lse, score),
         lambda: sv.attention_weights(q[:0], cache, 0, zero, none, zero, lse[:0], score[:0]),
         sv.attention_weights_error, (27, 0, -1)),
        (lambda: sv.kv_evict(cache, score, i32(8), bad, 4),
         lambda: sv.kv_evict(cache, score[:0], zero, none, 4), sv.kv_evict_error, (27, 0, -1)),
        (lambda: sv.logprobs(x, i32(100)),
         lambda: sv.logprobs(x[:0], zero), sv.logprobs_error, (20, -1, 0)),
    ]
    for failing, empty, error, want in calls:
        failing()
        assert error() == want
        empty()
        assert error() == (0, -1, -1)
        failing()
        assert error() == want
        side = torch.cuda.Stream()   # a workspace that was never written
        with torch.cuda.stream(side):
            empty()
            assert error() == (0, -1, -1)


def test_a_refused_call_is_not_the_last_one():
    cache = torch.zeros(4, 1, 2, 16, 128, dtype=torch.bfloat16, device=DEV)
    q = torch.zeros(1, 2, 64, dtype=torch.bfloat16, device=DEV)
    sv.attention(q, cache, 0, i32(8), i32(99).view(1, 1), i32(0))
    with torch.cuda.stream(torch.cuda.Stream()):   # a workspace that was never written
        with pytest.raises(sv.SpecVerifyError):
            sv.attention(q, cache, 0, i32(8), i32(1).view(1, 1), i32(0), scale=float("nan"))
    assert sv.attention_error() == (27, 0, -1)
