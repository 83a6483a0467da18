"""Windows and budgets past 32 bits: the C entries take 32-bit numbers, which the
binding must not wrap."""

import pytest
import torch

import speculative_decoding_verification_13_gb300 as sv

pytestmark = pytest.mark.gpu
DEV = "cuda"


def test_numbers_past_32_bits_do_not_wrap():
    g = torch.Generator(device=DEV).manual_seed(1)
    i32 = dict(dtype=torch.int32, device=DEV)
    cache = torch.randn(20, 1, 2, 16, 128, device=DEV, generator=g).bfloat16()
    q = torch.randn(1, 4, 64, device=DEV, generator=g).bfloat16()
    n, k = torch.tensor([300], **i32), torch.tensor([0], **i32)
    table = torch.arange(20, **i32)[None]
    want = sv.attention(q, cache, 0, n, table, k)
    for window in (2 ** 31, 2 ** 32, 2 ** 32 + 7, 2 ** 40 + 1):
        got = sv.attention(q, cache, 0, n, table, k, window=window)
        assert torch.equal(want[0], got[0]) and torch.equal(want[1], got[1])
    score = torch.rand(1, 320, device=DEV, generator=g)
    before = cache.clone()
    for budget in (2 ** 31, 2 ** 32 + 7):
        with pytest.raises(ValueError):
            sv.kv_evict(cache, score, n, table, budget)
    assert n.tolist() == [300] and torch.equal(cache, before)
