"""An expired wait in the kernels of attention over prompts and over trees, in the form
that faults nothing: with the test switch set, one wait of one block, on a barrier
nothing arrives on, runs out after its short limit.  The call reports SV_ERR_TIMEOUT,
the block's rows are NaN, and the next calls are as before."""

import random

import pytest
import torch

import speculative_decoding_verification_13_gb300 as sv

pytestmark = pytest.mark.gpu
DEV = "cuda"
SV_ERR_TIMEOUT = 24


@pytest.fixture
def expire():
    lib = sv.load_library()
    yield lib.spec_test_expire_wait
    lib.spec_test_expire_wait(0)


def check(expire, block, call, error):
    want, want_lse = call()
    assert error() == (0, -1, -1)
    out, lse = torch.full_like(want, 7), torch.full_like(want_lse, 7)
    expire(block + 1)
    call(out=out, out_lse=lse)
    assert error() == (SV_ERR_TIMEOUT, -1, -1)
    expire(0)
    failed = torch.isnan(lse)
    assert failed.any() and not failed.all()
    assert torch.isnan(out[failed]).all()
    assert torch.equal(out[~failed], want[~failed]) and torch.equal(lse[~failed], want_lse[~failed])
    for _ in range(3):
        again = call()
        assert error() == (0, -1, -1)
        assert torch.equal(want, again[0]) and torch.equal(want_lse, again[1])


@pytest.mark.parametrize("D,dtype", [(128, torch.bfloat16), (64, torch.float16),
                                     (256, torch.bfloat16), (80, torch.bfloat16)])
@pytest.mark.parametrize("block", [0, 1, 77, 151])
def test_prompt_attention_reports_an_expired_wait_and_recovers(expire, D, dtype, block):
    g = torch.Generator(device=DEV).manual_seed(3)
    n = [3000, 1, 700, 0, 1500, 90]
    at = torch.tensor([0] + n, device=DEV).cumsum(0).int()
    q, k, v = (torch.randn(sum(n), h, D, device=DEV, generator=g).to(dtype) for h in (16, 4, 4))
    check(expire, block, lambda **kw: sv.prompt_attention(q, k, v, at, **kw),
          sv.prompt_attention_error)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("block", [0, 77])
def test_tree_attention_reports_an_expired_wait_and_recovers(expire, D, block):
    g, rng = torch.Generator(device=DEV).manual_seed(4), random.Random(4)
    n, k, S, Hk = [60000, 5, 300, 14000], [63, 0, 40, 20], 16, 2
    pages = [-(-x // S) for x in n]
    table = torch.full((4, max(pages)), -1, dtype=torch.int32)
    at = 0
    for b, c in enumerate(pages):
        table[b, :c] = torch.arange(at, at + c)
        at += c
    cache = torch.randn(at, 1, 2, S, Hk * D, device=DEV, generator=g).bfloat16()
    spec = torch.randn(4, 64, 1, 2, Hk * D, device=DEV, generator=g).bfloat16()
    q = torch.randn(sum(k) + 4, Hk * 4, D, device=DEV, generator=g).bfloat16()
    parent = [rng.randrange(max(j, 1)) for x in k for j in range(x + 1)]
    i32 = dict(dtype=torch.int32, device=DEV)
    args = (q, cache, 0, torch.tensor(n, **i32), table.to(DEV), torch.tensor(k, **i32),
            torch.tensor(parent, **i32), spec)
    check(expire, block, lambda **kw: sv.tree_attention(*args, **kw), sv.tree_attention_error)
