"""An expired wait in the operators' kernels, in the form that faults nothing:
with the test switch set, one wait of one block, on a barrier nothing arrives on,
runs out after its short limit.  The call reports SV_ERR_TIMEOUT, its copies
land, and the next calls are as before."""

import time

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


def batch(D, dtype, seed=3):
    """Long and short requests: parts of one over many blocks, several in a block."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    n, k, S, Hk = [60000, 5, 300, 0, 14000], [3, 0, 15, 1, 7], 16, 2
    pages = [-(-x // S) for x in n]
    table = torch.full((5, max(pages)), -1, dtype=torch.int32)
    at = 0
    for b, c in enumerate(pages):
        table[b, :c] = torch.arange(at, at + c)
        at += c
    cache = torch.randn(at, 1, 2, S, Hk * D, device=DEV, generator=g).to(dtype)
    spec = torch.randn(5, 16, 1, 2, Hk * D, device=DEV, generator=g).to(dtype)
    q = torch.randn(sum(k) + 5, Hk * 4, D, device=DEV, generator=g).to(dtype)
    i32 = dict(dtype=torch.int32, device=DEV)
    return (q, cache, 0, torch.tensor(n, **i32), table.to(DEV), torch.tensor(k, **i32)), spec


@pytest.mark.parametrize("D,dtype", [(128, torch.bfloat16), (64, torch.float16),
                                     (256, torch.bfloat16)])
@pytest.mark.parametrize("block", [0, 1, 77, 151])
def test_attention_reports_an_expired_wait_and_recovers(expire, D, dtype, block):
    args, spec = batch(D, dtype)
    want = sv.attention(*args, spec)
    assert sv.attention_error()[0] == 0
    t0 = time.perf_counter()
    expire(block + 1)
    sv.attention(*args, spec)
    assert sv.attention_error() == (SV_ERR_TIMEOUT, -1, -1)
    assert time.perf_counter() - t0 < 5
    expire(0)
    for _ in range(3):
        again = sv.attention(*args, spec)
        assert sv.attention_error()[0] == 0
        assert torch.equal(want[0], again[0]) and torch.equal(want[1], again[1])


@pytest.mark.parametrize("D,dtype", [(128, torch.bfloat16), (64, torch.float16),
                                     (256, torch.bfloat16)])
@pytest.mark.parametrize("block", [0, 1, 40, 77, 151])
def test_no_row_of_an_expired_call_holds_anything_but_its_result_or_nan(expire, D, dtype, block):
    args, spec = batch(D, dtype)
    want, want_lse = sv.attention(*args, spec)
    # other outputs and parts in the buffers
    sv.attention(-args[0], *args[1:], spec)
    out, lse = torch.full_like(want, 7), torch.full_like(want_lse, 7)
    expire(block + 1)
    sv.attention(*args, spec, out=out, out_lse=lse)
    assert sv.attention_error()[0] == SV_ERR_TIMEOUT
    failed = torch.isnan(lse)
    assert failed.any() and not failed.all()
    assert torch.isnan(out[failed]).all()
    assert torch.equal(out[~failed], want[~failed]) and torch.equal(lse[~failed], want_lse[~failed])


@pytest.mark.parametrize("D,dtype", [(128, torch.bfloat16), (64, torch.float16),
                                     (256, torch.bfloat16)])
@pytest.mark.parametrize("block", [0, 1, 40, 151])
def test_weights_report_an_expired_wait_and_recover(expire, D, dtype, block):
    args, spec = batch(D, dtype)
    lse = sv.attention(*args, spec)[1]
    score = torch.rand(5, 60100, device=DEV)
    call = lambda: sv.attention_weights(*args, lse, score, spec,
                                        out_score=torch.full_like(score, 7))
    want = call()
    assert sv.attention_weights_error()[0] == 0
    t0 = time.perf_counter()
    expire(block + 1)
    got = call()
    assert sv.attention_weights_error() == (SV_ERR_TIMEOUT, -1, -1)
    assert time.perf_counter() - t0 < 5
    left = (got == 7) & (want != 7)     # positions that the block did not come to
    assert left.any() and not left.all()
    assert torch.equal(got[~left], want[~left])
    expire(0)
    for _ in range(3):
        assert torch.equal(call(), want)
        assert sv.attention_weights_error()[0] == 0


# one block a row, in several waves; clusters of 8, 4 and 2 blocks
@pytest.mark.parametrize("rows,V,dtype,cluster", [
    (700, 50257, torch.bfloat16, 1), (200, 40000, torch.float32, 1),
    (3, 151936, torch.bfloat16, 8), (30, 151936, torch.float32, 4), (8, 32000, torch.float32, 2)])
@pytest.mark.parametrize("n_top", [0, 20])
def test_logprobs_fail_the_row_of_an_expired_wait_only(expire, rows, V, dtype, cluster, n_top):
    g = torch.Generator(device=DEV).manual_seed(rows)
    x = torch.randn(rows, V, device=DEV, generator=g).to(dtype)
    tok = torch.randint(0, V, (rows,), dtype=torch.int32, device=DEV, generator=g)
    take = 6 if n_top else 4
    want = sv.logprobs(x, tok, None, n_top)[:take]
    assert sv.logprobs_error()[0] == 0
    for block in sorted({0, cluster - 1, rows // 2 * cluster, rows * cluster - 1}):
        t0 = time.perf_counter()
        expire(block + 1)
        got = sv.logprobs(x, tok, None, n_top)[:take]
        assert sv.logprobs_error() == (SV_ERR_TIMEOUT, -1, block // cluster)
        assert time.perf_counter() - t0 < 5
        other = torch.arange(rows, device=DEV) != block // cluster
        for a, b in zip(want, got):
            assert torch.equal(a[other], b[other])
            failed = b[~other]
            assert (torch.isnan(failed) if failed.is_floating_point() else failed == -1).all()
        expire(0)
        again = sv.logprobs(x, tok, None, n_top)[:take]
        assert sv.logprobs_error()[0] == 0
        assert all(torch.equal(a, b) for a, b in zip(want, again))
