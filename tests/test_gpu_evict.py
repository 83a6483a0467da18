"""Eviction on the GPU against the oracle (oracle/evict.py), bit-exact: the whole
cache, the scores, the lengths and the kept positions."""

import numpy as np
import pytest
import torch

import speculative_decoding_verification_13_gb300 as sv
from oracle import evict as oe

pytestmark = pytest.mark.gpu
DEV = "cuda"


def case(seed, n, S, layers, E, dtype=torch.bfloat16, ties=False, extra=3):
    g = torch.Generator().manual_seed(seed)
    need = [-(-x // S) for x in n]
    pool = sum(need) + extra
    order = torch.randperm(pool, generator=g).tolist()
    table = torch.full((len(n), max(need) + 1), -1, dtype=torch.int32)
    for b, c in enumerate(need):
        table[b, :c] = torch.tensor([order.pop() for _ in range(c)], dtype=torch.int32)
    cache = torch.randn(pool, layers, 2, S, E, generator=g).to(dtype)
    score = torch.randn(len(n), max(n) + 3, generator=g).exp()
    if ties:
        score = (score * 2).round()
    for b, x in enumerate(n):
        score[b, x:] = 0
    return n, table, cache, score


def bits(t):
    return t.cpu().contiguous().view(torch.int16 if t.element_size() == 2 else torch.int32).numpy()


def same(a, b):
    assert np.array_equal(a.view(np.int32), b.view(np.int32))


def run(n, table, cache, score, budget, sinks, recent, out=False):
    kv_len = torch.tensor(n, dtype=torch.int32)
    d = dict(cache=cache.to(DEV), score=score.to(DEV), kv_len=kv_len.to(DEV), table=table.to(DEV))
    ref_c, ref_s = bits(cache).copy(), score.numpy().copy()
    kw, dst, dt = {}, None, None
    if out:
        need = [-(-min(x, budget) // cache.shape[3]) for x in n]
        pages = torch.randperm(sum(need) + 2, generator=torch.Generator().manual_seed(1)).tolist()
        out_table = torch.full((len(n), max(1, max(need))), -1, dtype=torch.int32)
        for b, c in enumerate(need):
            out_table[b, :c] = torch.tensor([pages.pop() for _ in range(c)], dtype=torch.int32)
        out_cache = torch.zeros((sum(need) + 2,) + cache.shape[1:], dtype=cache.dtype)
        kw = dict(out_cache=out_cache.to(DEV), out_table=out_table.to(DEV),
                  out_score=d["score"].clone(),
                  out_len=torch.zeros(len(n), dtype=torch.int32, device=DEV))
        dst, dt = bits(out_cache).copy(), out_table.numpy()
    lengths, kept = sv.kv_evict(d["cache"], d["score"], d["kv_len"], d["table"], budget, sinks,
                                recent, with_kept=True, **kw)
    code = sv.kv_evict_error()[:2]
    want_len, want_kept, st = oe.kv_evict(ref_c, ref_s, n, table.numpy(), budget, sinks, recent,
                                          dst, dt)
    assert np.array_equal(lengths.cpu().numpy(), want_len)
    assert np.array_equal(kept.cpu().numpy(), want_kept)
    same((kw["out_score"] if out else d["score"]).cpu().numpy(), ref_s)
    assert np.array_equal(bits(kw["out_cache"]) if out else bits(d["cache"]),
                          dst if out else ref_c)
    if out:
        assert np.array_equal(bits(d["cache"]), bits(cache)) and d["kv_len"].tolist() == n
        same(d["score"].cpu().numpy(), score.numpy())
    bad = np.nonzero(st)[0]
    assert code == ((0, -1) if len(bad) == 0 else (st[bad[0]], bad[0]))
    return st


B16, F16, F32 = torch.bfloat16, torch.float16, torch.float32


@pytest.mark.parametrize("out", [False, True])
@pytest.mark.parametrize("n,S,layers,E,dtype,budget,sinks,recent", [
    ([700, 33, 1500, 1], 16, 3, 1024, B16, 128, 4, 32),
    ([90, 64, 65, 0], 7, 2, 64, F16, 64, 0, 0),
    ([50, 20], 1, 1, 8, B16, 17, 3, 14),               # nothing left to choose
    ([2500, 1024, 1025], 64, 1, 40, F32, 1000, 0, 1),
    ([40, 41], 16, 2, 520, B16, 1, 0, 0),              # one survivor, entries of 1040 bytes
    ([300], 16, 36, 1024, B16, 299, 4, 64),            # one position goes
])
def test_evict_matches_oracle(n, S, layers, E, dtype, budget, sinks, recent, out):
    assert not run(*case(sum(n), n, S, layers, E, dtype), budget, sinks, recent, out).any()


@pytest.mark.parametrize("out", [False, True])
def test_ties_infinities_and_nan(out):
    n, table, cache, score = case(5, [400, 3000], 16, 1, 64, ties=True)
    score[0, 50:60] = float("nan")
    score[0, 70:75] = float("inf")
    score[0, 80:200] = -float("inf")
    score[1, ::3] = 0.0
    score[1, 1::7] = -0.0
    assert not run(n, table, cache, score, 200, 2, 20, out).any()
    score[:] = 1.0
    assert not run(n, table, cache, score, 200, 2, 20, out).any()
    score[:] = float("nan")
    assert not run(n, table, cache, score, 390, 2, 20, out).any()


@pytest.mark.parametrize("out", [False, True])
def test_errors_touch_nothing(out):
    n, table, cache, score = case(7, [100, 90, 80, 70], 16, 2, 64)
    table[1, 2] = -1
    table[2, 4] = cache.shape[0]
    n = list(n)
    n[3] = 200          # past the block table and the scores
    st = run(n, table, cache, score, 60, 4, 8, out)
    assert st.tolist() == [0, 27, 27, 28]
    n[3] = -1
    assert run(n, table, cache, score, 60, 4, 8, out).tolist() == [0, 27, 27, 28]


def test_long_caches_and_strided_scores():
    n, table, cache, score = case(9, [40001, 12345], 16, 1, 8)
    assert not run(n, table, cache, score, 5000, 4, 100).any()
    wide = torch.zeros(2, score.shape[1] + 9, device=DEV)
    wide[:, :-9] = score.to(DEV)
    kv = torch.tensor(n, dtype=torch.int32, device=DEV)
    lengths, kept = sv.kv_evict(cache.to(DEV), wide[:, :-9], kv, table.to(DEV), 5000, 4, 100,
                                with_kept=True)
    want = [oe.choose(score[b].numpy(), n[b], 5000, 4, 100) for b in range(2)]
    assert kept.tolist() == want and lengths.tolist() == [5000, 5000]
    assert (wide[:, -9:] == 0).all()


def test_graph_and_refusals():
    n, table, cache, score = case(3, [200, 300], 16, 2, 64)
    d = [x.to(DEV) for x in (cache, score, torch.tensor(n, dtype=torch.int32), table)]
    out = dict(out_cache=torch.zeros_like(d[0]), out_table=d[3], out_score=torch.zeros_like(d[1]),
               out_len=torch.zeros(2, dtype=torch.int32, device=DEV))
    want = sv.kv_evict(*d, 50, 4, 10, with_kept=True, **out)[1].clone()
    kept = torch.zeros(2, 50, dtype=torch.int32, device=DEV)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        sv.kv_evict(*d, 50, 4, 10, out_kept=kept, **out)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(kept, want)
    with pytest.raises(ValueError):
        sv.kv_evict(*d, 0)
    with pytest.raises(ValueError):
        sv.kv_evict(*d, 10, 6, 5)
    with pytest.raises(ValueError):
        sv.kv_evict(*d, 10, out_cache=d[0])
    with pytest.raises(ValueError):
        sv.kv_evict(*d, 10, out_table=d[3], out_cache=d[0][:, :1].contiguous())
    with pytest.raises(TypeError):
        sv.kv_evict(d[0], d[1].half(), *d[2:], 10)


def test_the_own_pages_named_as_the_destination_are_in_place():
    # many blocks would copy at once between pages that lie over one another
    n, table, cache, score = case(13, [9001, 700, 2500], 16, 4, 1024)
    d = [x.to(DEV) for x in (cache, score, torch.tensor(n, dtype=torch.int32), table)]
    for dst in (None, d[0]):
        here = [x.clone() for x in d]
        if dst is not None:
            dst = here[0]
        lengths, kept = sv.kv_evict(*here, 2000, 4, 64, out_cache=dst, out_table=here[3],
                                    with_kept=True)
        assert sv.kv_evict_error()[0] == 0
        own = [x.clone() for x in d]
        want_lengths, want_kept = sv.kv_evict(*own, 2000, 4, 64, with_kept=True)
        assert torch.equal(lengths, want_lengths) and torch.equal(kept, want_kept)
        assert np.array_equal(bits(here[0]), bits(own[0])) and torch.equal(here[1], own[1])
