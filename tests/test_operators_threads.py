"""Operators called from several threads on one stream: the calls share their
stream's workspace and their kernels must not come between one another's."""

import threading
import time

import pytest
import torch

import speculative_decoding_verification_13_gb300 as sv
from speculative_decoding_verification_13_gb300 import operators as ops


def run_threads(*work):
    failures = []

    def guard(f):
        try:
            f()
        except BaseException as e:  # noqa: BLE001
            failures.append(e)

    threads = [threading.Thread(target=guard, args=(f,)) for f in work]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    if failures:
        raise failures[0]


def test_one_call_at_a_time_between_its_workspace_and_its_last_launch(monkeypatch):
    # without a GPU: a stand-in for the C entry that takes its time
    inside, most, made = [0], [0], []

    def entry(*args):
        inside[0] += 1
        most[0] = max(most[0], inside[0])
        time.sleep(0.002)
        inside[0] -= 1
        return 0

    def allocate(shape, dtype, dev, stream):
        time.sleep(0.002)
        made.append(shape)
        return torch.zeros(shape, dtype=dtype)

    lib = type("Lib", (), {"spec_attention": staticmethod(entry),
                           "spec_kv_evict": staticmethod(entry)})
    monkeypatch.setattr(ops, "_lib", lib)
    monkeypatch.setattr(ops, "_empty", allocate)
    monkeypatch.setattr(ops, "_workspace_size", lambda kind, dev, size: size[0])
    monkeypatch.setattr(ops, "_stream_of", lambda stream, dev: 1234)
    monkeypatch.setattr(ops, "_workspaces", {})
    monkeypatch.setattr(ops, "_last", {})
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: False)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    dev = torch.device("cuda", 0)
    run_threads(*[lambda kind=kind: [ops._launch(kind, dev, None, (512,), ()) for _ in range(10)]
                  for kind in ("attention", "kv_evict") * 2])
    assert most[0] == 1
    assert len(made) == 2   # one workspace a kind


@pytest.mark.gpu
def test_threads_on_one_stream_get_the_results_of_one():
    dev, i32 = "cuda", torch.int32
    g = torch.Generator(device=dev).manual_seed(1)

    def attention_case(B, n, Hk, D):
        S = 16
        pages = -(-n // S)
        cache = torch.randn(B * pages, 1, 2, S, Hk * D, device=dev, generator=g).bfloat16()
        q = torch.randn(B, 2 * Hk, D, device=dev, generator=g).bfloat16()
        table = torch.arange(B * pages, dtype=i32, device=dev).view(B, pages)
        args = (q, cache, 0, torch.full((B,), n, dtype=i32, device=dev), table,
                torch.zeros(B, dtype=i32, device=dev))
        return lambda: torch.cat([x.float().flatten() for x in sv.attention(*args)])

    def evict_case(B, n, budget):
        S, E = 16, 64
        pages = -(-n // S)
        cache = torch.randn(B * pages, 2, 2, S, E, device=dev, generator=g).bfloat16()
        score = torch.rand(B, n, device=dev, generator=g)
        table = torch.arange(B * pages, dtype=i32, device=dev).view(B, pages)
        n_ = torch.full((B,), n, dtype=i32, device=dev)

        def run():
            out = torch.zeros_like(cache)
            kept = sv.kv_evict(cache, score, n_, table, budget, 2, 5, out_cache=out,
                               out_table=table, out_score=torch.zeros_like(score),
                               out_len=torch.zeros_like(n_), with_kept=True)[1]
            return torch.cat([out.float().flatten(), kept.float().flatten()])
        return run

    for first, second in ((attention_case(1, 3000, 1, 64), attention_case(24, 700, 4, 128)),
                          (evict_case(1, 300, 50), evict_case(9, 900, 200)),
                          (attention_case(2, 2000, 2, 256), evict_case(3, 500, 77))):
        want = first(), second()
        torch.cuda.synchronize()

        def work(f, w):
            for _ in range(60):
                assert torch.equal(f(), w)

        run_threads(*[lambda f=f, w=w: work(f, w) for f, w in
                      zip((first, second) * 2, want * 2)])
