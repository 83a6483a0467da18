"""Workspaces of kv_commit: its two kernels hand each other the list of entries to
copy in it, so that calls that may run at the same time must not share one: calls on
two streams, a captured call and the stream's other ones, chains and paths."""

import threading
import time
import types

import numpy as np
import pytest
import torch

import speculative_decoding_verification_13_gb300 as sv
from oracle.kv import kv_commit as oracle_commit
from speculative_decoding_verification_13_gb300 import operators as ops

DEV = "cuda"


# ------------------------------------------------- without a GPU: a stand-in library
@pytest.fixture
def lib(monkeypatch):
    """A library that notes (entry, stream, workspace, bytes) of every call."""
    x = types.SimpleNamespace(calls=[], inside=0, most=0, read=[])

    def entry(name):
        def run(*args):
            x.inside += 1
            x.most = max(x.most, x.inside)
            time.sleep(0.001)
            stream, _, ws, nbytes = args[-4:]
            x.calls.append((name, getattr(stream, "value", stream), getattr(ws, "value", ws),
                            nbytes))
            x.inside -= 1
            return 0
        return run

    def get_error(ws, stream, *out):
        x.read.append((getattr(ws, "value", ws), getattr(stream, "value", stream)))
        return 0

    fake = types.SimpleNamespace(
        spec_kv_commit=entry("chain"), spec_kv_commit_path=entry("path"),
        spec_kv_commit_workspace_size=lambda B: 512 * max(B, 1),
        spec_kv_commit_path_workspace_size=lambda B: 1024 * max(B, 1),
        spec_verify_get_error=get_error)
    monkeypatch.setattr(ops, "_lib", fake)
    monkeypatch.setattr(sv, "load_library", lambda: fake)
    monkeypatch.setattr(ops, "_workspaces", {})
    monkeypatch.setattr(ops, "_last", {})
    monkeypatch.setattr(ops, "_sizes", {})
    monkeypatch.setattr(sv, "_kv_ws", {}, raising=False)
    monkeypatch.setattr(ops, "_empty", lambda shape, dtype, dev, s: torch.empty(shape, dtype=dtype))
    monkeypatch.setattr(torch.Tensor, "is_cuda", True)      # tensors here are the host's
    monkeypatch.setattr(torch.cuda, "current_device", lambda: None)
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: x.capturing)
    monkeypatch.setattr(torch.cuda, "device", lambda dev: __import__("contextlib").nullcontext())
    x.capturing = False
    return x


def commit(B, stream, path=False):
    i = torch.zeros(B, dtype=torch.int32)
    sv.kv_commit(torch.zeros(2, 1, 2, 4, 8), torch.zeros(B, 2, 1, 2, 8), i, i, i.clone(),
                 torch.zeros(B, 2, dtype=torch.int32), types.SimpleNamespace(cuda_stream=stream),
                 **(dict(path=i) if path else {}))


def test_streams_have_workspaces_of_their_own(lib):
    for stream in (7, 8, 7, 8):
        commit(3, stream)
    ws = [c[2] for c in lib.calls]
    assert [c[1] for c in lib.calls] == [7, 8, 7, 8]
    assert ws[0] == ws[2] and ws[1] == ws[3] and ws[0] != ws[1]


def test_a_captured_call_keeps_its_workspace_to_itself(lib):
    commit(3, 7)
    lib.capturing = True
    commit(3, 7)
    lib.capturing = False
    commit(3, 7)
    assert lib.calls[0][2] == lib.calls[2][2] != lib.calls[1][2]


def test_a_path_does_not_take_the_workspace_of_a_chain(lib):
    commit(3, 7)
    commit(40, 7, path=True)      # larger
    commit(3, 7)
    assert [c[0] for c in lib.calls] == ["chain", "path", "chain"]
    assert lib.calls[0][2] == lib.calls[2][2] != lib.calls[1][2]
    assert lib.calls[1][3] >= 40 * 1024


def test_one_call_at_a_time_between_its_workspace_and_its_last_launch(lib):
    threads = [threading.Thread(target=lambda p=p: [commit(3, 7, p) for _ in range(10)])
               for p in (False, True, False, True)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert len(lib.calls) == 40 and lib.most == 1


def test_the_error_is_the_last_calls(lib, monkeypatch):
    monkeypatch.setattr(torch, "device", lambda d: types.SimpleNamespace(index=None))
    commit(3, 7)
    commit(5, 8, path=True)
    sv.kv_commit_error(types.SimpleNamespace(cuda_stream=8))
    commit(3, 7)
    sv.kv_commit_error(types.SimpleNamespace(cuda_stream=7))
    assert lib.read == [(lib.calls[1][2], 8), (lib.calls[2][2], 7)]


# ------------------------------------------------------------------------ on the GPU
def case(seed, B, path):
    """Arguments on the GPU, and what the oracle makes of them."""
    rng = np.random.default_rng(seed)
    S, layers, E = 8, 2, 64
    k = rng.integers(0, 30, B).astype(np.int32)
    L = np.array([rng.integers(-1, x + 1) for x in k], np.int32)
    n = rng.integers(0, 40, B).astype(np.int32)
    cols = 10
    table = rng.permutation(B * cols).astype(np.int32).reshape(B, cols)
    g = torch.Generator().manual_seed(seed)
    cache = torch.randint(-2 ** 31, 2 ** 31 - 1, (B * cols, layers, 2, S, E), generator=g,
                          dtype=torch.int32)
    spec = torch.randint(-2 ** 31, 2 ** 31 - 1, (B, 30, layers, 2, E), generator=g,
                         dtype=torch.int32)
    moved, nodes = spec.numpy().copy(), None
    if path:
        nodes = np.full(int(k.sum()) + B, -1, np.int32)
        t = 0
        for b in range(B):
            walk = np.sort(rng.choice(k[b] + 1, L[b] + 1, replace=False))
            nodes[t:t + L[b] + 1] = walk
            moved[b, :L[b] + 1] = spec.numpy()[b, walk]
            t += k[b] + 1
    want = cache.numpy().copy()
    length, _ = oracle_commit(moved, L, k, n, table, want, S)
    args = [torch.as_tensor(x).to(DEV) for x in (cache, spec, L, k, n, table)]
    kw = {"path": torch.as_tensor(nodes).to(DEV)} if path else {}
    return args, kw, want, length


def fresh(x):
    args, kw, want, length = x
    return [args[0].clone(), *args[1:4], args[4].clone(), args[5]], kw


@pytest.mark.gpu
def test_two_streams_at_once():
    cases = [case(1, 200, False), case(2, 33, True), case(3, 7, False), case(4, 300, True)]
    streams = [torch.cuda.Stream() for _ in cases]
    for _ in range(10):
        runs = [fresh(c) for c in cases]
        torch.cuda.synchronize()
        for (args, kw), s in zip(runs, streams):
            sv.kv_commit(*args, s, **kw)
        torch.cuda.synchronize()
        for (args, _), (_, _, want, length) in zip(runs, cases):
            assert np.array_equal(args[0].cpu().numpy(), want)
            assert np.array_equal(args[4].cpu().numpy(), length)
    assert sv.kv_commit_error() == (0, -1, -1)


@pytest.mark.gpu
@pytest.mark.parametrize("captured,between", [(False, True), (True, False)])
def test_a_captured_commit_replayed_after_larger_ones(captured, between):
    small, large = case(5, 20, captured), case(6, 400, between)
    start, kw = fresh(small)
    args, _ = fresh(small)
    sv.kv_commit(*args, **kw)                       # the stream's own, before the capture
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        sv.kv_commit(*args, **kw)
    side = torch.cuda.Stream()
    for _ in range(3):
        args[0].copy_(start[0])
        args[4].copy_(start[4])
        other, other_kw = fresh(large)
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            graph.replay()
        sv.kv_commit(*other, **other_kw)
        torch.cuda.synchronize()
        for got, (_, _, want, length) in ((args, small), (other, large)):
            assert np.array_equal(got[0].cpu().numpy(), want)
            assert np.array_equal(got[4].cpu().numpy(), length)
    del graph
