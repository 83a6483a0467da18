"""Refusals of the calls for prompts, trees and tables (no GPU): the C entry points
reject bad arguments before touching the device, the binding rejects tensors that
do not fit."""

import ctypes

import pytest
import torch

import speculative_decoding_verification_13_gb300 as sv
from speculative_decoding_verification_13_gb300 import build as cuda_build
from speculative_decoding_verification_13_gb300 import operators as ops

P = ctypes.c_void_p
A, B_, C, W = P(0x10000), P(0x20000), P(0x30000), P(0x40000)   # never dereferenced
BIG = 1 << 40


@pytest.fixture(scope="module")
def lib():
    cuda_build.build()
    return ops._library()


def call(f, base, **kw):
    a = dict(base)
    assert set(kw) <= set(a), kw
    a.update(kw)
    return f(*a.values())


def refused(f, base, code, *many):
    for kw in many:
        assert call(f, base, **kw) == code, kw


def test_prompt_attention(lib):
    f = lib.spec_prompt_attention
    base = dict(q=A, qr=1024, qh=64, k=A, kr=1024, kh=64, v=A, vr=1024, vh=64, dtype=1, rows=10,
                Hq=8, Hk=2, D=64, offsets=A, scale=1.0, window=0, out=C, lse=C, stream=None, batch=2,
                ws=None, nbytes=0)
    assert call(f, base) == 4                                   # all fine but the workspace
    assert call(f, base, ws=P(0x30010), nbytes=BIG) == 4
    assert call(f, base, rows=0) == 0 and call(f, base, batch=0) == 0
    refused(f, base, 1, dict(batch=-1), dict(rows=-1), dict(rows=2 ** 31 - 256), dict(window=-1),
            dict(D=0), dict(Hk=0), dict(Hq=0), dict(Hq=7), dict(scale=float("nan")),
            dict(scale=float("inf")), dict(q=None), dict(k=None), dict(v=None), dict(offsets=None),
            dict(out=None), dict(lse=None))
    refused(f, base, 2, dict(dtype=3), dict(D=257), dict(Hq=131072, Hk=65536),
            dict(q=P(0x10001)), dict(out=P(0x30001)), dict(k=P(0x10002), dtype=0),
            dict(rows=2 ** 30, Hq=2048, Hk=1))
    assert lib.spec_prompt_attention_workspace_size(-1) == 0


def test_tree_attention(lib):
    desc = sv._KvCache(A, 4, 2, 16, 256, 2)
    f = lib.spec_tree_attention
    base = dict(cache=ctypes.byref(desc), dtype=1, layer=0, Hk=2, q=A, qts=1024, qhs=128, Hq=8,
                rows=3, spec=B_, slots=4, k=A, parent=A, n=A, table=A, cols=2, scale=1.0, window=0,
                out=C, lse=C, stream=None, batch=1, ws=None, nbytes=0)
    assert call(f, base) == 4
    assert call(f, base, batch=0, rows=0) == 0
    refused(f, base, 1, dict(parent=None), dict(spec=None), dict(layer=2), dict(Hk=3), dict(rows=0),
            dict(window=-1), dict(slots=0), dict(q=None), dict(out=None), dict(lse=None),
            dict(scale=float("nan")), dict(dtype=0))
    refused(f, base, 2, dict(dtype=7), dict(spec=P(0x20008)))
    assert lib.spec_tree_attention_workspace_size(-1, 64) == 0


def test_verify_tree_greedy(lib):
    f = lib.spec_verify_tree_greedy
    base = dict(argmax=A, drafts=A, parent=A, k=A, accept=C, tokens=C, path=C, stream=None, batch=2,
                rows=5, vocab=100, ws=None, nbytes=0)
    assert call(f, base) == 4 and call(f, base, ws=P(0x30010), nbytes=BIG) == 4
    assert call(f, base, batch=0, rows=0, ws=W, nbytes=BIG) == 0
    refused(f, dict(base, ws=W, nbytes=BIG), 1, dict(batch=-1), dict(rows=1), dict(rows=2 ** 31 - 1),
            dict(vocab=0), dict(argmax=None), dict(drafts=None), dict(parent=None), dict(k=None),
            dict(accept=None), dict(tokens=None), dict(path=None))
    assert lib.spec_verify_tree_greedy_workspace_size(-1) == 0


def test_kv_commit_path(lib):
    desc = sv._KvCache(A, 4, 2, 16, 256, 2)
    f = lib.spec_kv_commit_path
    base = dict(cache=ctypes.byref(desc), spec=B_, slots=4, accept=A, k=A, path=A, rows=5, n=A,
                table=A, cols=2, stream=None, batch=2, ws=None, nbytes=0)
    assert call(f, base) == 4
    assert call(f, base, nbytes=lib.spec_kv_commit_workspace_size(2), ws=W) == 4   # a chain's size
    assert call(f, base, batch=0, rows=0, ws=W, nbytes=BIG) == 0
    refused(f, dict(base, ws=W, nbytes=BIG), 1, dict(path=None), dict(rows=1), dict(batch=-1),
            dict(slots=0), dict(accept=None), dict(k=None), dict(n=None), dict(table=None))
    assert lib.spec_kv_commit_path_workspace_size(-1) == 0


def test_kv_reserve(lib):
    f = lib.spec_kv_reserve
    base = dict(table=A, out=A, cols=4, held=A, out_held=A, length=A, free=A, out_free=A,
                capacity=9, count=A, out_count=A, page=16, stream=None, batch=2, ws=None, nbytes=0)
    assert call(f, base) == 4 and call(f, base, ws=P(0x30010), nbytes=BIG) == 4
    assert call(f, base, batch=0, ws=W, nbytes=BIG) == 0
    refused(f, dict(base, ws=W, nbytes=BIG), 1, dict(batch=-1), dict(cols=-1), dict(page=0),
            dict(capacity=-1), dict(capacity=2 ** 31 - 1), dict(table=None), dict(out=None),
            dict(held=None), dict(out_held=None), dict(length=None), dict(free=None),
            dict(out_free=None), dict(count=None), dict(out_count=None))
    assert lib.spec_kv_reserve_workspace_size(-1, 4) == 0
    assert lib.spec_kv_reserve_workspace_size(4, -1) == 0


def test_kv_slots(lib):
    f = lib.spec_kv_slots
    base = dict(table=A, cols=4, start=A, count=A, rows=5, page=16, slots=C, request=C, position=C,
                offsets=C, stream=None, batch=2, ws=None, nbytes=0)
    assert call(f, base) == 4 and call(f, base, ws=P(0x30010), nbytes=BIG) == 4
    refused(f, dict(base, ws=W, nbytes=BIG), 1, dict(batch=-1), dict(cols=-1), dict(page=0),
            dict(rows=-1), dict(rows=2 ** 31 - 1), dict(table=None), dict(start=None),
            dict(count=None), dict(slots=None), dict(request=None), dict(position=None),
            dict(offsets=None))
    refused(f, dict(base, ws=W, nbytes=BIG), 2, dict(slots=P(0x30004)))
    assert lib.spec_kv_slots_workspace_size(-1, 4) == 0
    assert lib.spec_kv_slots_workspace_size(4, -1) == 0


def test_kv_write(lib):
    f = lib.spec_kv_write

    def desc(data=A, pages=4, layers=2, S=16, E=256, es=2):
        return ctypes.byref(sv._KvCache(data, pages, layers, S, E, es))
    base = dict(cache=desc(), layer=0, Hk=2, k=A, kr=256, kh=128, v=A, vr=256, vh=128, slots=A,
                rows=3, stream=None, ws=None, nbytes=0)
    assert call(f, base, rows=0) == 0
    refused(f, base, 1, dict(layer=2), dict(layer=-1), dict(Hk=0), dict(Hk=3), dict(rows=-1),
            dict(rows=2 ** 31 - 1), dict(k=None), dict(v=None), dict(slots=None),
            dict(cache=desc(data=None)), dict(cache=desc(layers=0)), dict(cache=desc(S=0)),
            dict(cache=desc(pages=-1)), dict(cache=desc(E=0)), dict(cache=desc(es=1)))
    refused(f, base, 2, dict(k=P(0x10001)), dict(v=P(0x10001)), dict(slots=P(0x10004)),
            dict(cache=desc(data=P(0x10001))))
    assert lib.spec_kv_write_workspace_size(-1) == 0


def test_status_texts(lib):
    assert "tree" in sv.strerror(29) and "free pages" in sv.strerror(30)
    assert sv.ERROR_NAMES[29] == "SV_ERR_DATA_TREE" and sv.ERROR_NAMES[30] == "SV_ERR_DATA_POOL"


def test_binding_refuses_what_is_not_on_the_gpu(lib):
    i = torch.zeros(2, dtype=torch.int32)
    q, kv, cache = torch.zeros(1, 4, 32), torch.zeros(1, 2, 32), torch.zeros(2, 1, 2, 4, 64)
    for f in (lambda: sv.prompt_attention(q, kv, kv, i),
              lambda: sv.tree_attention(q, cache, 0, i, i[:, None], i, i, cache),
              lambda: sv.verify_tree_greedy(i, i, i, i, 10),
              lambda: sv.kv_reserve(i[:, None], i, i, i, i[:1], 16),
              lambda: sv.kv_slots(i[:, None], i, i, 4, 16),
              lambda: sv.kv_write(cache, 0, kv, kv, torch.zeros(1, dtype=torch.int64))):
        with pytest.raises(TypeError):
            f()
    with pytest.raises(ValueError):
        sv.tree_attention(q, cache, 0, i, i[:, None], i, i, None)
