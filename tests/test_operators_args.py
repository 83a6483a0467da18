"""Refusals of the attention, eviction and log-probability calls (no GPU): the
C entry points reject bad arguments before touching the device, the binding
rejects tensors that do not fit."""

import ctypes
import os
import re

import pytest
import torch

import speculative_decoding_verification_13_gb300 as sv
from speculative_decoding_verification_13_gb300 import build as cuda_build
from speculative_decoding_verification_13_gb300 import operators as ops

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
P = ctypes.c_void_p
A, B_, C = P(0x10000), P(0x20000), P(0x30000)  # never dereferenced


@pytest.fixture(scope="module")
def lib():
    cuda_build.build()
    return ops._library()


def test_every_entry_point_of_the_header_is_exported(lib):
    src = open(os.path.join(ROOT, "include", "specverify.h")).read()
    src = re.sub(r"/\*.*?\*/", "", src, flags=re.S)
    names = set(re.findall(r"\b(spec_\w+)\s*\(", src))
    assert set(ops._SIGNATURES) <= names
    for name in names:
        assert hasattr(lib, name), name


def desc(data=A, pages=4, layers=2, S=16, E=256, es=2):
    return sv._KvCache(data, pages, layers, S, E, es)


def attention(lib, d=None, **kw):
    a = dict(dtype=1, layer=0, kv_heads=2, q=A, qts=1024, qhs=128, q_heads=8, rows=3, spec=B_,
             slots=4, k=A, n=A, table=A, cols=2, scale=1.0, window=0, out=C, lse=C, batch=1,
             ws=None, nbytes=0)
    a.update(kw)
    d = desc() if d is None else d
    return lib.spec_attention(ctypes.byref(d), a["dtype"], a["layer"], a["kv_heads"], a["q"],
                              a["qts"], a["qhs"], a["q_heads"], a["rows"], a["spec"], a["slots"],
                              a["k"], a["n"], a["table"], a["cols"], a["scale"], a["window"],
                              a["out"], a["lse"], None, a["batch"], a["ws"], a["nbytes"])


def test_attention_argument_errors(lib):
    assert attention(lib) == 4                                # all fine but the workspace
    assert attention(lib, ws=P(0x30010), nbytes=1 << 40) == 4
    assert attention(lib, batch=0, rows=0) == 0
    for kw in (dict(layer=2), dict(layer=-1), dict(kv_heads=0), dict(kv_heads=3),
               dict(q_heads=7), dict(q_heads=0), dict(rows=0), dict(rows=1 << 31), dict(batch=-1),
               dict(batch=0), dict(window=-1), dict(scale=float("nan")),
               dict(scale=float("inf")), dict(cols=-1), dict(slots=0), dict(q=None), dict(k=None),
               dict(n=None), dict(table=None), dict(out=None), dict(lse=None), dict(dtype=0)):
        assert attention(lib, **kw) == 1, kw
    for d in (desc(layers=0), desc(S=0), desc(pages=-1), desc(E=0), desc(data=None)):
        assert attention(lib, d) == 1
    assert attention(lib, dtype=7) == 2
    assert attention(lib, desc(E=1024)) == 2                  # heads of 512
    assert attention(lib, desc(E=24)) == 2                    # heads of 24 bytes
    assert attention(lib, desc(data=P(0x10008))) == 2
    assert attention(lib, spec=P(0x10008)) == 2


def test_attention_weights_argument_errors(lib):
    def call(score=A, ss=64, out=C, os_=64, cols=64, batch=2, rows=3, lse=A):
        d = desc()
        return lib.spec_attention_weights(ctypes.byref(d), 1, 0, 2, A, 1024, 128, 8, rows, B_, 4,
                                          A, A, A, 2, 1.0, 0, lse, None, score, ss, out, os_, cols,
                                          None, batch, None, 0)
    assert call() == 4
    assert call(batch=0, rows=0) == 0
    assert call(score=None) == 1 and call(out=None) == 1 and call(lse=None) == 1
    assert call(ss=63) == 1 and call(os_=63) == 1 and call(cols=-1) == 1
    assert call(out=A, os_=80) == 1                           # one buffer, two strides


def test_evict_argument_errors(lib):
    def call(d=None, dst=None, **kw):
        a = dict(table=A, cols=4, dt=None, dcols=0, score=A, ss=64, sc=64, out=A, os_=64, oc=64,
                 n=A, m=A, budget=8, sinks=1, recent=2, batch=2, ws=P(0x40000), nbytes=1 << 30)
        a.update(kw)
        d = desc() if d is None else d
        return lib.spec_kv_evict(ctypes.byref(d), a["table"], a["cols"],
                                 ctypes.byref(dst) if dst is not None else None, a["dt"],
                                 a["dcols"], a["score"], a["ss"], a["sc"], a["out"], a["os_"],
                                 a["oc"], a["n"], a["m"], a["budget"], a["sinks"], a["recent"],
                                 None, None, a["batch"], a["ws"], a["nbytes"])
    assert call(batch=0) == 0
    for kw in (dict(budget=0), dict(sinks=-1), dict(recent=-1), dict(sinks=7), dict(batch=-1),
               dict(sc=-1), dict(ss=63), dict(out=C, os_=63), dict(os_=80), dict(cols=-1),
               dict(n=None), dict(m=None), dict(table=None), dict(score=None), dict(out=None)):
        assert call(**kw) == 1, kw
    assert call(ws=None) == 4 and call(ws=P(0x40010)) == 4 and call(nbytes=64) == 4
    assert call(batch=65536) == 2
    assert call(desc(E=4)) == 2 and call(desc(data=P(0x10008))) == 2
    assert call(dst=desc(layers=3), dt=A, dcols=4) == 1
    assert call(dst=desc(S=8), dt=A, dcols=4) == 1
    assert call(dst=desc(), dt=None, dcols=4) == 1
    assert call(dst=desc(data=P(0x10008)), dt=A, dcols=4) == 2
    assert lib.spec_kv_evict_workspace_size(-1, 8) == 0
    assert lib.spec_kv_evict_workspace_size(4, 0) == 0


def test_logprobs_argument_errors(lib):
    def call(x, n_top=0, ws=P(0x40000), nbytes=1 << 30, tok=None, top=None):
        return lib.spec_logprobs(ctypes.byref(x), A, None, n_top, C, C, C, C, tok, top, None, ws,
                                 nbytes)
    L = sv._Logits
    assert call(L(None, 1, 100, 0, 100)) == 0
    assert call(L(A, 7, 100, 4, 100)) == 2 and call(L(A, 2, 100, 4, 100)) == 2
    assert call(L(A, 1, 0, 4, 100)) == 1 and call(L(A, 1, 100, -1, 100)) == 1
    assert call(L(A, 1, 100, 4, 99)) == 1 and call(L(A, 1, 100, 4, 0)) == 1
    assert call(L(None, 1, 100, 4, 100)) == 1
    assert call(L(A, 1, (1 << 22) + 1, 1, 1 << 23)) == 2
    assert call(L(P(0x10001), 1, 100, 4, 100)) == 2
    assert call(L(P(0x10002), 0, 100, 4, 100)) == 2
    assert call(L(A, 1, 100, 4, 100), n_top=33) == 2 and call(L(A, 1, 100, 4, 100), n_top=-1) == 1
    assert call(L(A, 1, 100, 4, 100), n_top=3) == 1
    assert call(L(A, 1, 100, 4, 100), ws=None) == 4 and call(L(A, 1, 100, 4, 100), nbytes=8) == 4
    assert lib.spec_logprobs_workspace_size(-1) == 0

    def grad(x, tokens=A, m=A, ls=A, ent=A, gl=A, gh=A, out=C, stride=100):
        return lib.spec_logprobs_grad(ctypes.byref(x), tokens, None, m, ls, ent, gl, gh, out,
                                      stride, None)
    x = L(A, 1, 100, 4, 100)
    assert grad(L(None, 1, 100, 0, 100)) == 0
    for kw in (dict(tokens=None), dict(m=None), dict(ls=None), dict(ent=None), dict(out=None),
               dict(stride=99), dict(out=A, stride=104)):
        assert grad(x, **kw) == 1, kw
    assert grad(x, out=P(0x30001)) == 2


def test_binding_refuses_what_is_not_on_the_gpu(lib):
    i = torch.zeros(1, dtype=torch.int32)
    cache = torch.zeros(2, 1, 2, 4, 64)
    with pytest.raises(TypeError):
        sv.attention(torch.zeros(1, 2, 32), cache, 0, i, i[:, None], i)
    with pytest.raises(TypeError):
        sv.attention_weights(torch.zeros(1, 2, 32), cache, 0, i, i[:, None], i, None, None)
    with pytest.raises(TypeError):
        sv.kv_evict(cache, torch.zeros(1, 4), i, i[:, None], 2)
    with pytest.raises(TypeError):
        sv.logprobs(torch.zeros(1, 8), i)
    with pytest.raises(TypeError):
        sv.logprobs_grad(torch.zeros(1, 8), i, None, None, None, None)
