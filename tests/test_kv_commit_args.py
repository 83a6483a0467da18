"""Refusals of kv_commit's binding (no GPU: tensors of the host pass for the GPU's, and
a stand-in for the library): the kernels read and write as many entries as the batch
has requests, whatever the tensors hold."""

import types

import pytest
import torch

import speculative_decoding_verification_13_gb300 as sv
from test_kv_commit_workspaces import lib  # noqa: F401


def arguments(B=3):
    i = torch.zeros(B, dtype=torch.int32)
    return dict(cache=torch.zeros(2, 1, 2, 4, 8), spec=torch.zeros(B, 2, 1, 2, 8), accept_len=i,
                k_per_req=i, kv_len=i.clone(), block_table=torch.zeros(B, 2, dtype=torch.int32),
                stream=types.SimpleNamespace(cuda_stream=7))


@pytest.mark.parametrize("path", [False, True])
def test_tensors_that_are_shorter_than_the_batch(lib, path):  # noqa: F811
    more = dict(path=torch.zeros(3, dtype=torch.int32)) if path else {}
    sv.kv_commit(**arguments(), **more)
    assert len(lib.calls) == 1
    for name in ("accept_len", "k_per_req", "kv_len", "block_table"):
        a = arguments()
        with pytest.raises(ValueError, match=name):
            sv.kv_commit(**{**a, name: a[name][:2]}, **more)
        longer = torch.cat([a[name], a[name]])
        sv.kv_commit(**{**a, name: longer}, **more)
    assert len(lib.calls) == 5


def test_what_is_missing_or_on_the_host(lib, monkeypatch):  # noqa: F811
    for name in ("accept_len", "k_per_req", "kv_len"):
        with pytest.raises(ValueError, match=name):
            sv.kv_commit(**{**arguments(), name: None})
    monkeypatch.setattr(torch.Tensor, "is_cuda", False)
    with pytest.raises(TypeError):
        sv.kv_commit(**arguments())
    assert not lib.calls


def test_a_table_of_no_page_may_be_left_out(lib):  # noqa: F811
    sv.kv_commit(**{**arguments(), "block_table": None})
    assert len(lib.calls) == 1
