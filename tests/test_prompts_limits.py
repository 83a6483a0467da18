"""Calls whose counts a 32-bit number would not hold are refused before the device is
touched (no GPU): sums that wrap could pass a check and be used as places."""

import ctypes

import pytest

import speculative_decoding_verification_13_gb300 as sv
from test_prompts_args import A, B_, C, call, lib, refused  # noqa: F401

MOST = (2 ** 31 - 1) // 64   # requests of 64 nodes


@pytest.mark.parametrize("batch,code", [(MOST, 4), (MOST + 1, 2), (2 ** 31 - 2, 2)])
def test_trees(lib, batch, code):  # noqa: F811
    desc = sv._KvCache(A, 4, 2, 16, 256, 2)
    rows = max(batch, 2 ** 30)
    assert lib.spec_verify_tree_greedy(A, A, A, A, C, C, C, None, batch, rows, 100, None, 0) == code
    assert lib.spec_tree_attention(ctypes.byref(desc), 1, 0, 2, A, 1024, 128, 8, rows, B_, 4, A, A,
                                   A, A, 2, 1.0, 0, C, C, None, batch, None, 0) == code
    assert lib.spec_kv_commit_path(ctypes.byref(desc), B_, 4, A, A, A, rows, A, A, 2, None, batch,
                                   None, 0) == code


def test_prompts(lib):  # noqa: F811
    f = lib.spec_prompt_attention
    base = dict(q=A, qr=1024, qh=64, k=A, kr=1024, kh=64, v=A, vr=1024, vh=64, dtype=1, rows=10,
                Hq=64, Hk=64, D=64, offsets=A, scale=1.0, window=0, out=C, lse=C, stream=None,
                batch=2 ** 24, ws=None, nbytes=0)
    assert call(f, base) == 4
    refused(f, base, 2, dict(batch=2 ** 25), dict(batch=2 ** 20, Hq=4096, Hk=4096),
            dict(batch=2 ** 31 - 2))
