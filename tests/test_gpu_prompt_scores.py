"""Attention over prompts and over trees where scores are large, fall or grow along the
sequence, so that the running maximum moves in most tiles, in some, or by less than a
rescaling takes; scales that leave a row one weight, that are negative or 0; products
that no 32-bit number holds.

Outputs and lse are compared with the oracle's in 64 bits, to the tolerances that the
headers of test_gpu_prompt.py and test_gpu_tree.py derive: they are relative to the
largest sum of |q k| scale of the row, which the oracle gives, so that they hold for any
scale while the error of a score, (D + 4) 2^-24 of that sum, stays small beside 1 (the
exponential of twice it is taken as 1 + that: at most 0.25 here, checked below, where
the square adds an eighth)."""

import math

import numpy as np
import pytest
import torch

import speculative_decoding_verification_13_gb300 as sv
from oracle import prompt as op
from test_gpu_prompt import check, gpu, i32, make
from test_gpu_tree import Case
from test_gpu_tree import check as check_tree

pytestmark = pytest.mark.gpu
DEV = "cuda"
B16, F16, F32 = torch.bfloat16, torch.float16, torch.float32


def small_errors(q, want):
    assert 2 * (q.shape[2] + 4) * 2.0 ** -24 * want[3].max() <= 0.25


@pytest.mark.parametrize("scale", [12.0, 3.0, -0.1, -3.0, 1e-6, 0.0])
@pytest.mark.parametrize("dtype,D,G", [(B16, 128, 2), (F16, 128, 4), (F16, 64, 3), (B16, 256, 2),
                                       (B16, 80, 1), (F32, 64, 2), (B16, 20, 2)])
def test_outputs_at_any_scale(dtype, D, G, scale):
    # products are of the order of 2 sqrt(D), the largest sum of |q k| of a row 1.7 D: at scale
    # 12 and D = 256 that is 5200, whose error is 0.08
    q, k, v, at = make(4 + D, [200, 140], 1, G, D, dtype)
    out, lse = sv.prompt_attention(*gpu(q, k, v), i32(at), scale=scale)
    assert sv.prompt_attention_error() == (0, -1, -1)
    want = op.prompt_attention(q, k, v, at, scale=scale, magnitude=True)
    small_errors(q, want)
    check(q, at, out, lse, want)


def ramp(kind, n):
    """A score's part that all queries have in common, by the key's place."""
    x = torch.arange(n, dtype=torch.float64)
    return {"grows": x / 2,                    # 64 a tile of 128: rescaled in every tile
            "falls": -x / 2,
            "slowly": x / 40,                  # 3.2 a tile, 4.6 binary: in every other one
            "jumps": (x >= 500) * 70.0 + (x >= 640) * 5.0 + (x >= 800) * 4.0,
            "waves": 60 * torch.sin(x / 50)}[kind]


@pytest.mark.parametrize("kind", ["grows", "falls", "slowly", "jumps", "waves"])
@pytest.mark.parametrize("dtype,D,G,window", [(B16, 128, 2, 0), (F16, 128, 1, 0), (F16, 64, 4, 300),
                                              (B16, 256, 1, 0), (F16, 256, 2, 200), (F32, 64, 2, 0),
                                              (B16, 144, 3, 0)])
def test_maxima_that_move(kind, dtype, D, G, window):
    lengths = [900, 300]
    q, k, v, at = (x.clone() if torch.is_tensor(x) else x for x in make(D, lengths, 1, G, D, dtype))
    # column 0 carries the common part: q holds 8, k the rest of it at scale 1 / 8
    q[:, :, 0] = 8
    for a, n in zip(at, lengths):
        k[a:a + n, 0, 0] = ramp(kind, n).to(dtype)
    out, lse = sv.prompt_attention(*gpu(q, k, v), i32(at), scale=0.125, window=window)
    assert sv.prompt_attention_error() == (0, -1, -1)
    want = op.prompt_attention(q, k, v, at, scale=0.125, window=window, magnitude=True)
    small_errors(q, want)
    check(q, at, out, lse, want)


@pytest.mark.parametrize("kind", ["grows", "falls", "slowly", "jumps"])
@pytest.mark.parametrize("k,D,G,dtype", [([63, 40], 128, 4, B16), ([63, 50], 64, 4, F16),
                                         ([5, 0], 128, 2, F16), ([30, 9], 256, 1, B16),
                                         ([20, 3], 64, 2, F32)])
def test_maxima_that_move_over_the_cache(kind, k, D, G, dtype):
    n = [900, 333]
    c = Case(D + len(kind), n, k, 1, G, D, 16, dtype)
    c.q[:, :, 0] = 8
    for b in range(2):
        values = ramp(kind, n[b] + k[b] + 1).to(dtype)
        for p in range(n[b]):
            c.cache[c.table[b, p // 16], c.layer, 0, p % 16, 0] = values[p]
        c.spec[b, :k[b] + 1, c.layer, 0, 0] = values[n[b]:]
    out, lse = c.run(scale=0.125)
    assert sv.tree_attention_error() == (0, -1, -1)
    want = c.oracle(scale=0.125)
    small_errors(c.q, want)
    check_tree(c, out, lse, want)


@pytest.mark.parametrize("how", ["product", "key"])
@pytest.mark.parametrize("dtype,D,G", [(B16, 128, 2), (B16, 64, 4), (B16, 256, 1), (B16, 80, 2),
                                       (F32, 64, 2), (F32, 20, 1), (B16, 20, 2)])
def test_products_that_no_number_holds(dtype, D, G, how):
    # column 0 of q holds 1e20 and of k 0, but for two keys: one product is -1e40 or that of
    # an infinite key, its position weighs nothing; the other +1e40, its rows are NaN
    low, high = 150, 333
    q, k, v, at = (x.clone() if torch.is_tensor(x) else x
                   for x in make(D, [400, 170], 1, G, D, dtype))
    q[:, :, 0], k[:, :, 0] = 1e20, 0
    k[low, 0, 0], k[high, 0, 0] = (-1e20, 1e20) if how == "product" else (-math.inf, math.inf)
    out, lse = sv.prompt_attention(*gpu(q, k, v), i32(at))
    assert sv.prompt_attention_error() == (0, -1, -1)
    assert torch.isnan(out[high:400]).all() and torch.isnan(lse[high:400]).all()
    # the others as without the two positions: the oracle over the rest of the rows
    q[:, :, 0] = k[:, :, 0] = 0
    keep = [i for i in range(570) if i != low and not high <= i < 400]
    part = [x[keep] for x in (q, k, v)]
    ends = [0, high - 1, high - 1 + 170]
    want = op.prompt_attention(*part, ends, magnitude=True)
    check(part[0], ends, out[keep], lse[keep], want)
