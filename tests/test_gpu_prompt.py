"""Attention over packed prompts on the GPU against the oracle (oracle/prompt.py).

Tolerances.  A score is a sum of D products in 32 bits: its error is at most
e_s = (D + 4) 2^-24 sum |q k| scale, and the exponential adds 2^-21 of itself.  A
weight is off by that factor twice (score and maximum or sum), plus half a step of
the type where it is rounded for the product with v; the weighted sum of n values
adds n 2^-24; the result is rounded once.  Errors of `out` are relative to
sum w |v|, which the oracle gives."""

import math

import numpy as np
import pytest
import torch

import speculative_decoding_verification_13_gb300 as sv
from oracle import prompt as op

pytestmark = pytest.mark.gpu
DEV = "cuda"
B16, F16, F32 = torch.bfloat16, torch.float16, torch.float32


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def make(seed, lengths, Hk, G, D, dtype, before=0, behind=0):
    """q, k, v as slices of one projection (CPU), and offsets."""
    g = torch.Generator().manual_seed(seed)
    Hq = Hk * G
    qkv = torch.randn(before + sum(lengths) + behind, Hq + 2 * Hk, D, generator=g)
    qkv[:, :Hq] *= 2
    qkv = qkv.to(dtype)
    at = [before]
    for x in lengths:
        at.append(at[-1] + x)
    return qkv[:, :Hq], qkv[:, Hq:Hq + Hk], qkv[:, Hq + Hk:], at


def gpu(q, k, v):
    """The same slices on the GPU, of one tensor."""
    return torch.cat([q, k, v], 1).to(DEV).split([q.shape[1], k.shape[1], v.shape[1]], 1)


def check(q, at, out, lse, want):
    o, l, mag, size = want
    rows = slice(at[0], at[-1])
    out, lse = out.double().cpu().numpy()[rows], lse.double().cpu().numpy()[rows]
    o, l, mag, size = o[rows], l[rows], mag[rows], size[rows]
    D, keys = q.shape[2], max([1] + [b - a for a, b in zip(at, at[1:])])
    half = torch.finfo(q.dtype).eps / 2
    e_s = (D + 4) * 2.0 ** -24 * size + 2.0 ** -21
    weight = 2 * e_s + (half if half > 2.0 ** -20 else 0) + (keys + 8) * 2.0 ** -24
    tol = weight[..., None] * mag + half * (np.abs(o) + weight[..., None] * mag)
    assert (np.abs(out - o) <= tol + 1e-30).all(), np.max(np.abs(out - o) / (tol + 1e-30))
    tl = e_s + (keys + 8) * 2.0 ** -24 + 2.0 ** -23 * np.abs(l)
    assert (np.abs(lse - l) <= tl).all(), np.max(np.abs(lse - l) / tl)


CASES = [
    # lengths, KV heads, group, head, type, window
    ([1], 1, 1, 128, B16, 0),
    ([5, 0, 1, 130], 2, 4, 128, B16, 0),
    ([64, 128, 127, 129], 1, 4, 128, B16, 0),
    ([300, 1, 1, 1, 33], 2, 1, 128, B16, 0),                 # whole tiles without a mask
    ([257, 511], 1, 2, 128, F16, 0),
    ([140, 63], 2, 7, 128, B16, 0),                          # 126 rows a tile
    ([200], 1, 16, 64, B16, 0),
    ([90, 280, 3], 2, 4, 64, F16, 0),
    ([200, 70], 2, 4, 256, B16, 0),
    ([129, 31, 260], 1, 8, 256, F16, 0),
    ([260, 64], 1, 1, 256, B16, 100),
    ([150, 77], 2, 4, 80, B16, 0),                           # between 64, 128 and 256
    ([66, 130], 1, 3, 72, F16, 0),
    ([131], 2, 2, 144, B16, 0),
    ([100, 40], 1, 5, 40, F16, 0),
    ([60, 9], 2, 2, 8, B16, 0),
    ([400, 90, 2], 1, 4, 128, B16, 1),
    ([400, 90, 2], 1, 4, 128, B16, 70),
    ([500, 300], 1, 1, 128, B16, 129),
    ([300, 40], 2, 2, 64, F16, 200),
    ([40, 20], 1, 130, 64, B16, 0),                          # more heads than a tile has rows
    ([3, 5], 1, 128, 64, B16, 0),
    ([70, 0, 9, 64], 2, 3, 64, F32, 0),
    ([130, 20], 1, 2, 128, F32, 33),
    ([65], 1, 4, 256, F32, 0),
    ([50, 7], 2, 2, 12, F32, 0),
    ([70, 9], 1, 4, 20, B16, 0),                             # heads that do not lie on 16 bytes
    ([33, 64], 2, 1, 7, F16, 5),
    ([1] * 40 + [200] + [2] * 30, 2, 4, 128, B16, 0),        # more than 32 sequences
]


@pytest.mark.parametrize("case", CASES, ids=range(len(CASES)))
def test_prompt_attention_matches_oracle(case):
    lengths, Hk, G, D, dtype, window = case
    q, k, v, at = make(sum(lengths) + D, lengths, Hk, G, D, dtype)
    out, lse = sv.prompt_attention(*gpu(q, k, v), i32(at), window=window)
    assert sv.prompt_attention_error() == (0, -1, -1)
    check(q, at, out, lse, op.prompt_attention(q, k, v, at, window=window, magnitude=True))


@pytest.mark.parametrize("dtype,D", [(B16, 128), (B16, 20), (F32, 64)])
def test_rows_of_no_sequence_are_left_alone(dtype, D):
    q, k, v, at = make(3, [40, 100], 2, 4, D, dtype, before=5, behind=90)
    for x in (q, k, v):
        x[:5] = math.nan
        x[at[-1]:] = math.inf
    out, lse = torch.full(q.shape, 7, dtype=dtype, device=DEV), torch.full(q.shape[:2], 7.0).to(DEV)
    got = sv.prompt_attention(*gpu(q, k, v), i32(at), out=out, out_lse=lse)
    assert got[0] is out and got[1] is lse
    check(q, at, out, lse, op.prompt_attention(q, k, v, at, magnitude=True))
    for x in (out, lse):
        assert (x[:5] == 7).all() and (x[at[-1]:] == 7).all()


@pytest.mark.parametrize("dtype,D", [(B16, 128), (F16, 64), (B16, 256), (B16, 20), (F32, 64)])
def test_infinite_and_nan_values_reach_those_that_see_them(dtype, D):
    lengths, G, W = [300, 150], 2, 200
    q, k, v, at = make(9, lengths, 1, G, D, dtype)
    v[10, 0, 3], v[130, 0, 5], v[290, 0, 1], v[135, 0, 5] = math.inf, -math.inf, math.nan, math.inf
    v[300, 0, 2], k[449, 0, :] = math.nan, math.nan      # another sequence; the last token's key
    out, lse = sv.prompt_attention(*gpu(q, k, v), i32(at), window=W)
    out = out.float().cpu().numpy()
    clean = v.clone()
    clean[~torch.isfinite(clean)] = 0
    want, _ = op.prompt_attention(q, k, clean, at, window=W)
    for i in range(450):
        a = at[0] if i < 300 else at[1]
        see = range(max(a, i - W + 1), i + 1)
        for d in range(6):
            bad = [float(v[j, 0, d]) for j in see if not math.isfinite(v[j, 0, d])]
            for h in range(G):
                x = out[i, h, d]
                if i == 449:
                    assert math.isnan(x)
                elif not bad:
                    assert abs(x - want[i, h, d]) < 0.1, (i, h, d)
                elif len(set(bad)) == 1 and not math.isnan(bad[0]):
                    assert x == bad[0], (i, h, d)
                else:
                    assert math.isnan(x), (i, h, d)


def test_scores_of_any_size():
    # scales that make one weight of each row, and infinite products
    q, k, v, at = make(4, [200, 140], 1, 2, 128, B16)
    args = gpu(q, k, v)
    out, lse = sv.prompt_attention(*args, i32(at), scale=30.0)
    o, l = op.prompt_attention(q, k, v, at, scale=30.0)
    size = 30 * (q.double().abs() @ k[:, 0].double().abs().T.unsqueeze(0)).amax()
    assert np.abs(lse.double().cpu().numpy() - l).max() <= 132 * 2.0 ** -24 * float(size) + 1e-3
    out, lse = sv.prompt_attention(*args, i32(at), scale=0.0)      # all weights alike
    o, l = op.prompt_attention(q, k, v, at, scale=0.0)
    assert np.abs(out.double().cpu().numpy() - o).max() < 2.0 ** -7 * np.abs(o).max()
    out, lse = sv.prompt_attention(*args, i32(at), scale=-0.1)
    o, l = op.prompt_attention(q, k, v, at, scale=-0.1)
    assert np.abs(lse.double().cpu().numpy() - l).max() < 1e-4


@pytest.mark.parametrize("how", ["heads first", "k and v alike", "unaligned", "wide rows"])
def test_strides_are_free(how):
    lengths = [70, 129, 3]
    q, k, v, at = make(6, lengths, 2, 4, 128, B16)
    T = q.shape[0]
    if how == "heads first":
        a = [x.transpose(0, 1).contiguous().to(DEV).transpose(0, 1) for x in (q, k, v)]
    elif how == "k and v alike":
        v = k
        kd = k.to(DEV)
        a = [q.to(DEV), kd, kd]
    elif how == "unaligned":
        a = []
        for x in (q, k, v):
            flat = torch.zeros(x.numel() + 1, dtype=B16, device=DEV)
            flat[1:] = x.reshape(-1).to(DEV)
            a.append(flat[1:].view(x.shape))
    else:
        a = []
        for x in (q, k, v):
            wide = torch.full((T, x.shape[1], 131), math.nan, dtype=B16, device=DEV)
            wide[:, :, :128] = x.to(DEV)
            a.append(wide[:, :, :128])
    out, lse = sv.prompt_attention(*a, i32(at))
    check(q, at, out, lse, op.prompt_attention(q, k, v, at, magnitude=True))


def test_heads_that_share_keys_and_one_row():
    q, k, v, at = make(8, [1], 1, 8, 128, B16)
    out, lse = sv.prompt_attention(*gpu(q, k, v), i32(at))
    assert torch.equal(out.cpu(), v.expand(1, 8, 128))   # its own value alone


@pytest.mark.parametrize("dtype,D", [(B16, 128), (F32, 64)])
@pytest.mark.parametrize("bad", [[0, 50, 40, 90], [-1, 20, 90], [0, 20, 91], [0, 95, 90]])
def test_bad_offsets_fail_the_batch(dtype, D, bad):
    q, k, v, _ = make(5, [90], 2, 2, D, dtype)
    out, lse = sv.prompt_attention(*gpu(q, k, v), i32(bad))
    assert sv.prompt_attention_error() == (21, -1, -1)
    assert torch.isnan(out).all() and torch.isnan(lse).all()
    sv.prompt_attention(*gpu(q, k, v), i32([0, 90]))
    assert sv.prompt_attention_error() == (0, -1, -1)


def test_empty_calls():
    q, k, v, _ = make(5, [4], 2, 2, 64, B16)
    a = gpu(q, k, v)
    out = torch.full(q.shape, 3, dtype=B16, device=DEV)
    sv.prompt_attention(*a, i32([0]), out=out)                    # no sequence
    sv.prompt_attention(*a, i32([2, 2, 2]), out=out)              # empty ones
    assert (out == 3).all() and sv.prompt_attention_error() == (0, -1, -1)
    sv.prompt_attention(*[x[:0] for x in a], i32([0, 0]))
    assert sv.prompt_attention_error() == (0, -1, -1)


def test_long_sequences_repeat_bit_for_bit_and_in_a_graph():
    lengths = [2100, 1, 700]
    q, k, v, at = make(11, lengths, 2, 4, 128, B16)
    a, o = gpu(q, k, v), i32(at)
    first = sv.prompt_attention(*a, o)
    # a sample of rows against the oracle of their own
    for i in (0, 127, 128, 1000, 2099):
        want = op.prompt_attention(q[i:i + 1], k[i:i + 1], v[i:i + 1], [0, 1])
        s = (k[:i + 1, 1].double() @ q[i, 5].double()) * 128 ** -0.5
        w = torch.softmax(s, 0)
        got = first[0][i, 5].double().cpu()
        mag = w @ v[:i + 1, 1].double().abs()
        assert ((got - w @ v[:i + 1, 1].double()).abs() <= 2.0 ** -7 * mag + 1e-3 * mag).all()
        assert abs(float(first[1][i, 5]) - float(torch.logsumexp(s, 0))) < 1e-4
        assert want[0].shape == (1, 8, 128)
    second = sv.prompt_attention(*a, o)
    assert torch.equal(first[0], second[0]) and torch.equal(first[1], second[1])
    out, lse = torch.empty_like(first[0]), torch.empty_like(first[1])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        sv.prompt_attention(*a, o, out=out, out_lse=lse)
    for _ in range(2):
        out.zero_()
        sv.prompt_attention(*a, i32([0, 2801]))      # the stream's own workspace in between
        g.replay()
        assert torch.equal(first[0], out) and torch.equal(first[1], lse)


def test_another_stream():
    q, k, v, at = make(12, [300, 20], 2, 4, 128, B16)
    a, o = gpu(q, k, v), i32(at)
    want = sv.prompt_attention(*a, o)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = sv.prompt_attention(*a, o, stream=side)
    side.synchronize()
    assert torch.equal(want[0], got[0]) and torch.equal(want[1], got[1])
    assert sv.prompt_attention_error() == (0, -1, -1)


@pytest.mark.parametrize("D,Hk,G,window", [(128, 8, 4, 0), (64, 1, 7, 50), (256, 2, 2, 0)])
def test_hundreds_of_sequences(D, Hk, G, window):
    # every CTA has units of many sequences and of several lengths
    rng = np.random.default_rng(D)
    lengths = rng.integers(0, 60, 700).tolist()
    lengths[13], lengths[600] = 1500, 300
    q, k, v, at = make(1, lengths, Hk, G, D, B16)
    a = gpu(q, k, v)
    out, lse = sv.prompt_attention(*a, i32(at), window=window)
    assert sv.prompt_attention_error() == (0, -1, -1)
    want, mag = torch.empty(q.shape, dtype=torch.float64), torch.empty(q.shape, dtype=torch.float64)
    ref = torch.empty(q.shape[:2], dtype=torch.float64)
    for lo, hi in zip(at, at[1:]):
        x, K, V = (y[lo:hi].double() for y in (q, k, v))
        s = torch.einsum("ihgd,jhd->hgij", x.unflatten(1, (Hk, G)), K) * D ** -0.5
        i = torch.arange(hi - lo)
        see = (i[None] <= i[:, None]) & ((i[None] > i[:, None] - window) if window else True)
        s = s.masked_fill(~see, -math.inf)
        w = torch.softmax(s, -1)
        want[lo:hi] = torch.einsum("hgij,jhd->ihgd", w, V).flatten(1, 2)
        mag[lo:hi] = torch.einsum("hgij,jhd->ihgd", w, V.abs()).flatten(1, 2)
        ref[lo:hi] = torch.logsumexp(s, -1).permute(2, 0, 1).flatten(1)
    # a score is at most 60 here: e_s (D + 4) 2^-24 60 + 2^-21 at most 1e-3; a weight's half step
    weight = 2e-3 + 2.0 ** -8
    err = (out.double().cpu() - want).abs()
    assert (err <= weight * mag + 2.0 ** -8 * (want.abs() + weight * mag) + 1e-30).all()
    assert ((lse.double().cpu() - ref).abs() <= 1e-3 + 2.0 ** -20 * ref.abs()).all()
