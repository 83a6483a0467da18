"""Log probabilities, entropy, alternatives and the gradient on the GPU against
the oracle (oracle/logprobs.py).

Tolerances.  y = (x - m) / T is rounded three times (difference, scale, log2
units): 4 2^-24 |y|; an exponential adds 2^-21 of itself; a thread adds V / 256
terms in 32 bits.  With M = sum p |y| these give the bounds of `bounds`."""

import math

import numpy as np
import pytest
import torch

import speculative_decoding_verification_13_gb300 as sv
from oracle import logprobs as ol

pytestmark = pytest.mark.gpu
DEV = "cuda"
E = 2.0 ** -24


def bounds(lp, ls, p):
    V = len(p)
    y = np.where(p > 0, lp + ls, 0.0)
    M = (p * np.abs(y)).sum()
    adds = (V / 256 + 64) * E
    t_ls = 4 * E * M + 2.0 ** -21 + adds + 2 * E * abs(ls)
    t_h = t_ls * (1 + M) + (p * np.abs(y) * (4 * E * np.abs(y) + 2.0 ** -21)).sum() + adds * M + 1e-7
    return t_ls, t_h


def logits(seed, R, V, dtype, pad=0, spread=2.5):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(R, V + pad, generator=g) * spread).to(dtype)[:, :V]


def compare(x, tok, T, n_top, r):
    x = x.double().cpu().numpy()
    for i in range(len(x)):
        t = int(tok[i])
        if t == -1:
            assert all(torch.isnan(v[i]) for v in (r.logprob, r.entropy, r.max, r.logsum))
            continue
        Ti = 0 if T is None else float(T[i])
        lp, H, m, ls, wt, wl, lps, p = ol.row(x[i], t, Ti, n_top)
        t_ls, t_h = bounds(lps, ls, p)
        with np.errstate(over="ignore"):  # what 32 bits cannot hold is infinite in them
            lp, wl = float(np.float32(lp)), wl.astype(np.float32).astype(np.float64)
        assert float(r.max[i]) == m
        assert abs(float(r.logsum[i]) - ls) <= t_ls
        assert abs(float(r.entropy[i]) - H) <= t_h
        got = float(r.logprob[i])
        assert got == lp if math.isinf(lp) else abs(got - lp) <= t_ls + 5 * E * (abs(lp) + ls)
        if n_top:
            assert r.top_tokens[i].tolist() == wt.tolist()
            got = r.top_logprobs[i].double().cpu().numpy()
            f = np.isfinite(wl)
            assert (got[~f] == wl[~f]).all()
            assert (np.abs(got[f] - wl[f]) <= t_ls + 5 * E * (np.abs(wl[f]) + ls)).all()


def run(x, tok, T=None, n_top=0):
    d = x.to(DEV) if not x.is_cuda else x
    r = sv.logprobs(d, tok.to(DEV), None if T is None else T.to(DEV), n_top)
    assert sv.logprobs_error()[0] == 0
    compare(x, tok, T, n_top, r)
    return r


B16, F32 = torch.bfloat16, torch.float32


@pytest.mark.parametrize("R,V,dtype,pad,n_top,temps", [
    (1, 1, F32, 0, 1, False), (3, 2, B16, 0, 5, True), (2, 7, B16, 3, 32, False),
    (5, 31, F32, 1, 32, True), (4, 257, B16, 1, 20, False), (6, 1000, F32, 0, 5, True),
    (3, 4099, B16, 2, 32, True), (2, 32000, F32, 0, 0, False), (3, 50257, B16, 0, 20, True),
    (2, 50257, F32, 0, 1, True), (3, 151936, B16, 0, 20, False), (40, 151936, B16, 8, 32, True),
    (1, 400003, F32, 0, 20, False),
])
def test_logprobs_match_oracle(R, V, dtype, pad, n_top, temps):
    g = torch.Generator().manual_seed(V)
    x = logits(V + R, R, V, dtype, pad)
    tok = torch.randint(0, V, (R,), generator=g, dtype=torch.int32)
    tok[R // 2] = 0
    tok[-1] = V - 1
    if R > 3:
        tok[1] = -1
    T = torch.rand(R, generator=g) + 0.3 if temps else None
    if temps:
        T[0] = 0.0
    if R > 8:
        x = x[:9].clone()
        tok, T = tok[:9], None if T is None else T[:9]
    run(x.to(DEV) if R > 8 else x, tok, T, n_top)


@pytest.mark.parametrize("dtype", [F32, B16])
def test_rows_at_every_element_offset(dtype):
    V = 3001
    buf = logits(1, 1, 16 * (V + 40), dtype)[0].to(DEV)
    tok = torch.tensor([5], dtype=torch.int32)
    for off in range(9):
        x = buf[off:off + V][None]
        run(x, tok, None, 7)
    x = buf[1:1 + 16 * (V + 2)].view(16, V + 2)[:, :V]   # rows at alternating offsets
    run(x, torch.arange(16, dtype=torch.int32) * 100, None, 20)


@pytest.mark.parametrize("dtype", [F32, B16])
@pytest.mark.parametrize("V", [300, 5000, 70001])
def test_masks_ties_and_extremes(dtype, V):
    low = torch.finfo(dtype).min
    tok = torch.tensor([0, 1, 2, 3, 4, 5, 6, 7, 8], dtype=torch.int32)
    x = logits(V, 9, V, dtype)
    x[0] = 0.0                                   # a uniform row: all ties
    x[1] = low                                   # the type's lowest value everywhere
    x[2] = low
    x[2, 17:20] = 1.0                            # masked by it but for three
    x[3] = -math.inf
    x[3, [3, 40, V - 1]] = torch.tensor([1.0, 2.0, 2.0]).to(dtype)  # three tokens left
    x[4, ::2] = -math.inf
    x[5] = torch.linspace(-30, 30, V).to(dtype)  # rising: late maxima
    x[6] = torch.linspace(30, -30, V).to(dtype)
    x[7] = (x[7] * 2).round()                    # long ties below the top
    x[8] = 60000.0
    x[8, V // 2] = 60032.0 if dtype == F32 else 60416.0
    run(x, tok, None, 20)
    run(x, tok, torch.full((9,), 0.25), 32)


@pytest.mark.parametrize("R,V,dtype,n_top", [(4096, 98304, B16, 20), (3000, 50001, F32, 32)])
def test_many_waves_of_rows_repeat_bit_for_bit(R, V, dtype, n_top):
    """Far more rows than run at a time: rows that start while others end.  A call
    repeats to the bit, and every row's sum holds."""
    g = torch.Generator(device=DEV).manual_seed(R)
    x = (torch.randn(R, V, device=DEV, generator=g) * 2.5).to(dtype)
    tok = torch.randint(0, V, (R,), device=DEV, generator=g, dtype=torch.int32)
    first = sv.logprobs(x, tok, None, n_top)
    for _ in range(7):
        r = sv.logprobs(x, tok, None, n_top)
        for name in ("logprob", "entropy", "max", "logsum", "top_tokens", "top_logprobs"):
            assert torch.equal(getattr(r, name), getattr(first, name)), name
    for i in range(0, R, 256):
        d = x[i:i + 256].double()
        m = d.max(1, keepdim=True).values
        y = m - d
        e = torch.exp(-y)
        ls = torch.log(e.sum(1))
        M = (e * y).sum(1) / e.sum(1)
        tol = 4 * E * M + 2.0 ** -21 + (V / 256 + 64) * E + 2 * E * ls
        assert ((first.logsum[i:i + 256].double() - ls).abs() <= tol).all()


def test_zero_signs_tie():
    x = torch.full((1, 700), -5.0)
    x[0, 100::2] = 0.0
    x[0, 101::2] = -0.0
    r = run(x, torch.tensor([0], dtype=torch.int32), None, 6)
    assert r.top_tokens[0].tolist() == [100, 101, 102, 103, 104, 105]


def test_data_errors():
    x = logits(3, 8, 2000, B16)
    x[1, 1500] = math.nan
    x[2, 3] = math.inf
    x[3] = -math.inf
    tok = torch.tensor([4, 1, 1, 1, 2000, -2, 1, 1], dtype=torch.int32)
    T = torch.tensor([1, 1, 1, 1, 1, 1, -1.0, math.nan])
    r = sv.logprobs(x.to(DEV), tok.to(DEV), T.to(DEV), 3)
    assert sv.logprobs_error() == (22, -1, 1)
    for v in (r.logprob, r.entropy, r.max, r.logsum):
        assert torch.isnan(v).tolist() == [False] + [True] * 7
    assert (r.top_tokens[1:] == -1).all() and torch.isnan(r.top_logprobs[1:]).all()
    for rows, code in (([0, 4], 20), ([0, 5], 20), ([0, 6], 17), ([7], 17), ([3], 22)):
        i = torch.tensor(rows)
        sv.logprobs(x[i].to(DEV), tok[i].to(DEV), T[i].to(DEV))
        assert sv.logprobs_error() == (code, -1, len(rows) - 1)


def test_no_tokens_and_an_empty_batch():
    x = logits(3, 3, 500, F32)
    r = sv.logprobs(x.to(DEV), None, None, 4)
    assert torch.isnan(r.logprob).all()
    for i in range(3):
        assert r.top_tokens[i].tolist() == ol.row(x[i].double().numpy(), 0, 0, 4)[4].tolist()
    r = sv.logprobs(x[:0].to(DEV), None)
    assert r.logprob.shape == (0,) and r.top_tokens is None


def grad_check(x, tok, T, gl, gh, r, got):
    x = x.double().cpu().numpy()
    half = torch.finfo(got.dtype).eps / 2
    got = got.double().cpu().numpy()
    for i in range(len(x)):
        t = int(tok[i])
        if t == -1:
            assert (got[i] == 0).all()
            continue
        Ti = 0 if T is None else float(T[i])
        g, h = (0.0 if v is None else float(v[i]) for v in (gl, gh))
        want = ol.grad_row(x[i], t, Ti, g, h)
        _, H, _, ls, _, _, lps, p = ol.row(x[i], t, Ti, 0)
        t_ls, t_h = bounds(lps, ls, p)
        inv = 1.0 / Ti if Ti else 1.0
        a = np.abs(np.where(p > 0, lps, 0.0))
        size = p * (abs(g) + abs(h) * (abs(H) + a)) * inv
        rel = 4 * E * (a + ls) + 2.0 ** -21 + t_ls + 8 * E
        tol = size * rel + p * abs(h) * inv * (t_h + t_ls + 4 * E * (a + ls))
        tol[t] += 4 * E * abs(g) * inv
        tol += half * (np.abs(want) + tol) + 1e-38
        assert (np.abs(got[i] - want) <= tol).all(), np.max(np.abs(got[i] - want) / tol)


@pytest.mark.parametrize("R,V,dtype,pad,temps,which", [
    (1, 1, F32, 0, False, "both"), (4, 13, B16, 1, True, "both"), (5, 1000, F32, 3, True, "lp"),
    (4, 4099, B16, 0, False, "entropy"), (3, 50257, F32, 0, True, "both"),
    (3, 50257, B16, 0, False, "lp"), (3, 151936, B16, 0, True, "both"),
])
def test_gradient_matches_oracle(R, V, dtype, pad, temps, which):
    g = torch.Generator().manual_seed(V + 1)
    x = logits(V, R, V, dtype, pad)
    if V > 20:
        x[0, 5:9] = -math.inf
        x[R - 1, 2] = torch.finfo(dtype).min
    tok = torch.randint(0, V, (R,), generator=g, dtype=torch.int32)
    if R > 3:
        tok[2] = -1
    T = torch.rand(R, generator=g) + 0.4 if temps else None
    gl = torch.randn(R, generator=g) if which != "entropy" else None
    gh = torch.randn(R, generator=g) if which != "lp" else None
    d = [None if v is None else v.to(DEV) for v in (x, tok, T, gl, gh)]
    r = sv.logprobs(d[0], d[1], d[2])
    args = (d[0], d[1], r.max, r.logsum, r.entropy if gh is not None else None, d[3], d[4], d[2])
    got = sv.logprobs_grad(*args)
    grad_check(x, tok, T, gl, gh, r, got)
    # another buffer whose rows lie elsewhere in their 16 bytes, then in place
    wide = torch.full((R, V + 3), 9.0, dtype=dtype, device=DEV)
    assert torch.equal(sv.logprobs_grad(*args, out=wide[:, 1:V + 1]), got)
    assert (wide[:, 0] == 9).all() and (wide[:, V + 1:] == 9).all()
    x2 = d[0].clone()
    sv.logprobs_grad(x2, *args[1:], out=x2)
    assert torch.equal(x2, got)


def test_gradient_equals_differences():
    # central differences of the GPU's own forward in 32 bits, over a short row: a
    # step of 2^-6 leaves 2^-12 of curvature and 2^-20 / 2^-6 of rounding
    x = logits(5, 1, 12, F32, spread=1.0).to(DEV)
    tok = torch.tensor([3], dtype=torch.int32, device=DEV)
    gl, gh = torch.tensor([0.8], device=DEV), torch.tensor([-0.5], device=DEV)
    r = sv.logprobs(x, tok)
    d = sv.logprobs_grad(x, tok, r.max, r.logsum, r.entropy, gl, gh)
    for i in range(12):
        up, dn = x.clone(), x.clone()
        up[0, i] += 2.0 ** -6
        dn[0, i] -= 2.0 ** -6
        a, b = sv.logprobs(up, tok), sv.logprobs(dn, tok)
        f = (0.8 * (a.logprob - b.logprob) - 0.5 * (a.entropy - b.entropy)) * 32
        assert abs(float(d[0, i]) - float(f)) < 2.0 ** -11


def test_gradient_of_bad_rows():
    x = logits(3, 4, 100, F32).to(DEV)
    x[1, 3] = math.nan
    tok = torch.tensor([4, 1, 100, 3], dtype=torch.int32, device=DEV)
    T = torch.tensor([1, 1, 1, -1.0], device=DEV)
    r = sv.logprobs(x, tok, T)
    one = torch.ones(4, device=DEV)
    got = sv.logprobs_grad(x, tok, r.max, r.logsum, r.entropy, one, None, T)
    assert torch.isfinite(got[0]).all() and torch.isnan(got[1:]).all()


def test_streams_graphs_and_refusals():
    x = logits(7, 33, 9000, B16).to(DEV)
    tok = torch.arange(33, dtype=torch.int32, device=DEV)
    want = sv.logprobs(x, tok, None, 5)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = sv.logprobs(x, tok, None, 5, stream=side)
    side.synchronize()
    for a, b in zip(want, got):
        assert torch.equal(a, b)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = sv.logprobs(x, tok, None, 5)
        d = sv.logprobs_grad(x, tok, got.max, got.logsum, got.entropy, got.logprob)
    graph.replay()
    torch.cuda.synchronize()
    for a, b in zip(want, got):
        assert torch.equal(a, b)
    assert torch.equal(d, sv.logprobs_grad(x, tok, want.max, want.logsum, None, want.logprob))
    with pytest.raises(ValueError):
        sv.logprobs(x, tok[:5])
    with pytest.raises(ValueError):
        sv.logprobs(x, tok, None, 33)
    with pytest.raises(ValueError):
        sv.logprobs(x.T, tok)
    with pytest.raises(TypeError):
        sv.logprobs(x.half(), tok)
    with pytest.raises(sv.SpecVerifyError):
        sv.logprobs(x[:1].expand(33, -1), tok)      # rows that share memory
    with pytest.raises(ValueError):
        sv.logprobs_grad(x, tok, want.max, want.logsum, None, None, want.entropy)
