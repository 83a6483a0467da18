"""Attention over the paged cache and its accumulated weights on the GPU against
the oracle (oracle/attention.py).

Tolerances.  A score is a sum of D products in 32 bits: its error is at most
e_s = (D + 4) 2^-24 sum |q K| scale, and the exponential adds 2^-21 of itself.
A weight is off by that factor (twice: score and maximum or lse), plus half a
step of the type where it is rounded for the matrix product with V; the
weighted sum of n values adds n 2^-24; the result is rounded once.  Errors of
`out` are relative to sum w |V|, which the oracle gives."""

import math

import numpy as np
import pytest
import torch

import speculative_decoding_verification_13_gb300 as sv
from oracle import attention as oa

pytestmark = pytest.mark.gpu
DEV = "cuda"


class Case:
    def __init__(self, seed, n, k, Hk, G, D, S, dtype, layers=2, spec=True, junk=True, cols=None):
        g = torch.Generator().manual_seed(seed)
        self.n, self.k, self.D, self.layer = n, k, D, layers - 1
        B, E = len(n), Hk * D
        need = [-(-x // S) for x in n]
        pool = sum(need) + 3
        order = torch.randperm(pool, generator=g).tolist()
        self.table = torch.full((B, cols or max(1, max(need) + 1)), -1, dtype=torch.int32)
        for b, c in enumerate(need):
            self.table[b, :c] = torch.tensor([order.pop() for _ in range(c)], dtype=torch.int32)
        self.cache = torch.randn(pool, layers, 2, S, E, generator=g).to(dtype)
        if junk:  # slots that hold no position of any request: anything may be there
            used = torch.zeros(pool, S, dtype=torch.bool)
            for b, x in enumerate(n):
                for p in range(x):
                    used[self.table[b, p // S], p % S] = True
            self.cache.permute(0, 3, 1, 2, 4)[~used] = math.nan
        self.q = (torch.randn(sum(k) + B, Hk * G, D, generator=g) * 2).to(dtype)
        self.spec = None
        if spec:
            self.spec = torch.randn(B, max(k) + 2, layers, 2, E, generator=g).to(dtype)
            for b, x in enumerate(k):
                self.spec[b, x + 1:] = math.nan
        self.kv_len = torch.tensor(n, dtype=torch.int32)
        self.k_per_req = torch.tensor(k, dtype=torch.int32)

    def gpu(self, q=None):
        spec = None if self.spec is None else self.spec.to(DEV)
        return (self.q.to(DEV) if q is None else q, self.cache.to(DEV), self.layer,
                self.kv_len.to(DEV), self.table.to(DEV), self.k_per_req.to(DEV)), spec

    def oracle(self, **kw):
        return oa.attention(self.q, self.cache, self.layer, self.n, self.table, self.k, self.spec,
                            magnitude=True, **kw)


def score_error(c, size):
    return (c.D + 4) * 2.0 ** -24 * size + 2.0 ** -21


def check(c, out, lse, want):
    out, lse = out.double().cpu().numpy(), lse.double().cpu().numpy()
    o, l, mag, size = want
    keys = max(c.n) + max(c.k) + 1
    half = torch.finfo(c.q.dtype).eps / 2
    weight = 2 * score_error(c, size) + (half if half > 2.0 ** -20 else 0) + (keys + 8) * 2.0 ** -24
    tol = weight[..., None] * mag + half * (np.abs(o) + weight[..., None] * mag)
    assert np.array_equal(np.isneginf(lse), np.isneginf(l))
    f = np.isfinite(l)
    assert (np.abs(out - o) <= tol + 1e-30).all(), np.max(np.abs(out - o) / (tol + 1e-30))
    tl = score_error(c, size) + (keys + 8) * 2.0 ** -24 + 2.0 ** -23 * np.abs(l)
    assert (np.abs(lse[f] - l[f]) <= tl[f]).all(), np.max(np.abs(lse[f] - l[f]) / tl[f])


B16, F16, F32 = torch.bfloat16, torch.float16, torch.float32
CASES = [
    # lengths, drafts, KV heads, group, head, page, type, spec, window
    ([17], [0], 1, 1, 128, 16, B16, True, 0),
    ([0, 1, 63, 64, 65, 130], [0, 0, 0, 0, 0, 0], 2, 4, 128, 16, B16, True, 0),
    ([5, 200, 0, 77], [3, 15, 7, 0], 2, 4, 128, 16, B16, True, 0),
    ([333, 64, 1], [32, 32, 32], 1, 8, 128, 64, B16, True, 0),       # 264 rows a head
    ([150, 90], [7, 2], 3, 7, 64, 7, F16, True, 0),                  # pages end inside tiles
    ([129, 40], [1, 4], 2, 2, 64, 1, B16, True, 0),                  # one position a page
    ([100, 31], [5, 0], 2, 1, 256, 32, F16, True, 0),
    ([100, 31, 2], [5, 0, 1], 1, 4, 80, 16, B16, True, 0),           # heads of other sizes
    ([70, 9], [2, 0], 2, 2, 8, 16, F16, True, 0),
    ([70, 9], [2, 3], 2, 3, 64, 16, F32, True, 0),
    ([50, 3], [4, 1], 1, 2, 256, 128, F32, True, 0),
    ([140, 300, 2], [3, 0, 5], 2, 4, 128, 16, B16, False, 0),        # entries cached already
    ([0, 2, 5], [0, 3, 2], 2, 2, 64, 16, F16, False, 0),             # tokens that see nothing
    ([200, 90, 0], [5, 15, 2], 2, 4, 128, 16, B16, True, 1),
    ([200, 90, 500], [5, 15, 0], 2, 4, 128, 16, B16, True, 70),
    ([200, 90, 3], [5, 15, 0], 2, 2, 64, 16, F32, False, 33),
    ([300, 131, 2], [5, 0, 15], 3, 4, 80, 16, F16, True, 0),         # between 64, 128 and 256
    ([400, 128, 70], [0, 32, 3], 2, 7, 96, 32, B16, True, 90),
    ([290, 129], [7, 1], 3, 2, 112, 7, B16, False, 0),
    ([300, 64, 9], [3, 0, 32], 3, 4, 144, 64, B16, True, 0),
    ([257, 90], [15, 2], 2, 8, 192, 16, F16, True, 65),
    ([200, 33], [0, 4], 1, 1, 240, 8, B16, True, 0),
    ([130, 90], [2, 0], 2, 2, 72, 16, F16, True, 0),                 # no multiple of 16
]


@pytest.mark.parametrize("case", CASES, ids=range(len(CASES)))
def test_attention_and_weights_match_oracle(case):
    n, k, Hk, G, D, S, dtype, spec, window = case
    c = Case(sum(n) + D, n, k, Hk, G, D, S, dtype, spec=spec)
    args, sp = c.gpu()
    out, lse = sv.attention(*args, sp, window=window)
    assert sv.attention_error()[0] == 0
    want = c.oracle(window=window)
    check(c, out, lse, want)
    # the weights, with the true lse so that only this call's error counts
    rng = np.random.default_rng(1)
    accept = np.array([rng.integers(-1, x + 1) for x in k], np.int32)
    accept[0] = k[0]
    cols = max(n) + max(k) + 2
    score = torch.rand(len(n), cols, generator=torch.Generator().manual_seed(5))
    truth = torch.as_tensor(want[1], dtype=torch.float32)
    ref = oa.weights(c.q, c.cache, c.layer, n, c.table, k, truth, score, c.spec, accept,
                     window=window)
    got = sv.attention_weights(*args, truth.to(DEV), score.to(DEV), sp,
                               torch.as_tensor(accept).to(DEV), window=window)
    assert sv.attention_weights_error()[0] == 0
    f = np.isfinite(want[1])
    top = float(want[3][f].max()) if f.any() else 0.0
    rel = 2 * score_error(c, top) + 2.0 ** -22 * (np.abs(want[1][f]).max() if f.any() else 0)
    terms = (max(k) + 1) * Hk * G
    tol = (rel + (terms + 4) * 2.0 ** -24) * ref + 1e-30
    err = np.abs(got.double().cpu().numpy() - ref)
    assert (err <= tol).all(), np.max(err / tol)
    for b, x in enumerate(n):   # beyond the positions nothing was written
        end = 0 if accept[b] < 0 else x + accept[b] + 1 if spec else x
        assert torch.equal(got[b, end:].cpu(), score[b, end:])


def test_long_context_is_split_and_joined():
    # one request over every SM: many partials a unit, joined in order
    c = Case(3, [20011], [3], 2, 4, 128, 16, B16, layers=1)
    args, sp = c.gpu()
    out, lse = sv.attention(*args, sp)
    q, K = c.q.double(), None
    kv = c.cache[c.table[0, :-(-20011 // 16)].long(), 0].transpose(0, 1).reshape(2, -1, 256)
    kv = torch.cat([kv[:, :20011], c.spec[0, :4, 0].transpose(0, 1)], 1).double()
    for hq in (0, 3, 4, 7):
        K, V = (kv[i, :, (hq // 4) * 128:(hq // 4 + 1) * 128] for i in (0, 1))
        for j in range(4):
            s = K[:20012 + j] @ q[j, hq] / math.sqrt(128)
            w = torch.softmax(s, 0)
            size = float((K.abs() @ q[j, hq].abs()).max()) / math.sqrt(128)
            rel = 2 * score_error(c, size) + 2.0 ** -8 + 20020 * 2.0 ** -24
            mag = w @ V[:20012 + j].abs()
            o = w @ V[:20012 + j]
            err = (out[j, hq].double().cpu() - o).abs()
            assert (err <= rel * mag + 2.0 ** -8 * (o.abs() + rel * mag)).all()
            want = float(torch.logsumexp(s, 0))
            assert abs(float(lse[j, hq]) - want) <= \
                score_error(c, size) + 20020 * 2.0 ** -24 + 2.0 ** -23 * abs(want)


def test_many_small_weights_in_half_precision():
    # one position holds most of the weight, 20000 hold 2^-20 of it each: below the
    # normal range of fp16 but for the scaling of the weights
    n, D = 20000, 64
    cache = torch.zeros(n // 16 + 1, 1, 2, 16, D, dtype=F16)
    flat = cache.permute(0, 3, 1, 2, 4)
    flat[..., 0, 0] = -13.8984375
    flat[..., 1, :] = 1.0
    flat[3, 5, 0, 0, 0] = 0.0
    flat[3, 5, 0, 1, :] = 0.0
    q = torch.zeros(1, 2, D, dtype=F16)
    q[..., 0] = 8.0
    i32 = torch.int32
    table = torch.arange(n // 16 + 1, dtype=i32)[None]
    out, lse = sv.attention(q.to(DEV), cache.to(DEV), 0, torch.tensor([n], dtype=i32, device=DEV),
                            table.to(DEV), torch.zeros(1, dtype=i32, device=DEV))
    total = 1 + (n - 1) * math.exp(-13.8984375)
    want = 1 - 1 / total
    # half a step for the weights, one for the result, n additions
    assert (out.double() - want).abs().max() <= want * (2 * 2.0 ** -11 + n * 2.0 ** -24 + 2.0 ** -20)
    assert (lse.double() - math.log(total)).abs().max() <= n * 2.0 ** -24 + 2.0 ** -20


def test_results_do_not_change_from_run_to_run():
    c = Case(9, [3000, 17, 700, 0], [7, 0, 3, 1], 4, 4, 128, 16, B16)
    args, sp = c.gpu()
    first = sv.attention(*args, sp)
    score = torch.zeros(4, 3100, device=DEV)
    w = sv.attention_weights(*args, first[1], score, sp, out_score=torch.zeros_like(score))
    for _ in range(3):
        again = sv.attention(*args, sp)
        assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])
        assert torch.equal(w, sv.attention_weights(*args, first[1], score, sp,
                                                   out_score=torch.zeros_like(score)))


@pytest.mark.parametrize("dtype,D", [(B16, 128), (F16, 64), (F32, 64)])
def test_strided_and_unaligned_queries(dtype, D):
    # q as a slice of a fused projection, off the 16-byte grid, heads apart
    c = Case(4, [90, 33], [3, 1], 2, 3, D, 16, dtype)
    rows = c.q.shape[0]
    wide = torch.zeros(rows, 3 * 6 * D + 5, dtype=dtype, device=DEV)
    q = wide[:, 3:3 + 6 * D].unflatten(1, (6, D))
    q.copy_(c.q)
    swapped = torch.zeros(6, rows, D + 1, dtype=dtype, device=DEV)[..., 1:].transpose(0, 1)
    swapped.copy_(c.q)
    for x in (q, swapped):
        args, sp = c.gpu(x)
        out, lse = sv.attention(*args, sp)
        check(c, out, lse, c.oracle())


def test_a_later_token_of_the_drafts_does_not_reach_an_earlier_one():
    # an infinite or NaN value of draft i is seen by tokens i.. only
    c = Case(6, [40], [5], 1, 2, 128, 16, B16)
    clean = c.oracle()
    for bad in (math.nan, math.inf):
        c.spec[0, 3, c.layer, 1, 5] = bad
        c.spec[0, 4, c.layer, 0] = math.nan
        args, sp = c.gpu()
        out, lse = sv.attention(*args, sp)
        o = out.double().cpu().numpy()
        keep = [x[:3] for x in clean]
        c.q, q = c.q[:3], c.q
        check(c, out[:3], lse[:3], keep)
        c.q = q
        assert not np.isfinite(o[3, :, 5]).any() and np.isfinite(o[3, :, 6]).all()
        assert np.isnan(o[4:]).all() and torch.isnan(lse[4:]).all()


@pytest.mark.parametrize("D", [80, 208])
def test_another_head_s_values_do_not_reach_a_narrow_head(D):
    # whole boxes of 128 bytes reach into the next head's entries
    c = Case(16, [640, 200], [3, 0], 2, 4, D, 16, B16)
    want = c.oracle()
    c.cache[..., D:] = math.nan
    c.spec[..., D:] = math.inf
    args, sp = c.gpu()
    out, lse = sv.attention(*args, sp)
    first = lambda x: x[:, :4]
    c.q = c.q[:, :4]
    check(c, first(out), first(lse), [first(x) for x in want])
    assert torch.isnan(lse[:, 4:]).all()
    score = torch.zeros(2, 700, device=DEV)
    got = sv.attention_weights(*args, torch.zeros_like(lse), score, sp,
                               out_score=torch.zeros_like(score))
    assert torch.isnan(got[0, :640]).all()


@pytest.mark.parametrize("dtype,D", [(B16, 80), (F16, 160)])
def test_narrow_heads_split_over_blocks_and_unaligned(dtype, D):
    c = Case(17, [3001, 50], [2, 1], 2, 3, D, 16, dtype)
    rows = c.q.shape[0]
    q = torch.zeros(6, rows, D + 1, dtype=dtype, device=DEV)[..., 1:].transpose(0, 1)
    q.copy_(c.q)
    args, sp = c.gpu(q)
    flat = torch.zeros(rows * 6 * D + 1, dtype=dtype, device=DEV)
    out, lse = sv.attention(*args, sp, out=flat[1:].view(rows, 6, D))
    check(c, out, lse, c.oracle())


@pytest.mark.parametrize("S", [8, 16, 64, 128, 24, 5])
@pytest.mark.parametrize("dtype,D", [(B16, 128), (F16, 64), (B16, 256), (F16, 80)])
def test_last_tiles_of_every_kind(S, dtype, D):
    # ends of the cache at, before and behind the edges of tiles, pages and boxes;
    # lengths and drafts off the 16-byte grid
    n = [127, 128, 129, 120, 64, 65, 8, 7, 255, 136, 0]
    k = [0, 3, 0, 15, 1, 7, 2, 0, 1, 8, 5]
    c = Case(S + D, n, k, 2, 2, D, S, dtype, layers=1)
    args, sp = c.gpu()
    wide = torch.zeros(2, len(n) + 1, dtype=torch.int32, device=DEV)
    wide[0, 1:], wide[1, 1:] = args[3], args[5]
    args = args[:3] + (wide[0, 1:], args[4], wide[1, 1:])
    out, lse = sv.attention(*args, sp)
    want = c.oracle()
    check(c, out, lse, want)
    score = torch.zeros(len(n), 300)
    truth = torch.as_tensor(want[1], dtype=torch.float32)
    ref = oa.weights(c.q, c.cache, c.layer, n, c.table, k, truth, score, c.spec)
    got = sv.attention_weights(*args, truth.to(DEV), score.to(DEV), sp)
    f = np.isfinite(want[1])
    rel = 2 * score_error(c, float(want[3][f].max())) + 2.0 ** -22 * np.abs(want[1][f]).max()
    tol = (rel + (16 * 4 + 4) * 2.0 ** -24) * ref + 1e-30
    assert (np.abs(got.double().cpu().numpy() - ref) <= tol).all()


def test_data_errors_fail_their_request_only():
    c = Case(8, [40, 100, 30, 20], [1, 2, 0, 3], 2, 2, 128, 16, B16)
    want = c.oracle()
    args, sp = c.gpu()
    table, kv_len = args[4], args[3]
    off = [0, 2, 5, 6, 10]
    table[1, 3] = -1                      # a page in the middle of request 1
    kv_len[2] = -5                        # a negative length
    out, lse = sv.attention(*args, sp)
    assert sv.attention_error()[:2] == (27, 1)
    nan = torch.isnan(lse).all(1).cpu().tolist()
    assert nan == [False] * 2 + [True] * 4 + [False] * 4
    assert torch.isnan(out[off[1]:off[3]]).all()
    for b in (0, 3):
        s = slice(off[b], off[b + 1])
        assert np.abs(out[s].double().cpu().numpy() - want[0][s]).max() < 0.1
    table[1, 3] = c.cache.shape[0]        # past the pool
    sv.attention(*args, sp)
    assert sv.attention_error()[:2] == (27, 1)
    # the weights leave what they cannot compute
    score = torch.ones(4, 128, device=DEV)
    got = sv.attention_weights(*args, torch.zeros_like(lse), score, sp,
                               out_score=torch.full_like(score, 7))
    assert sv.attention_weights_error()[:2] == (27, 1)
    assert (got[2] == 7).all() and (got[1, 48:64] == 7).all() and (got[1, :48] != 7).all()


def test_a_batch_that_does_not_fit_its_rows_fails_whole():
    c = Case(8, [40, 100], [1, 2], 2, 2, 64, 16, F16)
    args, sp = c.gpu()
    args[5][0] = 2
    out, lse = sv.attention(*args, sp)
    assert sv.attention_error()[0] == 21 and torch.isnan(out).all() and torch.isnan(lse).all()
    args[5][0], args[5][1] = 1, 33
    out, lse = sv.attention(*args, sp)
    assert sv.attention_error()[:2] == (16, 1) and torch.isnan(out).all() and torch.isnan(lse).all()
    score = torch.ones(2, 128, device=DEV)
    assert (sv.attention_weights(*args, lse, score, sp) == 1).all()


def test_weights_errors():
    c = Case(8, [40, 60], [1, 2], 2, 2, 64, 16, F16)
    args, sp = c.gpu()
    _, lse = sv.attention(*args, sp)
    score = torch.ones(2, 61, device=DEV)            # request 1 ends at 63
    sv.attention_weights(*args, lse, score, sp)
    assert sv.attention_weights_error()[:2] == (28, 1)
    assert (score[1] == 1).all() and (score[0, :42] > 1).all() and (score[0, 42:] == 1).all()
    acc = torch.tensor([2, 0], dtype=torch.int32, device=DEV)
    sv.attention_weights(*args, lse, score, sp, acc)
    assert sv.attention_weights_error()[:2] == (26, 0)


def test_other_streams_and_graphs():
    c = Case(11, [500, 64], [3, 0], 2, 4, 128, 16, B16)
    args, sp = c.gpu()
    want = sv.attention(*args, sp)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = sv.attention(*args, sp, stream=side)
    side.synchronize()
    assert torch.equal(want[0], got[0])
    out, lse = torch.zeros_like(want[0]), torch.zeros_like(want[1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        sv.attention(*args, sp, out=out, out_lse=lse)
    args[0].mul_(0.5)
    graph.replay()
    want = sv.attention(*args, sp)
    torch.cuda.synchronize()
    assert torch.equal(out, want[0]) and torch.equal(lse, want[1])


def test_many_requests_and_an_empty_batch():
    n = [(i * 37) % 90 for i in range(700)]
    k = [(i * 5) % 4 for i in range(700)]
    c = Case(12, n, k, 1, 2, 64, 16, F16, layers=1, junk=False)
    args, sp = c.gpu()
    out, lse = sv.attention(*args, sp)
    check(c, out, lse, c.oracle())
    e = torch.zeros(0, dtype=torch.int32, device=DEV)
    out, lse = sv.attention(args[0][:0], args[1], 0, e, args[4][:0], e)
    assert out.shape == (0, 2, 64) and lse.shape == (0, 2)


def test_binding_refusals():
    c = Case(1, [40], [1], 2, 2, 64, 16, F16)
    args, sp = c.gpu()
    q, cache, layer, n, table, k = args
    with pytest.raises(ValueError):
        sv.attention(q, cache, 2, n, table, k, sp)
    with pytest.raises(ValueError):
        sv.attention(q[..., :63], cache, layer, n, table, k, sp)
    with pytest.raises(ValueError):
        sv.attention(q, cache, layer, n, table, k, sp[:, :, :1].contiguous())
    with pytest.raises(ValueError):
        sv.attention(q, cache, layer, n, table, k, sp, window=-1)
    with pytest.raises(TypeError):
        sv.attention(q.float(), cache, layer, n, table, k, sp)
    with pytest.raises(TypeError):
        sv.attention(q, cache, layer, n.long(), table, k, sp)
    with pytest.raises(ValueError):
        sv.attention(q, cache, layer, n, table.T, k, sp)
    with pytest.raises(ValueError):
        sv.attention(q, cache, layer, n, table, k, sp, out=torch.empty_like(q)[:1])
    with pytest.raises(ValueError):
        sv.attention_weights(*args, torch.zeros(3, 4, device=DEV), torch.zeros(1, 64, device=DEV))


@pytest.mark.parametrize("dtype,D", [(B16, 128), (F16, 64), (F32, 64)])
@pytest.mark.parametrize("window", [2 ** 31 - 1, 2 ** 31 - 256, 2 ** 31 - 257, 1 << 30])
def test_the_widest_windows_hide_nothing(dtype, D, window):
    # tokens in front of the first position among them: their window starts at about
    # -2^31, which has to stay in 32 bits
    n, k = [2, 0, 40, 300], [32, 3, 32, 1]
    c = Case(18, n, k, 2, 2, D, 16, dtype, spec=False)
    args, _ = c.gpu()
    out, lse = sv.attention(*args, window=window)
    assert sv.attention_error()[0] == 0
    check(c, out, lse, c.oracle())
    zero = torch.zeros(4, 310, device=DEV)
    got = [sv.attention_weights(*args, lse, zero, window=w, out_score=torch.zeros_like(zero))
           for w in (0, window)]
    assert sv.attention_weights_error()[0] == 0
    assert torch.equal(*got)


@pytest.mark.parametrize("dtype,D", [(B16, 128), (F16, 64), (B16, 256)])
def test_a_missing_page_of_a_whole_tile_fails_its_rows_every_time(dtype, D):
    # the page is noted by the warp that loads, for those that wait for the tile
    n = [128 * i for i in (1, 2, 3, 9, 40)]
    c = Case(19, n, [0] * 5, 2, 4, D, 16, dtype, layers=1, junk=False)
    args, sp = c.gpu()
    want, want_lse = sv.attention(*args, sp)
    for b, page in ((0, 7), (1, 8), (2, 23), (3, 71), (4, 0)):
        table = args[4].clone()
        table[b, page] = -1
        for _ in range(40):
            out, lse = sv.attention(*args[:4], table, args[5], sp)
            assert torch.isnan(out[b]).all() and torch.isnan(lse[b]).all()
            other = torch.arange(5, device=DEV) != b
            assert torch.equal(out[other], want[other]) and torch.equal(lse[other], want_lse[other])
        assert sv.attention_error()[:2] == (27, b)
