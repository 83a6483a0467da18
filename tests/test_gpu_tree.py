"""Trees of drafts on the GPU against the oracles (oracle/tree.py): attention over
the paged cache, greedy verification, and the commit of the accepted path.

Attention's tolerances are those of tests/test_gpu_attention.py: a score's error is
at most (D + 4) 2^-24 sum |q K| scale, twice (score and maximum or sum), 2^-21 for
the exponential, half a step of the type for a weight that is rounded for the
product, n 2^-24 for sums of n, half a step for the result."""

import math
import random

import numpy as np
import pytest
import torch

import speculative_decoding_verification_13_gb300 as sv
from oracle import kv as okv
from oracle import tree as ot

pytestmark = pytest.mark.gpu
DEV = "cuda"
B16, F16, F32 = torch.bfloat16, torch.float16, torch.float32


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def trees(rng, k, kind="any"):
    parent = []
    for n in k:
        parent.append(rng.choice([-1, 0, 5]))   # node 0's is not read
        for j in range(1, n + 1):
            parent.append(j - 1 if kind == "chain" else 0 if kind == "star" else
                          rng.randint(max(0, j - 5), j - 1))
    return parent


class Case:
    def __init__(self, seed, n, k, Hk, G, D, S, dtype, kind="any", layers=2):
        g, rng = torch.Generator().manual_seed(seed), random.Random(seed)
        self.n, self.k, self.layer = n, k, layers - 1
        B, E = len(n), Hk * D
        need = [-(-x // S) for x in n]
        pool = sum(need) + 3
        order = torch.randperm(pool, generator=g).tolist()
        self.table = torch.full((B, max(1, max(need) + 1)), -1, dtype=torch.int32)
        for b, c in enumerate(need):
            self.table[b, :c] = torch.tensor([order.pop() for _ in range(c)], dtype=torch.int32)
        self.cache = torch.randn(pool, layers, 2, S, E, generator=g).to(dtype)
        used = torch.zeros(pool, S, dtype=torch.bool)   # other slots hold anything
        for b, x in enumerate(n):
            for p in range(x):
                used[self.table[b, p // S], p % S] = True
        self.cache.permute(0, 3, 1, 2, 4)[~used] = math.nan
        self.q = (torch.randn(sum(k) + B, Hk * G, D, generator=g) * 2).to(dtype)
        self.spec = torch.randn(B, max(k) + 2, layers, 2, E, generator=g).to(dtype)
        for b, x in enumerate(k):
            self.spec[b, x + 1:] = math.nan
        self.parent = trees(rng, k, kind)

    def run(self, **kw):
        return sv.tree_attention(self.q.to(DEV), self.cache.to(DEV), self.layer, i32(self.n),
                                 self.table.to(DEV), i32(self.k), i32(self.parent),
                                 self.spec.to(DEV), **kw)

    def oracle(self, **kw):
        return ot.attention(self.q, self.cache, self.layer, self.n, self.table, self.k,
                            self.parent, self.spec, magnitude=True, **kw)


def check(c, out, lse, want, rows=slice(None)):
    out, lse = out.double().cpu().numpy()[rows], lse.double().cpu().numpy()[rows]
    o, l, mag, size = (x[rows] for x in want)
    keys, D = max(c.n) + max(c.k) + 1, c.q.shape[2]
    half = torch.finfo(c.q.dtype).eps / 2
    e_s = (D + 4) * 2.0 ** -24 * size + 2.0 ** -21
    weight = 2 * e_s + (half if half > 2.0 ** -20 else 0) + (keys + 8) * 2.0 ** -24
    tol = weight[..., None] * mag + half * (np.abs(o) + weight[..., None] * mag)
    assert (np.abs(out - o) <= tol + 1e-30).all(), np.max(np.abs(out - o) / (tol + 1e-30))
    tl = e_s + (keys + 8) * 2.0 ** -24 + 2.0 ** -23 * np.abs(l)
    assert (np.abs(lse - l) <= tl).all(), np.max(np.abs(lse - l) / tl)


CASES = [
    # lengths, drafts, KV heads, group, head, page, type, window, kind
    ([17], [0], 1, 1, 128, 16, B16, 0, "any"),
    ([0, 5, 200, 77], [3, 15, 7, 0], 2, 4, 128, 16, B16, 0, "any"),
    ([150, 300, 64], [63, 20, 33], 1, 4, 128, 16, B16, 0, "any"),     # 256 rows a head
    ([90, 128, 3], [63, 63, 40], 1, 1, 128, 64, B16, 0, "any"),
    ([333, 64, 1], [31, 40, 12], 1, 8, 64, 7, F16, 0, "star"),
    ([100, 31], [24, 40], 2, 1, 256, 32, F16, 0, "any"),
    ([100, 31, 2], [5, 0, 63], 1, 4, 80, 16, B16, 0, "any"),
    ([70, 9], [24, 3], 2, 3, 64, 16, F32, 0, "any"),
    ([70, 9], [63, 10], 2, 2, 8, 16, F16, 0, "any"),
    ([200, 90, 3], [30, 15, 63], 2, 4, 128, 16, B16, 1, "any"),       # each sees itself alone
    ([200, 90, 3], [30, 15, 63], 2, 4, 128, 16, B16, 3, "chain"),
    ([200, 90, 500], [63, 15, 0], 2, 4, 128, 16, B16, 70, "any"),
    ([200, 40], [20, 40], 2, 2, 64, 16, F32, 4, "any"),
    ([300, 64], [50, 33], 3, 4, 144, 64, B16, 0, "any"),
    ([130, 127, 126, 65], [1, 2, 3, 63], 2, 2, 64, 16, B16, 0, "chain"),
    # many rows a request: both row tiles of the kernel for them, its heads and groups
    ([100, 31, 2], [45, 63, 30], 1, 4, 80, 16, B16, 0, "any"),
    ([300, 0, 127], [50, 63, 39], 2, 4, 96, 7, F16, 40, "chain"),
    ([129, 40], [20, 31], 1, 16, 128, 16, B16, 5, "any"),
    ([260, 5, 1000], [3, 9, 0], 1, 128, 64, 64, F16, 0, "star"),
    ([1500, 257, 0, 3], [63, 32, 31, 30], 3, 8, 128, 128, F16, 0, "any"),
]


@pytest.mark.parametrize("case", CASES, ids=range(len(CASES)))
def test_tree_attention_matches_oracle(case):
    n, k, Hk, G, D, S, dtype, window, kind = case
    c = Case(sum(n) + D, n, k, Hk, G, D, S, dtype, kind)
    out, lse = c.run(window=window)
    assert sv.tree_attention_error() == (0, -1, -1)
    check(c, out, lse, c.oracle(window=window))


@pytest.mark.parametrize("dtype,D", [(B16, 128), (F32, 64)])
def test_a_chain_is_attention(dtype, D):
    c = Case(3, [200, 31, 0], [15, 32, 4], 2, 4, D, 16, dtype, "chain")
    out, lse = c.run(window=90)
    args = (c.q.to(DEV), c.cache.to(DEV), c.layer, i32(c.n), c.table.to(DEV), i32(c.k))
    o, l = sv.attention(*args, c.spec.to(DEV), window=90)
    assert torch.equal(out, o) and torch.equal(lse, l)


@pytest.mark.parametrize("dtype,D", [(B16, 128), (F16, 256), (F32, 64)])
def test_a_torn_tree_fails_its_request_alone(dtype, D):
    k = [15, 40, 3, 7]
    c = Case(5, [200, 31, 0, 90], k, 2, 4, D, 16, dtype)
    want = c.oracle()
    at = np.cumsum([0] + [x + 1 for x in k])
    for b, j, up in ((1, 3, 3), (2, 2, -1), (1, 40, 63)):
        torn = list(c.parent)
        torn[at[b] + j] = up
        good, c.parent = c.parent, torn
        out, lse = c.run()
        assert sv.tree_attention_error() == (29, b, -1)
        c.parent = good
        rows = np.arange(at[-1])
        bad = (rows >= at[b]) & (rows < at[b + 1])
        assert torch.isnan(out[torch.tensor(bad)]).all() and torch.isnan(lse[torch.tensor(bad)]).all()
        check(c, out, lse, want, rows[~bad])


def test_other_errors_of_trees():
    c = Case(6, [40, 50], [10, 5], 2, 2, 128, 16, B16)
    c.table[1, 2] = -1
    out, _ = c.run()
    assert sv.tree_attention_error() == (27, 1, -1)
    assert torch.isnan(out[11:]).all() and torch.isfinite(out[:11]).all()
    c.k = [10, 64]
    c.run()
    assert sv.tree_attention_error()[0] == 16
    c.k = [10, 4]
    out, lse = c.run()
    assert sv.tree_attention_error()[0] == 21
    assert torch.isnan(out).all() and torch.isnan(lse).all()


def test_infinite_values_of_other_branches_stay_there():
    # nodes 1 and 2 hang from node 0: neither sees the other
    for dtype, D in ((B16, 128), (F16, 64), (B16, 256), (F32, 64)):
        c = Case(8, [37], [4], 1, 2, D, 16, dtype)
        c.parent = [-1, 0, 0, 1, 2]
        c.spec[0, 1, c.layer, 1, 5], c.spec[0, 2, c.layer, 1, 6] = math.inf, math.nan
        c.spec[0, 4, c.layer, 1, 7] = -math.inf
        out, _ = c.run()
        out = out.float().cpu().numpy()[:, :, 5:9]
        inf, nan, fin = np.isinf(out), np.isnan(out), np.isfinite(out)
        assert fin[0].all() and fin[:, :, 3].all()
        assert inf[1, :, 0].all() and inf[3, :, 0].all() and fin[2, :, 0].all() and fin[4, :, 0].all()
        assert nan[2, :, 1].all() and nan[4, :, 1].all() and fin[1, :, 1].all() and fin[3, :, 1].all()
        assert (out[4, :, 2] == -math.inf).all() and fin[:4, :, 2].all()


# ------------------------------------------- many rows: two row tiles over the same keys
def ancestors(parent, j):
    path = [j]
    while path[-1]:
        path.append(parent[path[-1]])
    return path


@pytest.mark.parametrize("dtype,D,G", [(B16, 128, 4), (F16, 64, 8), (B16, 80, 4)])
def test_a_torn_tree_of_many_rows_fails_its_request_alone(dtype, D, G):
    k = [63, 50, 3, 60]
    c = Case(15, [3000, 31, 0, 90], k, 1, G, D, 16, dtype)   # the first lies in several parts
    want = c.oracle()
    at = np.cumsum([0] + [x + 1 for x in k])
    for b, j, up in ((0, 63, 63), (0, 1, -1), (3, 60, 61), (2, 2, 2)):
        torn = list(c.parent)
        torn[at[b] + j] = up
        good, c.parent = c.parent, torn
        out, lse = c.run()
        assert sv.tree_attention_error() == (29, b, -1)
        c.parent = good
        rows = np.arange(at[-1])
        bad = (rows >= at[b]) & (rows < at[b + 1])
        assert torch.isnan(out[torch.tensor(bad)]).all() and torch.isnan(lse[torch.tensor(bad)]).all()
        check(c, out, lse, want, rows[~bad])


def test_other_errors_of_trees_of_many_rows():
    k = [60, 63, 55]
    c = Case(16, [1500, 50, 700], k, 2, 4, 128, 16, B16)
    want = c.oracle()
    rows = np.arange(sum(k) + 3)
    first = rows < 61
    for column, page in ((40, -1), (93, c.cache.shape[0]), (0, -7)):
        keep = int(c.table[0, column])
        c.table[0, column] = page
        out, lse = c.run()
        assert sv.tree_attention_error() == (27, 0, -1)
        c.table[0, column] = keep
        assert torch.isnan(out[:61]).all() and torch.isnan(lse[:61]).all()
        check(c, out, lse, want, rows[~first])
    for n in (-1, 10 ** 6):
        c.n[1], keep = n, c.n[1]
        out, lse = c.run()
        assert sv.tree_attention_error() == (28, 1, -1)
        c.n[1] = keep
        second = (rows >= 61) & (rows < 125)
        assert torch.isnan(out[61:125]).all()
        check(c, out, lse, want, rows[~second])
    for bad, code in (([60, 64, 54], 16), ([60, 63, 54], 21)):
        c.k = bad
        out, lse = c.run()
        assert sv.tree_attention_error()[0] == code
        assert torch.isnan(out).all() and torch.isnan(lse).all()


@pytest.mark.parametrize("dtype,D", [(B16, 128), (F16, 64), (F16, 112)])
def test_values_that_are_no_numbers_among_many_rows(dtype, D):
    n, W = 2000, 40
    c = Case(17, [n], [63], 1, 4, D, 16, dtype)
    parent, L = c.parent, c.layer
    for node, col, x in ((5, 5, math.inf), (9, 6, math.nan), (20, 7, -math.inf)):
        c.spec[0, node, L, 1, col] = x
    at = lambda p: (int(c.table[0, p // 16]), L, 1, p % 16)   # noqa: E731  (V of position p)
    c.cache[at(100)][9] = math.inf        # before every window
    c.cache[at(n - 5)][10] = -math.inf    # seen from positions below n - 5 + W
    c.cache[at(300)][11] = math.nan
    c.cache[int(c.table[0, 18]), L, 0] = math.nan   # keys of positions 288 to 303
    out, lse = c.run(window=W)
    out = out.float().cpu().numpy()
    assert torch.isfinite(lse).all()
    for j in range(64):
        path = ancestors(parent, j)
        seen = path[:W]
        here = out[j]
        assert np.isfinite(here[:, [i for i in range(D) if i not in (5, 6, 7, 10)]]).all()
        for node, col, test in ((5, 5, lambda x: x == math.inf), (9, 6, np.isnan),
                                (20, 7, lambda x: x == -math.inf)):
            assert (test if node in seen else np.isfinite)(here[:, col]).all(), (j, node)
        sees = n - 5 > n + len(path) - 1 - W
        assert ((here[:, 10] == -math.inf) if sees else np.isfinite(here[:, 10])).all(), j


def test_strided_queries_in_a_graph_and_twice():
    c = Case(9, [700, 90], [40, 63], 2, 4, 128, 16, B16)
    want = c.run()
    wide = torch.zeros(c.q.shape[0], c.q.shape[1], 200, dtype=B16, device=DEV)
    wide[:, :, :128] = c.q.to(DEV)
    args = (wide[:, :, :128], c.cache.to(DEV), c.layer, i32(c.n), c.table.to(DEV), i32(c.k),
            i32(c.parent), c.spec.to(DEV))
    out, lse = torch.empty_like(want[0]), torch.empty_like(want[1])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        sv.tree_attention(*args, out=out, out_lse=lse)
    for _ in range(2):
        out.zero_()
        g.replay()
        c.run()
        assert torch.equal(out, want[0]) and torch.equal(lse, want[1])


@pytest.mark.parametrize("dtype,D,k", [(B16, 128, [63, 40]), (F16, 64, [3, 9]), (B16, 256, [20, 5]),
                                       (F32, 64, [30, 5])])
def test_outputs_beside_memory_that_is_not_aligned(dtype, D, k):
    c = Case(11, [5000, 90], k, 2, 4, D, 16, dtype)      # the first lies in several parts
    want = c.run()
    buf = torch.full((want[0].numel() + 2,), 7, dtype=dtype, device=DEV)
    out = buf[1:-1].view(want[0].shape)
    c.run(out=out, out_lse=want[1].clone())
    assert torch.equal(out, want[0]) and buf[0] == 7 and buf[-1] == 7


# ----------------------------------------------------------------- verification
def verify_case(seed, k, V, agree=0.7):
    rng = random.Random(seed)
    parent = trees(rng, k)
    argmax, drafts, t = [], [], 0
    for n in k:
        tokens = [rng.randrange(V) for _ in range(n + 1)]
        best = [rng.randrange(V) for _ in range(n + 1)]
        for j in range(1, n + 1):
            if rng.random() < agree:
                best[parent[t + j]] = tokens[j]
        drafts += tokens[1:]
        argmax += best
        t += n + 1
    return argmax, drafts, parent


@pytest.mark.parametrize("B,k_max,V", [(1, 0, 10), (1, 63, 50), (7, 5, 1000), (9, 63, 3),
                                       (300, 24, 151936), (4097, 15, 40)])
def test_verify_tree_matches_oracle(B, k_max, V):
    rng = random.Random(B)
    k = [rng.randint(0, k_max) for _ in range(B)]
    k[-1] = k_max
    argmax, drafts, parent = verify_case(B + k_max, k, V)
    got = sv.verify_tree_greedy(i32(argmax), i32(drafts), i32(parent), i32(k), V)
    assert sv.verify_tree_greedy_error() == (0, -1, -1)
    for x, y in zip(got, ot.verify_greedy(argmax, drafts, parent, k)):
        assert np.array_equal(x.cpu().numpy(), y)


def test_a_chain_verifies_as_verify_greedy():
    rng = random.Random(2)
    k = [rng.randint(0, 32) for _ in range(50)]
    argmax, drafts, _ = verify_case(3, k, 4)
    parent = trees(rng, k, "chain")
    a, t, _ = sv.verify_tree_greedy(i32(argmax), i32(drafts), i32(parent), i32(k), 4)
    b, u = sv.verify_greedy_from_argmax(i32(argmax), i32(drafts), i32(k), 4)
    assert torch.equal(a, b) and torch.equal(t, u)


def test_the_lowest_child_of_a_token_is_taken():
    got = sv.verify_tree_greedy(i32([5, 9, 7, 1]), i32([5, 5, 7]), i32([-1, 0, 0, 2]), i32([3]), 10)
    assert [x.tolist() for x in got] == [[1], [5, 9, -1, -1], [0, 1, -1, -1]]


def test_verify_tree_errors():
    k = [3, 5, 2]
    argmax, drafts, parent = verify_case(5, k, 20)
    want = ot.verify_greedy(argmax, drafts, parent, k)
    for name, at, value, code, b in (("parent", 5, 1, 29, 1), ("parent", 11, -1, 29, 2),
                                     ("drafts", 0, 20, 20, 0), ("argmax", 9, -1, 20, 1)):
        x = dict(argmax=list(argmax), drafts=list(drafts), parent=list(parent))
        x[name][at] = value
        acc, tok, path = sv.verify_tree_greedy(i32(x["argmax"]), i32(x["drafts"]),
                                               i32(x["parent"]), i32(k), 20)
        assert sv.verify_tree_greedy_error() == (code, b, -1)
        lo, hi = (0, 4, 10, 13)[b:b + 2]
        assert acc[b] == -1 and (tok[lo:hi] == -1).all() and (path[lo:hi] == -1).all()
        keep = np.r_[0:lo, hi:13]
        assert np.array_equal(tok.cpu().numpy()[keep], want[1][keep])
    for bad, code in (([3, 64, 2], 16), ([3, -1, 2], 16), ([3, 4, 2], 21)):
        got = sv.verify_tree_greedy(i32(argmax), i32(drafts), i32(parent), i32(bad), 20)
        assert sv.verify_tree_greedy_error()[0] == code
        assert all((x == -1).all() for x in got)
    none = i32([])
    sv.verify_tree_greedy(none, none, none, none, 20)
    assert sv.verify_tree_greedy_error() == (0, -1, -1)


# ----------------------------------------------------------------------- commit
@pytest.mark.parametrize("B,dtype", [(1, B16), (40, F16), (1025, F32)])
def test_commit_of_the_accepted_path(B, dtype):
    rng, g = random.Random(B), torch.Generator().manual_seed(B)
    S, layers, E = 4, 2, 16
    k = [rng.randint(0, 63 if B < 100 else 9) for _ in range(B)]
    argmax, drafts, parent = verify_case(B, k, 30, 0.9)
    n = [rng.randint(0, 11) for _ in range(B)]
    accept, _, path = ot.verify_greedy(argmax, drafts, parent, k)
    accept[0] = accept[0] if B == 1 else -1
    cols = (11 + 64) // S + 1
    table = torch.randperm(B * cols, generator=g).int().view(B, cols)
    cache = torch.randn(B * cols, layers, 2, S, E, generator=g).to(dtype)
    spec = torch.randn(B, max(k) + 1, layers, 2, E, generator=g).to(dtype)
    # the oracle's commit of a chain, from the path's entries
    ints = torch.int16 if cache.element_size() == 2 else torch.int32
    ref, moved = cache.view(ints).numpy().copy(), spec.view(ints).numpy().copy()
    t = 0
    for b, x in enumerate(k):
        for i in range(max(0, accept[b] + 1)):
            moved[b, i] = spec.view(ints).numpy()[b, path[t + i]]
        t += x + 1
    length, _ = okv.kv_commit(moved, accept, k, n, table.numpy(), ref, S)
    c, kv_len = cache.to(DEV), i32(n)
    sv.kv_commit(c, spec.to(DEV), i32(accept.tolist()), i32(k), kv_len, table.to(DEV),
                 path=i32(path.tolist()))
    assert sv.kv_commit_error()[0] == 0
    assert np.array_equal(c.cpu().view(ints).numpy(), ref)
    assert np.array_equal(kv_len.cpu().numpy(), length)


def test_commit_errors_of_paths():
    k, n = [3, 2], [1, 0]
    cache = torch.zeros(4, 1, 2, 8, 8, device=DEV)
    spec = torch.ones(2, 4, 1, 2, 8, device=DEV)
    table = i32([[0, 1], [2, 3]])
    for path, kk, code, grown in (([0, 4, -1, -1, 0, -1, -1], k, 29, [1, 1]),
                                  ([0, -1, -1, -1, 0, -1, -1], k, 29, [1, 1]),
                                  ([0, 1, -1, -1, 0, -1, -1], [3, 3], 21, [1, 0]),
                                  ([0, 1, -1, -1, 0, -1, -1], [64, 2], 16, [1, 0])):
        c, kv_len = cache.clone(), i32(n)
        sv.kv_commit(c, spec, i32([1, 0]), i32(kk), kv_len, table, path=i32(path))
        assert sv.kv_commit_error()[0] == code
        assert kv_len.tolist() == grown
        assert float(c[:2].sum()) == 0 and float(c[2:].sum()) == 16 * (grown[1] == 1)
