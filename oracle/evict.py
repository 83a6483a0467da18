"""Oracle of eviction from the paged KV cache by accumulated attention weight.

TEST INFRASTRUCTURE ONLY: the plain definition in numpy loops.  Only tests/ and
__graft_entry__.smoke() may use it; the CUDA library never does.

A request of n > budget positions keeps its first `sinks`, its last `recent`
and the highest scores among the others (lowest position on ties, NaN below
every number).  Kept positions keep their order and move to positions 0 ..
budget - 1 in every layer, K and V; the scores move along, the rest of them
becomes 0.
"""

from __future__ import annotations

import numpy as np

EVICT_OK = 0
EVICT_ERR_PAGE = 27
EVICT_ERR_LENGTH = 28


def choose(score, n, budget, sinks, recent):
    """The kept positions of one request, increasing."""
    if n <= budget:
        return list(range(n))
    others = range(sinks, n - recent)

    def rank(p):
        s = float(score[p])
        return (1, 0.0, p) if s != s else (0, -s, p)

    best = sorted(others, key=rank)[:budget - sinks - recent]
    return sorted(list(range(sinks)) + best + list(range(n - recent, n)))


def kv_evict(cache, score, kv_len, table, budget, sinks, recent, dst=None, dst_table=None):
    """In place in `cache` (or `dst`) and `score`.  Returns (lengths, kept, status)."""
    S = cache.shape[3]
    B = len(kv_len)
    out = cache if dst is None else dst
    to = table if dst is None else dst_table
    lengths = np.array(kv_len, np.int64).copy()
    kept = np.full((B, budget), -1, np.int32)
    status = np.zeros(B, np.int32)
    for b in range(B):
        n = int(kv_len[b])
        m = min(n, budget)
        if n < 0 or n > score.shape[1] or n > table.shape[1] * S or m > to.shape[1] * S:
            status[b] = EVICT_ERR_LENGTH
        elif any(not 0 <= table[b, c] < cache.shape[0] for c in range(-(-n // S))) or \
                any(not 0 <= to[b, c] < out.shape[0] for c in range(-(-m // S))):
            status[b] = EVICT_ERR_PAGE
        if status[b]:
            if dst is not None:
                lengths[b] = -1
            continue
        keep = choose(score[b], n, budget, sinks, recent)
        moved = [cache[table[b, p // S], :, :, p % S].copy() for p in keep]
        for i, e in enumerate(moved):
            out[to[b, i // S], :, :, i % S] = e
        values = [score[b, p] for p in keep]
        score[b, :n] = 0
        score[b, :len(keep)] = values
        kept[b, :len(keep)] = keep
        lengths[b] = len(keep)
    return lengths.astype(np.int32), kept, status
