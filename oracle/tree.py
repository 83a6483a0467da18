"""Oracles of trees of drafts: their attention over the paged cache, their greedy
verification, and the path that the cache's commit takes.

TEST INFRASTRUCTURE ONLY: plain definitions in numpy loops.  Only tests/ and
__graft_entry__.smoke() may use it; the CUDA library never does.

Node 0 of a request is its last emitted token, nodes 1 .. k its drafts; node j
hangs from the earlier node parent[j].  A node lies one position behind its parent,
node 0 at position kv_len, and sees the cached positions, its ancestors and itself
(with a window W the last W positions of these).  Greedy verification walks from
node 0 to the child whose token is the target's argmax at the node, the lowest such
child, until there is none.
"""

from __future__ import annotations

import numpy as np

from .attention import as_f64, entry


def way(parent, j):
    """Nodes from node 0 to node j."""
    path = [j]
    while path[0] > 0:
        path.insert(0, int(parent[path[0]]))
    return path


def attention(q, cache, layer, kv_len, table, k_per_req, parent, spec, scale=None, window=0,
              magnitude=False):
    """As oracle.attention.attention, over trees."""
    q, cache, spec = as_f64(q), as_f64(cache), as_f64(spec)
    rows, Hq, D = q.shape
    Hk = cache.shape[4] // D
    scale = D ** -0.5 if scale is None else scale
    out, lse = np.zeros((rows, Hq, D)), np.full((rows, Hq), -np.inf)
    mag, size = np.zeros((rows, Hq, D)), np.zeros((rows, Hq))
    t = 0
    for b, (n, k) in enumerate(zip(kv_len, k_per_req)):
        n, k = int(n), int(k)
        for j in range(k + 1):
            path = way(parent[t:t + k + 1], j)
            at = n + len(path) - 1
            seen = [(p, p) for p in range(n)] + [(n + d, n + x) for d, x in enumerate(path)]
            seen = [key for pos, key in seen if not window or pos > at - window]
            kv = np.stack([entry(cache, spec, table, b, p, n, layer) for p in seen])
            for hq in range(Hq):
                h = hq // (Hq // Hk)
                K, V = kv[:, 0, h * D:(h + 1) * D], kv[:, 1, h * D:(h + 1) * D]
                s = K @ q[t + j, hq] * scale
                top = s.max()
                w = np.exp(s - top)
                lse[t + j, hq] = top + np.log(w.sum())
                w /= w.sum()
                out[t + j, hq] = w @ V
                mag[t + j, hq] = w @ np.abs(V)
                size[t + j, hq] = (np.abs(K) @ np.abs(q[t + j, hq])).max() * abs(scale)
        t += k + 1
    return (out, lse, mag, size) if magnitude else (out, lse)


def verify_greedy(argmax, drafts, parent, k_per_req):
    """(accept_len [B], tokens [rows], path [rows])."""
    accept, tokens, paths, t = [], [], [], 0
    for b, k in enumerate(k_per_req):
        k = int(k)
        path = [0]
        while True:
            best = argmax[t + path[-1]]
            nxt = [j for j in range(1, k + 1)
                   if parent[t + j] == path[-1] and drafts[t - b + j - 1] == best]
            if not nxt:
                break
            path.append(nxt[0])
        rest = [-1] * (k + 1 - len(path))
        accept.append(len(path) - 1)
        tokens += [int(argmax[t + j]) for j in path] + rest
        paths += path + rest
        t += k + 1
    return np.array(accept, np.int32), np.array(tokens, np.int32), np.array(paths, np.int32)
