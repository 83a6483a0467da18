"""Oracle of attention over the paged KV cache and of its accumulated weights.

TEST INFRASTRUCTURE ONLY: the plain definition in numpy loops (float64).  Only
tests/ and __graft_entry__.smoke() may use it; the CUDA library never does.

Request b has query tokens j = 0 .. k_b (the last emitted token and its drafts)
and sees, per KV head h, the keys of its cached positions 0 .. kv_len_b - 1
(page block_table[b, p // S], slot p % S) and, with a speculative buffer, its
entries as positions kv_len_b + i.  Token j sits at kv_len_b + j (with the
buffer) or kv_len_b - 1 - k_b + j (without: its entry is cached already), sees
the positions up to its own and with a window W only the last W of them:

  s_p = scale q . K_p,  lse = ln sum_p exp s_p,  out = sum_p exp(s_p - lse) V_p,
  score[b, p] += sum over the counted tokens and heads of exp(s_p - lse).

A token that sees nothing has out 0 and lse -inf.
"""

from __future__ import annotations

import numpy as np


def as_f64(x):
    import torch
    return x.detach().to("cpu", torch.float64).numpy() if isinstance(x, torch.Tensor) \
        else np.asarray(x, np.float64)


def position(n, k, j, with_spec):
    return n + j if with_spec else n - 1 - k + j


def visible(n, k, j, with_spec, window):
    """Positions token j sees, as a range."""
    at = position(n, k, j, with_spec)
    lo = max(0, at - window + 1) if window > 0 else 0
    return range(lo, max(lo, at + 1))


def entry(cache, spec, table, b, p, n, layer):
    """[2, E] of position p of request b."""
    if p >= n:
        return spec[b, p - n, layer]
    S = cache.shape[3]
    return cache[int(table[b][p // S]), layer, :, p % S]


def attention(q, cache, layer, kv_len, table, k_per_req, spec=None, scale=None, window=0,
              magnitude=False):
    """Returns (out, lse); with magnitude also sum_p w |V_p| and max_p scale sum |q K_p|."""
    q, cache = as_f64(q), as_f64(cache)
    spec = None if spec is None else as_f64(spec)
    rows, Hq, D = q.shape
    Hk = cache.shape[4] // D
    scale = D ** -0.5 if scale is None else scale
    out, lse = np.zeros((rows, Hq, D)), np.full((rows, Hq), -np.inf)
    mag, size = np.zeros((rows, Hq, D)), np.zeros((rows, Hq))
    t = 0
    for b, (n, k) in enumerate(zip(kv_len, k_per_req)):
        for j in range(int(k) + 1):
            see = visible(int(n), int(k), j, spec is not None, window)
            if len(see):
                kv = np.stack([entry(cache, spec, table, b, p, int(n), layer) for p in see])
                for hq in range(Hq):
                    h = hq // (Hq // Hk)
                    K, V = kv[:, 0, h * D:(h + 1) * D], kv[:, 1, h * D:(h + 1) * D]
                    s = K @ q[t, hq] * scale
                    top = s.max()
                    w = np.exp(s - top)
                    lse[t, hq] = top + np.log(w.sum())
                    w /= w.sum()
                    out[t, hq] = w @ V
                    mag[t, hq] = w @ np.abs(V)
                    size[t, hq] = (np.abs(K) @ np.abs(q[t, hq])).max() * abs(scale)
            t += 1
    return (out, lse, mag, size) if magnitude else (out, lse)


def weights(q, cache, layer, kv_len, table, k_per_req, lse, score, spec=None, accept_len=None,
            scale=None, window=0):
    q, cache, lse = as_f64(q), as_f64(cache), as_f64(lse)
    spec = None if spec is None else as_f64(spec)
    score = as_f64(score).copy()
    rows, Hq, D = q.shape
    Hk = cache.shape[4] // D
    scale = D ** -0.5 if scale is None else scale
    t = 0
    for b, (n, k) in enumerate(zip(kv_len, k_per_req)):
        last = int(k) if accept_len is None else int(accept_len[b])
        for j in range(last + 1):
            for p in visible(int(n), int(k), j, spec is not None, window):
                e = entry(cache, spec, table, b, p, int(n), layer)
                for hq in range(Hq):
                    h = hq // (Hq // Hk)
                    s = e[0, h * D:(h + 1) * D] @ q[t + j, hq] * scale
                    score[b, p] += np.exp(s - lse[t + j, hq])
        t += int(k) + 1
    return score
