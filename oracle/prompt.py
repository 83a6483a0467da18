"""Oracle of causal attention over packed prompts.

TEST INFRASTRUCTURE ONLY: the plain definition in numpy loops (float64).  Only
tests/ and __graft_entry__.smoke() may use it; the CUDA library never does.

Sequence b has rows offsets[b] .. offsets[b + 1] - 1.  Its token i sees its tokens
max(0, i - W + 1) .. i (all up to i without a window):

  s_j = scale q_i . k_j,  lse = ln sum_j exp s_j,  out = sum_j exp(s_j - lse) v_j.
"""

from __future__ import annotations

import numpy as np

from .attention import as_f64


def prompt_attention(q, k, v, offsets, scale=None, window=0, magnitude=False):
    """(out, lse), NaN for rows of no sequence; with magnitude also sum_j w |v_j| and
    max_j scale sum |q k_j|."""
    q, k, v = as_f64(q), as_f64(k), as_f64(v)
    rows, Hq, D = q.shape
    G = Hq // k.shape[1]
    scale = D ** -0.5 if scale is None else scale
    out, lse = np.full((rows, Hq, D), np.nan), np.full((rows, Hq), np.nan)
    mag, size = np.zeros((rows, Hq, D)), np.zeros((rows, Hq))
    for a, e in zip(offsets[:-1], offsets[1:]):
        for i in range(int(a), int(e)):
            lo = max(int(a), i - window + 1) if window else int(a)
            for h in range(Hq):
                K, V = k[lo:i + 1, h // G], v[lo:i + 1, h // G]
                s = K @ q[i, h] * scale
                top = s.max()
                w = np.exp(s - top)
                lse[i, h] = top + np.log(w.sum())
                w /= w.sum()
                out[i, h] = w @ V
                mag[i, h] = w @ np.abs(V)
                size[i, h] = (np.abs(K) @ np.abs(q[i, h])).max() * abs(scale)
    return (out, lse, mag, size) if magnitude else (out, lse)
