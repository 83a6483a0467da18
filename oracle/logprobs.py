"""Oracle of the log probabilities of given tokens, the entropy, the most likely
alternatives and the gradient with respect to the logits.

TEST INFRASTRUCTURE ONLY: the plain definition in numpy (float64).  Only tests/
and __graft_entry__.smoke() may use it; the CUDA library never does.

With z = x / T (T = 1 where it is 0 or not given), p = softmax(z), t the row's
token: log p_t, H = -sum p ln p (0 ln 0 = 0), the largest logits in order
(lowest index on ties, probability 0 left out), and for a loss with gradients
g of log p_t and h of H

  dL/dx_y = (1/T) (g ([y = t] - p_y) - h p_y (ln p_y + H)).
"""

from __future__ import annotations

import numpy as np


def row(x, token, T, n_top):
    """(logprob, entropy, max, logsum, tokens [n_top], logprobs [n_top], log p [V], p)."""
    x = np.asarray(x, np.float64)
    T = np.float64(T) if T else 1.0
    m = x.max()
    y = (x - m) / T
    logsum = np.log(np.exp(y).sum())
    lp = y - logsum
    p = np.exp(lp)
    H = -(p[p > 0] * lp[p > 0]).sum()
    order = [i for i in np.lexsort((np.arange(len(x)), -x)) if x[i] > -np.inf][:n_top]
    tok = np.full(n_top, -1, np.int32)
    top = np.full(n_top, -np.inf)
    tok[:len(order)] = order
    top[:len(order)] = lp[order]
    return (lp[token] if token >= 0 else np.nan), H, m, logsum, tok, top, lp, p


def grad_row(x, token, T, g, h):
    _, H, _, _, _, _, lp, p = row(x, token, T, 0)
    T = np.float64(T) if T else 1.0
    one = np.zeros_like(p)
    one[token] = 1.0
    with np.errstate(invalid="ignore"):
        ent = np.where(p > 0, p * (lp + H), 0.0)
    return (g * (one - p) - h * ent) / T
