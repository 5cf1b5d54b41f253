"""Page keys, page scores, page selection and the attention over selected pages, in fp64.

TEST INFRASTRUCTURE: only tests/ use this file. It shares no code with the CUDA path.

Reading: blocks are the cache's 64-position pages; a page's key is the mean of its rows [c ; k_r]; a token's
score of a page is the sum over its heads of the softmax, over the pages it sees, of sm_scale q · key;
all heads of a token attend the same pages, since all of them read the same latent rows.
"""
from __future__ import annotations

import math

import numpy as np

from . import mla_oracle as O

f64 = np.float64
PAGE = 64


def visible_pages(seqlen, s_q, t):
    """Pages with a position below seqlen - s_q + t + 1."""
    vis = seqlen - s_q + t + 1
    return max(0, -(-vis // PAGE))


def page_keys(rows):
    """Mean row of every page of rows [L, W] (the last page's mean is over the rows it has)."""
    rows = np.asarray(rows, f64)
    return np.stack([rows[p:p + PAGE].mean(0) for p in range(0, len(rows), PAGE)])


def page_scores(q, keys, sm_scale):
    """score [n] of keys [n, W] for the heads q [H, W] of one token."""
    if len(keys) == 0:
        return np.zeros(0)
    u = sm_scale * (np.asarray(q, f64) @ np.asarray(keys, f64).T)
    e = np.exp(u - u.max(1, keepdims=True))
    return (e / e.sum(1, keepdims=True)).sum(0)


def select(scores, k, n_first, n_recent):
    """Ascending indices of the min(k, n) kept pages: the first n_first and last n_recent, then by score
    (ties to the lower index, NaN below every number)."""
    n = len(scores)

    def order(p):
        s = float(scores[p])
        forced = p < n_first or p >= n - n_recent
        return (0 if forced else 1, 1 if math.isnan(s) else 0, 0.0 if math.isnan(s) else -s, p)

    # forced pages never compete: their own order among themselves does not matter (all are kept)
    return sorted(sorted(range(n), key=order)[:min(k, n)])


def sparse_decode(q_abs, c, k_r, pages, visible, sm_scale):
    """One token: q_abs [H, d_c + d_r] over the positions below `visible` of the listed pages of the rows c
    [L, d_c], k_r [L, d_r]. Returns (o_lat [H, d_c], lse [H]); zeros and -inf when nothing is attended."""
    pos = np.concatenate([np.arange(p * PAGE, min(p * PAGE + PAGE, visible)) for p in pages]).astype(int) \
        if len(pages) else np.zeros(0, int)
    H, d_c = len(q_abs), c.shape[1]
    if len(pos) == 0:
        return np.zeros((H, d_c)), np.full(H, -np.inf)
    o, lse = O.absorbed_decode(np.asarray(q_abs, f64)[None], np.asarray(c, f64)[pos], np.asarray(k_r, f64)[pos],
                               len(pos), sm_scale)
    return o[0], lse[0]
