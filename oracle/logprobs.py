"""Log probabilities of given tokens, entropy and top alternatives (fp64
oracle): p = softmax(l / T) of a row, where an id at -infinity has p = 0.

Test infrastructure only; see the package docstring.
"""
from __future__ import annotations

import numpy as np


def token_logprobs(logits, tokens, k: int, temperature: float = 1.0):
    """Rows of logits [R, V] (float64-convertible), tokens [R] (-1: not
    scored).  Returns dict(logp [R], entropy [R], top_ids [R, k], top_logp
    [R, k], bad [R]): bad rows (a NaN, +infinity or no finite logit) and
    rows that are not scored hold NaN and -1; a token outside [0, V) has a NaN
    logp."""
    l = np.asarray(logits, dtype=np.float64)
    R, V = l.shape
    out = dict(logp=np.full(R, np.nan), entropy=np.full(R, np.nan),
               top_ids=np.full((R, k), -1, np.int64), top_logp=np.full((R, k), np.nan),
               bad=np.zeros(R, bool))
    for r in range(R):
        t = int(tokens[r])
        if t == -1:
            continue
        x = l[r]
        if np.isnan(x).any() or not np.isfinite(x.max()):
            out["bad"][r] = True
            continue
        d = (x - x.max()) / temperature
        e = np.exp(d)
        lp = d - np.log(e.sum())
        p = np.exp(lp)
        if 0 <= t < V:
            out["logp"][r] = lp[t]
        out["entropy"][r] = -(p[p > 0] * lp[p > 0]).sum()
        ids = np.lexsort((np.arange(V), -(x + 0.0)))[:k]
        out["top_ids"][r] = ids
        out["top_logp"][r] = lp[ids]
    return out
