"""Distillation from a teacher's k best ids, loss and gradient (fp64 oracle).

Test infrastructure only; see the package docstring.
"""
from __future__ import annotations

import numpy as np


def distill(logits, top_ids, top_logp, inv_map=None, rest: bool = True, temperature: float = 1.0,
            grad_loss=None):
    """logits [R, K], top_ids and top_logp [R, k].  Returns dict(loss [R], grad [R,
    K], p, pull [R, K], mass, left, lnq [R], bad [R]): p = softmax(z / T); pull:
    what the teacher adds to the gradient of each id (before weight and 1 / T; minus for
    listed ids); mass and left: the teacher's on the kept entries and apart from
    them.  Rows that are flagged are NaN."""
    z = np.asarray(logits, dtype=np.float64)
    R, K = z.shape
    k = top_ids.shape[1]
    out = dict(loss=np.zeros(R), grad=np.zeros((R, K)), p=np.zeros((R, K)), pull=np.zeros((R, K)),
               mass=np.zeros(R), left=np.zeros(R), lnq=np.zeros(R), bad=np.zeros(R, bool))
    V = K if inv_map is None else len(inv_map)
    for r in range(R):
        at, lnt, bad, given = [], [], False, False
        for i in range(k):
            t = int(top_ids[r, i])
            if t == -1:
                continue
            if t < 0 or t >= V:
                bad = True
                continue
            j = t if inv_map is None else int(inv_map[t])
            if j == -1:
                continue
            if j < 0 or j >= K:
                bad = True
                continue
            given = True
            if z[r, j] == -np.inf:
                continue
            lp = float(top_logp[r, i])
            bad |= j in at or not lp < 80.0
            at.append(j)
            lnt.append(lp)
        if given and (np.isnan(z[r]).any() or z[r].max() == np.inf):
            bad |= len(at) > 0
        if bad:
            out["bad"][r] = True
            for n in ("loss", "grad"):
                out[n][r] = np.nan
            continue
        if not at:
            continue
        at, lnt = np.array(at), np.array(lnt)
        with np.errstate(divide="ignore"):
            d = (z[r] - z[r].max()) / temperature
            lse = np.log(np.exp(d).sum())
            lnp = d - lse
            un = np.ones(K, bool)
            un[at] = False
            t = np.exp(lnt)
            a = t.sum()
            b, lnq = 0.0, 0.0
            if rest and un.any() and d[un].max() > -np.inf:
                b = max(0.0, 1.0 - a)
                # (relative to their own maximum: of lnp - lnq nothing is left where both are far from 0)
                share = np.exp((z[r][un] - z[r][un].max()) / temperature)
                lnq = d[un].max() + np.log(share.sum()) - lse
                share /= share.sum()
            scale = 1.0 if rest else (1.0 / a if a > 0 else 0.0)
            if not (a + b > 0 and scale > 0):
                continue
            pos = t > 0
            loss = scale * (t[pos] * (lnt[pos] - lnp[at][pos])).sum()
            if not rest:
                loss -= np.log(a)
            if b > 0:
                loss += b * (np.log(b) - lnq)
        p = np.exp(lnp)
        pull = np.zeros(K)
        pull[at] = -t * scale
        if b > 0:
            pull[un] = -b * share
        A = (a + b) * scale
        w = 1.0 if grad_loss is None else float(grad_loss[r])
        out["loss"][r] = loss
        out["grad"][r] = (A * p + pull) * w / temperature
        out["p"][r], out["pull"][r] = A * p, pull
        out["mass"][r], out["left"][r], out["lnq"][r] = a * scale, b, lnq
    return out
