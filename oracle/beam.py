"""One step of beam search and the reordering of states (fp64 oracle).

Test infrastructure only; see the package docstring.
"""
from __future__ import annotations

import numpy as np


def beam_select(logits, scores, n: int, temperature: float = 1.0, trim_ids=None, done=None, end_id: int = -1):
    """logits [B, W, K], scores [B, W] (float64-convertible).  Returns dict(scores,
    parent, tokens, done [B, n], bad, gap [B]): candidates of beam w are its
    score + log softmax(logits / T); ids and beams at -infinity have none, beams
    that have ended one.  bad: a beam with a NaN or +infinity.  gap: the smallest
    nonzero distance between candidates of two beams that decides the order."""
    l = np.asarray(logits, dtype=np.float64)
    s = np.asarray(scores, dtype=np.float64)
    B, W, K = l.shape
    out = dict(scores=np.full((B, n), -np.inf), parent=np.full((B, n), -1, np.int64),
               tokens=np.full((B, n), -1, np.int64), done=np.zeros((B, n), bool), bad=np.zeros((B, W), bool),
               gap=np.full(B, np.inf))
    for b in range(B):
        cands = []  # (score, beam, index, token, ended)
        for w in range(W):
            if s[b, w] == -np.inf:
                continue
            if not np.isfinite(s[b, w]):
                out["bad"][b, w] = True
                continue
            if done is not None and done[b][w]:
                cands.append((s[b, w], w, 0, end_id, True))
                continue
            x = l[b, w]
            if np.isnan(x).any() or x.max() == np.inf:
                out["bad"][b, w] = True
                continue
            if x.max() == -np.inf:
                continue
            d = (x - x.max()) / temperature
            v = d - np.log(np.exp(d).sum()) + s[b, w]
            order = np.lexsort((np.arange(K), -(x + 0.0)))[:n]
            for j in order:
                if x[j] > -np.inf:
                    t = int(trim_ids[j]) if trim_ids is not None else int(j)
                    cands.append((v[j], w, int(j), t, end_id >= 0 and t == end_id))
        # within a beam the order is that of the logits: a stable sort on the score keeps it
        cands.sort(key=lambda c: -c[0])
        for i, (v, w, _, t, e) in enumerate(cands[:n]):
            out["scores"][b, i], out["parent"][b, i], out["tokens"][b, i], out["done"][b, i] = v, w, t, e
        for x, y in zip(cands[:n], cands[1:n + 1]):
            if x[1] != y[1] and x[0] != y[0]:
                out["gap"][b] = min(out["gap"][b], x[0] - y[0])
    return out


def beam_reorder(state, parent, out, dim: int = 0, lengths=None, len_dim=None):
    """numpy arrays; returns a copy of `out` with the parents' states in its slots."""
    src, dst = np.asarray(state), np.array(out)
    for b in range(parent.shape[0]):
        for i, p in enumerate(parent[b]):
            if p < 0 or p >= src.shape[dim + 1]:
                continue
            at = [slice(None)] * src.ndim
            at[dim] = b
            if lengths is not None:
                at[len_dim] = slice(0, max(0, int(lengths[b])))
            at[dim + 1] = i
            to = tuple(at)
            at[dim + 1] = int(p)
            dst[to] = src[tuple(at)]
    return dst
