"""Cases, plain forms and 64-bit definitions of the drafter's beam search and of its distillation.

* ``select``: one step of beam search over beams and vocabulary.  Each sequence's
  W beams with their scores and rows of logits give the N best continuations by
  score + log softmax(logits / T) (``vt_beam_select``).
* ``reorder``: the states of the beams (hidden states, token histories, caches)
  moved to the beams that continue them (``vt_beam_reorder``).
* ``loss``: distillation from a teacher's k best ids and their log probabilities,
  as ``vt_token_logprobs`` returns them, over the drafter's (trimmed) vocabulary
  (``vt_distill_loss``).
* ``grad``: the gradient of that loss with respect to the drafter's logits, from
  the statistics that the loss kept (``vt_distill_grad``).
* ``train``: loss and gradient in one call, as a training step wants them
  (``vt_distill_loss_grad``).

``run`` computes the plain forms with elementary torch operations where
``own`` is false, and calls the library where it is true.
"""
from __future__ import annotations

import math
import random

import torch

own = False


# ------------------------------------------------------------------- cases
def listed():
    return [
        # the first level of one draft tree: the root's eight best, where latency counts
        {"name": "select-root", "op": "select", "B": 1, "W": 1, "N": 8, "K": 32768, "dtype": "f32", "T": 1.0,
         "pad": 0, "masked": 0.0, "trimmed": True, "ends": False},
        # a deeper level of the drafting batch's trees: eight beams each over the trimmed vocabulary
        {"name": "select-trees", "op": "select", "B": 16, "W": 8, "N": 8, "K": 32768, "dtype": "f32", "T": 1.0,
         "pad": 0, "masked": 0.0, "trimmed": True, "ends": False},
        # constrained beam search: most ids masked with -inf, finished beams, odd sizes behind a padded stride
        {"name": "select-masked", "op": "select", "B": 13, "W": 5, "N": 7, "K": 32003, "dtype": "bf16", "T": 1.3,
         "pad": 13, "masked": 0.97, "trimmed": False, "ends": True},
        # the wide batch of the large drafting workload
        {"name": "select-large", "op": "select", "B": 256, "W": 8, "N": 8, "K": 38016, "dtype": "f32", "T": 0.7,
         "pad": 0, "masked": 0.0, "trimmed": True, "ends": False},
        # token histories of ragged beams: rows of four bytes, odd numbers of them
        {"name": "reorder-history", "op": "reorder", "kind": "history", "B": 50, "W": 5, "S": 1031},
        # keys and values of a drafter of one layer, half full on average
        {"name": "reorder-cache", "op": "reorder", "kind": "cache", "B": 16, "W": 8, "heads": 8, "S": 1024, "D": 64},
        # evaluation on the positions of the verification workload over the whole vocabulary
        {"name": "loss-verify", "op": "loss", "B": 16, "gamma": 6, "K": 128256, "dtype": "f32", "k": 8, "T": 1.0,
         "pad": 0, "trimmed": False, "rest": True, "emitted": True},
        # evaluation on every position of the large workload over the trimmed vocabulary
        {"name": "loss-large", "op": "loss", "B": 256, "gamma": 8, "K": 38016, "dtype": "bf16", "k": 20, "T": 0.7,
         "pad": 0, "trimmed": True, "rest": False, "emitted": False},
        # a small ragged batch: no size a multiple of anything, a padded stride
        {"name": "grad-ragged", "op": "grad", "B": 29, "gamma": 6, "K": 10007, "dtype": "f32", "k": 5, "T": 1.3,
         "pad": 9, "trimmed": True, "rest": True, "emitted": True},
        # the backward pass over every position of the large workload
        {"name": "grad-large", "op": "grad", "B": 256, "gamma": 8, "K": 38016, "dtype": "bf16", "k": 20, "T": 0.7,
         "pad": 0, "trimmed": True, "rest": True, "emitted": False},
        # a training batch over the trimmed vocabulary, fp32 logits as the drafter's head gives them
        {"name": "train-trimmed", "op": "train", "B": 256, "gamma": 7, "K": 32768, "dtype": "f32", "k": 32, "T": 1.0,
         "pad": 0, "trimmed": True, "rest": True, "emitted": False},
        # a training batch over a whole vocabulary with a long list; positions behind the last emitted token hold -1
        {"name": "train-full", "op": "train", "B": 128, "gamma": 7, "K": 128256, "dtype": "bf16", "k": 100, "T": 2.0,
         "pad": 0, "trimmed": False, "rest": False, "emitted": True},
    ]


_MOST_SELECT = 256 * 8 * 38016  # elements of the largest listed cases
_MOST_DISTILL = 256 * 8 * 32768
_MOST_CACHE = 2 * 16 * 8 * 8 * 1024 * 64


def _log_int(rng: random.Random, lo: int, hi: int) -> int:
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng: random.Random):
    op = rng.choice(["select", "select", "reorder", "loss", "grad", "train"])
    T = rng.choice([0.7, 1.0, 1.3, 2.0])
    dtype = rng.choice(["f32", "bf16"])
    pad = rng.choice([0, 0, rng.randint(1, 64)])
    if op == "select":
        W, K = rng.choice([1, rng.randint(2, 16), rng.randint(2, 32)]), _log_int(rng, 500, 152064)
        B = _log_int(rng, 1, max(1, min(256, _MOST_SELECT // (W * K))))
        return {"op": op, "B": B, "W": W, "N": rng.randint(1, 32) if rng.random() < 0.5 else min(32, max(W, 2)), "K": K,
                "dtype": dtype, "T": T, "pad": pad, "masked": rng.choice([0.0, 0.0, 0.5, 0.97]),
                "trimmed": rng.random() < 0.5, "ends": rng.random() < 0.5}
    if op == "reorder":
        kind = rng.choice(["history", "hidden", "cache", "cache"])
        W = rng.randint(2, 32)
        if kind == "history":
            return {"op": op, "kind": kind, "B": _log_int(rng, 1, 256), "W": W, "S": _log_int(rng, 1, 4096)}
        if kind == "hidden":
            return {"op": op, "kind": kind, "B": _log_int(rng, 1, 256), "W": W, "S": _log_int(rng, 256, 4096)}
        heads, D = rng.choice([1, 2, 8]), rng.choice([64, 80, 128])
        S = _log_int(rng, 1, 2048)
        B = _log_int(rng, 1, max(1, min(64, _MOST_CACHE // (2 * W * heads * S * D))))
        return {"op": op, "kind": kind, "B": B, "W": W, "heads": heads, "S": S, "D": D}
    gamma, K = rng.randint(0, 8), _log_int(rng, 500, 152064)
    B = _log_int(rng, 1, max(1, min(256, _MOST_DISTILL // ((gamma + 1) * K))))
    return {"op": op, "B": B, "gamma": gamma, "K": K, "dtype": dtype, "k": _log_int(rng, 1, 128), "T": T, "pad": pad,
            "trimmed": rng.random() < 0.5, "rest": rng.random() < 0.5, "emitted": rng.random() < 0.5}


def _size(case) -> int:
    return 4 if case["dtype"] == "f32" else 2


def _lengths(case):
    """The sequences' lengths, in an order that the seed decides: from S / B to S."""
    return [max(1, case["S"] * (b + 1) // case["B"]) for b in range(case["B"])]


def _distinct(W: int) -> int:
    """Beams of W that continue: about what independent choices leave."""
    return max(1, (5 * W + 4) // 8)


def _accepted(case, b: int) -> int:
    """Drafted tokens accepted in sequence b: every count from none to all in turn."""
    return b % (case["gamma"] + 1) if case["emitted"] else case["gamma"]


def work(case):
    op = case["op"]
    if op == "select":
        R, K, N = case["B"] * case["W"], case["K"], case["N"]
        live = R - (case["B"] * (case["W"] // 4) if case["ends"] else 0)
        # per element: a comparison for the list, a difference, a scale, an exponential, a sum
        return {"bytes": live * K * _size(case) + 4 * R + 12 * case["B"] * N, "flops": 5 * live * K}
    if op == "reorder":
        W, kind = case["W"], case["kind"]
        rows = case["B"] if kind == "hidden" else sum(_lengths(case))
        size = 2 * case["S"] if kind == "hidden" else 4 if kind == "history" else 2 * case["heads"] * case["D"] * 2
        return {"bytes": rows * size * (_distinct(W) + W) + 4 * case["B"] * W, "flops": 0}
    R, K, k = case["B"] * (case["gamma"] + 1), case["K"], case["k"]
    live = sum(_accepted(case, b) + 1 for b in range(case["B"]))
    teacher = R * k * 8
    if op == "loss":
        return {"bytes": live * K * _size(case) + teacher + R * 20, "flops": 5 * live * K}
    # rows that are not scored are written (zeros), not read
    return {"bytes": (live + R) * K * _size(case) + teacher + R * (8 if op == "train" else 20),
            "flops": (9 if op == "train" else 4) * live * K}


# ------------------------------------------------------------------- inputs
def _logits(case, rows, g, dev):
    """Rows of logits with a Zipf(1.1) rank bias under normal noise, behind a padded stride."""
    K = case["K"]
    perm = torch.randperm(K, generator=g, device=dev)
    bias = torch.empty(K, dtype=torch.float32, device=dev)
    bias[perm] = -3.3 * torch.arange(1, K + 1, dtype=torch.float32, device=dev).log()
    dt = torch.float32 if case["dtype"] == "f32" else torch.bfloat16
    x = torch.empty((rows, K + case["pad"]), dtype=dt, device=dev).normal_(0.0, 2.0, generator=g)[:, :K]
    x += bias
    return x


def _trim(K, g, dev):
    """K ascending ids of a vocabulary four times as large, and each id's place among them (-1: none)."""
    ids = torch.randperm(4 * K, generator=g, device=dev)[:K].sort().values
    inv = torch.full((4 * K,), -1, dtype=torch.int32, device=dev)
    inv[ids] = torch.arange(K, dtype=torch.int32, device=dev)
    return ids.to(torch.int32), inv


def _temperature(case) -> float:
    """The case's temperature as the fp32 value that the calls take."""
    return float(torch.tensor(case["T"], dtype=torch.float32))


def _prepare_select(case, g, dev):
    B, W, N, K = case["B"], case["W"], case["N"], case["K"]
    logits = _logits(case, B * W, g, dev)
    if case["masked"] > 0.0:
        logits.masked_fill_(torch.rand((B * W, K), generator=g, device=dev) < case["masked"], -math.inf)
    scores = torch.empty((B, W), dtype=torch.float32, device=dev).normal_(-12.0, 2.0, generator=g)
    scores = scores.sort(dim=1, descending=True).values.contiguous()
    trim_ids = _trim(K, g, dev)[0] if case["trimmed"] else None
    state = {"op": "select", "logits": logits.unflatten(0, (B, W)), "scores": scores, "N": N, "T": _temperature(case),
             "trim_ids": trim_ids, "done": None, "end_id": -1,
             "out_scores": torch.empty((B, N), dtype=torch.float32, device=dev),
             "out_parent": torch.empty((B, N), dtype=torch.int32, device=dev),
             "out_tokens": torch.empty((B, N), dtype=torch.int32, device=dev), "out_done": None,
             "status": torch.empty(1, dtype=torch.int32, device=dev)}
    if case["ends"]:
        # a quarter of the beams has ended; the end's id is a frequent one
        done = torch.rand((B, W), generator=g, device=dev).argsort(dim=1) < W // 4
        end = int(logits[0].float().argmax())
        state.update(done=done, end_id=int(trim_ids[end]) if trim_ids is not None else end,
                     out_done=torch.empty((B, N), dtype=torch.bool, device=dev))
    return state


def _prepare_reorder(case, g, dev):
    B, W, kind = case["B"], case["W"], case["kind"]
    if kind == "history":
        shape, dim, len_dim = (B, W, case["S"]), 0, 2
    elif kind == "hidden":
        shape, dim, len_dim = (B, W, case["S"]), 0, None
    else:
        shape, dim, len_dim = (2, B, W, case["heads"], case["S"], case["D"]), 1, 4
    if kind == "history":
        state, out = (torch.randint(0, 128256, shape, generator=g, device=dev, dtype=torch.int32) for _ in range(2))
    else:
        state, out = (torch.empty(shape, dtype=torch.bfloat16, device=dev).normal_(0.0, 1.0, generator=g)
                      for _ in range(2))
    # the first D of a shuffled row of beams continue at least once, the others not
    D = _distinct(W)
    order = torch.rand((B, W), generator=g, device=dev).argsort(dim=1)
    pick = torch.randint(0, D, (B, W), generator=g, device=dev)
    pick[:, :D] = torch.arange(D, device=dev)
    pick = pick.gather(1, torch.rand((B, W), generator=g, device=dev).argsort(dim=1))
    parent = order.gather(1, pick).to(torch.int32)
    lengths = None
    if len_dim is not None:
        lengths = torch.tensor(_lengths(case), dtype=torch.int32, device=dev)
        lengths = lengths[torch.randperm(B, generator=g, device=dev)]
    return {"op": "reorder", "state": state, "out": out, "parent": parent, "dim": dim, "lengths": lengths,
            "len_dim": len_dim, "status": torch.empty(1, dtype=torch.int32, device=dev)}


def _prepare_distill(case, g, dev):
    B, n, K, k = case["B"], case["gamma"] + 1, case["K"], case["k"]
    R = B * n
    logits = _logits(case, R, g, dev)
    trim_ids, inv_map = _trim(K, g, dev) if case["trimmed"] else (None, None)
    ids = torch.empty((R, k), dtype=torch.int64, device=dev)
    logp = torch.empty((R, k), dtype=torch.float32, device=dev)
    step = max(1, (1 << 26) // K)
    for r in range(0, R, step):  # the teacher agrees with the drafter up to noise
        t = logits[r:r + step].float()
        t = t + torch.empty_like(t).normal_(0.0, 1.0, generator=g)
        top = (t / case["T"]).log_softmax(dim=1).topk(k, dim=1)
        ids[r:r + step], logp[r:r + step] = top.indices, top.values
    if case["trimmed"]:
        # one in ten of the teacher's ids is not in the drafter's vocabulary
        other = (inv_map < 0).nonzero()[:, 0]
        at = torch.randint(0, len(other), (R, 1), generator=g, device=dev)
        at = (at + torch.arange(k, device=dev)) % len(other)
        lost = torch.rand((R, k), generator=g, device=dev) < 0.1
        ids = torch.where(lost, other[at], trim_ids.long()[ids])
    count = torch.tensor([_accepted(case, b) for b in range(B)], device=dev)
    count = count[torch.randperm(B, generator=g, device=dev)]
    skip = (torch.arange(n, device=dev)[None, :] > count[:, None]).view(R, 1)
    ids, logp = ids.masked_fill(skip, -1).to(torch.int32), logp.masked_fill(skip, math.nan)
    weight = torch.rand(R, generator=g, device=dev) * (2.0 / R)
    state = {"op": case["op"], "logits": logits, "top_ids": ids, "top_logp": logp, "inv_map": inv_map,
             "rest": case["rest"], "T": _temperature(case), "weight": weight,
             "loss": torch.empty(R, dtype=torch.float32, device=dev),
             "stats": torch.empty((R, 5), dtype=torch.float32, device=dev),
             "status": torch.empty(1, dtype=torch.int32, device=dev)}
    if case["op"] != "loss":
        state["grad"] = torch.empty((R, K + case["pad"]), dtype=logits.dtype, device=dev)[:, :K]
    if case["op"] == "grad":
        # the statistics that the loss kept for its backward pass
        state["stats"].copy_(_plain_distill({**state, "op": "loss"})["stats"])
    return state


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(int(seed))
    make = {"select": _prepare_select, "reorder": _prepare_reorder}.get(case["op"], _prepare_distill)
    return make(case, g, dev)


# ------------------------------------------------------------- plain forms
def _plain_select(s):
    B, W, K = s["logits"].shape
    N = s["N"]
    n = min(N, K)
    x = s["logits"].float()
    # one integer key per id: the order of the logit above, the lower id first below
    i = (x + 0.0).view(torch.int32)
    key = (i ^ ((i >> 31) & 0x7FFFFFFF)).long() << 32
    key += 0xFFFFFFFF - torch.arange(K, device=x.device)
    ids = 0xFFFFFFFF - (key.topk(n, dim=2).values & 0xFFFFFFFF)
    # scores in 64 bits: two beams' candidates may be as near as 32 bits tell apart
    m = x.amax(dim=2, keepdim=True).double()
    lse = ((x.double() - m) / s["T"]).exp().sum(dim=2, keepdim=True).log()
    cand = (x.gather(2, ids).double() - m) / s["T"] - lse + s["scores"].double()[:, :, None]
    cand = torch.where(x.gather(2, ids) == -math.inf, -math.inf, cand)
    tok = s["trim_ids"].long()[ids] if s["trim_ids"] is not None else ids
    if s["done"] is not None:
        # a beam that has ended continues once, as it is
        first = torch.arange(n, device=x.device) == 0
        stay = torch.where(first, s["scores"].double()[:, :, None], -math.inf)
        cand = torch.where(s["done"][:, :, None], stay, cand)
        tok = torch.where(s["done"][:, :, None], s["end_id"], tok)
    cand = torch.nn.functional.pad(cand.reshape(B, W * n), (0, N), value=-math.inf)
    best = torch.sort(cand, dim=1, descending=True, stable=True)
    score, at = best.values[:, :N], best.indices[:, :N].clamp(max=W * n - 1)
    none = score == -math.inf
    parent = torch.where(none, -1, at // n)
    tokens = torch.where(none, -1, tok.reshape(B, W * n).gather(1, at))
    out = {"scores": score.float(), "parent": parent.to(torch.int32), "tokens": tokens.to(torch.int32)}
    if s["done"] is not None:
        out["done"] = (s["done"].gather(1, parent.clamp(min=0)) | (tokens == s["end_id"])) & ~none
    return out


def _plain_reorder(s):
    state, out, d = s["state"], s["out"], s["dim"]
    at = s["parent"].long()
    at = at.view((1,) * d + at.shape + (1,) * (state.dim() - d - 2))
    moved = torch.take_along_dim(state, at, dim=d + 1)
    if s["lengths"] is not None:
        S = state.shape[s["len_dim"]]
        pos = torch.arange(S, device=state.device).view((S,) + (1,) * (state.dim() - s["len_dim"] - 1))
        n = s["lengths"].view((-1,) + (1,) * (state.dim() - d - 1))
        moved = torch.where(pos < n, moved, out)
    return {"out": out.copy_(moved)}


def _teacher(s):
    """The teacher's entries that the drafter can have: their places, logits and probabilities."""
    ids, x = s["top_ids"].long(), s["logits"]
    place = ids.clamp(min=0)
    if s["inv_map"] is not None:
        place = s["inv_map"].long()[place]
    z = x.gather(1, place.clamp(min=0)).float()
    kept = (ids >= 0) & (place >= 0) & (z > -math.inf)
    logp = torch.where(kept, s["top_logp"], -math.inf)
    t = logp.double().exp()  # the rest of the mass is what 64 bits leave of 1
    return place.clamp(min=0), z, kept, logp, t


def _plain_distill(s):
    x, T = s["logits"].float(), s["T"]
    place, z, kept, logp, t = _teacher(s)
    a = t.sum(dim=1)
    scored = kept.any(dim=1)
    if s["op"] == "grad":
        m, m_rest, c_all, c_rest, c_t = s["stats"].unbind(1)
    else:
        # the listed ids apart from the others, so that neither's sum is a difference
        hide = torch.zeros_like(x).scatter_add_(1, place, kept.float()) > 0
        others = x.masked_fill(hide, -math.inf)
        m_rest = others.amax(dim=1)
        m = torch.maximum(m_rest, torch.where(kept, z, -math.inf).amax(dim=1))
        any_rest = m_rest > -math.inf
        m_rest = torch.where(any_rest, m_rest, 0.0)
        m = torch.where(m == -math.inf, 0.0, m)
        s_rest = ((others - m_rest[:, None]) / T).exp().sum(dim=1).double()
        down = (m_rest.double() - m) / T
        S = torch.where(any_rest, s_rest * down.exp(), 0.0)
        S = S + torch.where(kept, ((z.double() - m[:, None]) / T).exp(), 0.0).sum(dim=1)
        rest = (1.0 - a).clamp(min=0.0) * any_rest * s["rest"]
        scored = scored & ((a > 0) | (rest > 0))
        A = a + rest
        scale = torch.ones_like(a) if s["rest"] else 1.0 / torch.where(a > 0, a, 1.0)
        # ln(t / p) of each listed id and of the rest
        lnp = (z.double() - m[:, None]) / T - S.log()[:, None]
        loss = (t * torch.where(t > 0, logp - lnp, 0.0)).sum(dim=1) * scale + (A * scale) * scale.log()
        lnq = s_rest.log() + down - S.log()
        loss = loss + torch.where(rest > 0, rest * (rest.log() - lnq), 0.0)
        loss = torch.where(scored, loss, 0.0).float()
        c_all, c_t = A * scale / (S * T), scale / T
        c_rest = torch.where(any_rest, A * scale * down.exp() / S - rest / s_rest, 0.0) / T
        m, m_rest, c_all, c_rest, c_t = (torch.where(scored, v, 0.0).float() for v in (m, m_rest, c_all, c_rest, c_t))
        if s["op"] == "loss":
            return {"loss": loss, "stats": torch.stack((m, m_rest, c_all, c_rest, c_t), dim=1)}
    g = s["weight"]
    d = ((x - m_rest[:, None]) / T).exp() * (c_rest * g)[:, None]
    listed = (((z - m[:, None]) / T).exp() * c_all[:, None] - t.float() * c_t[:, None]) * g[:, None]
    listed = torch.where(kept, listed - d.gather(1, place), 0.0)
    d = torch.where(scored[:, None], d.scatter_add_(1, place, listed), 0.0)
    d = d.to(s["logits"].dtype)
    return {"grad": d} if s["op"] == "grad" else {"loss": loss, "grad": d}


def _plain(s):
    if s["op"] == "select":
        return _plain_select(s)
    if s["op"] == "reorder":
        return _plain_reorder(s)
    return _plain_distill(s)


# ------------------------------------------------------------- the library
def _library(s):
    import drafter_sampling_gb300 as vt
    if s["op"] == "select":
        if "workspace" not in s:
            B, W, K = s["logits"].shape
            s["workspace"] = torch.empty(vt.workspace_bytes("beam_select", B=B, W=W, K=K, n=s["N"]), dtype=torch.uint8,
                                         device=s["logits"].device)
        scores, parent, tokens, done, _ = vt.vt_beam_select(
            s["logits"], s["scores"], s["N"], temperature=s["T"], trim_ids=s["trim_ids"], done=s["done"],
            end_id=s["end_id"], out_scores=s["out_scores"], out_parent=s["out_parent"], out_tokens=s["out_tokens"],
            out_done=s["out_done"], dev_status=s["status"], workspace=s["workspace"])
        out = {"scores": scores, "parent": parent, "tokens": tokens}
        return out if done is None else {**out, "done": done}
    if s["op"] == "reorder":
        out, _ = vt.vt_beam_reorder(s["state"], s["parent"], out=s["out"], dim=s["dim"], lengths=s["lengths"],
                                    len_dim=s["len_dim"], dev_status=s["status"])
        return {"out": out}
    if s["op"] == "loss":
        loss, stats, _ = vt.vt_distill_loss(
            s["logits"], s["top_ids"], s["top_logp"], inv_map=s["inv_map"], rest=s["rest"], temperature=s["T"],
            out_loss=s["loss"], out_stats=s["stats"], dev_status=s["status"])
        return {"loss": loss, "stats": stats}
    if s["op"] == "grad":
        return {"grad": vt.vt_distill_grad(s["logits"], s["top_ids"], s["top_logp"], s["stats"], grad_loss=s["weight"],
                                           inv_map=s["inv_map"], temperature=s["T"], out_grad=s["grad"])}
    loss, grad, _, _ = vt.vt_distill_loss_grad(
        s["logits"], s["top_ids"], s["top_logp"], grad_loss=s["weight"], inv_map=s["inv_map"], rest=s["rest"],
        temperature=s["T"], out_loss=s["loss"], out_grad=s["grad"], out_stats=s["stats"], dev_status=s["status"])
    return {"loss": loss, "grad": grad}


def run(state):
    return _library(state) if own else _plain(state)


# ----------------------------------------------------------- 64-bit values
def _exact_select(s):
    B, W, K = s["logits"].shape
    N, dev = s["N"], s["logits"].device
    out = {"scores": torch.full((B, N), -math.inf, dtype=torch.float64, device=dev),
           "parent": torch.full((B, N), -1, dtype=torch.int32, device=dev),
           "tokens": torch.full((B, N), -1, dtype=torch.int32, device=dev)}
    ended = torch.zeros((B, N), dtype=torch.bool, device=dev)
    for b in range(B):
        total = torch.log_softmax(s["logits"][b].double() / s["T"], dim=1) + s["scores"][b].double()[:, None]
        name = s["trim_ids"].long() if s["trim_ids"] is not None else torch.arange(K, device=dev)
        name = name.expand(W, K)
        if s["done"] is not None and bool(s["done"][b].any()):
            over = s["done"][b]
            total[over] = -math.inf
            total[over, 0] = s["scores"][b][over].double()
            name = name.clone()
            name[over] = s["end_id"]
        flat = total.reshape(-1)
        at = flat.argsort(descending=True, stable=True)[:N]
        at = at[flat[at] > -math.inf]
        n = len(at)
        out["scores"][b, :n] = flat[at]
        out["parent"][b, :n] = (at // K).to(torch.int32)
        out["tokens"][b, :n] = name.reshape(-1)[at].to(torch.int32)
        if s["done"] is not None:
            ended[b, :n] = s["done"][b][at // K] | (name.reshape(-1)[at] == s["end_id"])
    return out if s["done"] is None else {**out, "done": ended}


def _exact_reorder(s):
    out, d = s["out"].clone(), s["dim"]
    for b, row in enumerate(s["parent"].tolist()):
        dst, src = out.select(d, b), s["state"].select(d, b)
        if s["lengths"] is not None:
            n = int(s["lengths"][b])
            dst, src = dst.narrow(s["len_dim"] - 1, 0, n), src.narrow(s["len_dim"] - 1, 0, n)
        for to, frm in enumerate(row):
            dst.select(d, to).copy_(src.select(d, frm))
    return {"out": out.double() if out.is_floating_point() else out}


def _exact_distill(s):
    """From the definition, row by row: the drafter's softmax against the teacher's listed ids."""
    R, T, dev = s["logits"].shape[0], s["T"], s["logits"].device
    loss = torch.zeros(R, dtype=torch.float64, device=dev)
    stats = torch.zeros((R, 5), dtype=torch.float64, device=dev)
    grad = torch.zeros(s["logits"].shape, dtype=torch.float64, device=dev) if s["op"] != "loss" else None
    ids = s["top_ids"].long()
    if s["inv_map"] is not None:
        ids = torch.where(ids >= 0, s["inv_map"].long()[ids.clamp(min=0)], -1)
    for r in (ids >= 0).any(dim=1).nonzero()[:, 0].tolist():
        y = s["logits"][r].double() / T
        use = (ids[r] >= 0) & (y[ids[r].clamp(min=0)] > -math.inf)
        if not bool(use.any()):
            continue
        at, lnt = ids[r][use], s["top_logp"][r][use].double()
        lnp = torch.log_softmax(y, dim=0)
        others = torch.ones_like(y, dtype=torch.bool)
        others[at] = False
        p, t = lnp.exp(), lnt.exp()
        b = max(0.0, 1.0 - float(t.sum())) if s["rest"] and bool((p[others] > 0).any()) else 0.0
        if not s["rest"]:
            lnt = lnt - torch.logsumexp(lnt, dim=0)
            t = lnt.exp()
        loss[r] = (t * (lnt - lnp[at])).sum()
        if b > 0:
            lnq = torch.logsumexp(lnp[others], dim=0)
            loss[r] += b * (math.log(b) - lnq)
        # the largest logit of all and of the others, and the factors of the exponentials relative to them
        stats[r, 0], stats[r, 2] = y.max() * T, (t.sum() + b) * lnp.max().exp() / T
        if bool((p[others] > 0).any()):
            stats[r, 1] = y[others].max() * T
            top = lnp[others].max().exp()
            stats[r, 3] = ((t.sum() + b) * top - b * top / p[others].sum()) / T
        stats[r, 4] = (1.0 if s["rest"] else 1.0 / float(s["top_logp"][r][use].double().exp().sum())) / T
        if grad is not None:
            g = p * (t.sum() + b)
            g[at] -= t
            if b > 0:
                g[others] -= b * (lnp[others] - lnq).exp()
            grad[r] = g * (float(s["weight"][r]) / T)
    if s["op"] == "loss":
        return {"loss": loss, "stats": stats}
    return {"grad": grad} if s["op"] == "grad" else {"loss": loss, "grad": grad}


def exact(case, seed):
    s = prepare(case, seed)
    if s["op"] == "select":
        return _exact_select(s)
    if s["op"] == "reorder":
        return _exact_reorder(s)
    return _exact_distill(s)
