"""Cases, plain forms and 64-bit definitions of three operators around the drafter's head.

* ``quantize``: a bf16 head [K, H] to e4m3 with one power-of-two scale per
  128 x 128 block (``vt_quantize_head``).
* ``logits``: the head product in 8-bit floating point.  The hidden states are
  quantised within the call, one scale per row and group of 128 columns, the
  weights carry one scale per 128 x 128 block (``vt_draft_logits_fp8``).
* ``step``: a greedy drafting step through the same product: the one-hot q and
  the drafted token ids (``vt_draft_step_fp8`` at temperature 0).
* ``logprobs``: log probabilities of given tokens under rows of logits, with
  the entropy of each row and its k best alternatives (``vt_token_logprobs``).

``run`` computes the plain forms with elementary torch operations where
``own`` is false, and calls the library where it is true.
"""
from __future__ import annotations

import math
import random

import torch

own = False

BLOCK = 128
E4M3_MAX = 448.0


# ------------------------------------------------------------------- cases
def listed():
    return [
        # the smallest head to quantise: a drafter of a few hundred columns, no size a multiple of 128
        {"name": "quantize-small", "op": "quantize", "K": 1000, "H": 576},
        # the trimmed head of the drafting workload
        {"name": "quantize-trimmed", "op": "quantize", "K": 32768, "H": 2048},
        # an untrimmed head, as a server quantises it once when it loads
        {"name": "quantize-full", "op": "quantize", "K": 128256, "H": 4096},
        # one sequence drafting: the latency of a single token
        {"name": "logits-one", "op": "logits", "B": 1, "K": 32768, "H": 2048, "T": 1.0},
        # the wide batch of the large drafting workload
        {"name": "logits-wide", "op": "logits", "B": 256, "K": 38016, "H": 4096, "T": 0.7},
        # scoring many positions at once (prompts, or a tree's nodes of a whole batch)
        {"name": "logits-many", "op": "logits", "B": 1000, "K": 38016, "H": 4096, "T": 1.0},
        # the drafting batch, greedy as draft trees are grown
        {"name": "step-batch", "op": "step", "B": 16, "K": 32768, "H": 2048},
        # ragged: no size a multiple of the tile, the group or 16
        {"name": "step-ragged", "op": "step", "B": 50, "K": 10007, "H": 1500},
        # a single position answered with its five best alternatives
        {"name": "logprobs-one", "op": "logprobs", "B": 1, "gamma": 0, "V": 128256, "dtype": "f32", "k": 5,
         "T": 1.0, "pad": 0, "masked": 0.0, "emitted": False},
        # the emitted tokens of the verification workload; positions after the last emitted token hold -1
        {"name": "logprobs-verify", "op": "logprobs", "B": 16, "gamma": 6, "V": 128256, "dtype": "f32", "k": 8,
         "T": 1.0, "pad": 0, "masked": 0.0, "emitted": True},
        # every position of the large verification workload
        {"name": "logprobs-large", "op": "logprobs", "B": 256, "gamma": 8, "V": 152064, "dtype": "bf16", "k": 20,
         "T": 0.7, "pad": 0, "masked": 0.0, "emitted": False},
        # constrained decoding: most ids masked with -inf, rows of odd length behind a padded stride
        {"name": "logprobs-masked", "op": "logprobs", "B": 13, "gamma": 3, "V": 32003, "dtype": "bf16", "k": 3,
         "T": 1.3, "pad": 13, "masked": 0.97, "emitted": True},
    ]


def _log_int(rng: random.Random, lo: int, hi: int) -> int:
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng: random.Random):
    op = rng.choice(["quantize", "logits", "logits", "step", "logprobs", "logprobs"])
    if op == "quantize":
        return {"op": op, "K": _log_int(rng, 500, 128256), "H": _log_int(rng, 300, 4096)}
    if op == "logits":
        return {"op": op, "B": _log_int(rng, 1, 1000), "K": _log_int(rng, 500, 38016), "H": _log_int(rng, 256, 4096),
                "T": rng.choice([0.7, 1.0, 1.3])}
    if op == "step":
        return {"op": op, "B": _log_int(rng, 1, 256), "K": _log_int(rng, 500, 38016), "H": _log_int(rng, 256, 4096)}
    return {"op": op, "B": _log_int(rng, 1, 256), "gamma": rng.randint(0, 8), "V": _log_int(rng, 1000, 152064),
            "dtype": rng.choice(["f32", "bf16"]), "k": rng.randint(0, 20), "T": rng.choice([0.7, 1.0, 1.3]),
            "pad": rng.choice([0, 0, rng.randint(1, 64)]), "masked": rng.choice([0.0, 0.0, 0.5, 0.97]),
            "emitted": rng.random() < 0.5}


def _blocks(n: int) -> int:
    return (n + BLOCK - 1) // BLOCK


def _accepted(case, b: int) -> int:
    """Drafted tokens accepted in sequence b: every count from none to all in turn."""
    return b % (case["gamma"] + 1) if case["emitted"] else case["gamma"]


def work(case):
    op = case["op"]
    if op == "quantize":
        K, H = case["K"], case["H"]
        return {"bytes": 3 * K * H + 4 * _blocks(K) * _blocks(H), "flops": 2 * K * H}
    if op in ("logits", "step"):
        B, K, H = case["B"], case["K"], case["H"]
        extra = 8 * B if op == "step" else 0
        return {"bytes": K * H + 4 * _blocks(K) * _blocks(H) + 2 * B * H + 4 * B * K + extra, "flops": 2 * B * K * H}
    R = case["B"] * (case["gamma"] + 1)
    scored = sum(_accepted(case, b) + 1 for b in range(case["B"]))
    size = 4 if case["dtype"] == "f32" else 2
    return {"bytes": scored * case["V"] * size + R * (12 + 8 * case["k"]), "flops": 6 * scored * case["V"]}


# ------------------------------------------------------------------- inputs
def _pow2(e):
    """2^e of an int32 tensor, -126 <= e <= 127, exactly."""
    return ((e + 127) << 23).view(torch.float32)


def _exponent(amax):
    """The smallest e >= -126 with amax <= 448 * 2^e, for fp32 amax >= 0."""
    m, x = torch.frexp(amax)  # amax = m * 2^x, 0.5 <= m < 1; 448 = 0.875 * 2^9
    return (x.to(torch.int32) - 9 + (m > 0.875).to(torch.int32)).clamp(min=-126)


def _quantize_weights(W):
    """(e4m3 [K, H], scales [K/128, H/128]) of a bf16 head, in fp32."""
    K, H = W.shape
    kb, hb = _blocks(K), _blocks(H)
    x = torch.zeros((kb * BLOCK, hb * BLOCK), dtype=torch.float32, device=W.device)
    x[:K, :H] = W
    x = x.view(kb, BLOCK, hb, BLOCK)
    e = _exponent(x.abs().amax(dim=(1, 3)))
    x = (x * _pow2(-e)[:, None, :, None]).view(kb * BLOCK, hb * BLOCK)
    return x[:K, :H].to(torch.float8_e4m3fn), _pow2(e)


def _row_stride(H: int) -> int:
    return (H + 15) // 16 * 16


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(int(seed))
    op = case["op"]
    if op == "quantize":
        K, H = case["K"], case["H"]
        W = torch.empty((K, H), dtype=torch.bfloat16, device=dev).normal_(0.0, 0.02, generator=g)
        return {"op": op, "W": W,
                "W8": torch.empty((K, _row_stride(H)), dtype=torch.float8_e4m3fn, device=dev)[:, :H],
                "w_scale": torch.empty((_blocks(K), _blocks(H)), dtype=torch.float32, device=dev)}
    if op in ("logits", "step"):
        B, K, H = case["B"], case["K"], case["H"]
        W = torch.empty((K, H), dtype=torch.bfloat16, device=dev).normal_(0.0, 0.02, generator=g)
        q, w_scale = _quantize_weights(W)
        W8 = torch.zeros((K, _row_stride(H)), dtype=torch.float8_e4m3fn, device=dev)[:, :H]
        W8.view(torch.uint8).copy_(q.view(torch.uint8))
        hidden = torch.empty((B, H), dtype=torch.bfloat16, device=dev).normal_(0.0, 1.0, generator=g)
        state = {"op": op, "hidden": hidden, "W8": W8, "w_scale": w_scale,
                 "out": torch.empty((B, K), dtype=torch.float32, device=dev)}
        if op == "logits":
            return {**state, "T": case["T"]}
        # the trimmed ids: K ascending ids of a four times larger vocabulary
        ids = torch.randperm(4 * K, generator=g, device=dev)[:K].sort().values.to(torch.int32)
        return {**state, "trim_ids": ids, "tokens": torch.empty(B, dtype=torch.int32, device=dev)}
    B, R, V = case["B"], case["gamma"] + 1, case["V"]
    dt = torch.float32 if case["dtype"] == "f32" else torch.bfloat16
    perm = torch.randperm(V, generator=g, device=dev)
    # a Zipf(1.1) rank bias under normal noise, as target logits over a vocabulary look
    bias = torch.empty(V, dtype=torch.float32, device=dev)
    bias[perm] = -3.3 * torch.arange(1, V + 1, dtype=torch.float32, device=dev).log()
    logits = torch.empty((B * R, V + case["pad"]), dtype=dt, device=dev).normal_(0.0, 2.0, generator=g)[:, :V]
    logits += bias
    # given tokens: frequent ids, log-uniform over the ranks
    u = torch.rand(B * R, generator=g, device=dev, dtype=torch.float64)
    tokens = perm[(u * math.log(V)).exp().long().clamp(1, V) - 1].to(torch.int32)
    if case["masked"] > 0.0:
        drop = torch.rand((B * R, V), generator=g, device=dev) < case["masked"]
        drop[torch.arange(B * R, device=dev), tokens.long()] = False
        logits.masked_fill_(drop, -math.inf)
    n = torch.tensor([_accepted(case, b) for b in range(B)], device=dev)
    n = n[torch.randperm(B, generator=g, device=dev)]
    tokens = tokens.view(B, R).masked_fill(torch.arange(R, device=dev)[None, :] > n[:, None], -1).view(B * R)
    k = case["k"]
    return {"op": op, "logits": logits, "tokens": tokens, "k": k, "T": case["T"],
            "logp": torch.empty(B * R, dtype=torch.float32, device=dev),
            "entropy": torch.empty(B * R, dtype=torch.float32, device=dev),
            "top_ids": torch.empty((B * R, k), dtype=torch.int32, device=dev),
            "top_logp": torch.empty((B * R, k), dtype=torch.float32, device=dev),
            "status": torch.empty(1, dtype=torch.int32, device=dev)}


# ------------------------------------------------------------- plain forms
def _plain_product(hidden, W8, w_scale):
    """Logits [B, K] at temperature 1 in fp32; every factor but the sums is exact."""
    B, H = hidden.shape
    K = W8.shape[0]
    hb = _blocks(H)
    x = torch.zeros((B, hb * BLOCK), dtype=torch.float32, device=hidden.device)
    x[:, :H] = hidden
    x = x.view(B, hb, BLOCK)
    e = _exponent(x.abs().amax(dim=2))
    x = (x * _pow2(-e)[:, :, None]).to(torch.float8_e4m3fn).float() * _pow2(e)[:, :, None]
    w = W8.float() * w_scale.repeat_interleave(BLOCK, 0)[:K].repeat_interleave(BLOCK, 1)[:, :H]
    return x.view(B, hb * BLOCK)[:, :H] @ w.t()


def _plain_logprobs(s):
    tok, k, T = s["tokens"].long(), s["k"], s["T"]
    skip = tok < 0
    x = s["logits"].float()
    m = x.amax(dim=1, keepdim=True)
    d = (x - m) / T
    ex = d.exp()
    S = ex.sum(dim=1)
    logS = S.log()
    entropy = logS - (ex * d.clamp(min=-1e4)).sum(dim=1) / S
    logp = d.gather(1, tok.clamp(min=0)[:, None])[:, 0] - logS
    nan = x.new_full((), math.nan)
    out = {"logp": torch.where(skip, nan, logp), "entropy": torch.where(skip, nan, entropy)}
    if k:
        # one integer key per id: the order of the logit above, the lower id first below
        i = (x + 0.0).view(torch.int32)
        key = (i ^ ((i >> 31) & 0x7FFFFFFF)).long() << 32
        key += 0xFFFFFFFF - torch.arange(x.shape[1], device=x.device)
        ids = 0xFFFFFFFF - (key.topk(k, dim=1).values & 0xFFFFFFFF)
        out["top_ids"] = torch.where(skip[:, None], -1, ids).to(torch.int32)
        out["top_logp"] = torch.where(skip[:, None], nan, d.gather(1, ids) - logS[:, None])
    return out


def _plain(s):
    if s["op"] == "quantize":
        W8, w_scale = _quantize_weights(s["W"])
        return {"W8": W8, "w_scale": w_scale}
    if s["op"] == "logits":
        return {"logits": _plain_product(s["hidden"], s["W8"], s["w_scale"]) / s["T"]}
    if s["op"] == "step":
        z = _plain_product(s["hidden"], s["W8"], s["w_scale"])
        top = z.amax(dim=1, keepdim=True)
        ids = torch.arange(z.shape[1], device=z.device)
        best = torch.where(z == top, ids, z.shape[1]).amin(dim=1)
        return {"q": (ids[None, :] == best[:, None]).float(), "tokens": s["trim_ids"][best]}
    return _plain_logprobs(s)


# ------------------------------------------------------------- the library
def _workspace(s, vt):
    if "workspace" not in s:
        (B, H), K = s["hidden"].shape, s["W8"].shape[0]
        s["workspace"] = torch.empty(vt.workspace_bytes("draft_fp8", B=B, H=H, K=K), dtype=torch.uint8,
                                     device=s["hidden"].device)
        s["status"] = torch.empty(1, dtype=torch.int32, device=s["hidden"].device)
    return s["workspace"]


def _library(s):
    import drafter_sampling_gb300 as vt
    if s["op"] == "quantize":
        W8, w_scale, _ = vt.vt_quantize_head(s["W"], W8=s["W8"], w_scale=s["w_scale"])
        return {"W8": W8, "w_scale": w_scale}
    if s["op"] == "logits":
        z = vt.vt_draft_logits_fp8(s["hidden"], s["W8"], s["w_scale"], s["T"], logits=s["out"],
                                   workspace=_workspace(s, vt))
        return {"logits": z}
    if s["op"] == "step":
        ws = _workspace(s, vt)
        q, tokens, _ = vt.vt_draft_step_fp8(s["hidden"], s["W8"], s["w_scale"], s["trim_ids"], None, 0.0, q=s["out"],
                                            tokens=s["tokens"], dev_status=s["status"], workspace=ws)
        return {"q": q, "tokens": tokens}
    logp, entropy, top_ids, top_logp, _ = vt.vt_token_logprobs(
        s["logits"], s["tokens"], k=s["k"], temperature=s["T"], out_logp=s["logp"], out_entropy=s["entropy"],
        out_top_ids=s["top_ids"], out_top_logp=s["top_logp"], dev_status=s["status"])
    if s["k"] == 0:
        return {"logp": logp, "entropy": entropy}
    return {"logp": logp, "entropy": entropy, "top_ids": top_ids, "top_logp": top_logp}


def run(state):
    return _library(state) if own else _plain(state)


# ----------------------------------------------------------- 64-bit values
def _exact_pow2(e):
    """2^e in fp64, from its bit pattern: a power function need not be exact."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _exact_e4m3(v):
    """The e4m3 value nearest to each |v| <= 448 (ties to even), in fp64."""
    _, x = torch.frexp(v)
    ulp = _exact_pow2((x - 1).clamp(min=-6) - 3)
    return torch.round(v / ulp) * ulp


def _exact_scale(amax):
    """The power of two s >= 2^-126 with amax <= 448 s, the smallest such, in fp64."""
    m, x = torch.frexp(amax / E4M3_MAX)
    e = torch.where(m == 0.5, x - 1, x)
    e = torch.where(amax == 0, torch.full_like(e, -126), e).clamp(min=-126)
    return _exact_pow2(e)


def _exact_quantize(W):
    K, H = W.shape
    W8 = torch.empty((K, H), dtype=torch.float64, device=W.device)
    scale = torch.empty((_blocks(K), _blocks(H)), dtype=torch.float64, device=W.device)
    for r in range(0, K, BLOCK):
        rows = W[r:r + BLOCK].double()
        col = torch.nn.functional.pad(rows.abs().amax(dim=0), (0, _blocks(H) * BLOCK - H))
        s = _exact_scale(col.view(-1, BLOCK).amax(dim=1))
        scale[r // BLOCK] = s
        W8[r:r + BLOCK] = _exact_e4m3(rows / s.repeat_interleave(BLOCK)[:H])
    return W8, scale


def _exact_product(hidden, W8, w_scale):
    z = torch.zeros((hidden.shape[0], W8.shape[0]), dtype=torch.float64, device=hidden.device)
    for g in range(_blocks(hidden.shape[1])):
        cols = slice(g * BLOCK, (g + 1) * BLOCK)
        x = hidden[:, cols].double()
        sx = _exact_scale(x.abs().amax(dim=1))
        x = _exact_e4m3(x / sx[:, None])
        sw = w_scale[:, g].double().repeat_interleave(BLOCK)[:W8.shape[0]]
        z += (x @ W8[:, cols].float().double().t()) * sx[:, None] * sw[None, :]
    return z


def _exact_logprobs(s):
    k = s["k"]
    out = {"logp": [], "entropy": [], "top_ids": [], "top_logp": []}
    for r in range(0, s["logits"].shape[0], 128):
        tok = s["tokens"][r:r + 128].long()
        x = s["logits"][r:r + 128].double() / s["T"]
        logp = x - torch.logsumexp(x, dim=1, keepdim=True)
        p = logp.exp()
        entropy = -torch.where(p > 0, p * logp, torch.zeros_like(p)).sum(dim=1)
        given = logp[torch.arange(len(tok), device=tok.device), tok.clamp(min=0)]
        # ids from the logits as given: a stable sort keeps the lower of equal ones first
        ids = torch.sort(s["logits"][r:r + 128].float(), dim=1, descending=True, stable=True).indices[:, :k]
        top = logp.gather(1, ids)
        skip = tok < 0
        given[skip], entropy[skip], ids[skip], top[skip] = math.nan, math.nan, -1, math.nan
        for name, v in (("logp", given), ("entropy", entropy), ("top_ids", ids.to(torch.int32)), ("top_logp", top)):
            out[name].append(v)
    names = ("logp", "entropy", "top_ids", "top_logp") if k else ("logp", "entropy")
    return {n: torch.cat(out[n]) for n in names}


def exact(case, seed):
    s = prepare(case, seed)
    if s["op"] == "quantize":
        W8, w_scale = _exact_quantize(s["W"])
        return {"W8": W8, "w_scale": w_scale}
    if s["op"] == "logits":
        return {"logits": _exact_product(s["hidden"], s["W8"], s["w_scale"]) / s["T"]}
    if s["op"] == "step":
        z = _exact_product(s["hidden"], s["W8"], s["w_scale"])
        best = z.argmax(dim=1)
        q = torch.zeros_like(z)
        q[torch.arange(len(best), device=z.device), best] = 1.0
        return {"q": q, "tokens": s["trim_ids"][best]}
    return _exact_logprobs(s)
