"""vt_token_logprobs against the fp64 oracle (oracle/logprobs.py).

Ids are compared exactly (the order is on the logits as given).  Values, with
u = 2^-24: (l - m) c, c and ln 2 are five roundings of |l - m| / T; a
probability's sum takes at most V / 256 additions in one thread and 16 more
joining threads, warps and blocks, each term off by the exponential's 2^-22
(4 u) and by |d| roundings of its argument, at most 3 log2(V) <= 66 u in the
weighted mean.  So |log p - ref| <= u (6 |l - m| / T + V / 256 + 90); the
entropy adds the same relative error of the mean of d: times (1 + ln V).
The reference is rounded to fp32 (u more, inside the 90).
"""
import numpy as np
import pytest

import oracle
import synthetic

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

LOWEST = -3.4028234663852886e38


@pytest.fixture(scope="module")
def vt():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import drafter_sampling_gb300 as m
    from drafter_sampling_gb300 import build
    build.build()
    m.lib()
    return m


def _check(vt, x, tokens, k, T=1.0, status=0):
    """x: a CUDA tensor [R, V]; compares every output of one call."""
    R, V = x.shape
    tok = torch.as_tensor(np.asarray(tokens, np.int32)).cuda()
    lp, en, ids, top, st = vt.vt_token_logprobs(x, tok, k=k, temperature=T)
    assert int(st.item()) == status
    h = x.float().cpu().numpy().astype(np.float64)
    ref = oracle.token_logprobs(h, tokens, k, T)
    u = 2.0 ** -24

    def close(got, want, dist, extra=1.0):
        got = got.astype(np.float64)
        with np.errstate(over="ignore"):      # (l - m) / T may lie beyond fp32
            want = np.asarray(want).astype(np.float32).astype(np.float64)
        assert np.array_equal(np.isnan(got), np.isnan(want))
        assert np.array_equal(np.isneginf(got), np.isneginf(want))
        m = np.isfinite(want)
        tol = u * (6 * dist + V / 256 + 90) * extra
        assert np.all(np.abs(got - want)[m] <= np.broadcast_to(tol, want.shape)[m])

    with np.errstate(invalid="ignore"):
        peak = np.max(np.where(np.isnan(h), -np.inf, h), axis=1)
        safe = np.clip(np.asarray(tokens), 0, V - 1)
        dist = np.nan_to_num(np.abs(h[np.arange(R), safe] - peak) / T, nan=0.0, posinf=0.0)
    close(lp.cpu().numpy(), ref["logp"], dist)
    close(en.cpu().numpy(), ref["entropy"], 0.0, 1 + np.log(V))
    if k:
        assert np.array_equal(ids.cpu().numpy(), ref["top_ids"])
        with np.errstate(invalid="ignore"):
            d = np.take_along_axis(h, np.clip(ref["top_ids"], 0, V - 1), 1) - peak[:, None]
        close(top.cpu().numpy(), ref["top_logp"], np.nan_to_num(np.abs(d) / T, posinf=0.0, nan=0.0))
    else:
        assert ids is None and top is None
    return lp, en, ids, top


def _rows(seed, R, V, dt, pad=0, lead=0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    buf = torch.randn(lead + R * (V + pad), generator=g, device="cuda") * 3.0
    return buf.to(dt)[lead:].view(R, V + pad)[:, :V]


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("R,V,k", [(1, 1, 1), (1, 1, 0), (2, 2, 2), (3, 7, 7), (1, 31, 31), (1, 32, 32),
                                   (5, 33, 32), (4, 100, 5), (2, 255, 1), (3, 2047, 20), (2, 2048, 8),
                                   (1, 8191, 32), (7, 8193, 5), (2, 16385, 0), (3, 32003, 20),
                                   (2, 70000, 8), (112, 1003, 8), (700, 513, 3)])
def test_random_rows(vt, R, V, k, dt):
    x = _rows(R + V, R, V, dt)
    _check(vt, x, synthetic.rng(V, 1).integers(0, V, R), k, 0.7)


@pytest.mark.parametrize("dt,V", [(torch.float32, 128256), (torch.bfloat16, 152064), (torch.float32, 400003)])
def test_long_rows(vt, dt, V):
    for R in (1, 3):
        _check(vt, _rows(V + R, R, V, dt), synthetic.rng(V, 2).integers(0, V, R), 20)


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("pad,lead", [(0, 1), (1, 0), (3, 2), (13, 5), (0, 3), (8, 0)])
def test_strides_and_alignment(vt, dt, pad, lead):
    for V in (5, 1003, 9001):
        _check(vt, _rows(V, 6, V, dt, pad, lead), synthetic.rng(V, 3).integers(0, V, 6), 5 if V > 5 else 3)


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("V", [40, 3000, 20000, 140000])
def test_ordered_and_tied_rows(vt, dt, V):
    up = torch.linspace(-20, 20, V, device="cuda")
    period = torch.arange(V, device="cuda") % 7
    x = torch.stack([up, up.flip(0), torch.zeros_like(up), period.float(), torch.full_like(up, LOWEST),
                     torch.where(period == 3, 2.0, -torch.inf)]).to(dt)
    if dt == torch.bfloat16:
        x[4] = torch.finfo(dt).min
    for k in (1, 8, 32):
        _check(vt, x, [0, V - 1, V // 2, 5, 7, 3], k)


@pytest.mark.parametrize("V", [20000, 200000])
def test_bounds_that_let_too_many_through(vt, V):
    # every 32nd group of eight threads sees low values only, so the first bound is low
    for dt, ve in ((torch.float32, 4), (torch.bfloat16, 8)):
        x = _rows(V, 2, V, dt).clone()
        ids = torch.arange(V, device="cuda")
        x[:, (ids // ve) % 256 // 8 == 5] = -100.0
        _check(vt, x, [1, 2], 32)
        _check(vt, x, [1, 2], 31)


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
def test_masks(vt, dt):
    V = 5000
    x = _rows(11, 8, V, dt).clone()
    x[0, 1:] = -torch.inf                     # one id left
    x[1, :] = -torch.inf                      # none left
    x[2, :4990] = -torch.inf                  # ten left, fewer than k
    x[3, ::2] = -torch.inf
    x[4, :] = torch.finfo(dt).min             # the lowest value everywhere
    x[5, 17:] = torch.finfo(dt).min           # ... and as a mask
    x[6, 7] = torch.finfo(dt).max
    x[7, 3] = -torch.inf                      # the given token is masked
    _check(vt, x, [0, 3, 4995, 3, 4999, 2, 7, 3], 20, 1.0, status=8)
    _check(vt, x[[0, 2, 3, 4, 5, 6, 7]], [0, 4995, 3, 4999, 2, 9, 3], 20, 0.5)


@pytest.mark.parametrize("where", [0, 2500, 4999])
def test_nan_and_infinity_flag_their_row_only(vt, where):
    x = _rows(12, 4, 5000, torch.float32).clone()
    x[1, where] = torch.nan
    x[2, where] = torch.inf
    lp, en, ids, top = _check(vt, x, [5, 6, 7, 8], 4, status=8)
    assert bool(torch.isnan(lp[1:3]).all()) and bool((ids[1:3] == -1).all())


def test_tokens_outside_and_unscored(vt):
    V = 3000
    x = _rows(13, 6, V, torch.float32).clone()
    x[1] = torch.nan                          # not scored: not read
    _check(vt, x, [5, -1, V, -2, 2147483647, V - 1], 3, status=1)
    _check(vt, x[:2], [5, -1], 3)
    y = torch.full((2, V), torch.nan, device="cuda")
    _check(vt, y, [-1, -1], 2)


def test_leading_shape_outputs_and_reuse(vt):
    B, G, V, k = 3, 4, 777, 6
    x = _rows(14, B * G, V, torch.float32).view(B, G, V)
    tok = torch.randint(0, V, (B, G), device="cuda", dtype=torch.int32)
    lp, en, ids, top, st = vt.vt_token_logprobs(x, tok, k=k)
    assert lp.shape == (B, G) and en.shape == (B, G) and ids.shape == (B, G, k) and top.shape == (B, G, k)
    # a position of every sequence: rows apart by a whole sequence's logits
    lp1, en1, ids1, _, _ = vt.vt_token_logprobs(x[:, 2], tok[:, 2].contiguous(), k=k)
    assert torch.equal(lp1, lp[:, 2]) and torch.equal(en1, en[:, 2]) and torch.equal(ids1, ids[:, 2])
    _, none, _, _, _ = vt.vt_token_logprobs(x, tok, want_entropy=False)
    assert none is None
    st.fill_(99)
    out = vt.vt_token_logprobs(x, tok, k=k, out_logp=lp, out_entropy=en, out_top_ids=ids, out_top_logp=top,
                               dev_status=st)
    assert out[0].data_ptr() == lp.data_ptr() and int(st.item()) == 0


def test_two_calls_give_the_same_bits(vt):
    x = _rows(15, 40, 60000, torch.bfloat16)
    tok = torch.randint(0, 60000, (40,), device="cuda", dtype=torch.int32)
    a, b = vt.vt_token_logprobs(x, tok, k=20), vt.vt_token_logprobs(x, tok, k=20)
    assert all(torch.equal(p, q) for p, q in zip(a, b))


def test_rows_beyond_32_bit_offsets(vt):
    if torch.cuda.mem_get_info()[0] < 16 << 30:
        pytest.skip("needs 16 GB")
    ld, R, V = 1 << 20, 3000, 1000              # 3 G elements of bf16: 6 GB
    buf = torch.empty((R, ld), dtype=torch.bfloat16, device="cuda")
    x = buf[:, :V]
    x.copy_(_rows(16, R, V, torch.bfloat16))
    tok = torch.randint(0, V, (R,), device="cuda", dtype=torch.int32)
    a, b = vt.vt_token_logprobs(x, tok, k=4), vt.vt_token_logprobs(x.contiguous(), tok, k=4)
    assert torch.equal(a[2], b[2])
    assert torch.allclose(a[0], b[0], rtol=0, atol=1e-5) and torch.allclose(a[1], b[1], rtol=0, atol=1e-5)


def test_binding_refusals(vt):
    x = torch.zeros((2, 50), device="cuda")
    tok = torch.zeros(2, dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError, match="k must"):
        vt.vt_token_logprobs(x, tok, k=33)
    with pytest.raises(TypeError, match="logits"):
        vt.vt_token_logprobs(x.double(), tok)
    with pytest.raises(ValueError, match="tokens"):
        vt.vt_token_logprobs(x, tok[:1])
    with pytest.raises(TypeError, match="tokens"):
        vt.vt_token_logprobs(x, tok.long())
    with pytest.raises(ValueError, match="stride"):
        vt.vt_token_logprobs(x.t().contiguous().t(), tok)
    with pytest.raises(ValueError, match="stride"):
        vt.vt_token_logprobs(torch.zeros((1, 50), device="cuda").expand(2, 50), tok)
    with pytest.raises(vt.VtError):
        vt.vt_token_logprobs(x, tok, temperature=0.0)
    with pytest.raises(ValueError, match="out_logp"):
        vt.vt_token_logprobs(x, tok, out_logp=torch.zeros(3, device="cuda"))


def test_side_stream_and_graph(vt):
    xs = [_rows(20 + i, 9, 40000, torch.float32) for i in range(3)]
    tok = torch.randint(0, 40000, (9,), device="cuda", dtype=torch.int32)
    want = [vt.vt_token_logprobs(x, tok, k=5) for x in xs]
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    got = [vt.vt_token_logprobs(x, tok, k=5, stream=s) for x in xs]
    s.synchronize()
    assert all(torch.equal(p, q) for a, b in zip(got, want) for p, q in zip(a, b))
    buf = xs[0].clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = vt.vt_token_logprobs(buf, tok, k=5)
    for x, w in zip(xs, want):
        buf.copy_(x)
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(out, w))


def test_more_rows_than_blocks_with_gaps(vt):
    # persistent blocks walk over scored, unscored, flagged and ragged rows in turn
    R, V = 2000, 20011
    x = _rows(21, R, V, torch.bfloat16, 5, 1).clone()
    tok = synthetic.rng(21, 1).integers(0, V, R).astype(np.int64)
    tok[::3] = -1
    tok[5] = V
    x[7, 11] = torch.nan
    x[10, 40:] = -torch.inf
    _check(vt, x, tok, 7, 0.9, status=9)


def test_temperature_extremes(vt):
    x = _rows(22, 4, 3000, torch.float32)
    _check(vt, x, [0, 1, 2, 3], 5, 100.0)
    _check(vt, x, [0, 1, 2, 3], 5, 0.05)
    y = x.clone()
    y[0, ::2] = -torch.inf
    for T in (1e-30, 1e30):       # the limits: one id, or all that are not masked, alike
        lp, en, ids, top, st = vt.vt_token_logprobs(y, torch.tensor([1, 1, 2, 3], dtype=torch.int32,
                                                                    device="cuda"), k=3, temperature=T)
        assert int(st.item()) == 0
        if T > 1:
            want = np.log([1500, 3000, 3000, 3000])
            assert np.allclose(en.cpu().numpy(), want, atol=1e-4)
            assert np.allclose(lp.cpu().numpy(), -want, atol=1e-4)
        else:
            assert bool((en == 0).all()) and bool((top[:, 0] == 0).all())


def test_draft_verify_and_report(vt):
    # the operators as they are used together: quantise the trimmed head, draft a block through it,
    # verify it against the target's logits, report the emitted tokens
    from oracle import fp8
    V, H, K, B, gamma = 6000, 384, 1500, 4, 3
    W = synthetic.head_weights(V, H, seed=31)
    ids = synthetic.rng(31, 2).permutation(V)[:K].astype(np.int32)
    dev = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()
    W_trim, trim_ids, inv_map, _ = vt.vt_trim_head(dev(W.view(np.int16)), dev(ids))
    W8, s, st = vt.vt_quantize_head(W_trim)
    assert int(st.item()) == 0
    r_trim, r_ids, _ = oracle.trim_head(W, ids)
    codes, scale = fp8.quantize_head(r_trim)
    assert np.array_equal(W8.view(torch.uint8).cpu().numpy(), codes)
    hidden = synthetic.hidden_states((gamma, B, H), seed=32)
    u = synthetic.uniforms(33, 1, (gamma, B))
    q = torch.empty((B, gamma, K), device="cuda")
    tok = torch.empty((B, gamma), dtype=torch.int32, device="cuda")
    for j in range(gamma):
        _, _, st = vt.vt_draft_step_fp8(dev(hidden[j].view(np.int16)), W8, s, trim_ids, dev(u[j]), 1.0,
                                        q=q[:, j], tokens=tok[:, j])
        assert int(st.item()) == 0
        z, _ = fp8.draft_logits_fp8(hidden[j], codes, scale, 1.0)
        # the drafter's own confidence: its logits and the drafted trimmed indices
        zl = vt.vt_draft_logits_fp8(dev(hidden[j].view(np.int16)), W8, s)
        at = inv_map[tok[:, j].long()].contiguous()
        lp, en, top, _, _ = vt.vt_token_logprobs(zl, at, k=5)
        ref = oracle.token_logprobs(z, at.cpu().numpy(), 5)
        assert np.allclose(lp.cpu().numpy(), ref["logp"], atol=1e-4)
        assert np.allclose(en.cpu().numpy(), ref["entropy"], atol=1e-4)
    # target logits near the drafter's, so that some tokens are accepted
    g = torch.Generator(device="cuda")
    g.manual_seed(34)
    logits = torch.randn((B, gamma + 1, V), generator=g, device="cuda")
    logits.scatter_(2, trim_ids.long()[None, None, :].expand(B, gamma, K),
                    q.log() + 0.5 * torch.randn((B, gamma, K), generator=g, device="cuda") + 8.0)
    ua, ur = synthetic.uniforms(35, 1, (B, gamma)), synthetic.uniforms(35, 2, (B, gamma + 1))
    out, n, _, st = vt.vt_verify(logits, q, inv_map, tok, dev(ua), dev(ur))
    assert int(st.item()) == 0 and bool((n > 0).any()) and bool((n < gamma).any())
    lp, en, top, top_lp, st = vt.vt_token_logprobs(logits, out, k=3)
    assert int(st.item()) == 0
    ref = oracle.token_logprobs(logits.view(-1, V).cpu().numpy(), out.view(-1).cpu().numpy(), 3)
    assert np.array_equal(top.view(-1, 3).cpu().numpy(), ref["top_ids"])
    assert np.allclose(lp.view(-1).cpu().numpy(), ref["logp"], atol=1e-5, equal_nan=True)
    assert np.allclose(en.view(-1).cpu().numpy(), ref["entropy"], atol=1e-4, equal_nan=True)


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("low", [-300.0, -np.inf])
@pytest.mark.parametrize("V", [2000, 40001])
def test_peaked_rows(vt, V, low, dt):
    """A peak and runners-up at distance d, in the peak's own 16 bytes, its thread's chunk, and elsewhere.

    With w = e^-d the row's S - 1 is a sum of w, and ln S and the entropy are w (1 + d) and the like.
    Relative to it: w's argument d log2(e) is off by two roundings, which is d 2^-23 of w; its exponential
    by 2^-22, once more when the runner-up's thread is rescaled to the peak; the sums and their joins, two
    products, the logarithm and the last additions by 20 roundings of 2^-24.  And in absolute terms by 16
    roundings of S, half a step of 2^-23 each: those of the additions to the peak's 1 in its thread's chunk,
    at most 7 in a 16-byte vector and 8 over the vectors, where they are added one by one.
    """
    peak = 1000
    near = [peak + 1, peak - 1, peak + 3, peak + 256 * (16 // dt.itemsize), 3, V - 2]
    for T in (1.0, 0.5):
        rows, given, dist = [], [], []
        for d in (2.0, 5.0, 12.0, 20.0, 40.0):
            for ids in [[i] for i in near if i < V] + [[peak + 1, 7], [peak - 1, peak + 1, V - 2]]:
                x = torch.full((V,), low)
                x[peak] = 6.0
                x[ids] = 6.0 - d * T
                rows.append(x)
                given.append(peak)
                dist.append(d)
        x = torch.stack(rows).to(dt).cuda()
        lp, en, _, _, st = vt.vt_token_logprobs(x, torch.tensor(given, dtype=torch.int32, device="cuda"), temperature=T)
        assert int(st.item()) == 0
        y = (x.double().cpu().numpy() - 6.0) / T
        y[:, peak] = -np.inf                                # the others, apart from the peak's 1
        w = np.exp(y)
        rest = w.sum(axis=1)                                # S - 1 with its digits
        want = -np.log1p(rest)
        entropy = np.log1p(rest) - np.where(w > 0, w * np.maximum(y, -1e9), 0.0).sum(axis=1) / (1 + rest)
        d = np.array(dist)
        rel = (d + 16) * 2.0 ** -23
        floor = 16 * 2.0 ** -24 * (1 + rest)
        lp, en = lp.cpu().numpy().astype(np.float64), en.cpu().numpy().astype(np.float64)
        assert np.all(np.abs(lp - want) <= rel * np.abs(want) + floor)
        assert np.all(np.abs(en - entropy) <= rel * entropy + floor * (1 + entropy))


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("R,V", [(3, 9), (3, 60000)])
def test_differences_beyond_fp32(vt, R, V, dt):
    # log p = (l - m) / T is finite where l - m alone is not: 6e38 apart, T = 4 and the largest T
    x = torch.full((R, V), -3e38)
    x[:, 4] = 3e38
    x[1, 5] = 0.0
    x = x.to(dt).cuda()
    _check(vt, x, [1, 5, 4], 5, 4.0)
    _check(vt, x, [1, 5, 4], 5, 1e30)
