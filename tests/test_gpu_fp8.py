"""The 8-bit head through the public entry points, against the fp64 oracle
(oracle/fp8.py).

Quantised values are defined bit for bit.  Logits: with u = 2^-23 (each
addition rounded or truncated to fp32), a sum of n terms in any order is
within n u A of the exact one, A the sum of the terms' magnitudes; here n =
H products, one addition per group and the two scale factors, 1/T and the
last rounding: |z - ref| <= (H + groups + 6) 2^-23 A.  On small integers every
product and sum is exact, so the logits must be equal bit for bit.
"""
import numpy as np
import pytest

import oracle
import synthetic
from oracle import fp8
from parity import assert_probs_close

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def vt():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import drafter_sampling_gb300 as m
    from drafter_sampling_gb300 import build
    build.build()
    m.lib()
    return m


def _dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def _bf(bits):
    return _dev(np.ascontiguousarray(bits).view(np.int16))


def _ints(g, shape, lo=-2, hi=3):
    return (g.integers(lo, hi, shape).astype(np.float32).view(np.uint32) >> 16).astype(np.uint16)


def _head(codes, scale):
    """Codes [K, H] behind a row stride that is a multiple of 16, poison in the padding."""
    K, H = codes.shape
    buf = torch.full((K, (H + 15) // 16 * 16 + 16), 0x7F, dtype=torch.uint8, device="cuda")
    buf[:, :H] = _dev(codes)
    return buf[:, :H], _dev(scale.astype(np.float32))


def _logit_bound(H, A):
    return (H + (H + 127) // 128 + 6) * 2.0 ** -23 * A


# ------------------------------------------------------------- quantising
@pytest.mark.parametrize("K,H", [(1, 1), (1, 128), (127, 129), (128, 128), (129, 16), (300, 1000),
                                 (257, 333), (1000, 576), (2048, 2048)])
def test_quantize_head_bit_exact(vt, K, H):
    g = synthetic.rng(K * 7 + H, 5)
    W = g.standard_normal((K, H)).astype(np.float32) * np.float32(0.02)
    W *= (10.0 ** g.integers(-3, 3, (K, 1))).astype(np.float32)
    bits = synthetic.to_bf16_bits(W)
    W8, s, st = vt.vt_quantize_head(_bf(bits))
    torch.cuda.synchronize()
    assert int(st.item()) == 0 and W8.dtype == torch.float8_e4m3fn and W8.stride(0) % 16 == 0
    codes, scale = fp8.quantize_head(bits)
    assert np.array_equal(W8.view(torch.uint8).cpu().numpy(), codes)
    assert np.array_equal(s.cpu().numpy().astype(np.float64), scale)


@pytest.mark.parametrize("K,H", [(1, 1), (3, 5), (129, 129), (200, 136), (130, 1001), (260, 254)])
@pytest.mark.parametrize("lead", [1, 2, 3, 4, 7])
def test_quantize_head_misaligned_rows(vt, K, H, lead):
    # rows that start at any 2-byte boundary, the last ending at the end of the allocation's data
    bits = synthetic.head_weights(K, H, seed=K + H + lead)
    flat = torch.zeros(lead + K * H, dtype=torch.int16, device="cuda")
    flat[lead:] = _bf(bits).view(-1)
    W8, s, st = vt.vt_quantize_head(flat[lead:].view(K, H))
    codes, scale = fp8.quantize_head(bits)
    assert int(st.item()) == 0 and np.array_equal(W8.view(torch.uint8).cpu().numpy(), codes)
    assert np.array_equal(s.cpu().numpy().astype(np.float64), scale)


def test_quantize_head_extremes(vt):
    # zero blocks, subnormals, the largest bf16, and 448 on the boundary of two scales
    blocks = [0.0, 1e-40, 3.3e38, 448.0, 450.0, 2.0 ** -118 * 1.75, 2.0 ** -130, 1.0]
    W = np.zeros((128, 128 * len(blocks)), np.float32)
    g = synthetic.rng(1, 5)
    for i, v in enumerate(blocks):
        W[:, 128 * i:128 * (i + 1)] = g.uniform(-1, 1, (128, 128)) * v
        W[5, 128 * i + 7] = v
    bits = synthetic.to_bf16_bits(W)
    W8, s, st = vt.vt_quantize_head(_bf(bits))
    codes, scale = fp8.quantize_head(bits)
    assert int(st.item()) == 0
    assert np.array_equal(s.cpu().numpy().astype(np.float64), scale)
    assert np.array_equal(W8.view(torch.uint8).cpu().numpy(), codes)


@pytest.mark.parametrize("bad", [np.nan, np.inf, -np.inf])
def test_quantize_head_flags_nonfinite(vt, bad):
    W = np.ones((200, 200), np.float32)
    W[150, 10] = bad
    W8, s, st = vt.vt_quantize_head(_dev(W).to(torch.bfloat16))
    assert int(st.item()) == 8
    assert float(s[0, 0]) == 2.0 ** -8 and bool((W8[:128].float() == 256.0).all())
    W8, s, st = vt.vt_quantize_head(torch.ones((200, 200), dtype=torch.bfloat16, device="cuda"),
                                    W8=W8, w_scale=s, dev_status=st)
    assert int(st.item()) == 0                      # the status word starts at zero again


def test_quantize_head_leaves_the_padding_alone(vt):
    buf = torch.full((130, 160), 0x55, dtype=torch.uint8, device="cuda")
    W = torch.randn((130, 133), device="cuda").to(torch.bfloat16)
    vt.vt_quantize_head(W, W8=buf[:, :133])
    assert bool((buf[:, 133:] == 0x55).all())


# ------------------------------------------------------------------ logits
SHAPES = [(1, 1, 1), (1, 128, 128), (2, 16, 5), (3, 127, 129), (7, 300, 1003), (16, 2048, 4096),
          (17, 129, 256), (32, 512, 700), (33, 1000, 777), (64, 96, 130), (65, 640, 513),
          (100, 264, 300), (128, 1100, 257), (129, 33, 640), (200, 2050, 400), (256, 128, 1300),
          (257, 256, 200), (300, 1500, 1007), (1000, 200, 300), (4096, 64, 140)]


# more tiles than CTAs that run at once, with fewer groups than stages and with more
MANY = [(3, 100, 45000), (3, 900, 41000), (40, 130, 45001), (64, 64, 50000), (100, 200, 45000),
        (256, 136, 45000), (256, 900, 20003), (300, 64, 30000), (1000, 64, 12000)]


@pytest.mark.parametrize("B,H,K", SHAPES + MANY + [(2, 65536, 130), (70, 65536, 130), (130, 20000, 300)])
def test_logits_integer_inputs_bit_exact(vt, B, H, K):
    g = synthetic.rng(B + H + K, 6)
    hid, W = _ints(g, (B, H)), _ints(g, (K, H))
    codes, scale = fp8.quantize_head(W)
    z = vt.vt_draft_logits_fp8(_bf(hid), *_head(codes, scale), 0.5)
    want = oracle.draft_logits(hid, W, 0.5)
    assert np.array_equal(z.cpu().numpy().astype(np.float64), want)


@pytest.mark.parametrize("every", [1, 2, 3, 1000])
@pytest.mark.parametrize("B,H,K", [(16, 300, 1000), (130, 300, 41000), (256, 130, 40100), (256, 4225, 700),
                                   (300, 128, 20000), (1000, 640, 10500)])
def test_logits_mixed_scales_bit_exact(vt, B, H, K, every):
    """Some blocks of rows have a scale that is no power of two, others none; all sums are exact."""
    g = synthetic.rng(B + H + K, 12)
    hid, W = _ints(g, (B, H)), _ints(g, (K, H))
    codes, scale = fp8.quantize_head(W)
    scale = scale.copy()
    rows = np.arange(scale.shape[0])[::every]
    scale[rows, rows % scale.shape[1]] *= 1.5
    scale[rows[1::3], 0] *= -0.75
    z, again = (vt.vt_draft_logits_fp8(_bf(hid), *_head(codes, scale), 0.5) for _ in range(2))
    ref, _ = fp8.draft_logits_fp8(hid, codes, scale, 0.5)
    assert np.array_equal(z.cpu().numpy(), ref.astype(np.float32))
    assert torch.equal(z, again)


@pytest.mark.parametrize("B,H,K", [s for s in SHAPES if s[0] <= 300])
def test_logits_random_inputs(vt, B, H, K):
    hid = synthetic.hidden_states((B, H), seed=B + K)
    W = synthetic.head_weights(K, H, seed=H)
    codes, scale = fp8.quantize_head(W)
    scale = scale * synthetic.rng(H, 7).uniform(0.5, 2.0, scale.shape).astype(np.float32)
    scale = scale.astype(np.float32).astype(np.float64)      # any fp32 scales, as another quantiser leaves
    ref, A = fp8.draft_logits_fp8(hid, codes, scale, 0.7)
    out = torch.full((B, K + 3), -7.0, device="cuda")
    z = vt.vt_draft_logits_fp8(_bf(hid), *_head(codes, scale), 0.7, logits=out)
    z = z.cpu().numpy().astype(np.float64)
    assert np.all(np.abs(z[:, :K] - ref) <= _logit_bound(H, A) + 1e-30)
    assert np.all(z[:, K:] == -7.0)                          # columns behind the head stay as they were


def test_logits_rows_of_very_different_scale(vt):
    # one row and one block of the head 2^40 above the others: the scales are per row, group and block
    B, H, K = 5, 640, 400
    g = synthetic.rng(9, 6)
    x = g.standard_normal((B, H)).astype(np.float32)
    x[2] *= 2.0 ** 40
    x[:, 128:256] *= 2.0 ** -30
    x[3] = 0
    W = g.standard_normal((K, H)).astype(np.float32)
    W[128:256] *= 2.0 ** -40
    hid, Wb = synthetic.to_bf16_bits(x), synthetic.to_bf16_bits(W)
    codes, scale = fp8.quantize_head(Wb)
    ref, A = fp8.draft_logits_fp8(hid, codes, scale, 1.0)
    z = vt.vt_draft_logits_fp8(_bf(hid), *_head(codes, scale)).cpu().numpy().astype(np.float64)
    assert np.all(np.abs(z - ref) <= _logit_bound(H, A) + 1e-30)
    assert np.all(z[3] == 0)


def test_nonfinite_hidden_rows_stay_apart(vt):
    B, H, K = 6, 384, 300
    hid = torch.randn((B, H), device="cuda").to(torch.bfloat16)
    W8, s, _ = vt.vt_quantize_head(torch.randn((K, H), device="cuda").to(torch.bfloat16))
    clean = vt.vt_draft_logits_fp8(hid, W8, s)
    dirty = hid.clone()
    dirty[1, 200], dirty[4, 3] = float("nan"), float("-inf")
    z = vt.vt_draft_logits_fp8(dirty, W8, s)
    rows = [0, 2, 3, 5]
    assert torch.equal(z[rows], clean[rows]) and bool(torch.isnan(z[[1, 4]]).all())
    ids = torch.arange(K, dtype=torch.int32, device="cuda")
    u = torch.full((B,), 0.5, device="cuda")
    for T in (1.0, 0.0):
        _, tok, st = vt.vt_draft_step_fp8(dirty, W8, s, ids, u, T)
        assert int(st.item()) == 8
        assert tok.cpu().numpy()[[1, 4]].tolist() == [-1, -1] and bool((tok[rows] >= 0).all())


def test_misaligned_hidden_and_odd_columns(vt):
    B, H, K = 9, 301, 260
    flat = torch.randn(B * H + 1, device="cuda").to(torch.bfloat16)
    hid = flat[1:].view(B, H)
    W8, s, _ = vt.vt_quantize_head(torch.randn((K, H), device="cuda").to(torch.bfloat16))
    assert torch.equal(vt.vt_draft_logits_fp8(hid, W8, s), vt.vt_draft_logits_fp8(hid.clone(), W8, s))


# -------------------------------------------------------- drafting on top
@pytest.mark.parametrize("B,H,K", [(1, 64, 200), (5, 300, 1003), (16, 2048, 4096), (64, 512, 2000),
                                   (100, 520, 3001), (256, 128, 1300), (300, 256, 700)] + MANY)
def test_greedy_step_integer_inputs_bit_exact(vt, B, H, K):
    g = synthetic.rng(B + H + K, 8)
    hid, W = _ints(g, (B, H)), _ints(g, (K, H))
    W[K // 2] = W[K // 3]
    ids = np.sort(g.permutation(3 * K)[:K]).astype(np.int32)
    q, tok, st = vt.vt_draft_step_fp8(_bf(hid), *_head(*fp8.quantize_head(W)), _dev(ids), None, 0.0)
    assert int(st.item()) == 0
    ref = oracle.draft_step_greedy(hid, W, ids)
    assert np.array_equal(tok.cpu().numpy(), ref["tokens"])
    want = np.zeros((B, K), np.float32)
    want[np.arange(B), ref["index"]] = 1.0
    assert np.array_equal(q.cpu().numpy(), want)


@pytest.mark.parametrize("gap", [0, 1, 4])
@pytest.mark.parametrize("B,H,K", [(1, 40, 1), (3, 64, 129), (16, 130, 260), (33, 128, 1003), (64, 256, 39000),
                                   (65, 128, 300), (256, 64, 1028), (130, 72, 515)])
def test_greedy_step_rows(vt, B, H, K, gap):
    """Equal, only negative and non-finite logits, in rows with a gap behind them."""
    g = synthetic.rng(B * K + H, 11)
    hid, W = _ints(g, (B, H), 1, 3), _ints(g, (K, H), -3, 0)  # every z is negative
    W[:, 1:] = 0
    hid[B // 2] = 0                                           # every z is 0: the lowest index
    bad = sorted({0, B - 1} - {B // 2})
    ids = np.sort(g.permutation(3 * K)[:K]).astype(np.int32)
    ref = oracle.draft_step_greedy(hid, W, ids)
    dirty = hid.copy()
    for n, b in enumerate(bad):
        dirty[b, H - 1 - n] = (0x7FC0, 0xFF80)[n]  # NaN, -inf
    q_all = torch.full((B, K + gap), -7.0, device="cuda")
    q, tok, st = vt.vt_draft_step_fp8(_bf(dirty), *_head(*fp8.quantize_head(W)), _dev(ids), None, 0.0,
                                      q=q_all[:, :K])
    assert int(st.item()) == (vt.VT_DEV_NONFINITE if bad else 0)
    want, tokens = np.zeros((B, K), np.float32), ref["tokens"].copy()
    want[np.arange(B), ref["index"]] = 1.0
    want[bad], tokens[bad] = 0.0, -1
    assert np.array_equal(q.cpu().numpy(), want)
    assert np.array_equal(tok.cpu().numpy(), tokens)
    assert bool((q_all[:, K:] == -7).all())


@pytest.mark.parametrize("B,H,K,T", [(1, 256, 1000, 1.0), (16, 512, 3001, 0.7), (130, 200, 700, 1.3),
                                     (300, 128, 500, 1.0), (5, 130, 45000, 1.0), (70, 64, 40001, 0.8),
                                     (140, 64, 20500, 1.0)])
def test_sampling_step(vt, B, H, K, T):
    hid, W = synthetic.hidden_states((B, H), seed=3), synthetic.head_weights(K, H, seed=4)
    u = synthetic.uniforms(5, 1, (B,))
    ids = np.sort(synthetic.rng(6, 1).permutation(2 * K)[:K]).astype(np.int32)
    codes, scale = fp8.quantize_head(W)
    q_all = torch.full((B, 2, K), -1.0, device="cuda")
    t_all = torch.full((B, 2), -5, dtype=torch.int32, device="cuda")
    _, _, st = vt.vt_draft_step_fp8(_bf(hid), *_head(codes, scale), _dev(ids), _dev(u), T,
                                    q=q_all[:, 1], tokens=t_all[:, 1])
    assert int(st.item()) == 0
    z, _ = fp8.draft_logits_fp8(hid, codes, scale, T)
    q, tok = q_all[:, 1].cpu().numpy(), t_all[:, 1].cpu().numpy()
    for b in range(B):
        p = np.exp(z[b] - z[b].max())
        p /= p.sum()
        assert_probs_close(q[b], p)
        r = oracle.inverse_cdf(p, u[b])
        if r.margin > 1e-5:
            assert tok[b] == ids[r.index], b
    assert bool((q_all[:, 0] == -1).all()) and bool((t_all[:, 0] == -5).all())


@pytest.mark.parametrize("B,H,K,k", [(1, 128, 40, 32), (5, 300, 1003, 8), (70, 256, 5000, 20)])
def test_topk_matches_the_logits(vt, B, H, K, k):
    # the ids are the k largest of the same product's logits, ties to the lower id
    hid, W = synthetic.hidden_states((B, H), seed=7), synthetic.head_weights(K, H, seed=8)
    codes, scale = fp8.quantize_head(W)
    h, (W8, s) = _bf(hid), _head(codes, scale)
    ids = torch.arange(K, dtype=torch.int32, device="cuda")
    out, logq, st = vt.vt_draft_topk_fp8(h, W8, s, ids, k, 0.7)
    assert int(st.item()) == 0
    z, A = fp8.draft_logits_fp8(hid, codes, scale, 0.7)
    tol = 2 * _logit_bound(H, A).max(axis=1)
    out, logq = out.cpu().numpy(), logq.cpu().numpy()
    for b in range(B):
        lp = z[b] - z[b].max()
        lp -= np.log(np.exp(lp).sum())
        assert np.all(np.abs(logq[b] - lp[out[b]]) <= 2 * tol[b] + 1e-5)
        assert np.all(z[b, out[b]] >= np.sort(z[b])[::-1][:k] - tol[b])
        assert len(set(out[b].tolist())) == k


@pytest.mark.parametrize("T", [1.0, 0.0])
@pytest.mark.parametrize("B,H,K,V,gamma", [(4, 256, 600, 2000, 3), (130, 128, 300, 700, 2)])
def test_block_graph_equals_the_calls(vt, B, H, K, V, gamma, T):
    # the captured block drafts and verifies exactly what the calls made one by one do, at every replay
    g = synthetic.rng(B, 9)
    trim = np.sort(g.permutation(V)[:K]).astype(np.int32)
    inv = np.full(V, -1, np.int32)
    inv[trim] = np.arange(K)
    trim, inv = _dev(trim), _dev(inv)
    W8, s, _ = vt.vt_quantize_head(_bf(synthetic.head_weights(K, H, seed=5)))
    hid = _bf(synthetic.hidden_states((gamma, B, H), seed=6))
    logits = torch.randn((B, gamma + 1, V), device="cuda")
    ud, ua, ur = (_dev(synthetic.uniforms(7, i, sh)) for i, sh in
                  enumerate([(gamma, B), (B, gamma), (B, gamma + 1)]))
    blk = vt.BlockGraph(hid, W8, trim, inv, logits, ud, ua, ur, T, w_scale=s)
    for seed in (6, 60):
        hid.copy_(_bf(synthetic.hidden_states((gamma, B, H), seed=seed)))
        blk.launch()
        q = torch.empty((B, gamma, K), device="cuda")
        tok = torch.empty((B, gamma), dtype=torch.int32, device="cuda")
        for j in range(gamma):
            _, _, st = vt.vt_draft_step_fp8(hid[j], W8, s, trim, ud[j], T, q=q[:, j], tokens=tok[:, j])
            assert int(st.item()) == 0
        out, n, acc, st = vt.vt_verify(logits, q, inv, tok, ua, ur, T)
        torch.cuda.synchronize()
        assert blk.dev_status.tolist() == [0, int(st.item())]
        for a, b in ((blk.q, q), (blk.draft_tokens, tok), (blk.out_tokens, out), (blk.out_num_accepted, n)):
            assert torch.equal(a, b)
    with pytest.raises(ValueError, match="trim_ids"):
        vt.BlockGraph(hid, W8, trim[:-1], inv, logits, ud, ua, ur, T, w_scale=s)


def test_binding_refusals(vt):
    hid = torch.zeros((2, 64), dtype=torch.bfloat16, device="cuda")
    W8, s, _ = vt.vt_quantize_head(torch.ones((40, 64), dtype=torch.bfloat16, device="cuda"))
    with pytest.raises(ValueError, match="disagree"):
        vt.vt_draft_logits_fp8(hid[:, :32].contiguous(), W8, s)
    with pytest.raises(ValueError, match="w_scale"):
        vt.vt_draft_logits_fp8(hid, W8, s.repeat(2, 1))
    with pytest.raises(ValueError, match="W8"):
        vt.vt_draft_logits_fp8(hid, W8.t().contiguous().t(), s)
    with pytest.raises(ValueError, match="W8"):                    # a row stride of 72
        vt.vt_draft_logits_fp8(hid, torch.empty((40, 72), dtype=torch.uint8, device="cuda")[:, :64], s)
    with pytest.raises(TypeError, match="W8"):
        vt.vt_draft_logits_fp8(hid, W8.float(), s)
    with pytest.raises(ValueError, match="logits"):
        vt.vt_draft_logits_fp8(hid, W8, s, logits=torch.empty((2, 39), device="cuda"))
    with pytest.raises(vt.VtError):
        vt.vt_draft_logits_fp8(hid, W8, s, 0.0)
    with pytest.raises(vt.VtError):
        vt.vt_draft_logits_fp8(hid, W8, s, workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
    with pytest.raises(ValueError, match="k must"):
        vt.vt_draft_topk_fp8(hid, W8, s, torch.arange(40, dtype=torch.int32, device="cuda"), 33)


def test_side_stream_and_graph(vt):
    B, H, K = 20, 700, 900
    W8, s, _ = vt.vt_quantize_head(torch.randn((K, H), device="cuda").to(torch.bfloat16))
    hid = [torch.randn((B, H), device="cuda").to(torch.bfloat16) for _ in range(3)]
    want = [vt.vt_draft_logits_fp8(h, W8, s) for h in hid]
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    got = [vt.vt_draft_logits_fp8(h, W8, s, stream=st) for h in hid]
    st.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    # two captured graphs with workspaces of their own, replayed on new inputs, in turn and together
    ins = [hid[0].clone(), hid[0].clone()]
    graphs, outs = [], []
    for x in ins:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(vt.vt_draft_logits_fp8(x, W8, s))
        graphs.append(g)
    for i in range(3):
        ins[0].copy_(hid[i])
        ins[1].copy_(hid[2 - i])
        torch.cuda.synchronize()
        graphs[0].replay()
        graphs[1].replay()
        torch.cuda.synchronize()
        assert torch.equal(outs[0], want[i]) and torch.equal(outs[1], want[2 - i])


def test_calls_on_two_streams_at_once(vt):
    # without an order between them; each call has a workspace of its own
    heads = []
    for i in range(2):
        W8, s, _ = vt.vt_quantize_head(torch.randn((5000, 1024), device="cuda").to(torch.bfloat16))
        heads.append((W8, s))
    ids = torch.arange(5000, dtype=torch.int32, device="cuda")
    hid = [torch.randn((b, 1024), device="cuda").to(torch.bfloat16) for b in (9, 200)]
    u = [torch.rand(b, device="cuda") for b in (9, 200)]
    want = [vt.vt_draft_step_fp8(hid[i], *heads[i], ids, u[i], 1.0) for i in range(2)]
    torch.cuda.synchronize()
    st = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [[], []]
    for _ in range(10):
        for i in range(2):
            got[i].append(vt.vt_draft_step_fp8(hid[i], *heads[i], ids, u[i], 1.0, stream=st[i]))
    torch.cuda.synchronize()
    for i in range(2):
        for q, tok, status in got[i]:
            assert torch.equal(q, want[i][0]) and torch.equal(tok, want[i][1]) and int(status.item()) == 0


@pytest.mark.parametrize("B,H,K", [(50, 300, 1003), (130, 300, 20000), (256, 4300, 21000)])
def test_wide_and_greedy_calls_captured_and_on_two_streams(vt, B, H, K):
    W8, s, _ = vt.vt_quantize_head(torch.randn((K, H), device="cuda").to(torch.bfloat16))
    ids = torch.arange(K, dtype=torch.int32, device="cuda")
    hid = [torch.randn((B, H), device="cuda").to(torch.bfloat16) for _ in range(2)]
    want = [(*vt.vt_draft_step_fp8(h, W8, s, ids, None, 0.0)[:2], vt.vt_draft_logits_fp8(h, W8, s)) for h in hid]
    x = hid[0].clone()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        q, tok, st = vt.vt_draft_step_fp8(x, W8, s, ids, None, 0.0)
        z = vt.vt_draft_logits_fp8(x, W8, s)
    for i in (1, 0, 1):
        x.copy_(hid[i])
        g.replay()
        torch.cuda.synchronize()
        assert int(st.item()) == 0
        assert all(torch.equal(a, b) for a, b in zip((q, tok, z), want[i]))
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = []
    for _ in range(5):
        for i in range(2):
            got.append((i, vt.vt_draft_step_fp8(hid[i], W8, s, ids, None, 0.0, stream=streams[i]),
                        vt.vt_draft_logits_fp8(hid[i], W8, s, stream=streams[i])))
    torch.cuda.synchronize()
    for i, (q, tok, st), z in got:
        assert int(st.item()) == 0
        assert all(torch.equal(a, b) for a, b in zip((q, tok, z), want[i]))
