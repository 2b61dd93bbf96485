"""vt_beam_select and vt_beam_reorder against the fp64 oracle (oracle/beam.py).

Parents, tokens and moved states are compared exactly.  Scores: ln S of a row is
good to 5e-6 (half of the distance within which the library sums again, see
vt_beam.cu), the rest is fp64, rounded once: |score - ref| <= 5e-6 + 2^-24 |ref|.
"""
import numpy as np
import pytest

from oracle.beam import beam_reorder, beam_select

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


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _inputs(seed, B, W, K, dt, pad=0, lead=0, spread=2.0):
    g = _gen(seed)
    buf = torch.randn(lead + B * W * (K + pad), generator=g, device="cuda") * spread
    x = buf.to(dt)[lead:].view(B, W, K + pad)[:, :, :K]
    return x, -10.0 + 2.0 * torch.randn((B, W), generator=g, device="cuda")


def _check(vt, x, s, n, T=1.0, status=0, trim=None, done=None, end_id=-1):
    sc, pa, tk, dn, st = vt.vt_beam_select(x, s, n, T, trim_ids=trim, done=done, end_id=end_id)
    host = lambda t: None if t is None else t.cpu().numpy()  # noqa: E731
    ref = beam_select(x.float().cpu().numpy(), host(s), n, float(np.float32(T)), host(trim), host(done), end_id)
    assert int(st.item()) == status
    assert (ref["gap"] > 2e-8).all(), "the inputs leave the order open"
    assert np.array_equal(pa.cpu().numpy(), ref["parent"])
    assert np.array_equal(tk.cpu().numpy(), ref["tokens"])
    if end_id >= 0:
        assert np.array_equal(dn.cpu().numpy().astype(bool), ref["done"])
    else:
        assert dn is None
    got, want = sc.cpu().numpy().astype(np.float64), ref["scores"]
    assert np.array_equal(np.isneginf(got), np.isneginf(want))
    f = np.isfinite(want)
    assert np.all(np.abs(got[f] - want[f]) <= 5e-6 + 2.0 ** -24 * np.abs(want[f]))
    return sc, pa, tk


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("B,W,K,n", [(1, 1, 1, 1), (1, 1, 1, 3), (2, 3, 2, 8), (1, 1, 31, 32), (3, 1, 32, 32),
                                     (1, 32, 33, 32), (4, 5, 100, 7), (2, 8, 1003, 8), (7, 2, 2048, 1), (1, 4, 8193, 16),
                                     (16, 8, 3000, 8), (3, 7, 32003, 5), (200, 3, 257, 4)])
def test_random_beams(vt, B, W, K, n, dt):
    x, s = _inputs(B + K, B, W, K, dt)
    _check(vt, x, s, n, 0.7)


@pytest.mark.parametrize("dt,K", [(torch.float32, 128256), (torch.bfloat16, 152064), (torch.float32, 400003)])
def test_long_rows(vt, dt, K):
    for B, W in ((1, 1), (1, 3)):
        x, s = _inputs(K + W, B, W, K, dt)
        _check(vt, x, s, 8)


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("pad,lead", [(0, 1), (1, 0), (3, 2), (13, 5), (0, 3), (8, 0)])
def test_strides_and_alignment(vt, dt, pad, lead):
    for K in (5, 1003, 9001):
        x, s = _inputs(K + pad, 3, 4, K, dt, pad, lead)
        _check(vt, x, s, 6)


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("K", [40, 3000, 20000, 140000])
def test_ordered_and_tied_rows(vt, dt, K):
    up = torch.linspace(-20, 20, K, device="cuda")
    period = torch.arange(K, device="cuda") % 7
    low = torch.full_like(up, torch.finfo(dt).min)
    peak = low.clone()
    peak[K // 2] = 1.0
    x = torch.stack([up, up.flip(0), torch.zeros_like(up), period.float(), low,
                     torch.where(period == 3, 2.0, -torch.inf), peak, -up.abs()]).to(dt)[None]
    s = -torch.arange(8, device="cuda").float()[None] * 0.31
    for n in (1, 8, 32):
        _check(vt, x, s, n)
        for w in range(8):
            _check(vt, x[:, w:w + 1], s[:, :1].contiguous(), n)


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("K", [7, 1003, 20011])
def test_equal_beams_tie_to_the_lower(vt, dt, K):
    # the same row behind four alignments: equal scores, whatever order it is read in
    g = _gen(K)
    row = (torch.randn(K, generator=g, device="cuda") * 3).to(dt)
    buf = torch.zeros((2, 6, K + 3), dtype=dt, device="cuda")
    x = buf[:, :, :K]
    x[:] = row
    s = torch.full((2, 6), -3.25, device="cuda")
    s[1] = torch.tensor([-5.0, -4.0, -4.0, -4.0, -5.0, -4.5], device="cuda")
    _check(vt, x, s, 32)
    _check(vt, x, s, 5)


def test_near_beams_are_ordered_in_64_bits(vt):
    # the same logits in other orders, so ln S differs in the sums' rounding alone, and scores
    # 2^-21 to 2^-18 apart: nearer than fp32 sums tell, either way round
    K = 5003
    g = _gen(3)
    row = torch.randn(K, generator=g, device="cuda") * 2
    x = torch.stack([row[torch.randperm(K, generator=g, device="cuda")] for _ in range(8)])[None]
    for step in (2.0 ** -21, -2.0 ** -21, 2.0 ** -18, -2.0 ** -18):
        s = (-5.0 + torch.arange(8, device="cuda").double() * step).float()[None]
        for n in (1, 5, 8, 32):
            _check(vt, x, s, n)


def test_masks_and_dead_beams(vt):
    x, s = _inputs(5, 6, 4, 700, torch.float32)
    x = x.clone()
    g = _gen(6)
    x[torch.rand(x.shape, generator=g, device="cuda") < 0.97] = -torch.inf
    x[1] = -torch.inf                       # a sequence with nothing left
    x[2, :3] = -torch.inf                   # one beam left
    x[3, 0, 5:] = -torch.inf                # few ids in one beam
    x[3, 1, :] = LOWEST
    s[3, 2], s[4, 0], s[5, :] = -torch.inf, -torch.inf, -torch.inf
    for n in (1, 4, 32):
        _check(vt, x, s, n)


def test_beams_that_have_ended(vt):
    x, s = _inputs(7, 9, 5, 300, torch.bfloat16)
    g = _gen(8)
    done = torch.rand((9, 5), generator=g, device="cuda") < 0.4
    done[0] = True
    done[1] = False
    s[2, 0], done[2, 0] = -torch.inf, True
    trim = torch.arange(300, dtype=torch.int32, device="cuda") * 3 + 1
    end = int(trim[x[1, 0].float().argmax()])
    for n in (1, 5, 32):
        _check(vt, x, s, n, trim=trim, done=done, end_id=end)
        _check(vt, x, s, n, trim=trim, done=done.to(torch.uint8) * 5, end_id=end)
        _check(vt, x, s, n, trim=trim, end_id=end)
    # rows of ended beams are not read
    x = x.clone()
    x[done] = float("nan")
    _check(vt, x, s, 5, trim=trim, done=done, end_id=end)


def test_nonfinite_beams_are_flagged(vt):
    for bad in (float("nan"), float("inf")):
        x, s = _inputs(9, 3, 3, 500, torch.float32)
        x = x.clone()
        x[1, 2, 77] = bad
        _check(vt, x, s, 4, status=vt.VT_DEV_NONFINITE)
        x, s = _inputs(9, 3, 3, 500, torch.float32)
        s[0, 1] = bad
        _check(vt, x, s, 4, status=vt.VT_DEV_NONFINITE)


@pytest.mark.parametrize("T", [1e-30, 1e-3, 0.5, 3.0, 1e4, 1e30])
def test_temperatures(vt, T):
    x, s = _inputs(10, 2, 3, 400, torch.float32)
    if T < 1e-10:
        s = torch.tensor([[-1.0, -2.0, -3.0]] * 2, device="cuda")   # beams apart: candidates are 1e30 apart
    elif T > 1e3:
        s = torch.tensor([[-1.0, -1.5, -9.0]] * 2, device="cuda")
        x = (torch.arange(400, device="cuda") % 40 * 16.0).expand(2, 3, 400).contiguous() + s[:, :, None]
    _check(vt, x, s, 6, T)


def test_spread_beyond_fp32(vt):
    x = torch.zeros((1, 2, 50), device="cuda")
    x[0, 0, 3], x[0, 0, 4], x[0, 1, 9] = 3e38, -3e38, 3.2e38
    _check(vt, x, torch.tensor([[-1.0, -2.0]], device="cuda"), 3, 1.0)
    _check(vt, x, torch.tensor([[-1.0, -2.0]], device="cuda"), 3, 1e30)


def test_many_rows_and_wide_sequences(vt):
    x, s = _inputs(11, 300, 32, 129, torch.float32)
    _check(vt, x, s, 32, 1.3)
    x, s = _inputs(12, 40, 31, 5000, torch.bfloat16)
    _check(vt, x, s, 9)


def test_select_outputs_and_refusals(vt):
    x, s = _inputs(13, 2, 3, 64, torch.float32)
    ws = torch.empty(vt.workspace_bytes("beam_select", B=2, W=3, K=64, n=4), dtype=torch.uint8, device="cuda")
    sc = torch.empty((2, 4), device="cuda")
    out = vt.vt_beam_select(x, s, 4, out_scores=sc, workspace=ws)
    assert out[0] is sc
    for kw in (dict(out_scores=sc[:, :3]), dict(out_parent=sc), dict(done=s), dict(workspace=ws[:8])):
        with pytest.raises((ValueError, TypeError, vt.VtError)):
            vt.vt_beam_select(x, s, 4, **kw)
    for args in ((x[0], s, 4), (x, s[:1], 4), (x, s, 33), (x, s, 0), (x.transpose(0, 1), s, 4), (x.double(), s, 4),
                 (x.expand(2, 3, 64)[:, :, ::2], s, 4)):
        with pytest.raises((ValueError, TypeError)):
            vt.vt_beam_select(*args)
    with pytest.raises(ValueError, match="end_id"):
        vt.vt_beam_select(x, s, 4, done=torch.zeros((2, 3), dtype=torch.bool, device="cuda"))


# ------------------------------------------------------------- reordering
def _parents(seed, B, W, n):
    g = _gen(seed)
    return torch.randint(0, W, (B, n), generator=g, device="cuda", dtype=torch.int32)


def _reorder(vt, state, parent, dim=0, lengths=None, len_dim=None, status=0):
    np_ = lambda t: t.view(torch.int16).cpu().numpy() if t.dtype == torch.bfloat16 else t.cpu().numpy()  # noqa: E731
    ln = lengths.cpu().numpy() if lengths is not None else None
    before = np_(state)
    # apart, into a buffer that holds something
    out = torch.full_like(state, 3)
    want = beam_reorder(before, parent.cpu().numpy(), np_(out), dim, ln, len_dim)
    got, st = vt.vt_beam_reorder(state, parent, out, dim, lengths, len_dim)
    assert got is out and int(st.item()) == status
    assert np.array_equal(np_(out), want) and np.array_equal(np_(state), before)
    # in place
    if parent.shape[1] <= state.shape[dim + 1]:
        want = beam_reorder(before, parent.cpu().numpy(), before, dim, ln, len_dim)
        got, st = vt.vt_beam_reorder(state, parent, dim=dim, lengths=lengths, len_dim=len_dim)
        assert got is state and int(st.item()) == status
        assert np.array_equal(np_(state), want)


@pytest.mark.parametrize("shape", [(1, 1, 1), (3, 2, 1), (2, 8, 2048), (16, 8, 8), (5, 32, 33), (4, 3, 1031), (1, 7, 65537)])
@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32, torch.uint8, torch.int64])
def test_reorder_rows(vt, shape, dt):
    B, W, H = shape
    state = (torch.rand(shape, generator=_gen(H), device="cuda") * 100).to(dt)
    _reorder(vt, state, _parents(H, B, W, W))


@pytest.mark.parametrize("dt,D", [(torch.bfloat16, 64), (torch.float32, 3), (torch.uint8, 5), (torch.bfloat16, 80)])
def test_reorder_caches(vt, dt, D):
    B, W, h, S = 5, 6, 3, 37
    g = _gen(D)
    lengths = torch.tensor([0, 1, 20, 37, 99], dtype=torch.int32, device="cuda")
    for shape, dim, ld in (((2, B, W, h, S, D), 1, 4), ((2, B, W, S, h, D), 1, 3), ((B, W, S, h, D), 0, 2),
                           ((B, W, h, S, D), 0, 3)):
        state = (torch.rand(shape, generator=g, device="cuda") * 100).to(dt)
        _reorder(vt, state, _parents(D, B, W, W), dim, lengths, ld)
        _reorder(vt, state, _parents(D + 1, B, W, W), dim)
    lengths[0] = -4
    state = (torch.rand((B, W, S), generator=g, device="cuda") * 100).to(dt)
    _reorder(vt, state, _parents(3, B, W, W), 0, lengths, 2)


def test_reorder_cycles_and_missing_parents(vt):
    state = torch.rand((4, 8, 100), generator=_gen(1), device="cuda")
    p = torch.tensor([[1, 2, 3, 4, 5, 6, 7, 0], [7, 6, 5, 4, 3, 2, 1, 0], [0, 1, 2, 3, 4, 5, 6, 7],
                      [-1, 0, -1, 0, 3, -1, 2, 2]], dtype=torch.int32, device="cuda")
    _reorder(vt, state, p)
    p[1, 3], p[2, 2] = 8, -2
    _reorder(vt, state, p, status=vt.VT_DEV_BAD_ID)


def test_reorder_other_numbers_of_beams(vt):
    state = torch.rand((3, 8, 50), generator=_gen(2), device="cuda")
    _reorder(vt, state, _parents(1, 3, 8, 5))              # fewer slots: the others stay
    one = torch.rand((3, 1, 50), generator=_gen(3), device="cuda")
    out = torch.zeros((3, 8, 50), device="cuda")
    p = torch.zeros((3, 7), dtype=torch.int32, device="cuda")
    vt.vt_beam_reorder(one, p, out)                        # the root's state to every beam
    assert torch.equal(out[:, :7], one.expand(3, 7, 50)) and not out[:, 7].any()


def test_reorder_strided_states(vt):
    wide = torch.rand((4, 6, 20, 24), generator=_gen(4), device="cuda")
    keep = wide.clone()
    view = wide[:, :, :, 4:12]
    _reorder(vt, view, _parents(5, 4, 6, 6))
    assert torch.equal(wide[:, :, :, :4], keep[:, :, :, :4]) and torch.equal(wide[:, :, :, 12:], keep[:, :, :, 12:])
    _reorder(vt, wide[:, :, :, 1:4], _parents(6, 4, 6, 6), 0, torch.tensor([3, 0, 20, 7], dtype=torch.int32, device="cuda"), 2)
    _reorder(vt, wide.transpose(0, 1)[:, :4], _parents(7, 6, 4, 4))


def test_reorder_refusals(vt):
    s = torch.zeros((4, 6, 8, 2), device="cuda")
    p = torch.zeros((4, 6), dtype=torch.int32, device="cuda")
    n = torch.zeros(4, dtype=torch.int32, device="cuda")
    flat = torch.zeros(1000, device="cuda")
    for args, kw in [((s, p[:3]), {}), ((s, p.long()), {}), ((s, p), dict(dim=3)), ((s, p), dict(lengths=n)),
                     ((s, p), dict(lengths=n, len_dim=1)), ((s, p), dict(lengths=n[:3], len_dim=2)),
                     ((s.transpose(2, 3), p), dict(lengths=n, len_dim=2)), ((s, p, s.half()), {}),
                     ((s, p, torch.zeros((4, 5, 8, 2), device="cuda")), {}),
                     ((s, p, torch.zeros((4, 6, 8, 1), device="cuda")), {}),
                     ((flat[:384].view(4, 6, 16), p, flat[8:392].view(4, 6, 16)), {}),
                     ((s, p, torch.zeros((4, 1, 8, 2), device="cuda").expand(4, 6, 8, 2)), {}),
                     ((s[:, :3].contiguous(), p), {}), ((s.cpu(), p), {}),
                     ((s, torch.zeros((4, 33), dtype=torch.int32, device="cuda")), {})]:
        with pytest.raises((ValueError, TypeError)):
            vt.vt_beam_reorder(*args, **kw)


# ------------------------------------------- streams, graphs, used together
def test_streams_and_graphs(vt):
    x, s = _inputs(20, 4, 5, 9000, torch.float32)
    state = torch.rand((4, 5, 640), device="cuda")
    want = [t.clone() for t in vt.vt_beam_select(x, s, 5)[:3]]
    moved = vt.vt_beam_reorder(state, want[1], torch.empty_like(state))[0]
    torch.cuda.synchronize()
    side = [torch.cuda.Stream() for _ in range(3)]
    got = []
    for st in side:
        with torch.cuda.stream(st):
            a = vt.vt_beam_select(x, s, 5)
            got.append((*a[:3], vt.vt_beam_reorder(state, a[1], torch.empty_like(state))[0]))
    own = vt.vt_beam_select(x, s, 5, stream=side[0])
    side[0].synchronize()
    got.append((*own[:3], moved))
    torch.cuda.synchronize()
    for g in got:
        for a, b in zip(g, (*want, moved)):
            assert torch.equal(a, b)
    # a step captured, its inputs changed between replays
    bufs = dict(out_scores=torch.empty((4, 5), device="cuda"), out_parent=torch.empty((4, 5), dtype=torch.int32, device="cuda"),
                out_tokens=torch.empty((4, 5), dtype=torch.int32, device="cuda"),
                dev_status=torch.empty(1, dtype=torch.int32, device="cuda"),
                workspace=torch.empty(vt.workspace_bytes("beam_select", B=4, W=5, K=9000, n=5), dtype=torch.uint8, device="cuda"))
    rs = torch.empty(1, dtype=torch.int32, device="cuda")
    xin, sin, out = x.clone(), s.clone(), torch.empty_like(state)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        vt.vt_beam_select(xin, sin, 5, **bufs)
        vt.vt_beam_reorder(state, bufs["out_parent"], out, dev_status=rs)
    for k in range(3):
        x2, s2 = _inputs(30 + k, 4, 5, 9000, torch.float32)
        xin.copy_(x2)
        sin.copy_(s2)
        graph.replay()
        torch.cuda.synchronize()
        a = vt.vt_beam_select(x2, s2, 5)
        assert torch.equal(a[0], bufs["out_scores"]) and torch.equal(a[1], bufs["out_parent"])
        assert torch.equal(vt.vt_beam_reorder(state, a[1], torch.empty_like(state))[0], out)


@pytest.mark.parametrize("fp8", [False, True])
def test_a_tree_grown_by_beams_is_verified(vt, fp8):
    """Draft a tree of three levels through a trimmed head, beams for nodes, and verify it
    greedily against a target: the path found is the one the oracle finds."""
    import oracle
    B, W, H, K, V, depth = 3, 8, 64, 500, 2000, 3
    g = _gen(40)
    head = (torch.randn((V, H), generator=g, device="cuda") * 0.3).to(torch.bfloat16)
    top = torch.randperm(V, generator=g, device="cuda")[:K].to(torch.int32)
    W_trim, trim_ids, _, st = vt.vt_trim_head(head, top)
    embed = torch.randn((V, H), generator=g, device="cuda")
    if fp8:
        W8, w_scale, _ = vt.vt_quantize_head(W_trim)
    hidden = torch.randn((B, 1, H), generator=g, device="cuda")
    state = torch.zeros((B, W, H), device="cuda")
    scores = torch.zeros((B, 1), device="cuda")
    last = torch.full((B, 1), -1, dtype=torch.int32, device="cuda")
    parents, tokens = [], []
    for d in range(depth):
        w = hidden.shape[1]
        h = hidden.reshape(B * w, H).to(torch.bfloat16)
        z = vt.vt_draft_logits_fp8(h, W8, w_scale) if fp8 else vt.vt_draft_logits(h, W_trim)
        sc, pa, tk, _, st = vt.vt_beam_select(z.view(B, w, K), scores, W, trim_ids=trim_ids)
        assert int(st.item()) == 0
        ref = beam_select(z.view(B, w, K).cpu().numpy(), scores.cpu().numpy(), W, 1.0, trim_ids.cpu().numpy())
        assert np.array_equal(pa.cpu().numpy(), ref["parent"]) and np.array_equal(tk.cpu().numpy(), ref["tokens"])
        # a node's parent: the context, or its beam's node of the level above
        parents.append(torch.full_like(pa, -1) if d == 0 else pa + (d - 1) * W)
        tokens.append(tk)
        hidden, st = vt.vt_beam_reorder(hidden.contiguous(), pa, state)
        hidden = 0.5 * hidden + embed[tk.long()]
        scores = sc
    parent, token = torch.cat(parents, 1).contiguous(), torch.cat(tokens, 1).contiguous()
    target = torch.randn((B, depth * W + 1, V), generator=g, device="cuda")
    for b in range(B):   # the target agrees with one path to the second level
        i = b
        j = int((parent[b, W:2 * W] == i).nonzero()[0]) if bool((parent[b, W:2 * W] == i).any()) else None
        target[b, 0, token[b, i]] = 50.0
        if j is not None:
            target[b, i + 1, token[b, W + j]] = 50.0
    out, n, path, st = vt.vt_verify_tree(target, parent, token)
    ref = oracle.verify_tree_greedy(target.cpu().numpy(), parent.cpu().numpy(), token.cpu().numpy())
    assert int(st.item()) == 0 and int(n.min()) >= 1
    assert np.array_equal(out.cpu().numpy(), ref.tokens) and np.array_equal(n.cpu().numpy(), ref.num_accepted)
