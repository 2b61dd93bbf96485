"""vt_distill_loss, vt_distill_grad and vt_distill_loss_grad against the fp64
oracle (oracle/distill.py).

With u = 2^-24: ln S of a row or of its unlisted ids is off by at most E =
u (V / 256 + 90), as the log probabilities' sums are (V / 256 additions in one
thread and 16 more joining, each weight off by the exponential's 4 u and by three
roundings of its argument, whose mean under the softmax is at most 22 u each).
What else enters the loss is fp64 or a pair of fp32 values (t and what it leaves
of 1: 2^-28).  So with A the teacher's mass that counts and b its rest
  |loss - ref| <= (A + 2 b + 1) E + 2^-26 (|ln b| + |ln q| + 1) (b > 0) + 2 u |ref| + 2^-26.
A gradient is a difference of A p_j and what the teacher pulls: each is off by
E and by its own exponential (4 u, and three roundings of |z - max| / T) and
roundings (6 u), the rest's pull by 2^-27 / q p_j more:
  |grad - ref| <= |w| / T ((A p + pull) (E + u (10 + 3 |d|)) + 2^-27 p / q) + 1e-37,
and the result's own rounding, u |ref| or 2^-8 |ref|.
"""
import numpy as np
import pytest

from oracle.distill import distill

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

LOWEST = -3.4028234663852886e38
U = 2.0 ** -24


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


def _inputs(seed, R, K, k, dt, pad=0, lead=0, trimmed=False, spread=3.0):
    """(logits, top_ids, top_logp, inv_map, weight): a teacher near the drafter."""
    g = _gen(seed)
    buf = torch.randn(lead + R * (K + pad), generator=g, device="cuda") * spread
    x = buf.to(dt)[lead:].view(R, K + pad)[:, :K]
    t = (x.float() + torch.randn(R, K, generator=g, device="cuda")).log_softmax(1).topk(k, 1)
    ids, lnt, inv = t.indices, t.values.contiguous(), None
    if trimmed:
        V = 2 * K + 3
        keep = torch.randperm(V, generator=g, device="cuda")[:K].sort().values
        inv = torch.full((V,), -1, dtype=torch.int32, device="cuda")
        inv[keep] = torch.arange(K, dtype=torch.int32, device="cuda")
        other = (inv < 0).nonzero()[:, 0]
        lost = torch.rand(R, k, generator=g, device="cuda") < 0.2
        ids = torch.where(lost, other[torch.arange(k, device="cuda") % len(other)], keep[ids])
    w = torch.randn(R, generator=g, device="cuda")
    return x, ids.to(torch.int32).contiguous(), lnt, inv, w


def _compare(x, ref, T, w, loss, stats, grad):
    R, K = x.shape
    z = x.float().cpu().numpy().astype(np.float64)
    E = U * (K / 256 + 90)
    bad = ref["bad"]
    got = loss.cpu().numpy().astype(np.float64).reshape(R)
    assert np.array_equal(np.isnan(got), bad)
    b, lnq = ref["left"], ref["lnq"]
    A = ref["mass"] + b
    with np.errstate(divide="ignore", invalid="ignore"):
        more = np.where(b > 0, 2.0 ** -26 * (np.abs(np.log(np.where(b > 0, b, 1.0))) + np.abs(lnq) + 1), 0.0)
        tol = (A + 2 * b + 1) * E + more + 2 * U * np.abs(ref["loss"]) + 2.0 ** -26
    assert np.all((np.abs(got - ref["loss"]) <= tol) | bad), np.nanmax(np.abs(got - ref["loss"]) - tol)
    s = stats.cpu().numpy().reshape(R, 5)
    assert np.array_equal(np.isnan(s).any(1), bad)
    if grad is None:
        return
    g = grad.float().cpu().numpy().astype(np.float64).reshape(R, K)
    assert np.array_equal(np.isnan(g).any(1), bad) and np.array_equal(np.isnan(g).all(1), bad)
    ok = ~bad
    with np.errstate(invalid="ignore", over="ignore"):
        # (a NaN here is in a row that is not read: its gradient is 0, and so is p)
        d = np.nan_to_num(np.minimum(np.where(np.isneginf(z), 0.0, (z.max(1, keepdims=True) - z) / T), 300.0))
        p, pull, r = ref["p"], np.abs(ref["pull"]), ref["grad"]
        q = np.exp(np.clip(lnq, -600, 0))[:, None]
        rest = np.where((b[:, None] > 0) & (ref["pull"] < 0), 2.0 ** -27 * np.minimum(p / q, 1.0), 0.0)
        tol = np.abs(w)[:, None] / T * ((p + pull) * (E + U * (10 + 3 * d)) + rest) + 1e-37
        tol += np.abs(r) * (2.0 ** -8 if x.dtype == torch.bfloat16 else U)
    assert np.all((np.abs(g - r) <= tol)[ok]), np.nanmax((np.abs(g - r) - tol)[ok])


def _check(vt, x, ids, lnt, inv=None, w=None, rest=True, T=1.0, status=0):
    """Every output of the three calls, apart, fused and in place."""
    kw = dict(inv_map=inv, temperature=T)
    loss, stats, st = vt.vt_distill_loss(x, ids, lnt, rest=rest, **kw)
    assert int(st.item()) == status
    grad = vt.vt_distill_grad(x, ids, lnt, stats, grad_loss=w, **kw)
    h = lambda t: None if t is None else t.cpu().numpy()  # noqa: E731
    R, K = x.shape[:-1].numel(), x.shape[-1]
    flat = lambda t: None if t is None else t.reshape(R, t.shape[-1])  # noqa: E731
    T32 = float(np.float32(T))
    wh = np.ones(R) if w is None else h(w).reshape(R).astype(np.float64)
    ref = distill(h(flat(x.float())), h(flat(ids)), h(flat(lnt)), h(inv), rest, T32, wh)
    _compare(flat(x), ref, T32, wh, loss, stats, flat(grad))
    l2, g2, s2, st = vt.vt_distill_loss_grad(x, ids, lnt, grad_loss=w, rest=rest, **kw)
    assert int(st.item()) == status
    _compare(flat(x), ref, T32, wh, l2, s2, flat(g2))
    # in place, the row's padding left alone
    for fused in (False, True):
        base = x
        if x.dim() == 2 and x.stride(0) > K:
            base = torch.as_strided(x, (R - 1, x.stride(0)), (x.stride(0), 1)) if R > 1 else x
        keep = base.clone()
        y = torch.empty(R * max(x.stride(-2), K) + 8, dtype=x.dtype, device="cuda")
        y.fill_(7)
        off = x.storage_offset() % 8
        y = torch.as_strided(y, x.shape, x.stride(), off)
        y.copy_(x)
        if fused:
            vt.vt_distill_loss_grad(y, ids, lnt, grad_loss=w, rest=rest, out_grad=y, **kw)
        else:
            vt.vt_distill_grad(y, ids, lnt, stats, grad_loss=w, out_grad=y, **kw)
        _compare(flat(x), ref, T32, wh, loss, stats, flat(y))
        assert torch.equal(base.nan_to_num(), keep.nan_to_num())
        if x.dim() == 2 and x.stride(0) > K and R > 1:
            gap = torch.as_strided(y, (R - 1, x.stride(0) - K), (x.stride(0), 1), y.storage_offset() + K)
            assert bool((gap == 7).all())
    return loss, grad


@pytest.mark.parametrize("rest", [True, False])
@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("R,K,k", [(1, 1, 1), (2, 2, 1), (3, 7, 7), (1, 33, 32), (4, 100, 5), (2, 130, 128),
                                   (3, 2047, 20), (2, 8193, 100), (1, 9000, 8), (5, 32003, 33), (300, 513, 3)])
def test_random_rows(vt, R, K, k, dt, rest):
    x, ids, lnt, inv, w = _inputs(R + K, R, K, k, dt)
    _check(vt, x, ids, lnt, inv, w, rest, 0.7)
    x, ids, lnt, inv, w = _inputs(R + K + 1, R, K, k, dt, trimmed=True)
    _check(vt, x, ids, lnt, inv, w, rest, 1.3)


@pytest.mark.parametrize("dt,K", [(torch.float32, 128256), (torch.bfloat16, 152064), (torch.float32, 400003),
                                  (torch.bfloat16, 1000003)])
def test_long_rows(vt, dt, K):
    for R in (1, 3):
        x, ids, lnt, inv, w = _inputs(K + R, R, K, 20, dt)
        _check(vt, x, ids, lnt, inv, w, R == 1)


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("pad,lead", [(0, 1), (1, 0), (3, 2), (13, 5), (0, 3), (8, 0)])
def test_strides_and_alignment(vt, dt, pad, lead):
    for K in (5, 1003, 9001):
        x, ids, lnt, inv, w = _inputs(K, 6, K, 4, dt, pad, lead)
        _check(vt, x, ids, lnt, inv, w)
        # a gradient behind another stride and alignment than the logits'
        for gp, gl in ((0, 0), (5, 1), (2, 3)):
            out = torch.full((gl + 6 * (K + gp),), 7.0, dtype=dt, device="cuda")
            view = out[gl:].view(6, K + gp)[:, :K]
            want = vt.vt_distill_loss_grad(x, ids, lnt, w)[1]
            got = vt.vt_distill_loss_grad(x, ids, lnt, w, out_grad=view)
            assert got[1] is view and torch.equal(view, want)
            stats = got[2]
            a = vt.vt_distill_grad(x, ids, lnt, stats, w)
            out.fill_(7.0)
            vt.vt_distill_grad(x, ids, lnt, stats, w, out_grad=view)
            assert torch.equal(view, a)
            assert bool((out[:gl] == 7).all())
            assert gp == 0 or bool((out[gl:].view(6, K + gp)[:, K:] == 7).all())


@pytest.mark.parametrize("dt,R,K,k,pad", [(torch.float32, 3000, 300, 3, 0), (torch.bfloat16, 1500, 5000, 40, 3),
                                          (torch.float32, 420, 20000, 20, 0), (torch.bfloat16, 200, 70001, 9, 1),
                                          (torch.float32, 3, 170001, 100, 0)])
def test_more_rows_than_run_at_once(vt, dt, R, K, k, pad):
    # blocks take several rows in turn, some of them not scored
    x, ids, lnt, inv, w = _inputs(K, R, K, k, dt, pad, trimmed=True)
    skip = torch.arange(R, device="cuda") % 5 > 2
    ids[skip] = -1
    lnt[skip] = float("nan")
    x[skip] = float("nan")
    _check(vt, x, ids, lnt, inv, w, R % 2 == 0)


@pytest.mark.parametrize("rest", [True, False])
def test_rows_do_not_depend_on_the_batch(vt, rest):
    # long rows in many turns of clusters, against the same rows a few at a time: each is within
    # the bound E of the exact value, and the gradients' c_all and c_rest with them
    R, K, k = 470, 128256, 12
    x, ids, lnt, _, w = _inputs(77, R, K, k, torch.float32)
    ids[torch.arange(R, device="cuda") % 7 > 4] = -1
    E = U * (K / 256 + 90)
    loss, stats, st = vt.vt_distill_loss(x, ids, lnt, rest=rest)
    assert int(st.item()) == 0
    l2, g2, s2, st = vt.vt_distill_loss_grad(x, ids, lnt, w, rest=rest, out_grad=x.clone())
    assert int(st.item()) == 0
    for r in range(0, R, 47):
        part = slice(r, r + 5)
        l1, g1, s1, _ = vt.vt_distill_loss_grad(x[part], ids[part].contiguous(), lnt[part].contiguous(),
                                                w[part].contiguous(), rest=rest)
        for l, s in ((loss, stats), (l2, s2)):
            assert torch.all((l[part] - l1).abs() <= 8 * E + 4 * U * l1.abs())
            assert torch.equal(s[part, :2], s1[:, :2])              # the largest logits: exact
            assert torch.all((s[part, 2:] - s1[:, 2:]).abs() <= 4 * E * s1[:, 2:].abs().amax(1, True))
        # the bound of a gradient entry, twice, with A p + pull <= 2 and |d| <= 40
        assert torch.all((g2[part] - g1).abs() <= 4 * w[part, None].abs() * (E + 130 * U) * g1.abs().amax(1, True).clamp(min=1e-3))


def test_batched_logits_and_no_weight(vt):
    x, ids, lnt, _, w = _inputs(3, 12, 700, 6, torch.float32)
    _check(vt, x.view(3, 4, 700), ids.view(3, 4, 6), lnt.view(3, 4, 6), None, w.view(3, 4))
    _check(vt, x, ids, lnt)


@pytest.mark.parametrize("rest", [True, False])
def test_rows_with_nothing_to_learn(vt, rest):
    R, K, k = 9, 500, 5
    x, ids, lnt, inv, w = _inputs(4, R, K, k, torch.float32, trimmed=True)
    x = x.clone()
    ids[0] = -1                                   # no entry
    lnt[0] = float("nan")
    x[0] = float("nan")                           # and not read
    ids[1] = (inv < 0).nonzero()[:k, 0].int()     # none that the drafter has
    place = inv[ids[2].long()].long()
    x[2, place[place >= 0]] = -torch.inf          # all of them masked
    lnt[3] = -torch.inf                           # no mass listed
    ids[4, 1:] = -1                               # one entry
    x[5] = -torch.inf                             # a row whose mask leaves nothing
    x[6, :] = LOWEST
    keep = inv[ids[7].long()].long()
    hide = torch.ones(K, dtype=torch.bool, device="cuda")
    hide[keep[keep >= 0]] = False
    x[7, hide] = -torch.inf                       # nothing but the listed ids
    x[8, hide] = LOWEST if rest else -1e30        # the others at the type's lowest value
    loss, grad = _check(vt, x, ids, lnt, inv, w, rest)
    zero = [0, 1, 2, 5] + ([] if rest else [3])
    assert not loss[zero].any() and not grad[zero].any()


@pytest.mark.parametrize("rest", [True, False])
@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("K", [40, 3000, 20000, 140000])
def test_ordered_and_peaked_rows(vt, dt, K, rest):
    up = torch.linspace(-20, 20, K, device="cuda")
    spike = torch.zeros_like(up)
    spike[K // 3] = 60.0
    far = torch.full_like(up, -90.0)
    far[:4] = torch.tensor([80.0, 79.0, 78.0, 100.0], device="cuda")
    x = torch.stack([up, up.flip(0), torch.zeros_like(up), spike, far, far.flip(0)]).to(dt)
    ids = torch.stack([torch.arange(4), torch.arange(4) + K - 4, torch.tensor([0, 9, K - 1, K // 2]),
                       torch.tensor([K // 3, 1, 2, 3]), torch.arange(4), torch.tensor([K - 9, 7, 8, K - 1])])
    lnt = torch.log(torch.tensor([0.4, 0.3, 0.2, 0.05])).repeat(6, 1).cuda()
    w = torch.linspace(-1, 1, 6, device="cuda")
    _check(vt, x, ids.int().cuda(), lnt, None, w, rest)


def test_teacher_masses(vt):
    # masses above, at and just below 1; tiny ones; a positive logarithm within rounding
    R, K = 6, 300
    x, ids, lnt, _, w = _inputs(6, R, K, 4, torch.float32)
    mass = torch.tensor([1.5, 1.0, 1.0 - 1e-6, 1e-20, 0.5, 1.0], device="cuda")
    lnt = torch.log(mass[:, None] * torch.tensor([0.7, 0.2, 0.0999, 0.0001], device="cuda"))
    lnt[5] = torch.tensor([1e-7, -30.0, -torch.inf, -60.0], device="cuda")
    for rest in (True, False):
        _check(vt, x, ids, lnt, None, w, rest)


@pytest.mark.parametrize("T", [1e-30, 0.01, 0.5, 4.0, 1e4, 1e30])
def test_temperatures(vt, T):
    x, ids, lnt, _, w = _inputs(7, 4, 400, 6, torch.float32)
    if T < 1e-10:
        # a drafter at 1e-30 is sure of its best id, and infinitely far from any other teacher
        ids[:, :] = -1
        ids[:, 2] = x.argmax(1).int()
        lnt = torch.zeros_like(lnt)
    for rest in (True, False):
        _check(vt, x, ids, lnt, None, w, rest, T)


def test_flags(vt):
    K, k = 600, 6
    for what, flag in (("id", vt.VT_DEV_BAD_ID), ("map", vt.VT_DEV_BAD_ID), ("twice", vt.VT_DEV_DUPLICATE_ID),
                       ("nan", vt.VT_DEV_NONFINITE), ("inf", vt.VT_DEV_NONFINITE), ("listed", vt.VT_DEV_NONFINITE),
                       ("logp", vt.VT_DEV_NONFINITE), ("big", vt.VT_DEV_NONFINITE)):
        x, ids, lnt, inv, w = _inputs(8, 3, K, k, torch.float32, trimmed=True)
        x, inv = x.clone(), inv.clone()
        kept = (inv[ids[1].long()] >= 0).nonzero()[:, 0]
        i, j = int(kept[0]), int(kept[-1])
        assert i != j
        unlisted = int((~torch.isin(torch.arange(K, device="cuda"), inv[ids[1].long()].long())).nonzero()[7])
        if what == "id":
            ids[1, 2] = inv.numel()
        elif what == "map":
            spare = int((~torch.isin(torch.arange(inv.numel(), device="cuda"), ids.long())).nonzero()[0])
            inv[spare] = K
            ids[1, 2] = spare
        elif what == "twice":
            ids[1, j] = ids[1, i]
        elif what == "nan":
            x[1, unlisted] = float("nan")
        elif what == "inf":
            x[1, unlisted] = float("inf")
        elif what == "listed":
            x[1, int(inv[ids[1, i].long()])] = float("nan")
        elif what == "logp":
            lnt[1, i] = float("nan")
        else:
            lnt[1, i] = 80.0
        for rest in (True, False):
            _check(vt, x, ids, lnt, inv, w, rest, status=flag)
    # what is not kept is not looked at
    x, ids, lnt, inv, w = _inputs(8, 3, K, k, torch.float32, trimmed=True)
    lost = inv[ids.long()] < 0
    assert bool(lost.any())
    lnt[lost] = float("nan")
    ids[lost & (torch.arange(k, device="cuda") % 2 == 0)] = -1
    _check(vt, x, ids, lnt, inv, w)


def test_gradient_against_differences(vt):
    # the loss's own central difference along the gradient, in fp64 of the oracle
    x, ids, lnt, inv, _ = _inputs(9, 5, 777, 9, torch.float32, trimmed=True)
    for rest in (True, False):
        _, stats, _ = vt.vt_distill_loss(x, ids, lnt, inv, rest, 2.0)
        g = vt.vt_distill_grad(x, ids, lnt, stats, inv_map=inv, temperature=2.0).cpu().numpy().astype(np.float64)
        z, h = x.cpu().numpy().astype(np.float64), 1e-4
        v = g / np.linalg.norm(g, axis=1, keepdims=True)
        at = lambda s: distill(z + s * v, ids.cpu().numpy(), lnt.cpu().numpy(), inv.cpu().numpy(), rest, 2.0)["loss"]  # noqa: E731
        d = (at(h) - at(-h)) / (2 * h)
        # truncation h^2 |f'''| / 6 < 1e-8; the gradient's own error, below 2e-5 of it (the bound above)
        assert np.allclose(d, np.linalg.norm(g, axis=1), rtol=2e-5, atol=1e-8)


def test_outputs_and_refusals(vt):
    x, ids, lnt, inv, w = _inputs(10, 4, 64, 5, torch.float32, trimmed=True)
    loss, stats = torch.empty(4, device="cuda"), torch.empty((4, 5), device="cuda")
    out = vt.vt_distill_loss(x, ids, lnt, inv, out_loss=loss, out_stats=stats)
    assert out[0] is loss and out[1] is stats
    for fn in (lambda *a, **k: vt.vt_distill_loss(*a, **k), lambda *a, **k: vt.vt_distill_grad(*a, stats, **k),
               lambda *a, **k: vt.vt_distill_loss_grad(*a, **k)):
        for args in ((x, ids[:3], lnt), (x, ids.long(), lnt), (x, ids, lnt[:, :4]), (x, ids, lnt.double()),
                     (x.double(), ids, lnt), (x.t(), ids, lnt), (x.cpu(), ids, lnt), (x[:, ::2], ids, lnt),
                     (x, ids.repeat(1, 30), lnt.repeat(1, 30)), (x, ids[:, :0], lnt[:, :0])):
            with pytest.raises((ValueError, TypeError)):
                fn(*args, inv_map=inv)
        with pytest.raises((ValueError, TypeError)):
            fn(x, ids, lnt, inv_map=inv.long())
        with pytest.raises(vt.VtError):
            fn(x, ids, lnt, inv_map=inv, temperature=0.0)
    for bad in (x[:3], x.bfloat16(), x.cpu()):
        with pytest.raises((ValueError, TypeError)):
            vt.vt_distill_grad(x, ids, lnt, stats, inv_map=inv, out_grad=bad)
    with pytest.raises((ValueError, TypeError)):
        vt.vt_distill_grad(x, ids, lnt, stats[:, :4], inv_map=inv)
    buf = torch.zeros(64 * 6, device="cuda")
    with pytest.raises(vt.VtError):
        vt.vt_distill_loss_grad(buf[:256].view(4, 64), ids, lnt, inv_map=inv, out_grad=buf[64:320].view(4, 64))


def test_streams_and_graphs(vt):
    x, ids, lnt, inv, w = _inputs(11, 40, 9000, 9, torch.float32, trimmed=True)
    want = [t.clone() for t in vt.vt_distill_loss_grad(x, ids, lnt, w, inv)[:3]]
    back = vt.vt_distill_grad(x, ids, lnt, want[2], w, inv)
    torch.cuda.synchronize()
    side = [torch.cuda.Stream() for _ in range(3)]
    got = []
    for s in side:
        with torch.cuda.stream(s):
            a = vt.vt_distill_loss(x, ids, lnt, inv)
            got.append((a[0], vt.vt_distill_grad(x, ids, lnt, a[1], w, inv)))
    got.append(vt.vt_distill_loss_grad(x, ids, lnt, w, inv, stream=side[0])[:2])
    torch.cuda.synchronize()
    for a, b in got[:3]:
        assert torch.equal(a, got[0][0]) and torch.equal(b, got[0][1])
    assert torch.equal(got[3][0], want[0]) and torch.equal(got[3][1], want[1])
    xin, loss, grad, stats = x.clone(), torch.empty_like(want[0]), torch.empty_like(x), torch.empty_like(want[2])
    g2, st = torch.empty_like(x), torch.zeros(1, dtype=torch.int32, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        vt.vt_distill_loss_grad(xin, ids, lnt, w, inv, out_loss=loss, out_grad=grad, out_stats=stats, dev_status=st)
        vt.vt_distill_grad(xin, ids, lnt, stats, w, inv, out_grad=g2)
    for k in range(3):
        x2 = _inputs(20 + k, 40, 9000, 9, torch.float32)[0]
        xin.copy_(x2)
        graph.replay()
        torch.cuda.synchronize()
        a = vt.vt_distill_loss_grad(x2, ids, lnt, w, inv)
        assert torch.equal(a[0], loss) and torch.equal(a[1], grad) and int(st.item()) == 0
        assert torch.equal(vt.vt_distill_grad(x2, ids, lnt, a[2], w, inv), g2)
    assert torch.equal(vt.vt_distill_grad(x, ids, lnt, want[2], w, inv), back)


def test_a_trimmed_head_learns_from_the_targets_alternatives(vt):
    """The target's k best from vt_token_logprobs, the drafter's logits from vt_draft_logits, loss
    and gradient, and the head's gradient by a product: all of it against the oracle."""
    R, H, V, K, k, T = 24, 64, 1200, 400, 16, 1.5
    g = _gen(50)
    head = (torch.randn((V, H), generator=g, device="cuda") * 0.2).to(torch.bfloat16)
    hidden = torch.randn((R, H), generator=g, device="cuda").to(torch.bfloat16)
    W_trim, trim_ids, inv_map, _ = vt.vt_trim_head(head, torch.randperm(V, generator=g, device="cuda")[:K].to(torch.int32))
    target = hidden.float() @ head.float().t() + torch.randn((R, V), generator=g, device="cuda")
    given = torch.zeros(R, dtype=torch.int32, device="cuda")
    given[5:8] = -1                      # positions behind the last emitted token
    _, _, ids, lnt, st = vt.vt_token_logprobs(target, given, k=k, temperature=T)
    assert int(st.item()) == 0
    z = vt.vt_draft_logits(hidden, W_trim)
    w = torch.full((R,), 1.0 / R, device="cuda")
    for rest in (True, False):
        loss, grad = _check(vt, z, ids, lnt, inv_map, w, rest, T)
        ref = distill(z.cpu().numpy(), ids.cpu().numpy(), lnt.cpu().numpy(), inv_map.cpu().numpy(), rest,
                      T, w.cpu().numpy())
        dW = (grad.t().double() @ hidden.double()).cpu().numpy()
        want = ref["grad"].T @ hidden.double().cpu().numpy()
        assert np.linalg.norm(dW - want) <= 2e-5 * np.linalg.norm(want)
        assert not loss[5:8].any() and not grad[5:8].any()


@pytest.mark.parametrize("call", ["vt_distill_loss", "vt_distill_loss_grad", "vt_beam_select"])
def test_the_first_call_of_a_process_may_be_captured(vt, call):
    import os
    import subprocess
    import sys
    code = f"""
import torch
import drafter_sampling_gb300 as vt
x = torch.randn((6, 5, 3000), device="cuda")
ids = torch.arange(6 * 5 * 2, device="cuda", dtype=torch.int32).view(6, 5, 2)
low = torch.full((6, 5, 2), -1.0, device="cuda")
torch.cuda.synchronize()
f = (lambda: vt.vt_beam_select(x, low[:, :, 0].contiguous(), 4)[:3]) if "{call}" == "vt_beam_select" else (
    lambda: vt.{call}(x, ids, low)[:2])
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    got = f()
g.replay()
torch.cuda.synchronize()
assert all(torch.equal(a, b) for a, b in zip(got, f()))
print("equal")
"""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "equal" in r.stdout, r.stderr[-2000:]
