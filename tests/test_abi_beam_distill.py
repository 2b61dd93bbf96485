"""Refusals of the beam search and distillation calls that the host decides
before any device work (no GPU needed)."""
import ctypes

import pytest


@pytest.fixture(scope="module")
def lib():
    from drafter_sampling_gb300 import build
    build.build()
    from drafter_sampling_gb300 import _lib
    return _lib.load()


FAKE = ctypes.c_void_p(256)
ODD = ctypes.c_void_p(258)
BIG = 1 << 30
NAN, INF = float("nan"), float("inf")


def _bad():
    from drafter_sampling_gb300 import _lib
    return _lib.VT_ERR_INVALID_ARG, _lib.VT_ERR_UNSUPPORTED, _lib.VT_ERR_WORKSPACE


def test_beam_select_refusals(lib):
    bad, _, ws = _bad()
    ok = dict(l=FAKE, dt=0, B=2, W=3, K=10, ld=10, s=FAKE, done=None, end=-1, trim=None, n=4, T=1.0, os=FAKE,
              op=FAKE, ot=FAKE, od=None, st=FAKE, ws=FAKE, nb=BIG)

    def call(**kw):
        a = {**ok, **kw}
        return lib.vt_beam_select(*(a[k] for k in ok), None)
    for kw in [dict(l=None), dict(s=None), dict(os=None), dict(op=None), dict(ot=None), dict(st=None), dict(dt=2),
               dict(dt=-1), dict(B=0), dict(W=0), dict(W=33), dict(K=0), dict(K=(1 << 22) + 1, ld=1 << 23),
               dict(ld=9), dict(n=0), dict(n=33), dict(B=1 << 20, W=32), dict(T=0.0), dict(T=-1.0), dict(T=NAN),
               dict(T=INF), dict(T=1e-31), dict(l=ODD), dict(end=-2), dict(done=FAKE, od=FAKE),
               dict(od=FAKE), dict(end=3, done=FAKE)]:
        assert call(**kw) == bad, kw
    for kw in [dict(ws=None), dict(ws=ctypes.c_void_p(264)), dict(nb=16)]:
        assert call(**kw) == ws, kw
    assert lib.vt_beam_select_workspace_bytes(2, 3, 10, 4) > 0
    for a in [(0, 3, 10, 4), (2, 0, 10, 4), (2, 33, 10, 4), (2, 3, 0, 4), (2, 3, 10, 0), (2, 3, 10, 33)]:
        assert lib.vt_beam_select_workspace_bytes(*a) == 0


def test_beam_reorder_refusals(lib):
    bad, unsupported, _ = _bad()
    five = lambda *v: (ctypes.c_int64 * 5)(*v)  # noqa: E731
    ok = dict(s=FAKE, o=ctypes.c_void_p(1 << 20), st=five(0, 64, 16, 0, 0), ost=five(0, 64, 16, 0, 0), outer=1, B=2,
              W=4, n=4, inner=1, pos=1, row=16, par=FAKE, len=None, dev=FAKE)

    def call(**kw):
        a = {**ok, **kw}
        return lib.vt_beam_reorder(*(a[k] for k in ok), None)
    for kw in [dict(s=None), dict(o=None), dict(st=None), dict(ost=None), dict(par=None), dict(dev=None),
               dict(outer=0), dict(B=0), dict(W=0), dict(W=33), dict(n=0), dict(n=33), dict(inner=0), dict(pos=0),
               dict(row=0), dict(st=five(0, -64, 16, 0, 0)), dict(ost=five(0, 64, -16, 0, 0)),
               dict(o=FAKE, ost=five(0, 64, 32, 0, 0)),         # in place with other strides
               dict(o=FAKE, n=5)]:                              # in place, more slots than beams
        assert call(**kw) == bad, kw
    assert call(row=1 << 41) == unsupported
    assert call(pos=1 << 39, row=1 << 39) == unsupported


def _distill_ok():
    return dict(l=FAKE, dt=0, R=2, K=10, ld=10, ids=FAKE, lp=FAKE, k=3, inv=None, V=10)


DISTILL_BAD = [dict(l=None), dict(ids=None), dict(lp=None), dict(dt=2), dict(R=0), dict(R=(1 << 24) + 1), dict(K=0),
               dict(K=(1 << 22) + 1, V=(1 << 22) + 1, ld=1 << 23), dict(ld=9), dict(k=0), dict(k=129), dict(V=0),
               dict(V=11), dict(V=0, inv=FAKE), dict(l=ODD), dict(T=0.0), dict(T=NAN), dict(T=INF), dict(T=-1.0)]


def test_distill_refusals(lib):
    bad, _, _ = _bad()
    grad = ctypes.c_void_p(1 << 20)
    loss_ok = {**_distill_ok(), "rest": 1, "T": 1.0, "loss": FAKE, "stats": FAKE, "st": FAKE}
    grad_ok = {**_distill_ok(), "T": 1.0, "stats": FAKE, "g": None, "grad": grad, "ldg": 10}
    both_ok = {**_distill_ok(), "rest": 1, "T": 1.0, "g": None, "loss": FAKE, "stats": FAKE, "grad": grad, "ldg": 10,
               "st": FAKE}
    for fn, ok, more in [(lib.vt_distill_loss, loss_ok, [dict(loss=None), dict(st=None), dict(rest=2)]),
                         (lib.vt_distill_grad, grad_ok, []),
                         (lib.vt_distill_loss_grad, both_ok, [dict(loss=None), dict(st=None), dict(rest=-1)])]:
        cases = DISTILL_BAD + more + [dict(stats=None), dict(stats=ODD)]
        if "grad" in ok:
            cases += [dict(grad=None), dict(ldg=9), dict(grad=ctypes.c_void_p((1 << 20) + 2)),
                      dict(grad=ctypes.c_void_p(260)),          # overlaps the logits, elsewhere
                      dict(grad=FAKE, ldg=12)]                  # in place with another stride
        for kw in cases:
            a = {**ok, **kw}
            assert fn(*(a[k] for k in ok), None) == bad, (fn, kw)


def test_binding_refusals_name_the_argument():
    torch = pytest.importorskip("torch")
    import drafter_sampling_gb300 as vt
    cpu = torch.zeros((2, 3, 8))
    ids = torch.zeros((2, 3, 1), dtype=torch.int32)
    with pytest.raises(ValueError, match="logits must be a CUDA"):
        vt.vt_beam_select(cpu, cpu[:, :, 0], 2)
    with pytest.raises(TypeError, match="logits"):
        vt.vt_beam_select(None, None, 2)
    with pytest.raises(ValueError, match="state must be a CUDA"):
        vt.vt_beam_reorder(cpu, ids[:, :, 0])
    for fn in (vt.vt_distill_loss, vt.vt_distill_loss_grad):
        with pytest.raises(ValueError, match="logits must be a CUDA"):
            fn(cpu, ids, cpu[:, :, :1])
    with pytest.raises(ValueError, match="logits must be a CUDA"):
        vt.vt_distill_grad(cpu, ids, cpu[:, :, :1], None)
    assert vt.workspace_bytes("beam_select", B=2, W=3, K=100, n=4) > 0


def test_layouts_of_states():
    """How a state's dimensions become (outer, B, W, inner, positions) and a row."""
    torch = pytest.importorskip("torch")
    from drafter_sampling_gb300 import _beam_parts

    def parts(t, d, n):
        ext, st, ost, row = _beam_parts("state", t.shape, t.stride(), t.stride(), d, n)
        assert st == ost
        return ext, st, row
    e = torch.empty
    assert parts(e(4, 3, 16), 0, None) == ((1, 4, 3, 1, 1), (0, 48, 16, 0, 0), 16)
    assert parts(e(2, 4, 3, 5, 7, 6), 1, 4) == ((2, 4, 3, 5, 7), (2520, 630, 210, 42, 6), 6)
    assert parts(e(2, 4, 3, 7, 5, 6), 1, 3) == ((2, 4, 3, 1, 7), (2520, 630, 210, 0, 30), 30)
    assert parts(e(4, 3, 9), 0, 2) == ((1, 4, 3, 1, 9), (0, 27, 9, 0, 1), 1)
    # layers and halves before the sequences walk with one stride
    assert parts(e(3, 2, 4, 3, 8), 2, None) == ((6, 4, 3, 1, 1), (96, 24, 8, 0, 0), 8)
    # a slice of a wider cache
    assert parts(e(4, 3, 9, 8)[:, :, :, :4], 0, None) == ((1, 4, 3, 9, 1), (0, 216, 72, 8, 0), 4)
    assert parts(e(4, 3), 0, None) == ((1, 4, 3, 1, 1), (0, 3, 1, 0, 0), 1)
    # two layouts: rows as long as both allow
    a, b = e(4, 3, 9, 8), e(4, 3, 9, 16)[:, :, :, :8]
    assert _beam_parts("state", a.shape, a.stride(), b.stride(), 0, None) == (
        (1, 4, 3, 9, 1), (0, 216, 72, 8, 0), (0, 432, 144, 16, 0), 8)
    for t, d, n in [(e(4, 3, 8, 2).transpose(2, 3), 0, 2), (e(3, 2, 4, 3, 8)[:, :1].expand(3, 2, 4, 3, 8), 2, None)]:
        with pytest.raises(ValueError, match="contiguous rows"):
            parts(t, d, n)
