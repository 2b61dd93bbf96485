"""Losses of logits whose difference, or its quotient by T, lies beyond fp32 while the loss does not.

Such a loss is sum t (ln t - ln p) or b ln q with differences that pairs of fp32 values hold to 2^-45, t to
2^-28 of itself and b = 1 - a, here at least 0.1, to 2^-28 a / b <= 2^-24.8 of itself; it is rounded once,
2^-24.  That is below 2^-23 |ref|.  Rows whose loss is ordinary are off by what their sums are: |loss -
ref| <= (A + 2 b + 1) E + 2^-25, A + 2 b <= 3.
"""
import numpy as np
import pytest

from oracle.distill import distill

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

LOWEST = {torch.float32: -3.4028234663852886e38, torch.bfloat16: -3.3895313892515355e38}


@pytest.fixture(scope="module")
def vt():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import drafter_sampling_gb300 as m
    from drafter_sampling_gb300 import build
    build.build()
    m.lib()
    return m


def _rows(dt):
    """(logits, top_ids, top_logp): masks at the type's lowest value among listed and unlisted ids."""
    K, low = 700, LOWEST[dt]
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    x = torch.randn((6, K), generator=g, device="cuda").to(dt)
    ids = torch.arange(5, dtype=torch.int32, device="cuda").repeat(6, 1) * 9
    lnt = torch.log(torch.tensor([0.02, 0.3, 0.2, 0.1, 0.28], device="cuda")).repeat(6, 1)
    x[0, ids[0, 0].long()] = low                    # a listed id masked
    x[1] = low                                      # all but listed ids masked
    x[1, ids[1].long()] = torch.arange(5, device="cuda").to(dt)
    x[2] = low                                      # one id left, which is listed
    x[2, 9] = 0.0
    x[3] = low                                      # one id left, which is not
    x[3, 1] = 2.0
    x[4, 100] = -low                                # one id above all others
    x[4, ids[4, 0].long()] = low
    x[5, ids[5, 1].long()] = -low                   # the same, listed
    x[5, 300:] = low
    lnt[4:] = torch.log(torch.tensor([1e-3, 2e-4, 3e-4, 1e-4, 5e-4], device="cuda"))
    return x, ids, lnt


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("T", [0.3, 0.7, 1.0, 2.0, 4.0, 100.0, 1e6, 1e30])
@pytest.mark.parametrize("rest", [True, False])
def test_differences_beyond_fp32(vt, dt, T, rest):
    x, ids, lnt = _rows(dt)
    h = lambda t: t.float().cpu().numpy()  # noqa: E731
    ref = distill(h(x), ids.cpu().numpy(), h(lnt), None, rest, float(np.float32(T)))["loss"]
    most = float(np.finfo(np.float32).max)
    big, over = ref <= most * (1 - 2.0 ** -22), ref > most * (1 + 2.0 ** -22)  # (between them either may come)
    assert big.any()
    loss, stats, st = vt.vt_distill_loss(x, ids, lnt, rest=rest, temperature=T)
    fused, _, s2, st2 = vt.vt_distill_loss_grad(x, ids, lnt, rest=rest, temperature=T)
    assert int(st.item()) == 0 and int(st2.item()) == 0
    E = 2.0 ** -24 * (700 / 256 + 90)     # what ln S may be off by, where it counts
    for got in (loss, fused):
        got = got.cpu().numpy().astype(np.float64)
        assert np.isposinf(got[over]).all()
        assert np.all(np.abs(got - ref)[big] <= 2.0 ** -23 * np.abs(ref[big]) + 4 * E + 2.0 ** -25)
    assert bool(stats.isfinite().all()) and bool(s2.isfinite().all())


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("T", [0.3, 0.7, 1.0, 4.0, 1e30])
@pytest.mark.parametrize("rest", [True, False])
def test_gradients_of_such_rows(vt, dt, T, rest):
    """Each is A p_j minus what the teacher pulls, both off by E, by their exponential (4 u, and three roundings
    of |z - max| / T, u = 2^-24) and by 6 roundings, the rest's pull by 2^-27 / q p_j more; then rounded
    to the logits' type."""
    x, ids, lnt = _rows(dt)
    u = 2.0 ** -24
    h = lambda t: t.float().cpu().numpy()  # noqa: E731
    T32 = float(np.float32(T))
    ref = distill(h(x), ids.cpu().numpy(), h(lnt), None, rest, T32)
    z = h(x).astype(np.float64)
    d = np.minimum((z.max(1, keepdims=True) - z) / T32, 300.0)
    E, q = u * (700 / 256 + 90), np.exp(np.clip(ref["lnq"], -600, 0))[:, None]
    more = np.where((ref["left"][:, None] > 0) & (ref["pull"] < 0), 2.0 ** -27 * np.minimum(ref["p"] / q, 1.0), 0.0)
    tol = ((ref["p"] + np.abs(ref["pull"])) * (E + u * (10 + 3 * d)) + more) / T32 + 1e-37
    tol += np.abs(ref["grad"]) * (2.0 ** -8 if dt == torch.bfloat16 else u)
    _, stats, _ = vt.vt_distill_loss(x, ids, lnt, rest=rest, temperature=T)
    for g in (vt.vt_distill_grad(x, ids, lnt, stats, temperature=T),
              vt.vt_distill_loss_grad(x, ids, lnt, rest=rest, temperature=T)[1]):
        assert np.all(np.abs(h(g).astype(np.float64) - ref["grad"]) <= tol)
