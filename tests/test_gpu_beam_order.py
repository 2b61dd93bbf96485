"""The order of vt_beam_select where candidates are nearer than the first sums tell apart.

Equal beams have equal scores, and equal scores tie to the lower beam, then to the lower id: what a
sequence returns then follows from the logits alone and is worked out here without any
softmax.  Rows whose logits are equal but for their places or a constant have one ln S, so their
candidates compare by score + logit - largest, which fp64 holds exactly for the values taken here.
Scores are within 5e-6 + 2^-24 |ref| (half of the distance within which the library sums again).
"""
import numpy as np
import pytest

from oracle.beam import beam_select

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


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _rows_of_one_sum(x, s):
    """(scores, parents, ids) of the 32 best of sequences whose rows all have the same softmax sum."""
    x, s = x.double().cpu().numpy(), s.double().cpu().numpy()
    B, W, K = x.shape
    m = x.max(2, keepdims=True)
    lnS = np.log(np.exp(x - m).sum(2))[:, :, None]
    key = (s[:, :, None] + (x - m)).reshape(B, W * K)
    at = np.argsort(-key, axis=1, kind="stable")[:, :32]
    score = (key.reshape(B, W, K) - lnS).reshape(B, W * K)
    return np.take_along_axis(score, at, 1), at // K, at % K


def _check(vt, x, s, counts):
    score, parent, ids = _rows_of_one_sum(x, s)
    for n in counts:
        sc, pa, tk, _, st = vt.vt_beam_select(x, s, n)
        assert int(st.item()) == 0
        pa, tk, sc = pa.cpu().numpy(), tk.cpu().numpy(), sc.cpu().numpy().astype(np.float64)
        h = min(n, score.shape[1])
        assert np.array_equal(pa[:, :h], parent[:, :h]), n
        assert np.array_equal(tk[:, :h], ids[:, :h]), n
        assert (pa[:, h:] == -1).all() and (tk[:, h:] == -1).all()
        assert np.all(np.abs(sc[:, :h] - score[:, :h]) <= 5e-6 + 2.0 ** -24 * np.abs(score[:, :h]))


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("W,K,pad", [(2, 1003, 1), (3, 20011, 3), (6, 20011, 3), (8, 32003, 0), (32, 5003, 1), (32, 1, 0)])
@pytest.mark.parametrize("tied", [False, True])
def test_equal_beams_at_every_cut(vt, W, K, pad, dt, tied):
    # the same row behind several alignments, with one best logit or with three
    g = _gen(W * K + tied)
    B = 12
    row = (torch.randn((B, 1, K), generator=g, device="cuda") * 3).to(dt)
    if tied:
        best = row.amax(2, keepdim=True)
        for at in (K // 5, K // 2, K - 1):
            row[:, :, at:at + 1] = best
    buf = torch.zeros((B, W, K + pad), dtype=dt, device="cuda")
    x = buf[:, :, :K]
    x[:] = row
    s = torch.full((B, W), -3.25, device="cuda")
    _check(vt, x, s, range(1, 33))


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
def test_equal_beams_among_others(vt, dt):
    # three groups of equal beams, their numbers mixed; only the groups' scores tell them apart
    g = _gen(5)
    B, W, K = 20, 12, 9001
    row = (torch.randn((B, 1, K), generator=g, device="cuda") * 2).to(dt)
    x = torch.zeros((B, W, K + 5), dtype=dt, device="cuda")[:, :, :K]
    x[:] = row
    s = torch.full((B, W), -4.0, device="cuda")
    s[:, 1::3], s[:, 2::3] = -3.5, -4.5
    _check(vt, x, s, (1, 2, 3, 4, 5, 7, 8, 11, 20, 32))


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
def test_equal_beams_in_other_orders_of_ids(vt, dt):
    # rows of the same logits in other places, and behind constants that the sum takes out again
    g = _gen(6)
    B, W, K = 10, 8, 6007
    row = (torch.randn((B, 1, K), generator=g, device="cuda") * 24).round().clamp(-127, 127) / 8.0
    perm = torch.rand((B, W, K), generator=g, device="cuda").argsort(2)
    x = row.expand(B, W, K).gather(2, perm)
    s = torch.full((B, W), -3.25, device="cuda")
    _check(vt, x.to(dt), s, (1, 2, 3, 5, 8, 9, 17, 32))
    up = (torch.arange(W, device="cuda") * 3 % 8).float()[None, :, None]
    _check(vt, (x + up).to(dt), s, (1, 2, 3, 5, 8, 9, 17, 32))


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
def test_scores_and_logits_of_one_total(vt, dt):
    # totals of score and logit that are equal by different terms
    g = _gen(7)
    B, W, K = 40, 8, 3001
    row = (torch.randn((B, 1, K), generator=g, device="cuda") * 24).round().clamp(-127, 127) / 8.0
    perm = torch.rand((B, W, K), generator=g, device="cuda").argsort(2)
    x = row.expand(B, W, K).gather(2, perm).to(dt)
    s = -3.0 - torch.randint(0, 12, (B, W), generator=g, device="cuda") / 8.0
    _check(vt, x, s, (1, 2, 3, 5, 8, 13, 32))


@pytest.mark.parametrize("n", [1, 2, 3, 4])
def test_ended_beams_at_the_cut(vt, n):
    # beams that have ended, a few fp32 steps from the candidates of equal live ones
    g = _gen(8)
    B, W, K = 32, 6, 20011
    row = torch.randn((B, 1, K), generator=g, device="cuda") * 2
    x = torch.zeros((B, W, K + 3), device="cuda")[:, :, :K]
    x[:] = row
    s = torch.full((B, W), -3.25, device="cuda")
    done = torch.zeros((B, W), dtype=torch.bool, device="cuda")
    done[:, 1] = done[:, 4] = True
    d = row[:, 0].double()
    best = (s[:, 0].double() + d.amax(1) - d.logsumexp(1)).float()
    step = (torch.arange(B, device="cuda") % 8 - 4).float()
    s[:, 1] = best + step * 2.0 ** -21
    s[:, 4] = best - step * 2.0 ** -21
    ref = beam_select(x.cpu().numpy(), s.cpu().numpy(), n, 1.0, None, done.cpu().numpy(), K + 1)
    clear = ref["gap"] > 2e-8            # (the others are left open by the calls' contract)
    assert clear.sum() >= B // 2
    _, pa, tk, dn, st = vt.vt_beam_select(x, s, n, done=done, end_id=K + 1)
    assert int(st.item()) == 0
    # equal live beams tie in the oracle's fp64 as they are the same row
    assert np.array_equal(pa.cpu().numpy()[clear], ref["parent"][clear])
    assert np.array_equal(tk.cpu().numpy()[clear], ref["tokens"][clear])
    assert np.array_equal(dn.cpu().numpy()[clear], ref["done"][clear])
