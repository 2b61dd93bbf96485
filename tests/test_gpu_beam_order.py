"""The order of vt_beam_select where candidates are nearer than the first sums tell apart.

Equal beams have equal scores, and equal scores tie to the lower beam, then to the lower id: what a
sequence returns then follows from the logits alone and is worked out here without any
softmax: the rows have one ln S, so their candidates compare by score + logit - largest.
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
