"""Gradients in the logits' place: the same bits as apart from them, the loss, statistics and status
of the call in place among them.

(What a row is computed from does not depend on where its gradient goes, so no tolerance is needed.)
"""
import pytest

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


def _same(a, b):
    return torch.equal(a.nan_to_num(nan=7.5), b.nan_to_num(nan=7.5)) and torch.equal(a.isnan(), b.isnan())


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("R,K,k,pad,lead", [(1, 1, 1, 0, 0), (3, 5, 3, 2, 1), (700, 37, 5, 0, 3), (2000, 1003, 20, 1, 2),
                                            (460, 20011, 128, 0, 1), (40, 128256, 100, 0, 0), (5, 300007, 40, 3, 1)])
@pytest.mark.parametrize("rest", [True, False])
def test_in_place_is_as_apart(vt, R, K, k, pad, lead, dt, rest):
    g = torch.Generator(device="cuda")
    g.manual_seed(R + K)

    def rows():
        return torch.empty(lead + R * (K + pad), dtype=dt, device="cuda")[lead:].view(R, K + pad)[:, :K]

    x = rows()
    x.copy_(torch.randn((R, K), generator=g, device="cuda") * 3)
    step = max(1, (1 << 26) // K)
    ids = torch.empty((R, k), dtype=torch.int32, device="cuda")
    for r in range(0, R, step):  # distinct ids, those at the rows' ends among them
        ids[r:r + step] = torch.rand((min(step, R - r), K), generator=g, device="cuda").topk(k, 1).indices.int()
    ids[:, 0] = torch.where((ids == 0).any(1), ids[:, 0], 0)
    ids[1::7] = -1
    lnt = (torch.rand((R, k), generator=g, device="cuda") / k).log()
    w = torch.randn(R, generator=g, device="cuda")
    if R > 20:
        x[5, K // 2] = float("nan")       # one row that is flagged
        ids[9, 0] = K                     # and another
    apart = vt.vt_distill_loss_grad(x, ids, lnt, w, rest=rest, out_grad=rows())
    y = rows()
    y.copy_(x)
    here = vt.vt_distill_loss_grad(y, ids, lnt, w, rest=rest, out_grad=y)
    assert here[1] is y
    for a, b in zip(apart, here):
        assert _same(a.float(), b.float())
    want = (vt.VT_DEV_NONFINITE | vt.VT_DEV_BAD_ID) if R > 20 else 0
    assert int(here[3].item()) == want
    loss, stats, st = vt.vt_distill_loss(x, ids, lnt, rest=rest)
    assert int(st.item()) == want
    apart = vt.vt_distill_grad(x, ids, lnt, stats, w, out_grad=rows())
    y.copy_(x)
    here = vt.vt_distill_grad(y, ids, lnt, stats, w, out_grad=y)
    assert here is y and _same(apart.float(), y.float())
