"""What the documentation of beam search and distillation says of the ends of their ranges."""
import numpy as np
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


def test_scores_below_fp32_keep_their_parents(vt):
    x = torch.tensor([[[3.0, 2.0, 1.0], [0.0, -1.0, -2.0]]], device="cuda")
    sc, pa, tk, _, st = vt.vt_beam_select(x, torch.tensor([[-1.0, -2.0]], device="cuda"), 8, temperature=1e-30)
    assert int(st.item()) == 0
    # candidates 1e30 apart are within fp32, 1e39 are not
    assert sc[0, :2].tolist() == [-1.0, -2.0] and pa[0].tolist() == [0, 1, 0, 1, 0, 1, -1, -1]
    sc, pa, tk, _, st = vt.vt_beam_select(x * 1e9, torch.tensor([[-1.0, -2.0]], device="cuda"), 8, temperature=1e-30)
    assert int(st.item()) == 0
    assert np.isneginf(sc[0, 2:].cpu().numpy()).all()
    assert pa[0].tolist() == [0, 1, 0, 1, 0, 1, -1, -1] and tk[0].tolist() == [0, 0, 1, 1, 2, 2, -1, -1]


def test_rows_that_keep_nothing_are_not_looked_at(vt):
    x = torch.randn((2, 50), device="cuda")
    inv = torch.full((100,), -1, dtype=torch.int32, device="cuda")
    inv[:50] = torch.arange(50, dtype=torch.int32, device="cuda")
    ids = torch.tensor([[70, 80], [3, 4]], dtype=torch.int32, device="cuda")
    lnt = torch.full((2, 2), -1.0, device="cuda")
    x[0, 9] = float("nan")
    for rest in (True, False):
        loss, grad, stats, st = vt.vt_distill_loss_grad(x, ids, lnt, inv_map=inv, rest=rest)
        assert int(st.item()) == 0 and float(loss[0]) == 0.0 and not grad[0].any() and not stats[0].any()
        loss, stats, st = vt.vt_distill_loss(x, ids, lnt, inv, rest)
        assert int(st.item()) == 0 and float(loss[0]) == 0.0
        assert not vt.vt_distill_grad(x, ids, lnt, stats, inv_map=inv)[0].any()


def test_autograd_goes_on_from_the_gradient(vt):
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    h = torch.randn((12, 16), generator=g, device="cuda")
    W = torch.randn((40, 16), generator=g, device="cuda").requires_grad_()
    z = h @ W.t()
    ids = torch.arange(24, dtype=torch.int32, device="cuda").view(12, 2)
    lnt = torch.full((12, 2), -1.0, device="cuda")
    loss, grad, stats, _ = vt.vt_distill_loss_grad(z, ids, lnt)
    assert not (loss.requires_grad or grad.requires_grad or stats.requires_grad)
    torch.autograd.backward(z, grad)
    want = grad.double().t() @ h.double()
    # 12 products summed in fp32 (or TF32's 2^-11 of each, where the product uses it)
    assert torch.all((W.grad.double() - want).abs() <= 2.0 ** -10 * (grad.double().abs().t() @ h.double().abs()))
