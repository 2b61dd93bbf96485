"""The 8-bit product for more than 64 rows, whose scales differ in every block
of the head and every group of the hidden states, against 64-bit products.

Exact cases: hidden states are integers in [-2, 2] times 2^e, e in [-2, 2]
drawn per row and group, weights such integers times a scale 2^f, f in [-2, 2],
drawn per block (times 1.5 or -0.75 in blocks of rows that take the other loop).
Every term is a multiple of 2^-6 and every sum of terms at most A, the sum of
their magnitudes; A < 2^18 (asserted) makes every partial sum, in any order
and on either side of a rounding, a 24-bit multiple of 2^-6, so the logits are
equal bit for bit.
"""
import numpy as np
import pytest

import synthetic
from oracle import fp8
from parity import assert_probs_close

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

# e4m3 codes of -2 .. 2
CODES = np.array([0xC0, 0xB8, 0x00, 0x38, 0x40], np.uint8)


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


def _case(B, H, K, other):
    """(hidden bf16, W8, w_scale, z fp64 [B, K] at temperature 1), on the GPU.
    other: every how many blocks of rows have scales that are no powers of two (0: none)."""
    g = synthetic.rng(B + H + K + other, 21)
    n, kb = -(-H // 128), -(-K // 128)
    x = g.integers(-2, 3, (B, H)).astype(np.float64)
    x *= np.repeat(2.0 ** g.integers(-2, 3, (B, n)), 128, 1)[:, :H]
    w = g.integers(-2, 3, (K, H))
    s = 2.0 ** g.integers(-2, 3, (kb, n))
    if other:
        s[::other] *= np.where(g.integers(0, 2, s[::other].shape) == 0, 1.5, -0.75)
    xd, wd = _dev(x), _dev(w.astype(np.int8)).double()
    wd *= _dev(s).repeat_interleave(128, 0)[:K].repeat_interleave(128, 1)[:, :H]
    assert float((xd.abs() @ wd.abs().T).max()) < 2.0 ** 18
    buf = torch.full((K, (H + 15) // 16 * 16 + 16), 0x7F, dtype=torch.uint8, device="cuda")
    buf[:, :H] = _dev(CODES[w + 2])
    return xd.bfloat16(), buf[:, :H], _dev(s.astype(np.float32)), xd @ wd.T


# 5, 17, 33, 65 and 100 groups; up to several items per CTA or pair; one and more chunks, odd and even
CASES = [(65, 600, 45000), (100, 2110, 700), (130, 2110, 41000), (256, 4200, 20003), (256, 640, 40100),
         (300, 8300, 15000), (384, 2110, 4001), (1000, 12800, 10007), (1000, 600, 9999)]


@pytest.mark.parametrize("other", [0, 1, 2, 5])
@pytest.mark.parametrize("B,H,K", CASES)
def test_logits_of_differing_scales_bit_exact(vt, B, H, K, other):
    hid, W8, s, z = _case(B, H, K, other)
    got = vt.vt_draft_logits_fp8(hid, W8, s, 0.5)
    assert torch.equal(got.double(), 2 * z)
    assert torch.equal(got, vt.vt_draft_logits_fp8(hid, W8, s, 0.5))


@pytest.mark.parametrize("other", [0, 3])
@pytest.mark.parametrize("B,H,K", CASES)
def test_greedy_step_of_differing_scales(vt, B, H, K, other):
    hid, W8, s, z = _case(B, H, K, other)
    ids = torch.arange(K, dtype=torch.int32, device="cuda") * 3
    q, tok, st = vt.vt_draft_step_fp8(hid, W8, s, ids, None, 0.0)
    first = (z == z.amax(1, keepdim=True)).int().argmax(1)      # the lowest of equal ones
    want = torch.zeros_like(q)
    want[torch.arange(B), first] = 1.0
    assert int(st.item()) == 0 and torch.equal(tok, ids[first]) and torch.equal(q, want)


@pytest.mark.parametrize("other", [0, 3])
@pytest.mark.parametrize("B,H,K", [c for c in CASES if c[0] * c[2] < 6e6])
def test_sampling_and_topk_of_differing_scales(vt, B, H, K, other):
    hid, W8, s, z = _case(B, H, K, other)
    T = float(z.std())
    ids = torch.arange(K, dtype=torch.int32, device="cuda")
    q, _, st = vt.vt_draft_step_fp8(hid, W8, s, ids, torch.full((B,), 0.5, device="cuda"), T)
    assert int(st.item()) == 0
    assert_probs_close(q.cpu().numpy(), torch.softmax(z / T, 1).cpu().numpy())
    out, logq, st = vt.vt_draft_topk_fp8(hid, W8, s, ids, 8, T)
    assert int(st.item()) == 0
    assert torch.equal(torch.gather(z, 1, out.long()), z.topk(8, dim=1).values)
    # z2 = z log2(e) / T is rounded three times and |z| / T <= 8 here, the sum and its logarithm to 1e-6
    lq = torch.gather(torch.log_softmax(z / T, 1), 1, out.long())
    assert float((logq - lq).abs().max()) <= 8 * 4 * 2.0 ** -24 + 1e-5


@pytest.mark.parametrize("other", [False, True])
@pytest.mark.parametrize("B,H", [(16, 4096), (64, 8192), (65, 4096), (128, 2048), (128, 8192), (256, 4096), (256, 8192),
                                 (300, 6000), (512, 4096)])
def test_logits_keep_the_digits_of_an_fp32_product(vt, B, H, other):
    """The stated accuracy, 1.5e-7 of the logits in the 2-norm on random inputs, with the quantiser's own scales
    and with others.  It is a mean over B x 1500 errors, so it hardly varies between inputs: a plain fp32 product
    has 0.6e-7 to 1.2e-7 for these H, and sums of 32 groups by the tensor cores would have 2.1e-7."""
    K = 1500
    hid, W = synthetic.hidden_states((B, H), seed=B + H), synthetic.head_weights(K, H, seed=H)
    W8, s, st = vt.vt_quantize_head(_dev(W.view(np.int16)))
    assert int(st.item()) == 0
    if other:
        s = s * 1.25                                             # exact, and no power of two
    w = W8.float().double() * s.double().repeat_interleave(128, 0)[:K].repeat_interleave(128, 1)[:, :H]
    ref = _dev(fp8.quantize_rows(hid)) @ w.T
    z = vt.vt_draft_logits_fp8(_dev(hid.view(np.int16)), W8, s)
    assert float((z.double() - ref).norm() / ref.norm()) <= 1.5e-7


@pytest.mark.parametrize("B,H", [(100, 640), (256, 640), (256, 4200), (300, 4200), (512, 2110)])
def test_rows_groups_and_blocks_of_very_different_scale(vt, B, H):
    """Powers of two from 2^-110 to 2^100 between rows, groups and blocks, and groups and blocks of zeros (whose
    scale is 2^-126): with A the sum of the terms' magnitudes, n roundings or cuts of 2^-23 A as in
    tests/test_gpu_fp8.py; a tenth of the rows are far from the others' scale."""
    K = 700
    g = synthetic.rng(B + H, 22)
    n, kb = -(-H // 128), -(-K // 128)
    ex = g.integers(-3, 4, (B, n)) + np.where(np.arange(B) % 10 == 3, g.integers(-110, 90, B), 0)[:, None]
    x = g.standard_normal((B, H)) * np.repeat(2.0 ** ex, 128, 1)[:, :H]
    x[:, 128:256] *= 2.0 ** -30
    x[5], x[7, 256:384] = 0.0, 0.0
    w = g.standard_normal((K, H)) * np.repeat(np.repeat(2.0 ** g.integers(-20, 21, (kb, n)), 128, 0)[:K], 128, 1)[:, :H]
    w[128:256] *= 2.0 ** -40
    w[256:384, :128] = 0.0
    hid, wb = synthetic.to_bf16_bits(x.astype(np.float32)), synthetic.to_bf16_bits(w.astype(np.float32))
    W8, s, st = vt.vt_quantize_head(_dev(wb.view(np.int16)))
    assert int(st.item()) == 0 and float(s.min()) == 2.0 ** -126
    wd = W8.float().double() * s.double().repeat_interleave(128, 0)[:K].repeat_interleave(128, 1)[:, :H]
    xd = _dev(fp8.quantize_rows(hid))
    ref, A = xd @ wd.T, xd.abs() @ wd.abs().T
    for other in (False, True):
        z = vt.vt_draft_logits_fp8(_dev(hid.view(np.int16)), W8, s * 1.5 if other else s).double()
        want = ref * 1.5 if other else ref
        bound = (H + n + 6) * 2.0 ** -23 * A * (1.5 if other else 1.0) + 1e-30
        assert bool(((z - want).abs() <= bound).all())
        assert bool((z[5] == 0).all())
