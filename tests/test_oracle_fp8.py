"""The 8-bit head's oracle on facts that do not come from it: e4m3's published
extremes, torch's e4m3 type, brute-force nearest values, hand-worked blocks."""
import numpy as np
import pytest

import synthetic
from oracle import fp8


def test_e4m3_table_extremes():
    t = fp8.e4m3_table()
    assert t[0x7E] == 448.0 and t[0x08] == 2.0 ** -6 and t[0x01] == 2.0 ** -9 and t[0x38] == 1.0
    assert np.isnan(t[0x7F]) and np.isnan(t[0xFF]) and np.signbit(t[0x80])
    assert np.all(np.diff(t[:127]) > 0)


def test_rounding_equals_torch_on_every_bf16_in_range():
    torch = pytest.importorskip("torch")
    bits = np.arange(1 << 16, dtype=np.uint32) << 16
    v = bits.view(np.float32)
    v = v[np.isfinite(v) & (np.abs(v) <= 448.0)]
    want = torch.from_numpy(v.copy()).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(fp8.to_e4m3(v), want)


def test_rounding_is_nearest_with_ties_to_even_codes():
    t = fp8.e4m3_table()[:127]
    mid = (t[1:] + t[:-1]) / 2
    codes = fp8.to_e4m3(mid)
    assert np.array_equal(codes, np.where(np.arange(126) % 2 == 0, np.arange(126), np.arange(1, 127)))
    assert np.array_equal(fp8.to_e4m3(np.nextafter(mid, 0)), np.arange(126))
    assert np.array_equal(fp8.to_e4m3(np.nextafter(mid, 500)), np.arange(1, 127))


def test_block_scale_by_hand():
    assert fp8.block_scale(448.0) == 1.0 and fp8.block_scale(448.5) == 2.0
    assert fp8.block_scale(224.0) == 0.5 and fp8.block_scale(0.0) == 2.0 ** -126
    assert fp8.block_scale(1.0) == 2.0 ** -8        # 1 / 2^-8 = 256 <= 448 < 512


def test_blocks_are_scaled_apart_and_within_half_a_step():
    g = synthetic.rng(3, 1)
    W = g.standard_normal((200, 150)) * np.where(np.arange(200) < 128, 1.0, 1e-3)[:, None]
    bits = synthetic.to_bf16_bits(W.astype(np.float32))
    codes, s = fp8.quantize_head(bits)
    assert s.shape == (2, 2) and np.all(s[0] > 100 * s[1])
    from oracle.vocabtrim import bf16_to_f64
    w, back = bf16_to_f64(bits), fp8.dequantize_head(codes, s)
    step = np.repeat(np.repeat(s, 128, 0)[:200], 128, 1)[:, :150] * 2.0 ** -9
    assert np.all(np.abs(back - w) <= np.maximum(np.abs(w) * 2.0 ** -4, step / 2))


def test_logits_on_exact_values_equal_the_plain_head():
    from oracle.vocabtrim import draft_logits
    g = synthetic.rng(4, 1)
    hid = (g.integers(-2, 3, (3, 300)).astype(np.float32).view(np.uint32) >> 16).astype(np.uint16)
    W = (g.integers(-2, 3, (130, 300)).astype(np.float32).view(np.uint32) >> 16).astype(np.uint16)
    z, A = fp8.draft_logits_fp8(hid, *fp8.quantize_head(W), 0.5)
    assert np.array_equal(z, draft_logits(hid, W, 0.5)) and np.all(A >= np.abs(z))
