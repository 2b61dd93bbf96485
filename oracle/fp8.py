"""The 8-bit head: e4m3 values with one power-of-two scale per block of 128
(fp64 oracle).

The format is the library's (include/vt.h, "The head in 8-bit floating
point"): e4m3 is the 8-bit float with 4 exponent bits (bias 7), 3 mantissa
bits, no infinities, NaN at all-ones, largest value 448.  A block's scale s is
the smallest power of two >= 2^-126 with max |block| <= 448 s; the stored
value is the e4m3 value nearest to W / s, ties to the even code.

Test infrastructure only; see the package docstring.
"""
from __future__ import annotations

import numpy as np

from .vocabtrim import bf16_to_f64

BLOCK = 128
E4M3_MAX = 448.0


def e4m3_table() -> np.ndarray:
    """The 256 values of e4m3 by code (NaN at 0x7f and 0xff)."""
    out = np.empty(256, dtype=np.float64)
    for code in range(256):
        e, m = (code >> 3) & 15, code & 7
        v = m / 8.0 * 2.0 ** -6 if e == 0 else (1.0 + m / 8.0) * 2.0 ** (e - 7)
        if e == 15 and m == 7:
            v = np.nan
        out[code] = -v if code & 128 else v
    return out


_POS = e4m3_table()[:127]  # 0 .. 448, ascending


def to_e4m3(v) -> np.ndarray:
    """Codes of the nearest e4m3 values, ties to the even code, |v| <= 448."""
    v = np.asarray(v, dtype=np.float64)
    a = np.abs(v)
    if not np.all(a <= E4M3_MAX):
        raise ValueError("|v| must not exceed 448")
    hi = np.clip(np.searchsorted(_POS, a), 0, 126)     # first value >= a
    lo = np.maximum(hi - 1, 0)
    dl, dh = a - _POS[lo], _POS[hi] - a
    code = np.where(dl < dh, lo, np.where(dh < dl, hi, np.where(lo % 2 == 0, lo, hi)))
    return (code | np.where(np.signbit(v), 128, 0)).astype(np.uint8)


def block_scale(amax: float) -> float:
    """The smallest power of two s >= 2^-126 with amax <= 448 s."""
    s = 2.0 ** -126
    while amax > E4M3_MAX * s:
        s *= 2.0
    return s


def quantize_head(W_bits):
    """(codes uint8 [K, H], scales fp64 [ceil(K/128), ceil(H/128)]) of a head
    given as bf16 bit patterns."""
    W = bf16_to_f64(W_bits)
    K, H = W.shape
    scale = np.empty((-(-K // BLOCK), -(-H // BLOCK)))
    codes = np.empty((K, H), dtype=np.uint8)
    for i in range(scale.shape[0]):
        for g in range(scale.shape[1]):
            blk = np.s_[i * BLOCK:(i + 1) * BLOCK, g * BLOCK:(g + 1) * BLOCK]
            scale[i, g] = block_scale(float(np.abs(W[blk]).max()))
            codes[blk] = to_e4m3(W[blk] / scale[i, g])
    return codes, scale


def quantize_rows(hidden_bits):
    """(dequantised hidden states fp64 [B, H]): the same rule per row and
    group of 128 columns."""
    x = bf16_to_f64(hidden_bits)
    out = np.empty_like(x)
    table = e4m3_table()
    for b in range(x.shape[0]):
        for h in range(0, x.shape[1], BLOCK):
            s = block_scale(float(np.abs(x[b, h:h + BLOCK]).max()))
            out[b, h:h + BLOCK] = table[to_e4m3(x[b, h:h + BLOCK] / s)] * s
    return out


def dequantize_head(codes, scale) -> np.ndarray:
    """fp64 [K, H] of e4m3 codes and block scales."""
    K, H = np.asarray(codes).shape
    s = np.repeat(np.repeat(np.asarray(scale, np.float64), BLOCK, 0)[:K], BLOCK, 1)[:, :H]
    return e4m3_table()[codes] * s


def draft_logits_fp8(hidden_bits, codes, scale, temperature: float):
    """(z fp64 [B, K], A [B, K]): the logits, and the sum of the magnitudes
    of their terms (what an error bound of a sum is relative to)."""
    x, W = quantize_rows(hidden_bits), dequantize_head(codes, scale)
    return (x @ W.T) / float(temperature), (np.abs(x) @ np.abs(W).T) / float(temperature)
